"""Lists of selected pages with gaps and mistakes in them: an entry is compared with the
nearest one in range before it, whatever lies between."""
import pytest
import torch

from test_gpu_paged_decode import Case

pytestmark = pytest.mark.gpu


def counted(entries, pages):
    """The list as the call counts it, and whether it holds a mistake."""
    got, last, bad = [], -1, False
    for x in entries:
        inside = 0 <= x < pages
        ok = inside and x > last
        bad |= x != -1 and not ok
        got.append(x if ok else -1)
        last = x if inside else last
    return got, bad


LISTS = [
    [3, -1, 3], [5, -1, 2], [0, 20, 3], [0, -1, -1, -1, 0, 6], [4, 99, -1, -7, 4, 5], [-1, -1, 2, -1, 2, 3],
    [-1, -1, -1, 6], [0, -1, 2, -1, -1, 5], [6, -1, -1, -1, -1, -1, 1], [1, 1 << 30, 2, 3], [2, -5, 1, 3],
    [1, -1, 2, 7, -1, 4, 6],
]


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("entries", LISTS, ids=lambda e: "_".join(str(x) for x in e))
def test_lists_with_gaps_and_mistakes(cuda_lib, dtype, entries):
    ra = cuda_lib
    c = Case(dtype, 1, 1, 4, 1, 64, 16, [100], seed=2)  # 7 pages
    want, bad = counted(entries, 7)
    got = ra.ra_paged_decode_attention(*c.args, selected=torch.tensor([[entries]], dtype=torch.int32).cuda(), **c.kw)
    assert ra.ra_get_device_status() == (ra.RA_ERR_DEVICE_BOUNDS if bad else ra.RA_OK)
    c.check(got, True, torch.tensor([[want]]))


@pytest.mark.parametrize("gap", [1, 40, 300])
def test_an_early_page_again_behind_a_long_gap(cuda_lib, gap):
    """The repeated entry lies in another warp's run than the first, tiles without a page between."""
    ra = cuda_lib
    c = Case("int8", 2, 1, 8, 2, 128, 32, [32 * (gap + 6), 50], seed=gap)
    sel = torch.full((2, 2, gap + 6), -1, dtype=torch.int32)
    sel[:, :, 0] = 1
    good = ra.ra_paged_decode_attention(*c.args, selected=sel.cuda(), **c.kw)
    c.check(good, True, sel)
    assert ra.ra_get_device_status() == ra.RA_OK
    again = sel.clone()
    again[0, :, gap + 1] = 1
    got = ra.ra_paged_decode_attention(*c.args, selected=again.cuda(), **c.kw)
    assert ra.ra_get_device_status() == ra.RA_ERR_DEVICE_BOUNDS
    assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])
    sel[0, :, gap + 1] = 2  # and one that ascends is none
    c.check(ra.ra_paged_decode_attention(*c.args, selected=sel.cuda(), **c.kw), True, sel)
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("gap", [5, 6, 7, 8, 9, 15, 16, 17, 18, 4096, 20000])
def test_gaps_of_every_length(cuda_lib, gap):
    """[1, gap, x]: x = 1 and x = 0 are recorded and count as no page, x = 2 counts."""
    ra = cuda_lib
    ps, D = 16, 64
    pages = gap + 4
    gen = torch.Generator().manual_seed(gap)
    kp, vp = (torch.randn((8, 1, ps, D), generator=gen).to(torch.bfloat16).cuda() for _ in "kv")
    q = torch.randn((1, 1, 2, D), generator=gen).to(torch.bfloat16).cuda()
    table = (torch.arange(pages, dtype=torch.int32) % 8)[None].contiguous().cuda()
    lens = torch.tensor([pages * ps], dtype=torch.int32).cuda()

    def call(*entries):
        sel = torch.full((1, 1, gap + 2), -1, dtype=torch.int32)
        for at, x in entries:
            sel[0, 0, at] = x
        got = ra.ra_paged_decode_attention(q, kp, vp, table, lens, selected=sel.cuda())
        return got, ra.ra_get_device_status()

    alone, status = call((0, 1))
    assert status == ra.RA_OK
    for x in (0, 1):
        got, status = call((0, 1), (gap + 1, x))
        assert status == ra.RA_ERR_DEVICE_BOUNDS
        assert torch.equal(got[0], alone[0]) and torch.equal(got[1], alone[1])
    for entries in (((0, 1), (gap + 1, 2)), ((gap, 1), (gap + 1, 2)), ((0, pages), (gap // 2, 1), (gap + 1, 2))):
        got, status = call(*entries)
        assert status == (ra.RA_ERR_DEVICE_BOUNDS if entries[0][1] == pages else ra.RA_OK)
        k, v = (x[1:3, 0].reshape(2 * ps, D).double() for x in (kp, vp))
        s = q[0, 0].double() @ k.T / 8.0
        assert torch.allclose(got[0][0, 0].double(), torch.softmax(s, 1) @ v, atol=1e-4)
        assert torch.allclose(got[1][0, 0].double(), torch.logsumexp(s, 1), atol=1e-5)
