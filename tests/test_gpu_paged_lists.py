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
