"""ra_page_select: what its scores may and may not depend on, the search in lists of
candidates, and the attention through its lists."""
import numpy as np
import pytest
import torch

from oracle import paged as P
from test_gpu_page_select import draw, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seq,new,n_sel", [([1000, 333], None, 9), ([16 * 40 + 5, 16 * 33], [2, 1], 12), ([700, 500], [0, 0], 5)])
@pytest.mark.parametrize("other", [float("nan"), float("inf"), 2.0 ** 100, -3.0])
def test_pages_of_other_sequences_do_not_count(cuda_lib, seq, new, n_sel, other):
    """The bounds of a page that is in no list (the cache's first among them) reach neither the
    indices nor anything that the call works out on its way: scores, group maxima and their
    error bounds in the workspace are the same, byte for byte."""
    ra = cuda_lib
    q, bounds, table = draw(2, 2, 8, 2, 128, 16, seq, 5)
    pages = bounds.shape[0]
    table = torch.where(table >= 0, table + 1, table).int()  # page 0, and the last two, are nobody's
    bounds = torch.cat((bounds[:1], bounds))
    need = ra.ra_page_select_workspace(2, 2, table.shape[1])
    lens = torch.tensor(seq, dtype=torch.int32).cuda()
    nl = None if new is None else torch.tensor(new, dtype=torch.int32).cuda()
    got = []
    for x in (1.0, other):
        b = bounds.clone()
        free = [p for p in range(pages + 1) if not (table == p).any()]
        assert 0 in free
        b[free] = x
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        sel = ra.ra_page_select(q.cuda(), b.cuda(), table.cuda(), lens, n_sel, 16, new_lens=nl, workspace=ws)
        want = P.select(f64(q), f64(bounds), 16, table.tolist(), seq, new if new is not None else [min(2, n) for n in seq], n_sel)
        assert np.array_equal(sel.cpu().numpy(), want)
        got.append(ws)
    assert torch.equal(*got)
    assert ra.ra_get_device_status() == ra.RA_OK


def spread(pages, Hkv, D, ps, seed, step=2.0 ** -6):
    """Bounds whose scores spread widely, on a grid that keeps 64-bit sums exact, pages in random
    places (the oracle's sort of all pages of a large cache, one head)."""
    gen = torch.Generator().manual_seed(seed)
    a, b = ((torch.randn((pages + 1, Hkv, D), generator=gen) * 64).round().clamp(-900, 900) * step for _ in "ab")
    gain = torch.exp2(torch.randint(-2, 2, (pages + 1, 1, 1), generator=gen).float())
    bounds = torch.stack((torch.minimum(a, b), torch.maximum(a, b)), 2) * gain[..., None]
    table = torch.randperm(pages + 1, generator=gen)[:pages].int()[None].contiguous()
    q = ((torch.randn((1, 1, 4 * Hkv, D), generator=gen) * 64).round() * step).to(torch.bfloat16)
    return q, bounds.to(torch.bfloat16), table


def ranked(q, bounds, table, n, new, ps, n_sel):
    """The oracle's choice for one sequence, vectorised: 64-bit scores, ties to the lower page."""
    D, Hkv, pages = q.shape[-1], bounds.shape[1], -(-n // ps)
    G, first = q.shape[2] // Hkv, (n - new) // ps
    sel = np.full((1, Hkv, n_sel), -1)
    for g in range(Hkv):
        lo, hi = (f64(bounds[table[0, :pages].long(), g, i]) for i in (0, 1))
        rows = f64(q[0, :new, g * G:(g + 1) * G]).reshape(-1, D)
        score = np.max([np.maximum(r * lo, r * hi).sum(1) for r in rows], axis=0)
        score[first:] = np.inf
        best = np.sort(np.lexsort((np.arange(pages), -score))[:n_sel])
        sel[0, g, :len(best)] = best
    return sel


# pages, n_sel: the search keeps a list of candidates where n_sel is at most a 16th of the pages and
# 2,816 or more are scored; it scans 8,192 of them at a time
@pytest.mark.parametrize("pages,n_sel", [(2818, 3), (4000, 20), (4003, 250), (8193, 2), (8200, 512), (16387, 512), (16500, 1030),
                                         (30001, 64)])
@pytest.mark.parametrize("Hkv,D,ps", [(1, 64, 16), (2, 128, 64)])
def test_the_best_of_very_many_pages(cuda_lib, pages, n_sel, Hkv, D, ps):
    ra = cuda_lib
    q, bounds, table = spread(pages, Hkv, D, ps, pages + n_sel)
    for n in (pages * ps, pages * ps - ps + 1):
        got = ra.ra_page_select(q.cuda(), bounds.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), n_sel, ps)
        assert np.array_equal(got.cpu().numpy(), ranked(q, bounds, table, n, 1, ps, n_sel))
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("pages,n_sel,equal", [(4000, 20, 30), (9000, 100, 300), (16387, 512, 700), (16387, 512, 2500), (5000, 40, 4000)])
@pytest.mark.parametrize("last", [0.0, 2.0 ** -20])
def test_ties_among_the_candidates(cuda_lib, pages, n_sel, equal, last):
    """Pages that are equal to the n_sel-th best one, or so close to it that fp32 cannot tell: from a
    few, ranked by their exact keys, to more than the list or the comparison holds."""
    ra = cuda_lib
    D, ps = 64, 16
    q, bounds, table = spread(pages, 1, D, ps, equal)
    lo, hi = (f64(bounds[table[0].long(), 0, i]) for i in (0, 1))
    rows = f64(q[0, 0])
    score = np.max([np.maximum(r * lo, r * hi).sum(1) for r in rows], axis=0)
    border = int(np.argsort(-score)[n_sel // 2])
    gen = torch.Generator().manual_seed(pages)
    q[..., 7] = q[..., 7].abs() + 1.0
    alike = bounds[table[0, border].long()].clone()
    alike[0, :, 7] = 0.0  # the column that tells them apart, if any does
    for i, p in enumerate(torch.randperm(pages, generator=gen)[:equal].tolist()):
        bounds[table[0, p].long()] = alike
        bounds[table[0, p].long(), 0, 1, 7] = last * (i % 5)
    n = pages * ps
    got = ra.ra_page_select(q.cuda(), bounds.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), n_sel, ps)
    assert np.array_equal(got.cpu().numpy(), ranked(q, bounds, table, n, 1, ps, n_sel))
    assert ra.ra_get_device_status() == ra.RA_OK


def test_every_page_selected_is_the_whole_cache(cuda_lib):
    """Lists of all pages take the tiles that no list takes (16 keys to a page: no tile more): bit for bit."""
    ra = cuda_lib
    from test_gpu_paged_decode import Case
    for dtype in ("bf16", "int8", "e4m3"):
        c = Case(dtype, 3, 2, 8, 2, 128, 16, [700, 33, 1600], seed=4)
        sel = torch.full((3, 2, c.table.shape[1]), -1, dtype=torch.int32)
        for b, n in enumerate(c.seq):
            sel[b, :, :-(-n // 16)] = torch.arange(-(-n // 16), dtype=torch.int32)
        a = ra.ra_paged_decode_attention(*c.args, **c.kw)
        b = ra.ra_paged_decode_attention(*c.args, selected=sel.cuda(), **c.kw)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert ra.ra_get_device_status() == ra.RA_OK
