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
