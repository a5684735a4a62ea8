"""ra_page_select against the fp64 oracle, index for index.

Both sum products of bf16 values; the drawn values lie within 2^20 of each
other, so the kernel's 64-bit sums are exact (16-bit products, 7 bits for 128
terms, 2 x 15 bits of range below 53) and so is the oracle's fsum: the indices
have to be the same, ties included."""
import numpy as np
import pytest
import torch

from oracle import paged as P

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def draw(B, Tq, Hq, Hkv, D, ps, seq, seed, levels=None):
    """q, bounds and a table; with `levels`, pages repeat a few bounds (ties)."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in seq]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=gen).to(torch.int32)
    table = torch.full((B, max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c

    def quantised(*shape):  # values on a grid of 2^-6 below 16: the exponents stay close
        return ((torch.randn(shape, generator=gen) * 64).round() / 64).clamp(-15, 15).to(torch.bfloat16)

    a, b = quantised(n_pages, Hkv, D), quantised(n_pages, Hkv, D)
    bounds = torch.stack((torch.minimum(a, b), torch.maximum(a, b)), 2)
    if levels:
        bounds = bounds[torch.randint(0, levels, (n_pages,), generator=gen)].contiguous()
    return quantised(B, Tq, Hq, D), bounds, table


@pytest.mark.parametrize("B,Tq,Hq,Hkv,D,ps,seq,new,n_sel,levels", [
    (1, 1, 4, 1, 64, 16, [1], None, 1, None),
    (1, 1, 4, 1, 64, 16, [400], None, 1, None),               # the new token's page alone
    (2, 1, 8, 2, 128, 16, [400, 33], None, 7, None),
    (3, 1, 8, 2, 64, 32, [1000, 0, 96], None, 3, None),       # an empty slot; exactly n_sel pages
    (2, 4, 8, 2, 128, 16, [1000, 17], None, 9, None),
    (2, 4, 8, 2, 128, 16, [1000, 17], [2, 0], 9, None),       # padded rows; an idle sequence
    (1, 16, 4, 1, 64, 16, [161], None, 2, None),              # 64 rows; new tokens on two pages: nothing else fits
    (1, 9, 7, 1, 128, 64, [5000], None, 20, None),            # 63 rows
    (2, 1, 4, 2, 64, 16, [4000, 2000], None, 40, 5),          # ties
    (1, 1, 2, 2, 64, 128, [128 * 50], None, 25, 1),           # all pages alike: the lowest
    (1, 1, 8, 2, 128, 16, [16 * 5003], None, 700, None),      # more pages than threads
    (1, 1, 1, 1, 64, 16, [16 * 1500], None, 1499, None),      # all but one
])
def test_page_select(cuda_lib, B, Tq, Hq, Hkv, D, ps, seq, new, n_sel, levels):
    ra = cuda_lib
    for seed in (0, 1):
        q, bounds, table = draw(B, Tq, Hq, Hkv, D, ps, seq, seed, levels)
        if seed:  # one sign: every score negative or every one positive
            q, bounds = q.abs(), -bounds.abs().flip(2).sort(2).values
        lens = torch.tensor(seq, dtype=torch.int32).cuda()
        nl = None if new is None else torch.tensor(new, dtype=torch.int32).cuda()
        got = ra.ra_page_select(q.cuda(), bounds.cuda(), table.cuda(), lens, n_sel, ps, new_lens=nl)
        want = P.select(f64(q), f64(bounds), ps, table.tolist(), seq,
                        new if new is not None else [min(Tq, n) for n in seq], n_sel)
        assert np.array_equal(got.cpu().numpy(), want)
    assert ra.ra_get_device_status() == ra.RA_OK


def test_subnormal_huge_and_zero_bounds(cuda_lib):
    """The moved exponent field covers subnormal bf16 and the ends of the range."""
    ra = cuda_lib
    D, ps, n = 64, 16, 40
    gen = torch.Generator().manual_seed(3)
    scale = torch.tensor([2.0 ** -130, 2.0 ** -126, 1.0, 2.0 ** 126, 0.0])
    for s in scale:
        b = (torch.randn((n, 1, D), generator=gen).double() * s.double()).float().to(torch.bfloat16)
        bounds = torch.stack((b, b), 2).contiguous()
        q = torch.zeros((1, 1, 1, D), dtype=torch.bfloat16)
        q[..., 5] = -3.0  # one column counts: the sums are exact at any exponent
        table = torch.randperm(n, generator=gen).to(torch.int32)[None].contiguous()
        lens = torch.tensor([n * ps], dtype=torch.int32).cuda()
        got = ra.ra_page_select(q.cuda(), bounds.cuda(), table.cuda(), lens, 11, ps)
        want = P.select(f64(q), f64(bounds), ps, table.tolist(), [n * ps], [1], 11)
        assert np.array_equal(got.cpu().numpy(), want), s
    assert ra.ra_get_device_status() == ra.RA_OK


def test_padding_rows_and_wide_tables(cuda_lib):
    """Query rows that are not real hold NaN; the table is far wider than the lengths."""
    ra = cuda_lib
    seq, new = [900, 333, 50], [2, 1, 3]
    q, bounds, table = draw(3, 3, 8, 2, 128, 16, seq, 7)
    want = P.select(f64(q), f64(bounds), 16, table.tolist(), seq, new, 9)
    for b, n in enumerate(new):
        q[b, n:] = float("nan")
    wide = torch.full((3, 60000), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    got = ra.ra_page_select(q.cuda(), bounds.cuda(), wide.cuda(), torch.tensor(seq, dtype=torch.int32).cuda(), 9, 16,
                            new_lens=torch.tensor(new, dtype=torch.int32).cuda())
    assert np.array_equal(got.cpu().numpy(), want)
    assert ra.ra_get_device_status() == ra.RA_OK


def test_scores_closer_than_fp32_can_tell(cuda_lib):
    """Pages whose scores differ by one unit of 2^-30 beside terms of 2^10: the fp32
    pass cannot order them, the exact sums do.  More of them than are compared in
    shared memory, too."""
    ra = cuda_lib
    D, ps = 64, 16
    gen = torch.Generator().manual_seed(9)
    for n in (100, 3000):
        b = torch.zeros((n, 1, D), dtype=torch.bfloat16)
        b[..., :8] = 1024.0
        b[..., 9] = torch.randint(0, 16, (n, 1), generator=gen).float().to(torch.bfloat16) * 2.0 ** -30
        b[..., 10] = torch.randint(0, 16, (n, 1), generator=gen).float().to(torch.bfloat16) * 2.0 ** -26
        bounds = torch.stack((b, b), 2).contiguous()
        q = torch.ones((1, 1, 2, D), dtype=torch.bfloat16)
        table = torch.randperm(n, generator=gen).to(torch.int32)[None].contiguous()
        for n_sel in (2, 37):
            got = ra.ra_page_select(q.cuda(), bounds.cuda(), table.cuda(), torch.tensor([n * ps], dtype=torch.int32).cuda(),
                                    n_sel, ps)
            want = P.select(f64(q), f64(bounds), ps, table.tolist(), [n * ps], [1], n_sel)
            assert np.array_equal(got.cpu().numpy(), want), (n, n_sel)
    assert ra.ra_get_device_status() == ra.RA_OK


def test_infinite_keys_and_queries(cuda_lib):
    """An infinite bound counts as 2^128; a row whose sum is NaN does not count."""
    ra = cuda_lib
    q, bounds, table = draw(1, 2, 4, 1, 64, 16, [16 * 40], 3)
    bounds[5, 0, 1, 7] = float("inf")
    bounds[9, 0, 0, 3] = -float("inf")
    want = P.select(f64(q), f64(bounds), 16, table.tolist(), [16 * 40], [2], 12)
    lens = torch.tensor([16 * 40], dtype=torch.int32).cuda()
    got = ra.ra_page_select(q.cuda(), bounds.cuda(), table.cuda(), lens, 12, 16)
    assert np.array_equal(got.cpu().numpy(), want)
    q2 = q.clone()
    q2[0, 1] = float("nan")  # the second token's rows count for nothing
    want = P.select(f64(q[:, :1]), f64(bounds), 16, table.tolist(), [16 * 40], [1], 12)
    lens.fill_(16 * 40)
    got = ra.ra_page_select(q2.cuda(), bounds.cuda(), table.cuda(), lens, 12, 16)
    last = (16 * 40 - 2) // 16
    assert last == 39 and np.array_equal(got.cpu().numpy(), want)
    assert ra.ra_get_device_status() == ra.RA_OK


def test_bad_pages_are_recorded(cuda_lib):
    ra = cuda_lib
    q, bounds, table = draw(2, 1, 4, 2, 64, 16, [300, 200], 0)
    lens = torch.tensor([300, 200], dtype=torch.int32).cuda()
    good = ra.ra_page_select(q.cuda(), bounds.cuda(), table.cuda(), lens, 5, 16)
    table[1, 3] = 1 << 20
    got = ra.ra_page_select(q.cuda(), bounds.cuda(), table.cuda(), lens, 5, 16)
    assert ra.ra_get_device_status() == ra.RA_ERR_DEVICE_BOUNDS
    assert torch.equal(got[0], good[0])
    assert (got[1] >= 0).all() and (got[1] < 13).all()


def test_in_a_graph_with_the_attention(cuda_lib):
    """append -> select -> sparse attention as one captured step, replayed token by
    token; with every page selected it is the dense call, bit for bit."""
    ra = cuda_lib
    gen = torch.Generator().manual_seed(4)
    B, Hq, Hkv, D, ps, S, n_sel = 2, 8, 2, 64, 16, 300, 6
    n_pages = 2 * 22
    table = torch.randperm(n_pages, generator=gen).to(torch.int32).view(B, -1).contiguous()
    ref = P.Cache(n_pages, Hkv, ps, D, "int8")
    k, v = (torch.randn((B, S, Hkv, D), generator=gen).to(torch.bfloat16) for _ in "kv")
    kp = torch.zeros((n_pages, Hkv, ps, D), dtype=torch.int8, device="cuda")
    vp = torch.zeros_like(kp)
    ks, vs = (torch.zeros((n_pages, Hkv, ps), device="cuda") for _ in "kv")
    bounds = torch.zeros((n_pages, Hkv, 2, D), dtype=torch.bfloat16, device="cuda")
    tab = table.cuda()
    lens = torch.tensor([S, S - 40], dtype=torch.int32).cuda()
    sc = dict(k_scales=ks, v_scales=vs)
    ra.ra_cache_append(k.cuda(), v.cuda(), kp, vp, tab, lens, new_lens=lens, key_bounds=bounds, **sc)
    P.append(ref, f64(k), f64(v), table.tolist(), [S, S - 40], [S, S - 40])
    k1, v1 = (torch.zeros((B, 1, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    q = torch.zeros((B, 1, Hq, D), dtype=torch.bfloat16, device="cuda")

    def step(n):
        ra.ra_cache_append(k1, v1, kp, vp, tab, lens, key_bounds=bounds, **sc)
        sel = ra.ra_page_select(q, bounds, tab, lens, n, ps)
        return sel, ra.ra_paged_decode_attention(q, kp, vp, tab, lens, selected=sel, **sc)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(n_sel)  # outside the capture first; the token is appended again below
    torch.cuda.current_stream().wait_stream(stream)
    P.append(ref, np.zeros((B, 1, Hkv, D)), np.zeros((B, 1, Hkv, D)), table.tolist(), [S, S - 40], [1, 1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sel, (out, lse) = step(n_sel)
    for t in range(1, 20):
        nk, nv = (torch.randn((B, 1, Hkv, D), generator=gen).to(torch.bfloat16) for _ in "kv")
        nq = torch.randn((B, 1, Hq, D), generator=gen).to(torch.bfloat16)
        k1.copy_(nk)
        v1.copy_(nv)
        q.copy_(nq)
        now = [S + t, S - 40 + t]
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        P.append(ref, f64(nk), f64(nv), table.tolist(), now, [1, 1])
        assert np.array_equal(f64(bounds), ref.bounds)
        want = P.select(f64(nq), ref.bounds, ps, table.tolist(), now, [1, 1], n_sel)
        assert np.array_equal(sel.cpu().numpy(), want)
        ro, rl = P.decode(f64(nq), ref, table.tolist(), now, [1, 1], True, want.tolist())
        assert np.allclose(f64(out), ro, atol=1e-4) and np.allclose(f64(lse), rl, atol=1e-4)
    every = ra.ra_page_select(q, bounds, tab, lens, 22, ps)
    a = ra.ra_paged_decode_attention(q, kp, vp, tab, lens, **sc)
    b = ra.ra_paged_decode_attention(q, kp, vp, tab, lens, selected=every, **sc)
    assert torch.allclose(a[0], b[0], atol=1e-5) and torch.allclose(a[1], b[1], atol=1e-5)
    assert ra.ra_get_device_status() == ra.RA_OK
