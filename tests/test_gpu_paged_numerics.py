"""ra_paged_decode_attention where its arithmetic is at its limits: long runs of one
warp, weights far below the largest, scores of minus infinity, tiny value scales, the
16-bit terms of the weights.  Each tolerance is derived at its test."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
DTYPES = ["bf16", "int8", "e4m3"]
# Sequences that keep every team of warps on runs of one whole sequence, whatever the
# form: as many as the most teams that a grid has.
MANY = 148 * 15


class Shared:
    """One sequence's pages (k, v [n, D] of one KV head), attended to by `B` sequences."""

    def __init__(self, ra, dtype, k, v, B, ps=128):
        n, D = k.shape
        pages = -(-n // ps)
        self.k_pages, self.v_pages = (torch.zeros((pages, 1, ps, D), dtype=TORCH[dtype], device="cuda") for _ in "kv")
        self.scales = {}
        if dtype != "bf16":
            self.scales = {w + "_scales": torch.zeros((pages, 1, ps), device="cuda") for w in "kv"}
        table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
        length = torch.tensor([n], dtype=torch.int32, device="cuda")
        rows = [x.to(torch.bfloat16).cuda().view(1, n, 1, D) for x in (k, v)]
        ra.ra_cache_append(*rows, self.k_pages, self.v_pages, table, length, **self.scales)
        kk, vv = ra.ra_cache_read(self.k_pages, self.v_pages, table, length, n, out_dtype=torch.float32, **self.scales)
        self.k, self.v = kk[0, :, 0].double(), vv[0, :, 0].double()  # what the cache stands for
        self.table, self.lens = table.expand(B, -1).contiguous(), length.expand(B).contiguous()

    def decode(self, ra, q, **kw):
        return ra.ra_paged_decode_attention(q, self.k_pages, self.v_pages, self.table, self.lens, **self.scales, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 12, 20, 40])
def test_sums_of_a_long_run_do_not_drift(cuda_lib, dtype, rows):
    """Keys of two kinds, so that the scores are 0 and -3/8 all but exactly and the output is a
    mean of 20,000 positive values with weights 1 and exp(-3/8): only sums can be wrong.  A
    tile's products take up to 6 steps that may cut (2^-23 of its sum each); its sum joins
    the 624 before it, and its weights theirs in l, with one rounding each (2^-24 of sums
    that only grow, all to one side at worst).  Weights are held to 2^-22 at least, their
    exponentials to 2^-21 (scores included) in the numerator and in l, division and output round
    once, and so does the logarithm."""
    ra = cuda_lib
    n, D = 20000, 64
    gen = torch.Generator().manual_seed(rows)
    k = torch.zeros((n, D))
    k[:, 1] = 1.0
    k[:, 0] = torch.randint(0, 2, (n,), generator=gen).float()
    c = Shared(ra, dtype, k, 0.5 + torch.rand((n, D), generator=gen), MANY)
    q = torch.zeros((MANY, 1, rows, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = -3.0
    out, lse = c.decode(ra, q, out_dtype=torch.float32)
    x = c.k @ q[0, 0, 0].double() / math.sqrt(D)
    want = torch.softmax(x, 0) @ c.v
    sums = 625 * 2.0 ** -24
    tol = 2 * sums + 6 * 2.0 ** -23 + 2.0 ** -22 + 2 * 2.0 ** -21 + 2 * 2.0 ** -24
    off = ((out.double() - want).abs() / want).max().item()
    assert off <= tol, f"off by {off:.3g}, {off / tol:.3g} tolerances"
    exact = torch.logsumexp(x, 0)
    assert (lse.double() - exact).abs().max() <= sums + 2.0 ** -21 + 2.0 ** -23 * exact
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 12, 20])
def test_a_long_tail_of_small_weights_counts(cuda_lib, dtype, rows):
    """One key, and 49,999 whose weights are 2^-25.15 of its own: 1.4e-3 of the result.  Each
    weight of an 8-bit cache is held to 2^-34 of the largest; its exponent of 25.15 (the
    score in binary units) to 2^-22 of itself and the exponential to 2^-21; a run's 1,563 tiles are
    added with one rounding each, in o and in l, where the first key's lane rounds at its 1."""
    ra = cuda_lib
    n, D = 50000, 64
    k, v = torch.zeros((n, D)), torch.ones((n, D))
    k[1:, 0], k[:, 1] = -1.0, 1.0
    v[0] = 0.0
    v[0, 5] = 1.0
    c = Shared(ra, dtype, k, v, MANY)
    q = torch.zeros((MANY, 1, rows, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 25.15 * math.log(2) * math.sqrt(D)
    out, lse = c.decode(ra, q, out_dtype=torch.float32)
    x = c.k @ q[0, 0, 0].double() / math.sqrt(D)
    want = torch.softmax(x, 0) @ c.v
    tail = want[0].item()
    assert 1e-3 < tail < 2e-3
    sums, each = 1563 * 2.0 ** -24, 25.5 * 2.0 ** -22 + 2.0 ** -21
    off = (out.double() - want).abs()
    only_tail = torch.arange(D, device="cuda") != 5
    tol = n * 2.0 ** -34 + tail * (2 * sums + each + 2.0 ** -22)
    assert off[..., only_tail].max() <= tol, f"off by {off[..., only_tail].max():.3g} where {tol:.3g} may be"
    assert off[..., 5].max() <= n * 2.0 ** -34 + 2 * sums + tail * each + 2.0 ** -21
    assert (lse.double() - torch.logsumexp(x, 0)).abs().max() <= sums + tail * each + 2.0 ** -22
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("n,ps,where", [
    (33, 16, [32]),                    # the newest key, in a tile of its own
    (1281, 16, [1280]),                # the same behind other warps' tiles
    (70, 32, list(range(32))),         # all of the first tile
    (600, 128, list(range(0, 600, 2))),
    (900, 64, list(range(800))),       # whole runs of other warps
])
@pytest.mark.parametrize("rows", [1, 12, 20])
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
def test_scores_of_minus_infinity_weigh_nothing(cuda_lib, n, ps, where, rows, odt):
    """Keys with an infinite column that the queries take with the other sign: weight 0,
    wherever a warp's run begins.  Odd rows have a 0 there (0 times infinity is NaN), and
    stay apart; a row all of whose keys are such is empty."""
    ra = cuda_lib
    D, pages = 64, -(-n // ps)
    gen = torch.Generator().manual_seed(n)
    k, v = torch.randn((pages * ps, D), generator=gen), torch.randn((pages * ps, D), generator=gen)
    k[:, 0] = 0.0
    k[where, 0] = -math.inf
    kp, vp = (x.to(torch.bfloat16).view(pages, 1, ps, D).cuda() for x in (k, v))
    q = torch.randn((1, 1, rows, D), generator=gen)
    q[..., 0] = 1.0
    odd = torch.arange(rows) % 2 == 1
    q[:, :, odd, 0] = 0.0
    q = q.to(torch.bfloat16)
    table = torch.arange(pages, dtype=torch.int32)[None].contiguous().cuda()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    out, lse = ra.ra_paged_decode_attention(q.cuda(), kp, vp, table, lens, out_dtype=odt)
    kd, vd = k[:n].to(torch.bfloat16).double(), v[:n].to(torch.bfloat16).double()
    x = q[0, 0, ~odd].double() @ kd.T / math.sqrt(D)
    assert torch.isneginf(x[:, where]).all()
    want, l = torch.softmax(x, 1) @ vd, torch.logsumexp(x, 1)
    # scores to (D + 4) 2^-24 of their terms, weights, exponentials and up to 600 / 8 sums of them, the output's rounding
    terms = (q[0, 0, ~odd].abs().double()[:, 1:].max() * kd[:, 1:].abs().sum(1).max()).item() / math.sqrt(D)
    dx = (D + 4) * 2.0 ** -24 * terms + 2.0 ** -21 + 80 * 2.0 ** -24
    tol = 2 * (dx + 2.0 ** -16) * vd.abs().max() + torch.finfo(odt).eps / 2 * want.abs()
    got, gl = out[0, 0, ~odd].cpu().double(), lse[0, 0, ~odd].cpu().double()
    assert (got - want).abs().le(tol).all()
    assert ((gl - l).abs() <= dx + 2.0 ** -23 * l.abs()).all()
    assert torch.isnan(out[0, 0, odd]).all()
    all_inf = torch.full_like(kp, -math.inf)
    q.fill_(1.0)
    out, lse = ra.ra_paged_decode_attention(q.cuda(), all_inf, vp, table, lens, out_dtype=odt)
    assert not out.any() and torch.isneginf(lse).all()
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", ["int8", "e4m3"])
@pytest.mark.parametrize("rows", [1, 12, 20])
@pytest.mark.parametrize("shift,growth", [(0, 16.9), (-13, 26.0)])
def test_tiny_values_do_not_overflow_the_sum(cuda_lib, dtype, rows, shift, growth):
    """Values of 2^-99, the smallest that an append keeps, and scores that grow by 16.9 binary
    units behind the first tile: 2^17 keys' worth of terms in l beside a first tile that the
    tiny scales let count 2^100.  Weight times scale is held to 2^-15 of the largest, the
    score (16.9 units) to 2^-22 of itself, sums as in the test of long runs.  With scales 2^-13
    smaller yet (no append's) the lse is still asked for."""
    ra = cuda_lib
    n, D = 20000, 64
    gen = torch.Generator().manual_seed(rows)
    k, v = torch.zeros((n, D)), (0.5 + 0.5 * torch.rand((n, D), generator=gen)) * 2.0 ** -99
    k[32:, 0], k[:, 1] = 1.0, 1.0
    v[:, 5] = 2.0 ** -99
    c = Shared(ra, dtype, k, v, MANY)
    assert 2.0 ** -109 <= c.scales["v_scales"][c.scales["v_scales"] > 0].min() < 2.0 ** -105
    c.scales["v_scales"] *= 2.0 ** shift
    q = torch.zeros((MANY, 1, rows, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = growth * math.log(2) * math.sqrt(D)
    out, lse = c.decode(ra, q, out_dtype=torch.float32)
    x = c.k @ q[0, 0, 0].double() / math.sqrt(D)
    each, sums = (growth + 1) * 2.0 ** -22 + 2.0 ** -21, 625 * 2.0 ** -24
    exact = torch.logsumexp(x, 0)
    assert (lse.double() - exact).abs().max() <= each + sums + 2.0 ** -23 * exact
    if shift == 0:
        want = torch.softmax(x, 0) @ c.v
        off = ((out.double() - want).abs() / c.v.max()).max().item()
        tol = 2.0 ** -15 + 2 * (each + sums) + 6 * 2.0 ** -23 + 2.0 ** -22
        assert off <= tol, f"off by {off:.3g}, {off / tol:.3g} tolerances"
    assert ra.ra_get_device_status() == ra.RA_OK


def cut(x, bits):
    """x (positive) cut off to its leading bits."""
    e = np.floor(np.log2(x)) - (bits - 1)
    return np.floor(x / 2.0 ** e) * 2.0 ** e


def nearest(x, bits):
    e = np.floor(np.log2(np.maximum(x, 1e-300))) - (bits - 1)
    return np.rint(x / 2.0 ** e) * 2.0 ** e


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 8, 12, 16, 32, 64])
@pytest.mark.parametrize("n,D", [(32, 64), (100, 128)])
def test_every_term_of_the_weights_is_there(cuda_lib, dtype, rows, n, D):
    """One key with weight 1 and value 0, the others with one weight w and value 1: out =
    (n - 1) w / (1 + (n - 1) w) shows w itself.  Each row's w is one that the leading bits
    alone (and, in bf16, two terms) hold as badly as they can; the bound lies below half of
    what either would be off.

    The bound: x = log2 w goes through three roundings (2^-24 of it), the exponential has
    2^-22, both scales' products 2^-24 each; they enter out and 1 + (n - 1) w alike, so out
    takes no more than their part.  Then the terms' own loss (2^-24, 2^-22 for f16), 6 products
    that may cut (2^-23), at most four parts and (100 / 32 + 7) sums in fp32, the
    division and the output: 20 roundings of 2^-24."""
    ra = cuda_lib
    big = 4.6 if n > 64 else 3.4  # (n - 1) w about 1
    grid = torch.arange(0.8 * big, 1.2 * big, 1 / 64).mul(math.sqrt(D)).to(torch.bfloat16).double().unique()
    a = grid.numpy() / math.sqrt(D)
    w = np.exp(-a)
    bits = 8 if dtype == "bf16" else 11
    one = cut(w, bits)
    two = one + nearest(w - one, 8)
    lost = np.abs(two - w) if dtype == "bf16" else np.abs(one - w)
    pick = np.sort(np.argsort(-lost / w)[:rows] if rows <= len(w) // 3 else np.argsort(-lost / w)[:len(w) // 3])
    pick = np.resize(pick, rows)
    k, v = torch.zeros((n, D)), torch.ones((n, D))
    k[1:, 0], k[:, 1] = -1.0, 1.0
    v[0] = 0.0
    v[0, 5] = 1.0
    c = Shared(ra, dtype, k, v, 2, ps=16)
    q = torch.zeros((2, 1, rows, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = grid[torch.tensor(pick)].to(torch.bfloat16).cuda()
    out, _ = c.decode(ra, q, out_dtype=torch.float32)
    out = out[:, 0].cpu().double().numpy()
    kk, vv = c.k.cpu().numpy(), c.v.cpu().numpy()
    assert np.array_equal(kk[1:, 0], -np.ones(n - 1)) and np.abs(vv[1:, 0] - 1).max() < 2.0 ** -23
    W = w[pick]
    want = (n - 1) * W / (1 + (n - 1) * W)
    tol = want * (np.log2(1 / W) * 3 * 2.0 ** -24 * math.log(2) + 2.0 ** -22 + 2 * 2.0 ** -24
                  + (2.0 ** -24 if dtype == "bf16" else 2.0 ** -22) + 6 * 2.0 ** -23 + 20 * 2.0 ** -24)
    off = np.abs(out[..., 0] - want)
    assert (off <= tol).all(), f"off by {(off / tol).max():.3g} tolerances"
    for terms in (one, two) if dtype == "bf16" else (one,):
        wrong = np.abs((n - 1) * terms[pick] / (1 + (n - 1) * W) - want)
        assert np.median(wrong / tol) > 2, "the bound does not tell"
    if dtype == "bf16":  # a bf16 output: its rounding, and two terms (2^-16)
        got = c.decode(ra, q, out_dtype=torch.bfloat16)[0][:, 0, :, 0].cpu().double().numpy()
        half = 2.0 ** -8 * want + tol + 2.0 ** -16 * want
        assert (np.abs(got - want) <= half).all()
    assert ra.ra_get_device_status() == ra.RA_OK
