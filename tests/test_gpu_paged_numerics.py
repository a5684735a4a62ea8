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
