"""ra_paged_decode_attention against the fp64 oracle.

Tolerances, from the arithmetic (per case, on the case's own values):
  scores   fp32 sums of D exact products of bf16 values, scaled: an error of at
           most dx = (D + 4) 2^-24 max_j s sum_d |q_d k_jd|;
  weights  2^dx ... and two bf16 terms (2^-17) for a bf16 output, three for fp32
           (2^-24), the exponential itself 2^-21;
  sums     n terms in fp32: n 2^-24;
so |out - exact| <= 2 (dx + w + 2^-21 + n 2^-24) max|v| + half a step of the
output type of |out|, and |lse - exact| <= dx + 2^-21 + n 2^-24 + 2^-23 |lse|."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as P

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Case:
    """A filled cache: the valid rows hold drawn tokens, every other row of the
    pages NaN (bf16) or random codes with NaN scales."""

    def __init__(self, dtype, B, Tq, Hq, Hkv, D, ps, seq, new=None, seed=0, extra=2):
        gen = torch.Generator().manual_seed(seed)
        self.seq, self.ps, self.dtype = seq, ps, dtype
        self.new = new if new is not None else [min(Tq, n) for n in seq]
        need = [-(-n // ps) for n in seq]
        n_pages = sum(need) + extra
        order = torch.randperm(n_pages, generator=gen).to(torch.int32)
        self.table = torch.full((B, max(max(need), 1)), -1, dtype=torch.int32)
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.ref = P.Cache(n_pages, Hkv, ps, D, dtype)
        T = max(max(seq), 1)
        gain = torch.exp(0.5 * torch.randn(D, generator=gen))
        k = (torch.randn((B, T, Hkv, D), generator=gen) * gain).to(torch.bfloat16)
        v = torch.randn((B, T, Hkv, D), generator=gen).to(torch.bfloat16)
        P.append(self.ref, f64(k), f64(v), self.table.tolist(), seq, seq)
        self.q = (1.5 * torch.randn((B, Tq, Hq, D), generator=gen)).to(torch.bfloat16)
        live = np.zeros((n_pages, ps), bool)
        for b, n in enumerate(seq):
            for p in range(n):
                live[int(self.table[b, p // ps]), p % ps] = True
        dead = torch.tensor(~live)[:, None, :].expand(n_pages, Hkv, ps)
        self.pages, self.scales = {}, {"k": None, "v": None}
        for w in "kv":
            if dtype == "bf16":
                x = torch.tensor(self.ref.value[w]).to(torch.bfloat16)
                x[dead] = float("nan")
                self.pages[w] = x.cuda()
            else:
                c = torch.tensor(self.ref.code[w])
                c[dead] = 0x7e
                s = torch.tensor(self.ref.scale[w]).float()
                s[dead] = float("nan")
                self.pages[w] = c.view(TORCH[dtype]).cuda()
                self.scales[w] = s.cuda()
        self.args = (self.q.cuda(), self.pages["k"], self.pages["v"], self.table.cuda(),
                     torch.tensor(seq, dtype=torch.int32).cuda())
        self.kw = dict(new_lens=None if new is None else torch.tensor(new, dtype=torch.int32).cuda(),
                       k_scales=self.scales["k"], v_scales=self.scales["v"])

    def expect(self, causal, selected=None):
        sel = None if selected is None else selected.cpu().tolist()
        return P.decode(f64(self.q), self.ref, self.table.tolist(), self.seq, self.new, causal, sel)

    def check(self, got, causal, selected=None, what=""):
        out, lse = got
        ro, rl = self.expect(causal, selected)
        D = self.q.shape[-1]
        q, k, v = np.abs(f64(self.q)), np.abs(self.ref.value["k"]), np.abs(self.ref.value["v"])
        dx = (D + 4) * 2.0 ** -24 * (q.reshape(-1, D).max(0) * k.reshape(-1, D).max(0)).sum() / math.sqrt(D)
        n = max(self.seq + [1]) * 2.0 ** -24
        w = 2.0 ** -17 if out.dtype == torch.bfloat16 else 2.0 ** -24
        half = torch.finfo(out.dtype).eps / 2
        tol = 2 * (dx + w + 2.0 ** -21 + n) * v.max() + half * np.abs(ro) * 1.01
        go, gl = f64(out), f64(lse)
        assert np.array_equal(np.isneginf(gl), np.isneginf(rl)), what
        assert np.isfinite(go).all(), what
        assert (np.abs(go - ro) <= tol).all(), f"{what}: out off by {np.max(np.abs(go - ro) / tol):.3g} tolerances"
        fin = np.isfinite(rl)
        off = np.abs(gl[fin] - rl[fin]) - (dx + 2.0 ** -21 + n + 2.0 ** -23 * np.abs(rl[fin]))
        assert (off <= 0).all(), f"{what}: lse off by {off.max():.3g} more than it may"
        assert (go[np.isneginf(rl)] == 0).all(), what


SHAPES = [
    # B, Tq, Hq, Hkv, D, ps, seq, new
    (1, 1, 1, 1, 64, 16, [1], None),
    (1, 1, 8, 2, 128, 16, [1000], None),
    (2, 1, 4, 4, 128, 32, [31, 33], None),
    (4, 1, 8, 1, 64, 64, [64, 0, 65, 200], None),
    (3, 4, 8, 2, 128, 16, [100, 3, 47], None),                 # fewer tokens than query rows
    (3, 4, 8, 2, 64, 128, [300, 128, 129], [2, 4, 1]),         # a padded batch
    (2, 5, 12, 3, 128, 32, [77, 160], [5, 0]),                 # 20 rows: two warps to a team; an idle sequence
    (1, 7, 14, 2, 64, 16, [333], None),                        # 49 rows: four warps
    (2, 1, 64, 1, 128, 64, [1500, 17], None),                  # 64 rows
    (2, 2, 32, 1, 128, 16, [700, 699], None),
    (5, 1, 7, 7, 128, 128, [1, 127, 128, 129, 640], None),
    (20, 1, 4, 2, 128, 16, [0, 0, 5, 900] + [33] * 15 + [0], None),
    (70, 2, 4, 4, 64, 32, [0] * 40 + [9, 2000] + [40] * 27 + [1], None),   # empty runs longer than a warp
]


@pytest.mark.parametrize("dtype", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in s[:6]))
@pytest.mark.parametrize("causal", [True, False])
def test_paged_decode(cuda_lib, dtype, shape, causal):
    ra = cuda_lib
    c = Case(dtype, *shape, seed=shape[0] + 7 * shape[1])
    for odt in (torch.bfloat16, torch.float32):
        got = ra.ra_paged_decode_attention(*c.args, causal=causal, out_dtype=odt, **c.kw)
        c.check(got, causal, what=str(odt))
        again = ra.ra_paged_decode_attention(*c.args, causal=causal, out_dtype=odt, **c.kw)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("D,ps,Hkv,G", [(128, 16, 2, 4), (64, 128, 1, 1), (128, 64, 3, 7)])
def test_many_cut_pairs(cuda_lib, dtype, D, ps, Hkv, G):
    """Long beside short: pairs cut over many teams, several pairs in one team's run."""
    ra = cuda_lib
    c = Case(dtype, 6, 1, Hkv * G, Hkv, D, ps, [9001, 40, 1, 0, 3333, 700], seed=4)
    got = ra.ra_paged_decode_attention(*c.args, out_dtype=torch.bfloat16, **c.kw)
    c.check(got, True)
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_selected_pages(cuda_lib, dtype, ps):
    ra = cuda_lib
    Hkv, n_sel = 2, 5
    c = Case(dtype, 4, 2, 8, Hkv, 128, ps, [ps * 20 + 3, ps * 3, 1, 0], seed=ps)
    gen = torch.Generator().manual_seed(ps)
    sel = torch.full((4, Hkv, n_sel), -1, dtype=torch.int32)
    for b, n in enumerate(c.seq):
        pages = -(-n // ps)
        for h in range(Hkv):
            m = min(n_sel, pages) - (1 if h and pages > 1 else 0)
            sel[b, h, :m] = torch.randperm(pages, generator=gen)[:m].sort().values.int()
    sel[0, 1] = torch.tensor([-1, 0, -1, 7, 20], dtype=torch.int32)  # no page, in the middle of a list
    for causal in (True, False):
        for odt in (torch.bfloat16, torch.float32):
            got = ra.ra_paged_decode_attention(*c.args, causal=causal, selected=sel.cuda(), out_dtype=odt, **c.kw)
            c.check(got, causal, sel)
    assert ra.ra_get_device_status() == ra.RA_OK
    none = torch.full_like(sel, -1).cuda()  # lists without a page: no row sees a key
    out, lse = ra.ra_paged_decode_attention(*c.args, selected=none, **c.kw)
    assert not out.any() and torch.isneginf(lse).all()
    assert ra.ra_get_device_status() == ra.RA_OK


def test_selected_lists_that_break_the_rule_are_recorded(cuda_lib):
    """An index out of range, the same one twice, a descending list: recorded, counted as no page."""
    ra = cuda_lib
    c = Case("bf16", 1, 1, 4, 1, 64, 16, [100], seed=2)
    for bad, same_as in (([0, 0, 3], [0, -1, 3]), ([5, 2, 6], [5, -1, 6]), ([1, 7, -1], [1, -1, -1]), ([-7, 2, 3], [-1, 2, 3])):
        sel = torch.tensor([[bad]], dtype=torch.int32)
        got = ra.ra_paged_decode_attention(*c.args, selected=sel.cuda(), **c.kw)
        assert ra.ra_get_device_status() == ra.RA_ERR_DEVICE_BOUNDS
        c.check(got, True, torch.tensor([[same_as]]))


def test_bad_table_and_lengths_are_recorded(cuda_lib):
    ra = cuda_lib
    c = Case("int8", 3, 2, 4, 2, 128, 16, [40, 70, 33], seed=3)
    good = ra.ra_paged_decode_attention(*c.args, **c.kw)
    assert ra.ra_get_device_status() == ra.RA_OK
    q, kp, vp, table, seq = c.args
    for value in (-1, kp.shape[0], 1 << 30):
        t = table.clone()
        t[1, 2] = value
        out, lse = ra.ra_paged_decode_attention(q, kp, vp, t, seq, **c.kw)
        assert ra.ra_get_device_status() == ra.RA_ERR_DEVICE_BOUNDS
        for b in (0, 2):  # the other sequences are as they were
            assert torch.equal(out[b], good[0][b]) and torch.equal(lse[b], good[1][b])
    for n in (-5, 10 ** 6):
        s = seq.clone()
        s[1] = n
        ra.ra_paged_decode_attention(q, kp, vp, table, s, **c.kw)
        assert ra.ra_get_device_status() == ra.RA_ERR_DEVICE_BOUNDS


def test_infinities_and_nan_of_tokens_behind_a_row(cuda_lib):
    """Causal rows of one call: a token's NaN key or infinite value reaches its own
    and later rows only."""
    ra = cuda_lib
    c = Case("bf16", 1, 4, 4, 2, 64, 16, [50], seed=6)
    where = int(c.table[0, 3]), 49 % 16  # the last token
    c.pages["v"][where[0], :, where[1]] = float("inf")
    c.pages["k"][where[0], 0, where[1]] = float("nan")
    out, lse = ra.ra_paged_decode_attention(*c.args, out_dtype=torch.float32, **c.kw)
    ro, rl = c.expect(True)
    assert np.allclose(f64(out)[:, :3], ro[:, :3], atol=1e-4) and np.allclose(f64(lse)[:, :3], rl[:, :3], atol=1e-4)
    assert torch.isnan(out[0, 3, :2]).all()                      # KV head 0: the key is NaN
    assert torch.isinf(out[0, 3, 2:]).all()                      # KV head 1: the value is infinite
    assert ra.ra_get_device_status() == ra.RA_OK


def test_a_nan_scale_is_a_nan_row(cuda_lib):
    ra = cuda_lib
    c = Case("int8", 1, 2, 2, 1, 128, 32, [90], seed=6)
    page = int(c.table[0, 2])
    c.scales["v"][page, 0, 89 % 32] = float("nan")  # the last token's value
    out, _ = ra.ra_paged_decode_attention(*c.args, out_dtype=torch.float32, **c.kw)
    assert torch.isfinite(out[0, 0]).all() and torch.isnan(out[0, 1]).all()


def test_scores_of_every_size(cuda_lib):
    """Scores in the thousands, both signs: the running maximum carries them."""
    ra = cuda_lib
    for sign in (1.0, -1.0):
        c = Case("bf16", 1, 1, 4, 2, 128, 16, [400], seed=9)
        c.q = (c.q.float() * 60 * sign).to(torch.bfloat16)
        c.args = (c.q.cuda(),) + c.args[1:]
        c.check(ra.ra_paged_decode_attention(*c.args, out_dtype=torch.float32, **c.kw), True)


@pytest.mark.parametrize("dtype", ["int8", "e4m3"])
@pytest.mark.parametrize("B,Tq,Hq,Hkv,D,ps,seq", [(2, 1, 4, 2, 128, 16, [20, 90]), (1, 3, 12, 2, 64, 64, [41]),
                                                  (3, 4, 32, 2, 128, 32, [70, 33, 7]), (1, 1, 8, 8, 64, 128, [130])])
def test_masked_codes_may_be_any_byte(cuda_lib, dtype, B, Tq, Hq, Hkv, D, ps, seq):
    """Memory never written holds every code, e4m3's without a value among them: the
    result is, bit for bit, that with other bytes there."""
    ra = cuda_lib
    c = Case(dtype, B, Tq, Hq, Hkv, D, ps, seq, seed=11)
    for causal in (True, False):
        want = ra.ra_paged_decode_attention(*c.args, causal=causal, out_dtype=torch.float32, **c.kw)
        c.check(want, causal)
        for byte in (0x7f, 0xff, 0x80):
            pages = {}
            for w in "kv":
                dead = torch.isnan(c.scales[w])[..., None]
                raw = c.pages[w].view(torch.uint8)
                pages[w] = torch.where(dead, torch.full_like(raw, byte), raw).view(TORCH[dtype])
            kept = {w: x.clone() for w, x in pages.items()}
            got = ra.ra_paged_decode_attention(c.args[0], pages["k"], pages["v"], *c.args[3:], causal=causal,
                                               out_dtype=torch.float32, **c.kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), hex(byte)
            for w in "kv":
                assert torch.equal(pages[w].view(torch.uint8), kept[w].view(torch.uint8))
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("Tq,Hq,D", [(1, 8, 128), (2, 8, 64), (7, 8, 128)])
@pytest.mark.parametrize("factor", [2.0 ** 40, 2.0 ** 100, float("inf"), float("nan"), 2.0 ** -60])
def test_rows_of_every_size_stand_side_by_side(cuda_lib, dtype, Tq, Hq, D, factor):
    """A row's result does not hang on the others of its KV head: rows 2^40 or 2^100
    larger, infinite ones, and rows so small that they weigh every key alike."""
    ra = cuda_lib
    c = Case(dtype, 2, Tq, Hq, 1, D, 32, [300, 77], seed=12)
    odd = torch.zeros((2, Tq, Hq), dtype=torch.bool)
    odd[:, :, 1::3] = True
    c.q[odd] = (c.q[odd].float() * factor).to(torch.bfloat16)
    got = ra.ra_paged_decode_attention(c.q.cuda(), *c.args[1:], out_dtype=torch.float32, **c.kw)
    shown = ~odd if not factor < 1 else torch.ones_like(odd)
    c.q[~shown] = 0.0  # the others' results are replaced by what a row of zeros has
    ro, rl = c.expect(True)
    out, lse = torch.tensor(ro, dtype=torch.float32), torch.tensor(rl, dtype=torch.float32)
    out[shown], lse[shown] = got[0].cpu()[shown], got[1].cpu()[shown]
    c.check((out, lse), True)
    rest = got[0].cpu()[~shown]
    if not math.isfinite(factor):
        assert torch.isnan(rest).all()
    assert ra.ra_get_device_status() == ra.RA_OK


def test_value_scales_of_every_size(cuda_lib):
    """Scales from subnormal ones to 2^100, and 0 beside others: the outputs are exact to a part of the
    largest value, and lse does not hang on them."""
    ra = cuda_lib
    for dtype in ("int8", "e4m3"):
        for exps in ((0,), (-97,), (100,), (-130,), (0, -40), (30, -30, 0)):
            c = Case(dtype, 1, 1, 8, 2, 128, 16, [200], seed=13)
            live = ~torch.isnan(c.scales["v"])
            n = live.shape[2]
            e = torch.tensor([exps[i % len(exps)] for i in range(n)], dtype=torch.float64)
            s = (c.scales["v"].cpu().double() * torch.exp2(e)).float()
            zero = [] if exps[0] < -80 else [5, 6]  # rows of zeros
            s[:, :, zero] = torch.where(live[:, :, zero].cpu(), torch.zeros_like(s[:, :, zero]), s[:, :, zero])
            c.scales["v"] = c.kw["v_scales"] = s.cuda()
            was = np.where(c.ref.scale["v"] > 0, c.ref.scale["v"], 1.0)
            c.ref.value["v"] = c.ref.value["v"] / was[..., None] * np.nan_to_num(f64(s))[..., None]
            codes = c.pages["v"].view(torch.uint8).cpu()
            codes[:, :, zero] = torch.where(live.cpu()[:, :, zero, None], torch.zeros_like(codes[:, :, zero]), codes[:, :, zero])
            c.args = c.args[:2] + (codes.view(TORCH[dtype]).cuda(),) + c.args[3:]
            got = ra.ra_paged_decode_attention(*c.args, out_dtype=torch.float32, **c.kw)
            if exps[0] == -130:  # below fp32's normal numbers: no result but 0 is asked for, and the lse
                assert (got[0].abs() < 2.0 ** -100).all()
                got = (torch.tensor(c.expect(True)[0], dtype=torch.float32), got[1])
            c.check(got, True, what=f"{dtype} {exps}")
    assert ra.ra_get_device_status() == ra.RA_OK


def test_offsets_past_32_bits(cuda_lib):
    """Pages whose byte and element offsets pass 2^32 and 2^31."""
    ra = cuda_lib
    D, Hkv, ps = 128, 2, 64
    for dtype, n_pages in (("bf16", 140000), ("int8", 140000)):  # 17.9M rows: 2.3G elements
        c = Case(dtype, 2, 1, 4, Hkv, D, ps, [200, 65], seed=1)
        small = c.pages["k"].shape[0]
        off = n_pages - small
        big, scales = {}, {"k": None, "v": None}
        for w in "kv":
            big[w] = torch.empty((n_pages, Hkv, ps, D), dtype=c.pages[w].dtype, device="cuda")
            big[w][off:] = c.pages[w]
            if dtype != "bf16":
                scales[w] = torch.empty((n_pages, Hkv, ps), device="cuda")
                scales[w][off:] = c.scales[w]
        table = torch.where(c.table >= 0, c.table + off, -1).int().cuda()
        lens = c.args[4]
        got = ra.ra_paged_decode_attention(c.args[0], big["k"], big["v"], table, lens, k_scales=scales["k"],
                                           v_scales=scales["v"], out_dtype=torch.bfloat16)
        c.check(got, True)
        gk, gv = ra.ra_cache_read(big["k"], big["v"], table, lens, 200, k_scales=scales["k"], v_scales=scales["v"],
                                  out_dtype=torch.float32)
        rk, rv = ra.ra_cache_read(c.pages["k"], c.pages["v"], c.table.cuda(), lens, 200, k_scales=c.scales["k"],
                                  v_scales=c.scales["v"], out_dtype=torch.float32)
        assert torch.equal(gk, rk) and torch.equal(gv, rv)
        new = torch.ones((2, 1, Hkv, D), dtype=torch.bfloat16, device="cuda")
        ra.ra_cache_append(new, new, big["k"], big["v"], table, lens, k_scales=scales["k"], v_scales=scales["v"])
        gk, _ = ra.ra_cache_read(big["k"], big["v"], table, lens, 200, k_scales=scales["k"], v_scales=scales["v"],
                                 out_dtype=torch.float32)
        assert torch.equal(gk[0, :199], rk[0, :199]) and torch.allclose(gk[0, 199], torch.ones(()).cuda())
        assert torch.allclose(gk[1, 64], torch.ones(()).cuda())
        assert ra.ra_get_device_status() == ra.RA_OK
        del big, scales, gk, gv, rk, rv
        torch.cuda.empty_cache()


def test_graph_stream_and_workspace(cuda_lib):
    """Two captured calls that share a workspace, replayed in turn with other
    lengths; a call on another stream; a workspace full of NaN."""
    ra = cuda_lib
    a = Case("bf16", 3, 1, 8, 2, 128, 16, [600, 100, 900], seed=1)
    b = Case("e4m3", 2, 3, 8, 1, 64, 32, [300, 1000], seed=2)
    need = max(ra.ra_paged_decode_workspace(3, 1, 8, 2, 128), ra.ra_paged_decode_workspace(2, 3, 8, 1, 64))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got, graphs = [], []
    for c in (a, b):
        ra.ra_paged_decode_attention(*c.args, workspace=ws, **c.kw)
    torch.cuda.synchronize()
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(ra.ra_paged_decode_attention(*c.args, workspace=ws, out_dtype=torch.bfloat16, **c.kw))
        graphs.append(g)
    for lens in ([600, 100, 900], [1, 0, 512], [599, 64, 33]):
        a.seq, a.new = lens, [min(1, n) for n in lens]
        a.args[4].copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(255)
        for g in graphs:
            g.replay()
        a.check(got[0], True)
        b.check(got[1], True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    res = ra.ra_paged_decode_attention(*b.args, stream=side, out_dtype=torch.bfloat16, **b.kw)
    side.synchronize()
    b.check(res, True)
    assert ra.ra_get_device_status() == ra.RA_OK


def test_a_large_batch_with_idle_sequences(cuda_lib):
    """More sequences than the walker's warp, several chunks of empty and idle ones between."""
    ra = cuda_lib
    seq = [(7 * b) % 53 if b % 3 else 0 for b in range(300)]
    new = [min(1, n) if b % 5 else 0 for b, n in enumerate(seq)]
    seq[137], new[137], seq[299], new[299] = 2500, 1, 41, 1
    c = Case("int8", 300, 1, 4, 2, 64, 16, seq, new, seed=5)
    got = ra.ra_paged_decode_attention(*c.args, out_dtype=torch.bfloat16, **c.kw)
    c.check(got, True)
    assert ra.ra_get_device_status() == ra.RA_OK


def test_a_table_much_wider_than_the_sequences(cuda_lib):
    ra = cuda_lib
    c = Case("e4m3", 2, 1, 8, 2, 128, 16, [100, 33], seed=5)
    wide = torch.full((2, 70000), -1, dtype=torch.int32)
    wide[:, :c.table.shape[1]] = c.table
    q, kp, vp, _, lens = c.args
    c.check(ra.ra_paged_decode_attention(q, kp, vp, wide.cuda(), lens, out_dtype=torch.bfloat16, **c.kw), True)
    k, _ = ra.ra_cache_read(kp, vp, wide.cuda(), lens, 40, first=80, k_scales=c.scales["k"], v_scales=c.scales["v"])
    assert not k[0, 20:].any() and not k[1].any() and k[0, :20].any()
    assert ra.ra_get_device_status() == ra.RA_OK


def test_two_streams_at_once(cuda_lib):
    """Calls that overlap, each with a workspace of its own."""
    ra = cuda_lib
    cases = [Case("bf16", 3, 1, 8, 2, 128, 16, [3000, 1000, 2500], seed=1),
             Case("int8", 3, 4, 8, 2, 128, 16, [2000, 2200, 300], seed=2)]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [torch.empty(ra.ra_paged_decode_workspace(3, c.q.shape[1], 8, 2, 128), dtype=torch.uint8, device="cuda") for c in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, st, w in zip(cases, streams, ws):
            with torch.cuda.stream(st):
                got.append(ra.ra_paged_decode_attention(*c.args, workspace=w, out_dtype=torch.bfloat16, **c.kw))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        cases[i % 2].check(g, True)
    assert ra.ra_get_device_status() == ra.RA_OK


def test_the_binding_refuses(cuda_lib):
    """Tensors of another type, shape, layout or device; outputs that do not fit; things that are no tensors."""
    ra = cuda_lib
    c = Case("int8", 2, 1, 4, 2, 64, 16, [40, 20], seed=1)
    q, kp, vp, table, lens = c.args
    ks, vs = c.scales["k"], c.scales["v"]

    def call(**kw):
        a = dict(q=q, k_pages=kp, v_pages=vp, page_table=table, seq_lens=lens, k_scales=ks, v_scales=vs)
        a.update(kw)
        return ra.ra_paged_decode_attention(**a)

    call()
    for bad in (dict(seq_lens=lens.long()), dict(seq_lens=lens.cpu()), dict(seq_lens=lens[:1]), dict(page_table=table.t()),
                dict(page_table=table[:, ::2]), dict(page_table=table[0]), dict(new_lens=lens.float()),
                dict(v_pages=vp.view(torch.uint8)), dict(v_pages=vp[:1]), dict(k_pages=kp[0]), dict(k_pages=kp.cpu()),
                dict(k_scales=None), dict(v_scales=None), dict(k_scales=ks[:, :1]), dict(k_scales=ks.half()),
                dict(q=q[0]), dict(q=q.transpose(2, 3)), dict(q=q[..., ::2]), dict(q=q.half()), dict(q=q.cpu()),
                dict(out=torch.empty(3, device="cuda")), dict(out=q.half()), dict(lse=torch.empty_like(q)),
                dict(out_dtype=torch.float16), dict(out_dtype="bf16"), dict(workspace=torch.empty(8)),
                dict(selected=lens), dict(selected=torch.zeros((2, 2, 2), device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q=3), dict(k_pages=None), dict(page_table=[1]), dict(selected="x"), dict(workspace=7)):
        with pytest.raises(TypeError):
            call(**bad)
    for bad, status in ((dict(q=q.float()), ra.RA_ERR_UNSUPPORTED), (dict(q=q[:, :, :3].contiguous()), ra.RA_ERR_INVALID_ARG),
                        (dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), ra.RA_ERR_WORKSPACE),
                        (dict(selected=torch.zeros((2, 2, 0), dtype=torch.int32, device="cuda")), ra.RA_ERR_INVALID_ARG)):
        with pytest.raises(ra.RAError) as e:
            call(**bad)
        assert e.value.status == status
    with pytest.raises(ra.RAError):
        ra.ra_cache_read(kp, vp, table, lens, 0, k_scales=ks, v_scales=vs)
    with pytest.raises(ValueError):
        ra.ra_cache_read(kp, vp, table, lens, 1 << 40, k_scales=ks, v_scales=vs)
    with pytest.raises(ValueError):
        ra.ra_cache_append(q, q, kp, vp, table, lens, k_scales=ks, v_scales=vs)  # four heads for two
    assert ra.ra_get_device_status() == ra.RA_OK


def test_given_outputs_and_streams(cuda_lib):
    """Outputs are written where they are given; on a given stream (object or handle)
    the workspace belongs to that stream, so calls one after another do not share it
    with the current stream's work."""
    ra = cuda_lib
    c = Case("bf16", 2, 2, 8, 2, 128, 32, [400, 900], seed=1)
    want = ra.ra_paged_decode_attention(*c.args, out_dtype=torch.bfloat16, **c.kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        out = torch.empty_like(want[0])
        lse = torch.empty_like(want[1])
        torch.cuda.synchronize()
        got = []
        for _ in range(20):
            got.append(ra.ra_paged_decode_attention(*c.args, stream=stream, out_dtype=torch.bfloat16, **c.kw))
            torch.empty(16 << 20, dtype=torch.uint8, device="cuda").fill_(255)  # the current stream's allocations
        r = ra.ra_paged_decode_attention(*c.args, stream=stream, out=out, lse=lse, **c.kw)
        assert r[0].data_ptr() == out.data_ptr() and r[1].data_ptr() == lse.data_ptr()
        torch.cuda.synchronize()
        for g in got + [(out, lse)]:
            assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def test_a_serving_run(cuda_lib):
    """Prompt, appended in chunks; then decoded token by token: the paged calls
    against the dense decode over the same (bf16) cache, and ra_ring_attention over
    the prefix read back."""
    ra = cuda_lib
    gen = torch.Generator().manual_seed(12)
    B, Hq, Hkv, D, ps, S, steps = 2, 8, 2, 128, 16, 96, 5
    k, v = (torch.randn((B, S + steps, Hkv, D), generator=gen).to(torch.bfloat16).cuda() for _ in "kv")
    q = torch.randn((B, S + steps, Hq, D), generator=gen).to(torch.bfloat16).cuda()
    n_pages = 2 * (-(-(S + steps) // ps))
    table = torch.randperm(n_pages, generator=gen).to(torch.int32).view(B, -1).contiguous().cuda()
    kp = torch.full((n_pages, Hkv, ps, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for s0, s1 in ((0, 41), (41, 43), (43, S)):
        lens.fill_(s1)
        ra.ra_cache_append(k[:, s0:s1].contiguous(), v[:, s0:s1].contiguous(), kp, vp, table, lens)
    rk, rv = ra.ra_cache_read(kp, vp, table, lens, S)
    assert torch.equal(rk, k[:, :S]) and torch.equal(rv, v[:, :S])
    full, _ = ra.ra_ring_attention(q[:, :S].contiguous(), rk, rv, 4, True)
    last, _ = ra.ra_paged_decode_attention(q[:, S - 1:S].contiguous(), kp, vp, table, lens)
    assert torch.allclose(full[:, S - 1:], last, atol=2e-2)
    for t in range(S, S + steps):
        lens.fill_(t + 1)
        one = slice(t, t + 1)
        ra.ra_cache_append(k[:, one].contiguous(), v[:, one].contiguous(), kp, vp, table, lens)
        got = ra.ra_paged_decode_attention(q[:, one].contiguous(), kp, vp, table, lens)
        want = ra.ra_decode_attention(q[:, one].contiguous(), k[:, :t + 1].contiguous(), v[:, :t + 1].contiguous())
        assert torch.allclose(got[0], want[0], atol=2e-2) and torch.allclose(got[1], want[1], atol=1e-4)
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", ["int8", "e4m3"])
def test_zero_values_of_a_long_cache(cuda_lib, dtype):
    """Every value 0 and scores that grow along the cache: outputs 0, lse that of the keys."""
    ra = cuda_lib
    n, D, ps = 300000, 64, 128
    pages = -(-n // ps)
    gen = torch.Generator().manual_seed(3)
    k = torch.randn((pages, 1, ps, D), generator=gen)
    k[..., 0] += torch.arange(pages * ps).view(pages, 1, ps) / n * 8
    q = torch.zeros((1, 1, 1, D))
    q[..., 0] = 30.0
    kp, ks = torch.zeros((pages, 1, ps, D), dtype=TORCH[dtype]).cuda(), torch.zeros((pages, 1, ps)).cuda()
    vp, vs = torch.zeros_like(kp), torch.zeros_like(ks)
    table = torch.arange(pages, dtype=torch.int32)[None].cuda()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    rows = k.permute(1, 0, 2, 3).reshape(1, pages * ps, 1, D)[:, :n].to(torch.bfloat16).cuda()
    ra.ra_cache_append(rows, torch.zeros_like(rows), kp, vp, table, lens, k_scales=ks, v_scales=vs)
    out, lse = ra.ra_paged_decode_attention(q.to(torch.bfloat16).cuda(), kp, vp, table, lens, k_scales=ks, v_scales=vs)
    assert not out.any() and not vs.any()
    back, _ = ra.ra_cache_read(kp, vp, table, lens, n, k_scales=ks, v_scales=vs, out_dtype=torch.float32)
    x = back[0, :, 0, 0].double() * 30.0 / math.sqrt(D)
    want = float(torch.logsumexp(x, 0))
    # scores to (D + 4) 2^-24 of their largest, a sum of n terms, the exponentials
    tol = (D + 4) * 2.0 ** -24 * float(x.abs().max()) + n * 2.0 ** -24 + 2.0 ** -20 * want
    assert abs(float(lse) - want) <= tol
    assert ra.ra_get_device_status() == ra.RA_OK


def test_calls_behind_copies_and_other_streams(cuda_lib):
    """A step whose lengths and rows come by copies, a fill and another stream's kernel
    right before it, eager and captured: the calls see what precedes them."""
    ra = cuda_lib
    B, Hkv, Hq, D, ps, width = 4, 2, 8, 128, 16, 40
    gen = torch.Generator().manual_seed(21)
    table = torch.randperm(B * width, generator=gen).view(B, width).int().cuda()
    kp, vp = (torch.zeros((B * width, Hkv, ps, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    q = torch.randn((B, 1, Hq, D), generator=gen).to(torch.bfloat16).cuda()
    lens, out, lse = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty((B, 1, Hq), device="cuda")
    k, v = (torch.empty((B, 1, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    ws = torch.empty(ra.ra_paged_decode_workspace(B, 1, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    host_len = torch.zeros(B, dtype=torch.int32).pin_memory()
    src = torch.empty((2, B, 1, Hkv, D), dtype=torch.bfloat16, device="cuda")

    def step():
        lens.copy_(host_len, non_blocking=True)   # a copy from the host
        k.copy_(src[0])                           # a copy on the device
        out.zero_()
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.mul(src[1], 1.0, out=v)         # a kernel of another stream
        here.wait_stream(side)
        ra.ra_cache_append(k, v, kp, vp, table, lens)
        ra.ra_paged_decode_attention(q, kp, vp, table, lens, out=out, lse=lse, workspace=ws)

    def run(go):
        kp.zero_()
        vp.zero_()
        gen.manual_seed(22)
        got = []
        for i in range(1, 60):
            torch.cuda.synchronize()
            host_len.copy_(torch.tensor([i, 2 * i, 3 * i, 7 * i if 7 * i <= width * ps else width * ps]).int())
            src.copy_(torch.randn(src.shape, generator=gen).to(torch.bfloat16))
            go()
            got.append((out.clone(), lse.clone()))
        torch.cuda.synchronize()
        return got

    want = run(lambda: (torch.cuda.synchronize(), step(), torch.cuda.synchronize()))
    eager = run(step)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    replayed = run(graph.replay)
    for got in (eager, replayed):
        for (a, b), (c, d) in zip(got, want):
            assert torch.equal(a, c) and torch.equal(b, d)
    # the last step against the formula
    rk, rv = ra.ra_cache_read(kp, vp, table, lens, int(lens.max()), out_dtype=torch.float32)
    n = int(lens[3])
    x = torch.einsum("hd,td->ht", q[3, 0, :4].double(), rk[3, :n, 0].double()) / math.sqrt(D)
    assert torch.allclose(torch.logsumexp(x, 1), lse[3, 0, :4].double(), atol=1e-4)
    assert ra.ra_get_device_status() == ra.RA_OK
