"""The paged key-value cache on the CPU: the oracle's own pins and the library's
refusals, which come back before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import attention as F
from oracle import paged as P


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import blockwise_exact_attention_block_b200 as mod
    return mod


FAKE = 1 << 20  # an aligned, non-null address; never dereferenced on these paths


def cache(ra, **kw):
    args = dict(k_pages=FAKE, v_pages=FAKE, k_scales=None, v_scales=None, key_bounds=None, dtype=ra.RA_BF16,
                n_pages=100, page_size=16, Hkv=2, D=128, page_table=FAKE, B=3, max_pages=10, seq_lens=FAKE,
                new_lens=None)
    args.update(kw)
    return ra.ra_paged_cache(*(args[n] for n, _ in ra.ra_paged_cache._fields_))


BAD_CACHE = [
    (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(k_pages=FAKE + 8), 1), (dict(v_pages=FAKE + 2), 1),
    (dict(k_scales=FAKE), 1),                                  # scales of a bf16 cache
    (dict(dtype=2), 1),                                        # an int8 cache without scales
    (dict(dtype=3, k_scales=FAKE), 1),
    (dict(dtype=2, k_scales=FAKE, v_scales=FAKE + 4), 1),      # misaligned scales
    (dict(dtype=0), 2), (dict(dtype=9), 1),
    (dict(key_bounds=FAKE + 4), 1),
    (dict(n_pages=0), 1), (dict(B=0), 1), (dict(max_pages=0), 1), (dict(Hkv=0), 1),
    (dict(page_size=48), 2), (dict(page_size=8), 2), (dict(page_size=256), 2), (dict(D=96), 2),
    (dict(n_pages=1 << 26, page_size=16), 2),                  # rows past 2^31
    (dict(max_pages=1 << 27), 2),                              # positions past 2^31
    (dict(page_table=None), 1), (dict(seq_lens=None), 1), (dict(page_table=FAKE + 2), 1), (dict(seq_lens=FAKE + 1), 1),
    (dict(new_lens=FAKE + 2), 1),
]


def append(ra, c, k=FAKE, v=FAKE, dtype=1, T=1):
    return ra._lib.ra_cache_append(ctypes.byref(c), k, v, dtype, T, None)


def read(ra, c, first=0, T=1, k=FAKE, v=FAKE, dtype=1):
    return ra._lib.ra_cache_read(ctypes.byref(c), first, T, k, v, dtype, None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_append_and_read_refuse_a_bad_cache(ra, kw, status):
    assert append(ra, cache(ra, **kw)) == status
    assert read(ra, cache(ra, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 8), 1), (dict(T=0), 1), (dict(T=-3), 1), (dict(dtype=0), 2),
    (dict(dtype=2), 1)])
def test_append_refuses(ra, kw, status):
    assert append(ra, cache(ra), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(first=-1), 1), (dict(T=0), 1), (dict(k=FAKE + 4), 1), (dict(v=FAKE + 8), 1), (dict(dtype=2), 1),
    (dict(dtype=3), 1), (dict(k=None, v=None), 0)])
def test_read_refuses(ra, kw, status):
    assert read(ra, cache(ra), **kw) == status


def test_null_cache(ra):
    assert ra._lib.ra_cache_append(None, FAKE, FAKE, 1, 1, None) == 1
    assert ra._lib.ra_cache_read(None, 0, 1, FAKE, FAKE, 1, None) == 1


def test_binding_refuses_tensors_on_the_host(ra):
    k = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ra.ra_cache_append(k[:1, 0, :1][None], k[:1, 0, :1][None], k, k, table, lens)
    with pytest.raises(ValueError):
        ra.ra_cache_read(k, k, table, lens, 4)


def decode(ra, c, q=FAKE, in_dtype=1, Tq=1, Hq=8, causal=1, selected=None, n_sel=0, out=FAKE, out_dtype=1, lse=FAKE,
           ws=FAKE, ws_bytes=1 << 40):
    return ra._lib.ra_paged_decode_attention(q, in_dtype, ctypes.byref(c), Tq, Hq, causal, selected, n_sel, out,
                                             out_dtype, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_paged_decode_refuses_a_bad_cache(ra, kw, status):
    assert decode(ra, cache(ra, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(out=None), 1), (dict(out=FAKE + 4), 1), (dict(lse=None), 1),
    (dict(lse=FAKE + 2), 1), (dict(in_dtype=0), 2), (dict(in_dtype=2), 1), (dict(out_dtype=2), 1), (dict(Tq=0), 1),
    (dict(Hq=7), 1), (dict(Hq=0), 1),
    (dict(Hq=66, Tq=2), 2),                                       # 33 heads x 2 tokens > 64 rows per KV head
    (dict(Hq=2, Tq=65), 2),
    (dict(Hq=2, Tq=1 << 30), 2),
    (dict(selected=FAKE, n_sel=0), 1), (dict(selected=FAKE, n_sel=-1), 1), (dict(selected=FAKE + 2, n_sel=4), 1),
    (dict(n_sel=4), 1),                                           # a count without a list
    (dict(ws=None), 3), (dict(ws_bytes=64), 3), (dict(ws=FAKE + 64), 1)])
def test_paged_decode_refuses(ra, kw, status):
    assert decode(ra, cache(ra), **kw) == status


def test_paged_decode_refuses_a_line_past_32_bits(ra):
    """Tiles of all (sequence, KV head) pairs by the table's width: a team's share of them is a 32-bit count."""
    wide = dict(page_size=128, n_pages=1000, max_pages=1 << 23)  # 2^25 tiles each
    assert decode(ra, cache(ra, B=1 << 14, Hkv=2, **wide)) == 2
    assert decode(ra, cache(ra, B=1 << 20, Hkv=8, page_size=64, max_pages=1 << 24)) == 2


def test_paged_decode_workspace(ra):
    # teams of a full grid: 8 warps an SM at least, 1, 2 or 4 to a team; two cut pairs each
    for Tq, Hq, Hkv, per in ((1, 8, 2, 8), (4, 32, 8, 8), (5, 4, 1, 4), (1, 64, 1, 2)):
        rows = Hq // Hkv * Tq
        n = ra.ra_paged_decode_workspace(3, Tq, Hq, Hkv, 128)
        assert n >= 148 * per * 2 * rows * (128 + 2) * 4 + 3 * Hkv * 8
    for bad in ((0, 1, 8, 2, 128), (1, 1, 8, 3, 128), (1, 1, 8, 2, 96), (1, 65, 8, 8, 128)):
        with pytest.raises(ra.RAError):
            ra.ra_paged_decode_workspace(*bad)


def select(ra, c, q=FAKE, in_dtype=1, Tq=1, Hq=8, n_sel=4, selected=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return ra._lib.ra_page_select(q, in_dtype, ctypes.byref(c), Tq, Hq, n_sel, selected, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(in_dtype=0), 2), (dict(in_dtype=3), 1), (dict(Tq=0), 1),
    (dict(Hq=7), 1), (dict(Hq=2, Tq=65), 2), (dict(n_sel=0), 1), (dict(n_sel=-1), 1),
    (dict(Tq=2, n_sel=1), 1), (dict(Tq=18, Hq=2, n_sel=2), 1),    # fewer than the new tokens' own pages
    (dict(selected=None), 1), (dict(selected=FAKE + 2), 1), (dict(ws=None), 3), (dict(ws_bytes=3 * 2 * 10 * 8 - 1), 3),
    (dict(ws=FAKE + 8), 1)])
def test_page_select_refuses(ra, kw, status):
    assert select(ra, cache(ra, key_bounds=FAKE), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(key_bounds=None), 1), (dict(key_bounds=FAKE + 8), 1), (dict(B=65536), 2), (dict(Hkv=65536), 2),
    (dict(page_size=24), 2), (dict(D=80), 2), (dict(page_table=None), 1), (dict(seq_lens=FAKE + 2), 1),
    (dict(n_pages=0), 1)])
def test_page_select_refuses_a_bad_cache(ra, kw, status):
    c = dict(dict(key_bounds=FAKE), **kw)
    assert select(ra, cache(ra, **c), Hq=8 if kw.get("Hkv", 2) == 2 else 65536) == status


def test_page_select_workspace(ra):
    assert ra.ra_page_select_workspace(3, 2, 10) >= 3 * 2 * 10 * 8
    with pytest.raises(ra.RAError):
        ra.ra_page_select_workspace(1, 0, 10)


# ------------------------------------------------------------- oracle pins

def test_e4m3_grid_is_the_types():
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.e4m3_values(), grid)


def test_quantise_worked_rows():
    x = np.array([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 3.0, -127.0])
    code, val, s = P.quantise(x, "int8")
    assert s == 1.0
    assert val.tolist() == [127, 0, 2, 2, 0, -2, 3, -127]
    assert code.tolist() == [127, 0, 2, 2, 0, 254, 3, 129]
    # e4m3 with scale 1: 17 lies between 16 and 18 (even code: 16), 19 between 18 and 20 (20)
    x = np.array([448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, 400.0])
    code, val, s = P.quantise(x, "e4m3")
    assert s == 1.0
    assert val.tolist() == [448, 16, 20, -16, 0, 2 * 2.0 ** -9, 0, 384]
    for bad in (np.nan, np.inf):
        c, v, s = P.quantise(np.array([1.0, bad]), "int8")
        assert np.isnan(s) and not c.any() and np.isnan(v).all()
    c, v, s = P.quantise(np.array([2.0 ** -101, 0.0]), "e4m3")
    assert s == 0 and not c.any() and not v.any()


def random_cache(rng, ps, seqs, Hkv, D, dtype="bf16"):
    need = [-(-n // ps) for n in seqs]
    order = rng.permutation(sum(need) + 2)
    table, at = [], 0
    for c in need:
        table.append(order[at:at + c].tolist())
        at += c
    ca = P.Cache(sum(need) + 2, Hkv, ps, D, dtype)
    T = max(seqs)
    k, v = (torch.tensor(rng.standard_normal((len(seqs), T, Hkv, D))).to(torch.bfloat16).double().numpy() for _ in "kv")
    P.append(ca, k, v, table, seqs, seqs)
    return ca, table, k, v


def test_oracle_decode_is_the_dense_one():
    rng = np.random.default_rng(0)
    seqs, Hkv, G, D, Tq = [37, 16, 5], 2, 2, 64, 3
    ca, table, k, v = random_cache(rng, 16, seqs, Hkv, D)
    q = rng.standard_normal((3, Tq, Hkv * G, D))
    for causal in (True, False):
        out, lse = P.decode(q, ca, table, seqs, [Tq] * 3, causal)
        allpages = [[list(range(-(-n // 16)))] * Hkv for n in seqs]
        o2, l2 = P.decode(q, ca, table, seqs, [Tq] * 3, causal, allpages)
        assert np.array_equal(out, o2) and np.array_equal(lse, l2)
        for b, n in enumerate(seqs):
            ro, rl = F.decode_attention(q[b:b + 1], k[b:b + 1, :n], v[b:b + 1, :n], causal, G)
            assert np.allclose(out[b], ro[0], atol=1e-12) and np.allclose(lse[b], rl[0], atol=1e-12)
            assert np.array_equal(P.read(ca, table, seqs, 0, n)[b], k[b, :n])


def test_oracle_bounds_bound_and_select_keeps_the_best():
    rng = np.random.default_rng(1)
    seqs, Hkv, G, D, ps = [130, 16], 2, 2, 64, 16
    ca, table, k, _ = random_cache(rng, ps, seqs, Hkv, D)
    q = rng.standard_normal((2, 1, Hkv * G, D))
    sel = P.select(q, ca.bounds, ps, table, seqs, [1, 1], 4)
    for b, n in enumerate(seqs):
        for g in range(Hkv):
            rows = q[b, 0, g * G:(g + 1) * G]
            bound = [max(np.maximum(r * ca.bounds[t, g, 0], r * ca.bounds[t, g, 1]).sum() for r in rows)
                     for t in table[b]]
            for p, top in enumerate(bound):  # no key of the page scores above its bound
                assert (k[b, p * ps:min(n, (p + 1) * ps), g] @ rows.T).max() <= top + 1e-12
            got = [p for p in sel[b, g] if p >= 0]
            last = (n - 1) // ps
            want = sorted(range(len(bound)), key=lambda p: (p != last, -bound[p]))[:4]
            assert got == sorted(want)
    assert sel[1].tolist() == [[0, -1, -1, -1]] * Hkv
