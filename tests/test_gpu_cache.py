"""ra_cache_append and ra_cache_read against the fp64 oracle of the paged cache.

Codes, scales and bounds are compared bit for bit: the scale is one correctly
rounded division, a code is the exact quotient rounded once, bounds are minima
and maxima of bf16 values.  Values read back are one fp32 product of the code
and the scale (compared bit for bit with the product that the host rounds), and
one more rounding for bf16."""
import numpy as np
import pytest
import torch

from oracle import paged as P

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def codes(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def tables(seq_lens, page_size, extra, gen):
    """A page table with its pages in random places and -1 behind each sequence."""
    need = [-(-n // page_size) for n in seq_lens]
    order = torch.randperm(sum(need) + extra, generator=gen).to(torch.int32)
    table = torch.full((len(seq_lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    return table, sum(need) + extra


class Device:
    """A cache on the GPU filled with a pattern, beside the oracle's."""

    def __init__(self, n_pages, Hkv, ps, D, dtype, bounds=True):
        shape = (n_pages, Hkv, ps, D)
        self.dtype = dtype
        self.k = torch.full(shape, 3, dtype=torch.float32).to(TORCH[dtype]).cuda()
        self.v = self.k.clone()
        self.ks = self.vs = None
        if dtype != "bf16":
            self.ks = torch.full(shape[:3], 7.0, device="cuda")
            self.vs = self.ks.clone()
        self.bounds = torch.full((n_pages, Hkv, 2, D), 5.0, dtype=torch.bfloat16, device="cuda") if bounds else None
        self.ref = P.Cache(n_pages, Hkv, ps, D, dtype)
        for w, t in (("k", self.k), ("v", self.v)):
            self.ref.value[w][:] = f64(t.float()) * (1.0 if dtype == "bf16" else 7.0)
            if dtype != "bf16":
                self.ref.code[w][:] = codes(t)
                self.ref.scale[w][:] = 7.0
        self.ref.bounds[:] = 5.0

    def kw(self):
        return dict(k_scales=self.ks, v_scales=self.vs)

    def check(self):
        for w, t, s in (("k", self.k, self.ks), ("v", self.v, self.vs)):
            if self.dtype == "bf16":
                assert np.array_equal(f64(t), self.ref.value[w], equal_nan=True), w
            else:
                got, want = codes(t), self.ref.code[w]
                if self.dtype == "e4m3":  # the sign of a zero is of no account
                    got, want = np.where(got == 128, 0, got), np.where(want == 128, 0, want)
                assert np.array_equal(got, want), f"{w}: {np.sum(got != want)} codes differ"
                assert np.array_equal(f64(s), self.ref.scale[w], equal_nan=True), w
        if self.bounds is not None:
            assert np.array_equal(f64(self.bounds), self.ref.bounds)


def draw(gen, *shape):
    return (torch.randn(shape, generator=gen) * torch.exp(torch.randn(shape[-1], generator=gen))).to(torch.bfloat16)


@pytest.mark.parametrize("dtype", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("B,T,Hkv,D,ps,seq,new", [
    (1, 1, 1, 64, 16, [1], [1]),                       # one token into an empty cache
    (1, 1, 3, 128, 16, [17], [1]),                     # the first row of a page
    (3, 1, 2, 128, 32, [1, 33, 64], None),             # decode step
    (4, 5, 2, 64, 16, [5, 20, 0, 37], [5, 3, 0, 1]),   # padded batch, an empty slot
    (2, 40, 8, 128, 16, [57, 40], [40, 39]),           # several pages, begun inside one
    (2, 300, 2, 64, 128, [411, 300], [300, 257]),      # eight warps to a unit
    (1, 129, 5, 128, 128, [130], [129]),
    (2, 70, 1, 128, 64, [3, 70], [2, 70]),
    (2, 9, 1, 64, 64, [4, 2], None),                   # fewer tokens than rows
])
def test_append(cuda_lib, dtype, B, T, Hkv, D, ps, seq, new):
    ra = cuda_lib
    gen = torch.Generator().manual_seed(hash((B, T, Hkv, D, ps)) & 0xffff)
    table, n_pages = tables(seq, ps, 3, gen)
    dev = Device(n_pages, Hkv, ps, D, dtype)
    k, v = draw(gen, B, T, Hkv, D), draw(gen, B, T, Hkv, D)
    news = new if new is not None else [min(T, n) for n in seq]
    args = (k.cuda(), v.cuda(), dev.k, dev.v, table.cuda(), torch.tensor(seq, dtype=torch.int32).cuda())
    nl = None if new is None else torch.tensor(new, dtype=torch.int32).cuda()
    ra.ra_cache_append(*args, new_lens=nl, key_bounds=dev.bounds, **dev.kw())
    P.append(dev.ref, f64(k), f64(v), table.tolist(), seq, news)
    dev.check()
    # the same step once more leaves the cache as it is (bounds only widen)
    ra.ra_cache_append(*args, new_lens=nl, key_bounds=dev.bounds, **dev.kw())
    dev.check()
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_rounds_as_exact_arithmetic(cuda_lib, dtype, D):
    """Ties, borders, ends of the range, zeros, tiny and huge rows, NaN and infinity."""
    ra = cuda_lib
    gen = torch.Generator().manual_seed(3)
    qmax = P.QMAX[dtype]
    rows = []
    grid = P.e4m3_values() if dtype == "e4m3" else np.arange(128.0)
    mids = (grid[1:] + grid[:-1]) / 2
    mids = torch.tensor(mids).to(torch.bfloat16)
    for e in (0, -20, 60, 3):  # scale 2^e: quotients on the borders themselves
        for s in (1.0, -1.0):
            for c in range(0, len(mids), D - 1):
                r = torch.zeros(D, dtype=torch.bfloat16)
                part = mids[c:c + D - 1]
                r[1:1 + len(part)] = part * s
                r[0] = qmax
                rows.append((r.double() * 2.0 ** e).to(torch.bfloat16))
    wide = torch.randn(600, D, generator=gen) * torch.exp(6 * torch.randn(600, D, generator=gen))
    rows += list(wide.to(torch.bfloat16))
    for x in (0.0, 2.0 ** -101, 2.0 ** -100, 2.0 ** -130, 3.38e38, -0.0):
        rows.append(torch.full((D,), x).to(torch.bfloat16))
    for x in (float("nan"), float("inf"), -float("inf")):
        r = torch.ones(D)
        r[D // 3] = x
        rows.append(r.to(torch.bfloat16))
    k = torch.stack(rows)[None, :, None]  # [1, T, 1, D]
    T, ps = k.shape[1], 64
    table, n_pages = tables([T], ps, 2, gen)
    dev = Device(n_pages, 1, ps, D, dtype)
    ra.ra_cache_append(k.cuda(), k.flip(1).contiguous().cuda(), dev.k, dev.v, table.cuda(),
                       torch.tensor([T], dtype=torch.int32).cuda(), key_bounds=dev.bounds, **dev.kw())
    P.append(dev.ref, f64(k), f64(k.flip(1)), table.tolist(), [T], [T])
    dev.check()
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", ["int8", "e4m3"])
def test_every_significand_against_every_scale(cuda_lib, dtype):
    """Codes of all bf16 significands, over 20 binades, in rows of all largest significands: what
    the choice between two codes can hang on, for the smallest scales, ordinary and the largest."""
    ra = cuda_lib
    D, ps = 128, 128
    m = torch.arange(128, 256, dtype=torch.float64)
    x = torch.cat([m * 2.0 ** -d for d in range(20)])                       # 2,560 values
    x = x * torch.where(torch.arange(len(x)) % 2 == 0, 1.0, -1.0)
    x = torch.cat([x, x.new_zeros(-len(x) % (D - 1))]).view(-1, D - 1)      # 21 rows
    rows = torch.zeros((128, len(x), D), dtype=torch.float64)
    rows[:, :, 0] = m[:, None]
    rows[:, :, 1:] = torch.where(x.abs() <= m[:, None, None], x, 0.0)
    rows = rows.view(-1, D)
    k = torch.cat([(rows * 2.0 ** e).to(torch.bfloat16) for e in (-107, -7, 120)])[None, :, None]
    T = k.shape[1]
    table = torch.arange(-(-T // ps), dtype=torch.int32)[None].contiguous()
    dev = Device(table.numel(), 1, ps, D, dtype, bounds=False)
    ra.ra_cache_append(k.cuda(), -k.cuda(), dev.k, dev.v, table.cuda(), torch.tensor([T], dtype=torch.int32).cuda(), **dev.kw())
    for got, scales, sign in ((dev.k, dev.ks, 1.0), (dev.v, dev.vs, -1.0)):
        code, value, scale = P.quantise(sign * f64(k[0, :, 0]), dtype)
        assert np.array_equal(f64(scales.view(-1)[:T]), scale)
        got = f64(got.view(-1, D)[:T].float())
        off = got != value / scale[:, None]
        assert not off.any(), f"{off.sum()} codes, first {np.argwhere(off)[0]}"
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", ["int8", "e4m3"])
def test_every_scale_is_correctly_rounded(cuda_lib, dtype):
    """All bf16 magnitudes from 2^-100 up as a row's largest value."""
    ra = cuda_lib
    bits = torch.arange(27 << 7, 0x7f80, dtype=torch.int32).to(torch.int16)  # 2^-100 ... the largest finite
    amax = bits.view(torch.bfloat16)
    D, ps, T = 64, 128, len(bits)
    k = torch.zeros((1, T, 1, D), dtype=torch.bfloat16)
    k[0, :, 0, 17] = amax
    table = torch.arange(-(-T // ps), dtype=torch.int32)[None].contiguous()
    dev = Device(table.numel(), 1, ps, D, dtype, bounds=False)
    ra.ra_cache_append(k.cuda(), -k.cuda(), dev.k, dev.v, table.cuda(), torch.tensor([T], dtype=torch.int32).cuda(), **dev.kw())
    want = (amax.double() / P.QMAX[dtype]).float()  # (no such quotient is near a tie of fp32: its bits repeat)
    for s in (dev.ks, dev.vs):
        assert torch.equal(s.cpu().view(-1)[:T], want)
    assert ra.ra_get_device_status() == ra.RA_OK


@pytest.mark.parametrize("dtype", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Hkv,D,ps,seq,first,T", [
    (1, 1, 64, 16, [1], 0, 1),
    (2, 3, 128, 16, [50, 7], 5, 40),       # first inside a page, an end inside the stretch
    (3, 2, 64, 128, [300, 0, 129], 128, 2),
    (2, 8, 128, 32, [64, 33], 0, 70),      # rows behind both ends
    (1, 2, 128, 64, [100], 500, 3),        # wholly behind the end
])
def test_read(cuda_lib, dtype, out, B, Hkv, D, ps, seq, first, T):
    ra = cuda_lib
    gen = torch.Generator().manual_seed(11)
    table, n_pages = tables(seq, ps, 2, gen)
    if dtype == "bf16":
        k, v = draw(gen, n_pages, Hkv, ps, D), draw(gen, n_pages, Hkv, ps, D)
        ks = vs = None
        val = {"k": k.float(), "v": v.float()}
    else:  # every code but the NaNs, scales of all sizes
        k, v = (torch.randint(0, 256, (n_pages, Hkv, ps, D), generator=gen, dtype=torch.uint8) for _ in "kv")
        if dtype == "e4m3":
            k, v = (torch.where((t & 127) == 127, t - 1, t) for t in (k, v))
        k, v = k.view(TORCH[dtype]), v.view(TORCH[dtype])
        ks, vs = (torch.exp(4 * torch.randn(n_pages, Hkv, ps, generator=gen)) for _ in "kv")
        val = {"k": k.float() * ks[..., None], "v": v.float() * vs[..., None]}
        ks, vs = ks.cuda(), vs.cuda()
    ref = P.Cache(n_pages, Hkv, ps, D, dtype)
    for w in "kv":
        ref.value[w][:] = val[w].to(out).double().numpy()
    gk, gv = ra.ra_cache_read(k.cuda(), v.cuda(), table.cuda(), torch.tensor(seq, dtype=torch.int32).cuda(), T,
                              first=first, k_scales=ks, v_scales=vs, out_dtype=out)
    assert gk.dtype == out and gk.shape == (B, T, Hkv, D)
    assert np.array_equal(f64(gk), P.read(ref, table.tolist(), seq, first, T, "k"))
    assert np.array_equal(f64(gv), P.read(ref, table.tolist(), seq, first, T, "v"))
    assert ra.ra_get_device_status() == ra.RA_OK


def test_device_integers_out_of_range_are_recorded(cuda_lib):
    """A page outside the cache, a length past the table, too many new tokens: the
    status word says so, the other sequences' results are right, nothing else is written."""
    ra = cuda_lib
    gen = torch.Generator().manual_seed(5)
    ps, Hkv, D, T = 16, 2, 64, 3
    seq, new = [20, 35, 9], [3, 2, 3]
    table, n_pages = tables(seq, ps, 2, gen)
    k, v = draw(gen, 3, T, Hkv, D), draw(gen, 3, T, Hkv, D)

    def step(table, seq, new):
        dev = Device(n_pages, Hkv, ps, D, "int8")
        ra.ra_cache_append(k.cuda(), v.cuda(), dev.k, dev.v, table.cuda(), torch.tensor(seq, dtype=torch.int32).cuda(),
                           new_lens=torch.tensor(new, dtype=torch.int32).cuda(), key_bounds=dev.bounds, **dev.kw())
        return dev

    bad = table.clone()
    bad[1, 2] = n_pages  # the page of sequence 1's new tokens
    dev = step(bad, seq, new)
    assert ra.ra_get_device_status() == ra.RA_ERR_DEVICE_BOUNDS
    P.append(dev.ref, f64(k), f64(v), table.tolist(), [20, 0, 9], [3, 0, 3])
    dev.check()
    for s, n in (([20, 35, -4], [3, 2, 0]), ([20, 35, 9], [3, 2, 4]), ([20, 35, 9], [3, 2, -1])):
        step(table, s, n)
        assert ra.ra_get_device_status() == ra.RA_ERR_DEVICE_BOUNDS
    seq_t = torch.tensor([20, 49, 9], dtype=torch.int32).cuda()  # 3 table entries of 16 rows hold 48
    dev = Device(n_pages, Hkv, ps, D, "bf16")
    ra.ra_cache_read(dev.k, dev.v, table.cuda(), seq_t, 8)
    assert ra.ra_get_device_status() == ra.RA_ERR_DEVICE_BOUNDS
    assert ra.ra_get_device_status() == ra.RA_OK


def test_append_in_a_graph_and_on_a_stream(cuda_lib):
    """A captured step replays with the lengths, table and tokens then in its buffers."""
    ra = cuda_lib
    gen = torch.Generator().manual_seed(8)
    ps, Hkv, D = 16, 2, 128
    table, n_pages = tables([40, 40], ps, 1, gen)
    dev = Device(n_pages, Hkv, ps, D, "e4m3")
    k, v = draw(gen, 2, 1, Hkv, D).cuda(), draw(gen, 2, 1, Hkv, D).cuda()
    seq = torch.tensor([1, 1], dtype=torch.int32).cuda()
    tab = table.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ra.ra_cache_append(k, v, dev.k, dev.v, tab, seq, key_bounds=dev.bounds, **dev.kw())
    torch.cuda.current_stream().wait_stream(side)
    P.append(dev.ref, f64(k), f64(v), table.tolist(), [1, 1], [1, 1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ra.ra_cache_append(k, v, dev.k, dev.v, tab, seq, key_bounds=dev.bounds, **dev.kw())
    for lens in ([2, 2], [3, 17], [33, 18], [34, 0]):
        nk, nv = draw(gen, 2, 1, Hkv, D), draw(gen, 2, 1, Hkv, D)
        k.copy_(nk)
        v.copy_(nv)
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        P.append(dev.ref, f64(nk), f64(nv), table.tolist(), lens, [min(1, n) for n in lens])
    dev.check()
    assert ra.ra_get_device_status() == ra.RA_OK
