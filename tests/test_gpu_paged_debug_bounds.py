"""The paged cache's kernels in the checked build: their edge cases break no check and
match the oracle; an index that is put out of range where it is checked (an
offset that only the checked build reads, from the environment) is recorded, its
access left out, and the next call is right again."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import os
import numpy as np
import torch
import blockwise_exact_attention_block_b200 as ra
from oracle import paged as P
from test_gpu_cache import Device, draw as tokens, f64, tables
from test_gpu_page_select import draw as pages_of
from test_gpu_paged_decode import SHAPES, Case

assert ra.ra_debug_build(), "the checked build was not loaded"

def clean(what):
    torch.cuda.synchronize()
    st, rec = ra.ra_get_device_status(), ra.ra_get_bounds_record()
    assert st == 0 and rec == (0, 0, 0), (what, ra.ra_status_string(st), rec)

def broken(what):
    torch.cuda.synchronize()
    st, (line, idx, lim) = ra.ra_get_device_status(), ra.ra_get_bounds_record()
    assert st == ra.RA_ERR_DEVICE_BOUNDS, (what, ra.ra_status_string(st))
    assert line > 0 and lim > 0 and idx >= 1 << 40, (what, line, idx, lim)

gen = torch.Generator().manual_seed(1)
for dtype in ("bf16", "int8", "e4m3"):
    for shape in SHAPES:
        for causal in (True, False):
            c = Case(dtype, *shape, seed=3)
            c.check(ra.ra_paged_decode_attention(*c.args, causal=causal, out_dtype=torch.bfloat16, **c.kw), causal)
            clean((dtype, shape))
    for T, Hkv, D, ps, seq, new in ((1, 3, 128, 16, [17, 1], [1, 1]), (5, 2, 64, 16, [5, 20], [5, 3]),
                                    (300, 2, 64, 128, [411, 300], [300, 257]), (40, 8, 128, 16, [57, 40], [40, 0])):
        table, n_pages = tables(seq, ps, 1, gen)
        dev = Device(n_pages, Hkv, ps, D, dtype)
        k, v = tokens(gen, 2, T, Hkv, D), tokens(gen, 2, T, Hkv, D)
        lens, nl = (torch.tensor(x, dtype=torch.int32).cuda() for x in (seq, new))
        ra.ra_cache_append(k.cuda(), v.cuda(), dev.k, dev.v, table.cuda(), lens, new_lens=nl, key_bounds=dev.bounds, **dev.kw())
        P.append(dev.ref, f64(k), f64(v), table.tolist(), seq, new)
        dev.check()
        for odt in (torch.bfloat16, torch.float32):
            for first, n in ((0, 1), (3, max(seq)), (10 ** 6, 5)):
                ra.ra_cache_read(dev.k, dev.v, table.cuda(), lens, n, first=first, out_dtype=odt, **dev.kw())
        clean((dtype, T, D, ps))
for B, Tq, Hq, Hkv, D, ps, seq, new, n_sel, levels in (
        (2, 4, 8, 2, 128, 16, [1000, 17], [2, 0], 9, None), (2, 1, 4, 2, 64, 16, [4000, 2000], None, 40, 5),
        (1, 1, 8, 2, 128, 16, [16 * 5003], None, 100, None), (1, 1, 2, 2, 64, 16, [16 * 4000], None, 25, 1)):
    q, bounds, table = pages_of(B, Tq, Hq, Hkv, D, ps, seq, 0, levels)
    lens = torch.tensor(seq, dtype=torch.int32).cuda()
    nl = None if new is None else torch.tensor(new, dtype=torch.int32).cuda()
    got = ra.ra_page_select(q.cuda(), bounds.cuda(), table.cuda(), lens, n_sel, ps, new_lens=nl)
    want = P.select(f64(q), f64(bounds), ps, table.tolist(), seq, new or [min(Tq, n) for n in seq], n_sel)
    assert np.array_equal(got.cpu().numpy(), want)
    clean(("select", seq))

c = Case("int8", 2, 1, 8, 2, 128, 16, [300, 40], seed=3)
q, kp, vp, table, lens = c.args
sc = dict(k_scales=c.scales["k"], v_scales=c.scales["v"])
kept = kp.clone()
new = tokens(gen, 2, 1, 2, 128).cuda()
sq, bounds, st = pages_of(1, 1, 4, 1, 64, 16, [16 * 40], 0)
calls = {
    "decode": lambda: ra.ra_paged_decode_attention(q, kp, vp, table, lens, **sc),
    "read": lambda: ra.ra_cache_read(kp, vp, table, lens, 300, **sc),
    "append": lambda: ra.ra_cache_append(new, new, kp, vp, table, lens, **sc),
    "select": lambda: ra.ra_page_select(sq.cuda(), bounds.cuda(), st.cuda(), torch.tensor([640], dtype=torch.int32).cuda(), 5, 16),
}
for name, call in calls.items():
    os.environ["RA_DEBUG_INJECT_PAGED"] = str(1 << 40)
    call()
    broken(name)
    assert torch.equal(kp, kept), name  # nothing was written
    os.environ["RA_DEBUG_INJECT_PAGED"] = "0"
    if name != "append":
        call()
        clean(name)
c.check(ra.ra_paged_decode_attention(q, kp, vp, table, lens, out_dtype=torch.float32, **sc), True)
calls["append"]()
assert not torch.equal(kp, kept)
clean("the calls after")
print("CHECKED BUILD OK")
'''


def test_paged_kernels_in_the_checked_build(cuda_lib):
    env = dict(os.environ, RA_DEBUG_BOUNDS="1", PYTHONPATH=os.pathsep.join((ROOT, os.path.join(ROOT, "tests"))))
    res = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, env=env, timeout=600)
    assert res.returncode == 0 and "CHECKED BUILD OK" in res.stdout, res.stdout[-2000:] + res.stderr[-4000:]
