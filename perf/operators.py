"""The serving operators over a paged key-value cache, as cases to be timed and checked.

Four operators, in the order of a serving step:

* ``append``: new keys and values go into the pages of a cache (bf16 as they are; int8 and e4m3 with one fp32 scale for
  each token and KV head), and the page bounds (smallest and largest key of each page and column) are kept with them.
  A cache in 8 bits is read back in the same pass, as the values that its codes stand for.
* ``read``: a stretch of the cache as dense keys and values, as a prompt's attention takes them.
* ``decode``: a few new tokens' attention over the whole paged cache.
* ``sparse``: the pages that the bounds' score selects for each KV head, and the attention over these pages alone.

Layouts: pages ``[n_pages, Hkv, page, D]``, scales ``[n_pages, Hkv, page]``, bounds ``[n_pages, Hkv, 2, D]`` (min, max),
page table ``[B, max_pages]``; ``seq_lens`` counts the step's new tokens in, ``new_lens`` is how many of a sequence's
token rows are real.
"""
import math

import torch

own = False

_QMAX = {"int8": 127.0, "e4m3": 448.0}
_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_TINY = 2.0 ** -100  # a row whose largest magnitude is below this is stored as zeros


# ---------------------------------------------------------------- the cases

def _case(name, op, B, T, Hq, Hkv, D, page, dtype, low, cap, **more):
    c = {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype,
         "low": low, "cap": cap, "empty": False, "ragged": False, "causal": True, "out": "bf16", "n_sel": 0, "first": 0}
    c.update(more)
    return c


def listed():
    return [
        # one decoded token for each of 64 running conversations, cache in bf16, bounds kept for page selection
        _case("append_step_64", "append", 64, 1, 32, 8, 128, 16, "bf16", 17, 1000),
        # a 24,000-token prompt (the 24k grouped-query shape) written in 8 bits, and read back
        _case("append_prompt_24k_int8", "append", 1, 24000, 32, 8, 128, 64, "int8", 24000, 24000, out="f32"),
        # chunked prefill of an odd batch: chunks of up to 2,049 tokens behind what is there already
        _case("append_chunk_ragged_e4m3", "append", 6, 2049, 8, 2, 64, 32, "e4m3", 2100, 5001, ragged=True, out="f32"),
        # a shared prefix of four sequences taken out of an int8 cache for a prompt's attention in bf16
        _case("read_prefix_24k_int8", "read", 4, 24000, 32, 8, 128, 16, "int8", 12000, 24000),
        # a short prefix, odd length and start
        _case("read_small_e4m3", "read", 2, 701, 8, 2, 64, 32, "e4m3", 500, 777, out="f32", first=13),
        # one token of one short conversation: latency
        _case("decode_step_1k", "decode", 1, 1, 8, 2, 128, 16, "bf16", 1000, 1000),
        # the long-context cache: one token against 1,048,576
        _case("decode_1m", "decode", 1, 1, 8, 2, 128, 64, "bf16", 1048576, 1048576),
        # the 24k batch with four proposed tokens each, int8 cache
        _case("decode_24k_int8", "decode", 8, 4, 32, 8, 128, 16, "int8", 9000, 24000, ragged=True),
        # a full serving batch, lengths from one token to 8,192 and a slot that is empty, e4m3 cache
        _case("decode_batch_e4m3", "decode", 64, 1, 32, 8, 128, 32, "e4m3", 1, 8192, empty=True),
        # heads of 64 without grouping, every key visible (scoring of a given continuation)
        _case("decode_mha_d64", "decode", 16, 3, 8, 8, 64, 128, "bf16", 700, 4096, causal=False),
        # one token against the 1M cache through its 512 best pages
        _case("sparse_1m", "sparse", 1, 1, 8, 2, 128, 64, "bf16", 1048576, 1048576, n_sel=512),
        # the 24k batch, int8, through 1/12 of its pages
        _case("sparse_24k_int8", "sparse", 8, 1, 32, 8, 128, 16, "int8", 2000, 24000, n_sel=128),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode", "sparse"])
    D = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "int8", "e4m3"])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    B = _log(rng, 1, 64)
    # at most 2^28 cached keys' values, as many as the 1M-token cases hold
    most = max(2, min(262144, (1 << 28) // (B * Hkv * D)))
    cap = _log(rng, min(200, most), most)
    low = rng.randint(1, cap)
    more = {"empty": B > 2 and rng.random() < 0.3, "ragged": rng.random() < 0.5, "causal": rng.random() < 0.75}
    if op == "append":
        T = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(cap, 8192)))
        more["out"] = "f32"
    elif op == "read":
        T = _log(rng, 1, cap)
        more["first"] = rng.randint(0, cap - T)
        more["out"] = rng.choice(["bf16", "f32"])
    else:
        T = rng.choice([1, 1, 1, 2, 3, 4, 6]) if group < 8 else 1
        if op == "sparse":
            pages = -(-cap // page)
            more["n_sel"] = 2 + _log(rng, 1, max(1, pages))
    return {k: v for k, v in _case("", op, B, min(T, cap), Hkv * group, Hkv, D, page, dtype, low, cap, **more).items()
            if k != "name"}


def _lens(case):
    """(tokens cached, new ones among them) of each sequence: spread over low .. cap by their ratio, the longest first."""
    B, low, cap, T = case["B"], max(1, case["low"]), case["cap"], case["T"]
    lens, news = [], []
    for b in range(B):
        x = ((b * 7) % B) / B  # any order but the sorted one
        n = cap if b == 0 else max(1, int(round(cap * (low / cap) ** x)))
        if case["empty"] and b == 1:
            n = 0
        lens.append(n)
        t = T - (b * 3) % T if case["ragged"] and case["op"] != "read" else T
        news.append(0 if case["op"] == "read" else min(t, n))
    return lens, news


# ---------------------------------------------------------------- the inputs

def _tokens(gen, shape):
    """Keys or values as a trained model makes them: columns of their own size and offset (the last two axes), in bf16."""
    tail = shape[-2:]
    gain = torch.exp(0.4 * torch.randn(tail, generator=gen, device="cuda"))
    mean = 0.5 * torch.randn(tail, generator=gen, device="cuda")
    x = torch.randn(shape, generator=gen, device="cuda")
    return x.mul_(gain).add_(mean).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    B, T, Hq, Hkv, D, ps = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"], case["page"]
    dt = case["dtype"]
    lens, news = _lens(case)
    max_pages = -(-case["cap"] // ps)
    need = [-(-n // ps) for n in lens]
    total = sum(need)
    n_pages = total + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    st = {"case": dict(case), "page_table": table,
          "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
          "new_lens": torch.tensor(news, dtype=torch.int32, device="cuda")}
    # the pages, as earlier steps left them
    pages = [_tokens(gen, (n_pages, ps, Hkv, D)).transpose(1, 2).contiguous() for _ in range(2)]
    scales = [None, None]
    st["key_bounds"] = torch.stack((pages[0].amin(2), pages[0].amax(2)), 2) if case["op"] in ("append", "sparse") else None
    if dt != "bf16":
        for i in range(2):
            amax = pages[i].abs().amax(-1).float()
            scales[i] = amax / _QMAX[dt]
            x = pages[i].float() / scales[i][..., None]
            pages[i] = x.round().to(torch.int8) if dt == "int8" else x.to(torch.float8_e4m3fn)
    st["k_pages"], st["v_pages"] = pages
    st["k_scales"], st["v_scales"] = scales
    if case["op"] == "append":
        st["k"], st["v"] = _tokens(gen, (B, T, Hkv, D)), _tokens(gen, (B, T, Hkv, D))
    elif case["op"] != "read":
        st["q"] = (1.5 * torch.randn((B, T, Hq, D), generator=gen, device="cuda")).to(torch.bfloat16)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    return {"append": _append, "read": _read, "decode": _decode, "sparse": _sparse}[c["op"]](st, c)


def _append(st, c):
    if own:
        import blockwise_exact_attention_block_b200 as ra
        ra.ra_cache_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["page_table"], st["seq_lens"],
                           new_lens=st["new_lens"], k_scales=st["k_scales"], v_scales=st["v_scales"],
                           key_bounds=st["key_bounds"])
        if c["dtype"] == "bf16":
            return {"k": st["k_pages"], "v": st["v_pages"], "bounds": st["key_bounds"]}
        k, v = ra.ra_cache_read(st["k_pages"], st["v_pages"], st["page_table"], st["seq_lens"], c["cap"],
                                k_scales=st["k_scales"], v_scales=st["v_scales"], out_dtype=torch.float32)
    else:
        _plain_append(st, c)
        if c["dtype"] == "bf16":
            return {"k": st["k_pages"], "v": st["v_pages"], "bounds": st["key_bounds"]}
        k, v = _plain_dense(st, c, "k", 0, c["cap"]), _plain_dense(st, c, "v", 0, c["cap"])
    return {"k": k, "v": v, "k_scales": st["k_scales"], "v_scales": st["v_scales"], "bounds": st["key_bounds"]}


def _read(st, c):
    if own:
        import blockwise_exact_attention_block_b200 as ra
        k, v = ra.ra_cache_read(st["k_pages"], st["v_pages"], st["page_table"], st["seq_lens"], c["T"], first=c["first"],
                                k_scales=st["k_scales"], v_scales=st["v_scales"], out_dtype=_TORCH[c["out"]])
    else:
        k = _plain_dense(st, c, "k", c["first"], c["T"]).to(_TORCH[c["out"]])
        v = _plain_dense(st, c, "v", c["first"], c["T"]).to(_TORCH[c["out"]])
    return {"k": k, "v": v}


def _decode(st, c):
    if own:
        import blockwise_exact_attention_block_b200 as ra
        out, lse = ra.ra_paged_decode_attention(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["seq_lens"],
                                                new_lens=st["new_lens"], k_scales=st["k_scales"], v_scales=st["v_scales"],
                                                causal=c["causal"], out_dtype=_TORCH[c["out"]])
        return {"out": out, "lse": lse}
    k = _plain_dense(st, c, "k", 0, c["cap"]).permute(0, 2, 1, 3)
    v = _plain_dense(st, c, "v", 0, c["cap"]).permute(0, 2, 1, 3)
    pos = torch.arange(c["cap"], device=k.device).expand(c["B"], c["Hkv"], -1)
    return _plain_attention(st, c, k, v, pos)


def _sparse(st, c):
    if own:
        import blockwise_exact_attention_block_b200 as ra
        sel = ra.ra_page_select(st["q"], st["key_bounds"], st["page_table"], st["seq_lens"], c["n_sel"], c["page"],
                                new_lens=st["new_lens"])
        out, lse = ra.ra_paged_decode_attention(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["seq_lens"],
                                                new_lens=st["new_lens"], k_scales=st["k_scales"], v_scales=st["v_scales"],
                                                causal=c["causal"], selected=sel, out_dtype=_TORCH[c["out"]])
        return {"selected": sel, "out": out, "lse": lse}
    sel = _plain_select(st, c)
    k, v = _plain_selected(st, c, "k", sel), _plain_selected(st, c, "v", sel)
    pos = sel.long()[..., None] * c["page"] + torch.arange(c["page"], device=sel.device)
    pos = torch.where(sel[..., None] >= 0, pos, 1 << 40).flatten(2)  # no page: beyond every length
    return {"selected": sel, **_plain_attention(st, c, k, v, pos)}


# ---------------------------------------------------------------- the plain forms

def _places(st, c, first, T):
    """(page, row in it, whether the cache holds it) of the positions first .. first + T - 1 of each sequence."""
    p = first + torch.arange(T, device=st["page_table"].device)
    held = p[None, :] < st["seq_lens"][:, None]
    logical = (p // c["page"]).clamp(max=st["page_table"].shape[1] - 1)
    return st["page_table"][:, logical].long().clamp(min=0), (p % c["page"])[None, :].expand_as(held), held


def _plain_dense(st, c, which, first, T):
    """[B, T, Hkv, D] in 32 bits: the cached values, zero behind a sequence's end."""
    page, row, held = _places(st, c, first, T)
    x = st[which + "_pages"][page, :, row].float()
    if st[which + "_scales"] is not None:
        x = x * st[which + "_scales"][page, :, row][..., None]
    return torch.where(held[:, :, None, None], x, 0.0)


def _plain_selected(st, c, which, sel):
    """[B, Hkv, n_sel * page, D] in 32 bits: the selected pages of each KV head."""
    B, Hkv, n = sel.shape
    logical = sel.long().clamp(min=0)
    page = torch.gather(st["page_table"][:, None, :].expand(-1, Hkv, -1), 2, logical).long().clamp(min=0)
    head = torch.arange(Hkv, device=sel.device)[None, :, None].expand_as(page)
    x = st[which + "_pages"][page, head].float()
    if st[which + "_scales"] is not None:
        x = x * st[which + "_scales"][page, head][..., None]
    return x.flatten(2, 3)


def _plain_limits(st, c):
    """[B, T]: keys below this position are visible; 0 for a token row that is not real."""
    t = torch.arange(c["T"], device=st["seq_lens"].device)[None, :]
    s, n = st["seq_lens"].long()[:, None], st["new_lens"].long()[:, None]
    return torch.where(t < n, s - n + t + 1 if c["causal"] else s.expand(-1, c["T"]), 0)


def _plain_attention(st, c, k, v, pos):
    """k, v [B, Hkv, S, D] in 32 bits, pos [B, Hkv, S]: softmax over the visible keys."""
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    q = st["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    s = q @ k.transpose(2, 3) * (1.0 / math.sqrt(D))
    lim = _plain_limits(st, c).repeat_interleave(G, 1)[:, None, :, None]
    s = torch.where(pos[:, :, None, :] < lim, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    tot = e.sum(-1, keepdim=True)
    out = (e @ v) / torch.where(tot == 0, 1.0, tot)
    lse = (m + torch.log(tot)).squeeze(-1)
    out = out.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = lse.view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)
    return {"out": out.to(_TORCH[c["out"]]), "lse": lse.contiguous()}


def _plain_quantise(x, dtype):
    """(codes, scales) of rows x in 32 bits.  The quotients are taken in 64 bits: 32 round some across a border."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax < _TINY, 0.0, (amax.double() / _QMAX[dtype]).float())
    t = x.double() / torch.where(scale == 0, 1.0, scale).double()[..., None]
    t = torch.where(scale[..., None] == 0, 0.0, t)
    if dtype == "int8":
        return t.round().clamp(-127, 127).to(torch.int8), scale
    # e4m3: 3 bits behind the leading one, steps of 2^-9 below 2^-6; round() goes to the even multiple of the step
    step = torch.exp2(torch.log2(t.abs().clamp(min=2.0 ** -6)).floor() - 3)
    return ((t / step).round() * step).clamp(-448, 448).float().to(torch.float8_e4m3fn), scale


def _plain_append(st, c):
    t = torch.arange(c["T"], device=st["k"].device)[None, :]
    b, t = torch.nonzero(t < st["new_lens"][:, None], as_tuple=True)
    pos = (st["seq_lens"].long() - st["new_lens"].long())[b] + t
    page, row = st["page_table"][b, pos // c["page"]].long(), pos % c["page"]
    k, v = st["k"][b, t], st["v"][b, t]
    if c["dtype"] == "bf16":
        st["k_pages"][page, :, row], st["v_pages"][page, :, row] = k, v
    else:
        (kc, ks), (vc, vs) = _plain_quantise(k.float(), c["dtype"]), _plain_quantise(v.float(), c["dtype"])
        st["k_pages"].view(torch.int8)[page, :, row] = kc.view(torch.int8)
        st["v_pages"].view(torch.int8)[page, :, row] = vc.view(torch.int8)
        st["k_scales"][page, :, row], st["v_scales"][page, :, row] = ks, vs
    fresh = page[row == 0]  # pages that the new tokens begin
    lo, hi = st["key_bounds"][:, :, 0].float(), st["key_bounds"][:, :, 1].float()
    lo[fresh], hi[fresh] = math.inf, -math.inf
    lo.index_reduce_(0, page, k.float(), "amin")
    hi.index_reduce_(0, page, k.float(), "amax")
    st["key_bounds"].copy_(torch.stack((lo, hi), 2))


def _plain_select(st, c):
    """The n_sel best pages of each KV head by the bounds' score, ascending, -1 behind.  Scores in 64 bits: two pages'
    may be close, and the products of bf16 values and their sums are then exact for all practical ranges."""
    B, T, Hq, Hkv, D, n = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["n_sel"]
    G, P = Hq // Hkv, st["page_table"].shape[1]
    q = st["q"].double().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    bounds = st["key_bounds"][st["page_table"].long().clamp(min=0)].double()  # [B, P, Hkv, 2, D]
    lo, hi = bounds[:, :, :, 0].permute(0, 2, 3, 1), bounds[:, :, :, 1].permute(0, 2, 3, 1)
    score = q.clamp(min=0) @ hi + q.clamp(max=0) @ lo  # the larger of q lo and q hi, summed over the columns
    real = torch.arange(T, device=q.device)[None, :] < st["new_lens"][:, None]
    score = torch.where(real.repeat_interleave(G, 1)[:, None, :, None], score, -math.inf).amax(2)  # [B, Hkv, P]
    p = torch.arange(P, device=q.device)[None, :]
    s, new = st["seq_lens"].long()[:, None], st["new_lens"].long()[:, None]
    there = p * c["page"] < s
    latest = there & (p >= (s - new).clamp(min=0) // c["page"]) & (new > 0)
    rank = torch.where(latest, 2, torch.where(there, 1, 0))[:, None, :].expand_as(score)
    score = torch.where(rank == 1, score, 0.0)
    by = torch.sort(score, dim=-1, descending=True, stable=True).indices
    by = by.gather(-1, torch.sort(rank.gather(-1, by), dim=-1, descending=True, stable=True).indices)
    by = by[..., :n]
    by = torch.where(there[:, None, :].expand(-1, Hkv, -1).gather(-1, by), by, P)
    by = torch.sort(by, dim=-1).values
    by = torch.nn.functional.pad(by, (0, n - by.shape[-1]), value=P)
    return torch.where(by < P, by, -1).to(torch.int32)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    lens, news = _lens(c)
    D, Hkv, T, G, ps = c["D"], c["Hkv"], c["T"], c["Hq"] // c["Hkv"], c["page"]
    row = 2 * D if c["dtype"] == "bf16" else D + 4  # bytes of one cached key or value
    out = 2 if c["out"] == "bf16" else 4
    if c["op"] == "append":
        n = sum(news)
        touched = sum(-(-s // ps) - (s - t) // ps for s, t in zip(lens, news) if t)
        b = 2 * n * Hkv * (2 * D + row) + 4 * D * Hkv * touched
        f = 2 * n * Hkv * D
        if c["dtype"] != "bf16":  # read back: what is there is read, the dense values are written
            b += 2 * Hkv * (sum(lens) * row + c["B"] * c["cap"] * D * 4)
            f += 2 * sum(lens) * Hkv * D
        return {"bytes": b, "flops": f}
    if c["op"] == "read":
        n = sum(max(0, min(s - c["first"], T)) for s in lens)
        return {"bytes": 2 * Hkv * (n * row + c["B"] * T * D * out), "flops": 2 * n * Hkv * D}
    tokens = lens if c["op"] == "decode" else [min(s, c["n_sel"] * ps) for s in lens]
    keys = sum(tokens)
    rows = c["B"] * T * c["Hq"]
    b = 2 * Hkv * keys * row + rows * (D * (2 + out) + 4)
    f = 4 * D * Hkv * G * sum(s * t for s, t in zip(tokens, news))
    if c["op"] == "sparse":
        pages = sum(-(-s // ps) for s in lens)
        b += pages * Hkv * 4 * D + 4 * c["B"] * Hkv * c["n_sel"]
        f += sum(-(-s // ps) * t for s, t in zip(lens, news)) * Hkv * G * 2 * D
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    st = prepare(case, seed)
    c = case
    lens, news = _lens(c)
    ps, Hkv, T = c["page"], c["Hkv"], c["T"]
    table = st["page_table"].tolist()

    def value(which):
        x = st[which + "_pages"].double()
        return x if st[which + "_scales"] is None else x * st[which + "_scales"].double()[..., None]

    def dense(pages, b, first, last):
        """[last - first, Hkv, D] of sequence b."""
        ids = torch.tensor(table[b][first // ps:-(-last // ps)], device=pages.device, dtype=torch.long)
        x = pages[ids].transpose(1, 2).reshape(-1, Hkv, c["D"])
        return x[first - first // ps * ps:][:last - first]

    if c["op"] == "append":
        return _exact_append(st, c, lens, news, table, value, dense)
    if c["op"] == "read":
        got = {}
        for which in ("k", "v"):
            pages = value(which)
            out = torch.zeros((c["B"], T, Hkv, c["D"]), dtype=torch.float64, device=pages.device)
            for b, n in enumerate(lens):
                last = min(n, c["first"] + T)
                if last > c["first"]:
                    out[b, :last - c["first"]] = dense(pages, b, c["first"], last)
            got[which] = out
        return got
    return _exact_attention(st, c, lens, news, table)


def _exact_append(st, c, lens, news, table, value, dense):
    ps = c["page"]
    bounds = st["key_bounds"].double()
    pages = {w: value(w) for w in ("k", "v")}
    scales = {w: None if st[w + "_scales"] is None else st[w + "_scales"].double() for w in ("k", "v")}
    for b, (n, new) in enumerate(zip(lens, news)):
        if not new:
            continue
        pos = torch.arange(n - new, n, device=bounds.device)
        page = torch.tensor(table[b], device=bounds.device, dtype=torch.long)[pos // ps]
        for w in ("k", "v"):
            x = st[w][b, :new].double()
            if c["dtype"] != "bf16":
                # the scale is held in fp32: that is part of the definition, and so is a zero row's zero scale
                s = (x.abs().amax(-1) / _QMAX[c["dtype"]]).float().double()
                d = torch.where(s == 0, 1.0, s)[..., None]
                if c["dtype"] == "int8":
                    y = torch.round(x / d)
                else:  # the nearest of the type's values; of two, the one with the even last bit
                    grid = torch.arange(0, 127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
                    mag = (x / d).abs()
                    hi = torch.searchsorted(grid, mag).clamp(max=126)
                    lo = (hi - 1).clamp(min=0)
                    dl, dh = mag - grid[lo], grid[hi] - mag
                    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
                    y = grid[pick] * torch.sign(x)
                scales[w][page, :, pos % ps] = s
                pages[w][page, :, pos % ps] = y * s[..., None]
            else:
                pages[w][page, :, pos % ps] = x
        for j in range((n - new) // ps, -(-n // ps)):
            a, z = max(n - new, j * ps), min(n, j * ps + ps)
            x = st["k"][b, a - (n - new):z - (n - new)].double()
            lo, hi = x.amin(0), x.amax(0)
            old = bounds[table[b][j]]
            if a > j * ps:
                lo, hi = torch.minimum(lo, old[:, 0]), torch.maximum(hi, old[:, 1])
            bounds[table[b][j]] = torch.stack((lo, hi), 1)
    if c["dtype"] == "bf16":
        return {"k": pages["k"], "v": pages["v"], "bounds": bounds}
    got = {"k_scales": scales["k"], "v_scales": scales["v"], "bounds": bounds}
    for w in ("k", "v"):
        got[w] = torch.zeros((c["B"], c["cap"], c["Hkv"], c["D"]), dtype=torch.float64, device=bounds.device)
        for b, n in enumerate(lens):
            got[w][b, :n] = dense(pages[w], b, 0, n)
    return got


def _exact_attention(st, c, lens, news, table):
    B, T, Hq, Hkv, D, ps = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    dev = st["q"].device
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=dev)
    sel = torch.full((B, Hkv, max(1, c["n_sel"])), -1, dtype=torch.int32, device=dev)
    for b, (n, new) in enumerate(zip(lens, news)):
        if not n:
            continue
        count = -(-n // ps)
        ids = torch.tensor(table[b][:count], device=dev, dtype=torch.long)
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            q = st["q"][b, :new, heads].double()
            mine = torch.arange(count, device=dev)
            if c["op"] == "sparse":
                lo, hi = st["key_bounds"][ids, h].double().unbind(1)
                s = torch.stack([torch.maximum(x * lo, x * hi).sum(-1) for x in q.reshape(-1, D)]).amax(0) if new else \
                    torch.full((count,), -math.inf, dtype=torch.float64, device=dev)
                if new:
                    s[(n - new) // ps:] = math.inf
                best = sorted(range(count), key=lambda j, s=s.tolist(): (-s[j], j))[:c["n_sel"]]
                mine = torch.tensor(sorted(best), device=dev, dtype=torch.long)
                sel[b, h, :len(best)] = mine.int()
            if not new:
                continue
            k, v = (st[w + "_pages"][ids[mine], h].double() for w in ("k", "v"))
            if st["k_scales"] is not None:
                k = k * st["k_scales"][ids[mine], h].double()[..., None]
                v = v * st["v_scales"][ids[mine], h].double()[..., None]
            k, v = k.reshape(-1, D), v.reshape(-1, D)
            pos = (mine[:, None] * ps + torch.arange(ps, device=dev)).reshape(-1)
            for i in range(new):
                seen = pos < (n - new + i + 1 if c["causal"] else n)
                s = torch.where(seen, q[i] @ k.T / math.sqrt(D), -math.inf)
                m = s.max(-1, keepdim=True).values
                if not bool(torch.isfinite(m).all()):
                    continue
                e = torch.exp(s - m)
                tot = e.sum(-1, keepdim=True)
                out[b, i, heads] = e @ torch.where(seen[:, None], v, 0.0) / tot
                lse[b, i, heads] = (m + torch.log(tot))[:, 0]
    return {"out": out, "lse": lse} if c["op"] == "decode" else {"selected": sel, "out": out, "lse": lse}
