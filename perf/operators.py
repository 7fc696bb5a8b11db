"""Cases of the chunk operators over the paged K/V cache: what is run, on which inputs, and the operators' plain forms.

The cache is a pool of 64-token pages; inside a page the (layer, kv head) chunks follow each other, a K region then a V region, each fp16, Q8_0
or FP8 (e4m3) in the framework's page layout. The operators: the plan of a ragged batch of new tokens (offsets, positions, pages, slots), the
append (rotary embedding, encoding, scatter into pages), the read-back of cached tokens, and the attention of the new tokens over their pages."""
import math
import random

import torch

own = False

HD = 128
PAGE = 64
F16, Q8, FP8 = 0, 1, 2
REGION = {F16: 16384, Q8: 8704, FP8: 8192}
THETA = 1e6
SECTIONS = {1: (64,), 3: (16, 24, 24)}
DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _case(op, name=None, **kw):
    c = {"op": op, "R": 1, "new_lo": 1, "new_hi": 1, "ctx_lo": 0, "ctx_hi": 0, "mix": 1, "n_q": 32, "n_kv": 8, "layers": 2, "layer": 1,
         "k_type": F16, "v_type": F16, "io": "f16", "inp": "f32", "axes": 1, "causal": True, "window": 0, "holes": False}
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step's bookkeeping for a full batch of 32 sequences: a launch's latency
        _case("plan", "plan step 32", R=32, ctx_lo=800, ctx_hi=30000, mix=3),
        # admission of a thousand ragged prompts at once: about a million tokens, bound by the writes
        _case("plan", "plan prompts 1024", R=1024, new_lo=1, new_hi=8192, ctx_hi=8192, mix=4),
        # eight sequences' next tokens into an fp16 cache, from the fp32 projections
        _case("append", "append step 8 f16", R=8, ctx_lo=800, ctx_hi=30000, mix=5),
        # long prompts into an FP8 cache, bf16 projections
        _case("append", "append prompts fp8", R=3, new_lo=3001, new_hi=8000, mix=6, k_type=FP8, v_type=FP8, io="bf16", inp="bf16"),
        # a prompt with images: three rotary axes; Q8_0, and the rows read back
        _case("append", "append image q8_0", R=2, new_lo=1207, new_hi=1331, ctx_lo=3, ctx_hi=700, mix=7, k_type=Q8, v_type=Q8, inp="f16", axes=3),
        # a few cached tokens in any order, some of them without a page; K and V of different types
        _case("read", "read 77 fp8/q8_0", R=1, new_lo=77, new_hi=77, mix=8, k_type=FP8, v_type=Q8, holes=True),
        # a long prefix out of a Q8_0 cache
        _case("read", "read 30000 q8_0", R=1, new_lo=30000, new_hi=30000, mix=9, k_type=Q8, v_type=Q8),
        # one sequence's next token over 2048 cached ones: latency
        _case("attention", "attention step 1 f16", R=1, ctx_lo=2048, ctx_hi=2048, mix=10),
        # the swarm: eight sequences of 800 to 30000 tokens, one new token each
        _case("attention", "attention step 8 q8_0", R=8, ctx_lo=800, ctx_hi=30000, mix=11, k_type=Q8, v_type=Q8, io="bf16"),
        # a 2048-token chunk of a long prompt: the tensor cores' rate
        _case("attention", "attention chunk 2048 f16", R=1, new_lo=2048, new_hi=2048, ctx_lo=30000, ctx_hi=30000, mix=12),
        # prompts and single tokens in one batch, a sliding window, an FP8 cache
        _case("attention", "attention mixed fp8", R=12, new_lo=1, new_hi=1500, ctx_hi=4000, mix=13, k_type=FP8, v_type=FP8, io="bf16", window=1024),
        # queries of five requests over another stream's states (no causal mask), eight query heads per kv head
        _case("attention", "attention cross f16", R=5, new_lo=33, new_hi=700, ctx_lo=1, ctx_hi=1500, mix=14, n_q=16, n_kv=2, causal=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "read", "attention", "attention", "attention"])
    mix = rng.randrange(1 << 20)
    n_kv = rng.choice([1, 2, 4, 8])
    kt, vt = rng.choice([(F16, F16), (F16, F16), (FP8, FP8), (Q8, Q8), (F16, FP8), (FP8, F16), (Q8, F16)])
    c = _case(op, mix=mix, n_kv=n_kv, n_q=n_kv * rng.choice([1, 2, 4, 4, 8]), layers=rng.choice([1, 2, 3]), layer=0, k_type=kt, v_type=vt)
    c["layer"] = rng.randrange(c["layers"])
    if op == "plan":
        hi = _log(rng, 1, 8000)
        c.update(R=_log(rng, 1, 1024), new_lo=rng.choice([0, 1, hi]), new_hi=hi, ctx_hi=_log(rng, 1, 8192))
    elif op == "append":
        hi = _log(rng, 1, 4000)
        c.update(R=_log(rng, 1, 4), new_lo=rng.choice([1, hi]), new_hi=hi, ctx_hi=_log(rng, 1, 8192), io=rng.choice(["f16", "bf16"]),
                 inp=rng.choice(["f32", "f16", "bf16"]), axes=rng.choice([1, 3]))
    elif op == "read":
        hi = _log(rng, 1, 30000)
        c.update(R=1, new_lo=hi, new_hi=hi, holes=rng.choice([False, True]))
    else:
        # a rounded Q8_0 code times its scale reaches the tensor cores in fp16: bf16 outputs there
        c["io"] = "bf16" if Q8 in (kt, vt) else rng.choice(["f16", "bf16"])
        hi = _log(rng, 1, 1500)
        R = max(1, min(_log(rng, 1, 32), 6000 // hi)) if hi > 1 else _log(rng, 1, 32)
        most = min(30000, 2_000_000_000 // (R * hi * max(c["n_q"], 8)) - hi)
        c.update(R=R, new_lo=rng.choice([1, hi]), new_hi=hi, ctx_hi=_log(rng, 1, max(1, most)), causal=rng.random() < 0.8)
        if c["causal"] and rng.random() < 0.3:
            c["window"] = _log(rng, 1, 4096)
    return c


def _lengths(c):
    """(cached, new) tokens of each request: the first of each the largest, the others spread over the range's logarithm."""
    r = random.Random(c["mix"])
    pick = lambda lo, hi: _log(r, max(lo, 1), max(hi, 1)) if r.random() < 0.9 or lo > 0 else lo  # noqa: E731
    new = [c["new_hi"]] + [pick(c["new_lo"], c["new_hi"]) for _ in range(c["R"] - 1)]
    ctx = [c["ctx_hi"]] + [min(c["ctx_hi"], pick(c["ctx_lo"], c["ctx_hi"])) for _ in range(c["R"] - 1)]
    return ctx, new


def _kv_lengths(c):
    """Keys of each request's attention: cached and new ones, or (no causal mask) the other stream's states."""
    ctx, new = _lengths(c)
    return [a + b for a, b in zip(ctx, new)] if c["causal"] else ctx


def _pairs(c):
    """Visible (query, key) pairs of one head and keys that some query sees, over all requests."""
    pairs = keys = 0
    for n, kv in zip(_lengths(c)[1], _kv_lengths(c)):
        if not c["causal"]:
            pairs, keys = pairs + n * kv, keys + kv
            continue
        a, w = kv - n, c["window"] or kv + 1
        first = max(0, a + 1 - w)
        keys += kv - first
        short = max(0, min(n, w - a))  # queries that the window does not cut
        pairs += short * a + short * (short + 1) // 2 + (n - short) * w
    return pairs, keys


def work(c):
    T = sum(_lengths(c)[1])
    tok = c["n_kv"] * (REGION[c["k_type"]] + REGION[c["v_type"]]) / PAGE  # bytes of one cached token
    if c["op"] == "plan":
        pages = sum(-(-(a + n) // PAGE) - -(-a // PAGE) for a, n in zip(*_lengths(c)))
        return {"bytes": 16 * c["R"] + 12 * T + 8 * pages, "flops": 0}
    if c["op"] == "append":
        size = 4 if c["inp"] == "f32" else 2
        return {"bytes": T * ((c["n_q"] + 2 * c["n_kv"]) * HD * size + c["n_q"] * HD * 2 + tok), "flops": T * (c["n_q"] + c["n_kv"]) * HD * 3}
    if c["op"] == "read":
        return {"bytes": T * (tok + 4 * c["n_kv"] * HD), "flops": 0}
    pairs, keys = _pairs(c)
    return {"bytes": 4 * T * c["n_q"] * HD + keys * tok, "flops": 4 * HD * c["n_q"] * pairs}


# ------------------------------------------------------------------ inputs
def _gen(c, seed):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + c["mix"])


def _values(kind, shape, g):
    """Random rows of a cached tensor as the cache holds them: (codes, scales or None)."""
    x = torch.randn(shape, generator=g, device=DEV).half()
    return _encode(kind, x)


def _encode(kind, x):
    """fp16 rows [..., 128] in storage form: fp16; e4m3 bytes (saturating); Q8_0 bytes (code + 128) and fp16 scales of 32."""
    if kind == F16:
        return x, None
    if kind == FP8:
        return x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), None
    b = x.float().unflatten(-1, (4, 32))
    d = b.abs().amax(-1, keepdim=True) / 127
    q = torch.where(d > 0, b / torch.where(d > 0, d, 1), 0).round().clamp(-127, 127) + 128
    return q.to(torch.uint8).flatten(-2), d.squeeze(-1).half()


def _decode(kind, codes, scales, to=torch.float32):
    if kind == F16:
        return codes.to(to)
    if kind == FP8:
        return codes.view(torch.float8_e4m3fn).to(to)
    return ((codes.to(to) - 128).unflatten(-1, (4, 32)) * scales.to(to).unsqueeze(-1)).flatten(-2)


def _pages(c, lengths, g):
    """Block tables of sequences of these lengths (pages in any order; -1 behind the last) and the number of pages."""
    n = [-(-x // PAGE) for x in lengths]
    total, width = sum(n) + 3, max(max(n), 1)
    order = torch.randperm(total, generator=g, device=DEV)
    ends = torch.tensor(n, device=DEV).cumsum(0)
    j = torch.arange(width, device=DEV)[None]
    counts = torch.tensor(n, device=DEV)[:, None]
    at = (ends[:, None] - counts + j).clamp(max=total - 1)
    return torch.where(j < counts, order[at], -1).int(), total


def _inputs(c, seed):
    """Everything of a case that its seed makes, before the cache's layout: the same tensors for prepare() and exact()."""
    g = _gen(c, seed)
    ctx, new = _lengths(c)
    T = sum(new)
    s = {"T": T, "ctx": torch.tensor(ctx, device=DEV, dtype=torch.int32), "new": torch.tensor(new, device=DEV, dtype=torch.int32)}
    if c["op"] == "plan":
        need = [-(-(a + n) // PAGE) for a, n in zip(ctx, new)]
        held = torch.tensor([-(-a // PAGE) for a in ctx], device=DEV)[:, None]
        width, total = max(need) + 1, sum(need) + 5
        order = torch.randperm(total, generator=g, device=DEV).int()
        j = torch.arange(width, device=DEV)[None]
        at = (held.cumsum(0) - held + j).clamp(max=total - 1)
        s["tables"] = torch.where(j < held, order[at], -1).int()
        s["free"] = order[int(held.sum()):].contiguous()
        return s
    lengths = _kv_lengths(c) if c["op"] == "attention" else [a + n for a, n in zip(ctx, new)]
    s["tables"], s["n_pages"] = _pages(c, lengths, g)
    s["kv_len"] = torch.tensor(lengths, device=DEV, dtype=torch.int32)
    s["cu"] = torch.cat([s["new"].new_zeros(1), s["new"].cumsum(0).int()])
    row = torch.repeat_interleave(torch.arange(c["R"], device=DEV), s["new"], output_size=T)
    pos = torch.arange(T, device=DEV) - s["cu"][row] + s["ctx"][row]
    if c["op"] != "attention":
        page = s["tables"][row, pos // PAGE].long()
        s["slots"] = page * PAGE + pos % PAGE
    if c["op"] == "append":
        s["pos"] = pos.int()[None].repeat(c["axes"], 1)
        if c["axes"] > 1:  # an image's rows and columns beside the time axis
            s["pos"][1:] += torch.randint(0, 64, (c["axes"] - 1, T), generator=g, device=DEV).int()
        s["qkv"] = torch.randn(T, (c["n_q"] + 2 * c["n_kv"]) * HD, generator=g, device=DEV).to(DTYPE[c["inp"]])
        return s
    if c["op"] == "read":
        s["slots"] = s["slots"][torch.randperm(T, generator=g, device=DEV)] if c["holes"] else s["slots"]
        if c["holes"]:
            s["slots"] = torch.where(torch.rand(T, generator=g, device=DEV) < 0.1, -1, s["slots"])
    # the cached tokens, each page's 64 of them in order
    shape = (s["n_pages"] * PAGE, c["n_kv"], HD)
    s["k"], s["v"] = _values(c["k_type"], shape, g), _values(c["v_type"], shape, g)
    if c["op"] == "attention":
        s["q"] = (1.3 * torch.randn(T, c["n_q"], HD, generator=g, device=DEV)).to(DTYPE[c["io"]])
    return s


def prepare(c, seed):
    s = _inputs(c, seed)
    s["case"] = c
    if c["op"] == "plan":
        i32 = dict(device=DEV, dtype=torch.int32)
        s.update(cu=torch.zeros(c["R"] + 1, **i32), kv_len=torch.zeros(c["R"], **i32), positions=torch.zeros(s["T"], **i32),
                 slots=torch.zeros(s["T"], device=DEV, dtype=torch.int64), taken=torch.zeros(2, **i32))
        return s
    page_bytes = c["layers"] * c["n_kv"] * (REGION[c["k_type"]] + REGION[c["v_type"]])
    s["pool"] = torch.zeros(s["n_pages"], page_bytes, device=DEV, dtype=torch.uint8)
    if "k" in s:
        every = torch.arange(s["n_pages"] * PAGE, device=DEV)
        _put(c, s["pool"], every, 0, *s.pop("k"))
        _put(c, s["pool"], every, 1, *s.pop("v"))
    if c["op"] == "append":
        s["q"] = torch.zeros(s["T"], c["n_q"], HD, device=DEV, dtype=DTYPE[c["io"]])
    if c["op"] in ("append", "read"):
        s["k_out"] = torch.zeros(s["T"], c["n_kv"], HD, device=DEV, dtype=torch.float16)
        s["v_out"] = torch.zeros_like(s["k_out"])
    if c["op"] == "attention":
        s["o"] = torch.zeros_like(s["q"])
    return s


# ------------------------------------------------------------------ plain forms
def _at(c, slots, v):
    """Bytes' places in the pool of K (v = 0) or V (v = 1) of these slots: elements [T, n_kv, 128] and scales [T, n_kv, 4]."""
    kind = c["v_type" if v else "k_type"]
    kb, vb = REGION[c["k_type"]], REGION[c["v_type"]]
    t = (slots % PAGE)[:, None, None]
    d = torch.arange(HD, device=DEV)
    b = torch.arange(4, device=DEV)
    head = torch.arange(c["n_kv"], device=DEV)[:, None] + c["layer"] * c["n_kv"]
    base = (slots // PAGE)[:, None, None] * (c["layers"] * c["n_kv"] * (kb + vb)) + head * (kb + vb) + v * kb
    if not v:
        e = t * 256 + (((d >> 3) ^ (t & 7)) << 4) + ((d & 7) << 1) if kind == F16 else t * 128 + (((d >> 4) ^ (t & 7)) << 4) + (d & 15)
        return base + e, base + 8192 + t * 8 + b * 2
    u = t & 31
    if kind == F16:
        e = ((t >> 5) * 128 + d) * 64 + (((u >> 3) ^ ((d >> 1) & 3)) << 4) + ((u & 7) << 1)
    else:
        e = ((t >> 5) * 128 + d) * 32 + (((u >> 4) ^ ((d >> 2) & 1)) << 4) + (u & 15)
    return base + e, base + 8192 + (((t >> 5) * 4 + b) * 32 + u) * 2


def _put(c, pool, slots, v, codes, scales):
    e, sc = _at(c, slots, v)
    if codes.dtype == torch.float16:
        pool.view(torch.float16).view(-1)[e >> 1] = codes
        return
    pool.view(-1)[e] = codes
    if scales is not None:
        pool.view(torch.float16).view(-1)[sc >> 1] = scales


def _get(c, pool, slots, v):
    kind = c["v_type" if v else "k_type"]
    e, sc = _at(c, slots, v)
    if kind == F16:
        return pool.view(torch.float16).view(-1)[e >> 1].float()
    return _decode(kind, pool.view(-1)[e], pool.view(torch.float16).view(-1)[sc >> 1] if kind == Q8 else None)


def _plain_plan(s):
    ctx, new = s["ctx"].long(), s["new"].long()
    R, T = ctx.numel(), s["T"]
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    held, need = (ctx + PAGE - 1) // PAGE, (ctx + new + PAGE - 1) // PAGE
    fresh = need - held
    first = fresh.cumsum(0) - fresh
    tables = s["tables"]
    j = torch.arange(tables.shape[1], device=DEV)[None]
    mine = (j >= held[:, None]) & (j < need[:, None])
    at = (first[:, None] + j - held[:, None]).clamp(0, s["free"].numel() - 1)
    tables.copy_(torch.where(mine, s["free"][at], tables))
    t = torch.arange(T, device=DEV)
    row = torch.searchsorted(cu, t, right=True) - 1
    pos = ctx[row] + t - cu[row]
    page = tables[row, pos // PAGE].long()
    s["cu"].copy_(cu)
    s["kv_len"].copy_(ctx + new)
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(page >= 0, page * PAGE + pos % PAGE, -1))
    s["taken"].copy_(torch.stack([fresh.sum(), cu[R]]))
    return {"tables": tables, "cu": s["cu"], "kv_len": s["kv_len"], "positions": s["positions"], "slots": s["slots"], "taken": s["taken"]}


def _axis(c):
    return torch.repeat_interleave(torch.arange(c["axes"], device=DEV), torch.tensor(SECTIONS[c["axes"]], device=DEV))


def _plain_append(c, s):
    x = s["qkv"].float().unflatten(-1, (-1, HD))
    i = torch.arange(64, device=DEV, dtype=torch.float64)
    turn = (s["pos"][_axis(c)].T.double() * THETA ** (-i / 64))  # 64 bits: far positions
    cos, sin = turn.cos().float()[:, None], turn.sin().float()[:, None]
    a, b = x[:, : c["n_q"] + c["n_kv"], :64], x[:, : c["n_q"] + c["n_kv"], 64:]
    y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    s["q"].copy_(y[:, : c["n_q"]])
    _put(c, s["pool"], s["slots"], 0, *_encode(c["k_type"], y[:, c["n_q"]:].half()))
    _put(c, s["pool"], s["slots"], 1, *_encode(c["v_type"], x[:, c["n_q"] + c["n_kv"]:].half()))


def _plain_read(c, s):
    there = (s["slots"] >= 0)[:, None, None]
    at = s["slots"].clamp(min=0)
    s["k_out"].copy_(torch.where(there, _get(c, s["pool"], at, 0), 0))
    s["v_out"].copy_(torch.where(there, _get(c, s["pool"], at, 1), 0))


def _plain_attention(c, s):
    R, Hk, G = c["R"], c["n_kv"], c["n_q"] // c["n_kv"]
    most, kv = max(_lengths(c)[1]), max(_kv_lengths(c))
    new, kv_len, cu = s["new"].long(), s["kv_len"].long(), s["cu"].long()
    i, j = torch.arange(most, device=DEV), torch.arange(kv, device=DEV)
    live = i[None] < new[:, None]
    q = s["q"][(cu[:R, None] + i).clamp(max=s["T"] - 1)].float()                      # [R, most, n_q, 128]
    q = q.unflatten(2, (Hk, G)).permute(0, 2, 3, 1, 4).reshape(R, Hk, G * most, HD)
    page = s["tables"][:, j // PAGE].long()
    slots = (page * PAGE + j % PAGE).clamp(min=0).reshape(-1)
    there = (j < kv_len[:, None]) & (page >= 0)                                       # [R, kv]
    k = _get(c, s["pool"], slots, 0).view(R, kv, Hk, HD).permute(0, 2, 3, 1)
    p = (q @ k).mul_(HD ** -0.5).view(R, Hk, G, most, kv)
    del k, q
    see = there[:, None] & live[:, :, None]
    if c["causal"]:
        at = (kv_len - new)[:, None] + i
        see &= j <= at[:, :, None]
        if c["window"]:
            see &= j > (at - c["window"])[:, :, None]
    p.masked_fill_(~see[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(m > -math.inf, m, 0)).exp_()
    p.div_(p.sum(-1, keepdim=True).clamp(min=1e-30))
    v = torch.where(there[:, :, None, None], _get(c, s["pool"], slots, 1).view(R, kv, Hk, HD), 0).transpose(1, 2)
    o = (p.view(R, Hk, G * most, kv) @ v).view(R, Hk, G, most, HD).permute(0, 3, 1, 2, 4).reshape(R, most, c["n_q"], HD)
    s["o"].copy_(o[live])
    return {"o": s["o"]}


# ------------------------------------------------------------------ one pass
def _typed(c, s):
    """What an append left in the cache: the pool itself where every byte of it is a value, else the appended rows read back."""
    if c["k_type"] == c["v_type"] == F16:
        return {"q": s["q"], "pool": s["pool"].view(torch.float16)}
    if c["k_type"] == c["v_type"] == FP8:
        return {"q": s["q"], "pool": s["pool"].view(torch.float8_e4m3fn)}
    return {"q": s["q"], "k": s["k_out"], "v": s["v_out"]}


def _same_types(c):
    return c["k_type"] == c["v_type"] and c["k_type"] != Q8


def _own_run(c, s):
    import quantized_decode_step_02_gb300 as z

    if c["op"] == "plan":
        z.chunk_plan(s["ctx"], s["new"], s["tables"], s["cu"], s["kv_len"], s["positions"], s["slots"], s["taken"], free_pages=s["free"])
        return {k: s[k] for k in ("tables", "cu", "kv_len", "positions", "slots", "taken")}
    if "cache" not in s:  # a program keeps these
        s["cache"] = z.KVPool(s["pool"], c["layers"], c["n_kv"], (c["k_type"], c["v_type"]))
        if c["op"] == "attention":
            s["workspace"] = torch.empty(z.chunk_attention_workspace_bytes(c["n_q"], c["n_kv"]), dtype=torch.uint8, device=DEV)
    if c["op"] == "append":
        z.chunk_append(s["cache"], c["layer"], s["qkv"], s["pos"], s["slots"], s["q"], rope_theta=THETA, sections=SECTIONS[c["axes"]])
        if not _same_types(c):
            z.chunk_read(s["cache"], c["layer"], s["slots"], s["k_out"], s["v_out"])
        return _typed(c, s)
    if c["op"] == "read":
        z.chunk_read(s["cache"], c["layer"], s["slots"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    z.chunk_attention(s["cache"], c["layer"], s["q"], s["o"], s["cu"], s["kv_len"], s["tables"], s["workspace"], causal=c["causal"], window=c["window"])
    return {"o": s["o"]}


def run(s):
    c = s["case"]
    if own:
        return _own_run(c, s)
    if c["op"] == "plan":
        return _plain_plan(s)
    if c["op"] == "append":
        _plain_append(c, s)
        if not _same_types(c):
            _plain_read(c, s)
        return _typed(c, s)
    if c["op"] == "read":
        _plain_read(c, s)
        return {"k": s["k_out"], "v": s["v_out"]}
    return _plain_attention(c, s)


# ------------------------------------------------------------------ in 64 bits
def exact(c, seed):
    if c["op"] == "plan":
        return None
    s = _inputs(c, seed)
    if c["op"] == "append":
        x = s["qkv"].double().unflatten(-1, (-1, HD))
        z = torch.complex(x[..., :64], x[..., 64:])[:, : c["n_q"] + c["n_kv"]]
        angle = torch.stack([s["pos"][a].double() * (THETA ** (-2.0 * i / HD)) for i, a in enumerate(_axis(c).tolist())], 1)
        z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
        y = torch.cat([z.real, z.imag], -1)
        if _same_types(c):
            return {"q": y[:, : c["n_q"]], "pool": None}
        kept = {}
        for name, kind, r in (("k", c["k_type"], y[:, c["n_q"]:]), ("v", c["v_type"], x[:, c["n_q"] + c["n_kv"]:])):
            h = r.half()
            if kind == Q8:
                b = h.double().unflatten(-1, (4, 32))
                d = b.abs().amax(-1, keepdim=True) / 127
                h = ((b / d.clamp(min=1e-300)).round() * d.half().double()).flatten(-2)
            elif kind == FP8:
                h = h.double().clamp(-448, 448).float().to(torch.float8_e4m3fn)
            kept[name] = h.double()
        return {"q": y[:, : c["n_q"]], **kept}
    if c["op"] == "read":
        at, hole = s["slots"].clamp(min=0), (s["slots"] < 0)[:, None, None]
        return {n: _decode(c[n + "_type"], s[n][0][at], s[n][1][at] if s[n][1] is not None else None, torch.float64).masked_fill(hole, 0) for n in ("k", "v")}
    out = torch.zeros(s["T"], c["n_q"], HD, device=DEV, dtype=torch.float64)
    G = c["n_q"] // c["n_kv"]
    for r, (n, kv, t0) in enumerate(zip(_lengths(c)[1], _kv_lengths(c), s["cu"].tolist())):
        if n == 0 or kv == 0:
            continue
        pages = s["tables"][r, : -(-kv // PAGE)].long()
        at = (pages[:, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten()[:kv]
        i, j = torch.arange(n, device=DEV)[:, None] + kv - n, torch.arange(kv, device=DEV)
        hide = (j > i) | (j <= i - c["window"] if c["window"] else j < 0) if c["causal"] else None
        for h in range(c["n_kv"]):
            k, v = (_decode(c[x + "_type"], s[x][0][at, h], s[x][1][at, h] if s[x][1] is not None else None, torch.float64) for x in ("k", "v"))
            for g in range(h * G, h * G + G):
                w = s["q"][t0:t0 + n, g].double() @ k.T / math.sqrt(HD)
                out[t0:t0 + n, g] = (w.masked_fill(hide, -math.inf) if hide is not None else w).softmax(-1) @ v
    return {"o": out}
