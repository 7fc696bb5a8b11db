"""The chunk operators on the GPU: the plan of a ragged batch (exact), the
append (bit-exact encodings against the CPU oracle, rotations against 64-bit
angles), the read-back (exact), the attention of new tokens over their pages
against the formula in 64 bits, and a run of them together on a decoder's own
cache.  Pools start as 0xFF bytes (NaN in every type), so anything read that
was never written shows."""
import numpy as np
import pytest

import oracle
import synth
from synth.model import ModelDesc, make_kv_history, make_tokens
from tests.helpers import cached_model, gpu, needs_cuda

pytestmark = [gpu, needs_cuda]

torch = pytest.importorskip("torch")
import quantized_decode_step_02_gb300 as z  # noqa: E402

DEV = "cuda"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}     # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}   # half a subnormal step


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------- plan
def _plan_ref(ctx, new, tables, free, T):
    """The plan by the definition, in Python integers."""
    tables = [list(r) for r in tables]
    P = len(tables[0]) if tables else 1
    ctx, new = [max(0, c) for c in ctx], [max(0, n) for n in new]
    cu, pos, slots, taken = [0], [], [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        for pg in range(-(-c // 64), min(P, -(-(c + n) // 64))):
            if pg < P:
                if free is not None:
                    tables[r][pg] = free[taken] if taken < len(free) else -1
                taken += 1
        for i in range(n):
            p = c + i
            e = tables[r][p // 64] if p // 64 < P else -1
            pos.append(p)
            slots.append(e * 64 + p % 64 if e >= 0 else -1)
        cu.append(len(pos))
    pad = T - len(pos)
    return tables, cu, [c + n for c, n in zip(ctx, new)], pos + [-1] * pad, slots + [-1] * pad, [taken, cu[-1]]


PLANS = {
    "one token": ([70], [1], 4, 0, 0),
    "page start": ([64], [1], 4, 0, 0),
    "empty cache": ([0], [130], 4, 0, 0),
    "nothing new": ([5, 64, 0], [0, 0, 0], 2, 0, 3),
    "no request": ([], [], 1, 0, 2),
    "ragged": ([0, 63, 64, 65, 1000, 7], [1, 1, 64, 200, 0, 3], 30, 0, 7),
    "negative lengths count as none": ([-5, 3], [4, -2], 2, 0, 1),
    "short free list": ([0, 0, 10], [100, 300, 100], 8, 3, 0),
    "past the table": ([100, 0], [200, 10], 3, 0, 0),
    "many requests": ([(37 * i) % 500 for i in range(1300)], [(i * i) % 7 for i in range(1300)], 9, 0, 11),
    "long": ([3], [9000], 150, 0, 100),
}


@pytest.mark.parametrize("assign", [True, False])
@pytest.mark.parametrize("name", PLANS)
def test_plan(name, assign):
    ctx, new, P, cut, pad = PLANS[name]
    rng = np.random.default_rng(len(name))
    R = len(ctx)
    pages = rng.permutation(20000)
    tables = np.full((R, P), -1)
    used = 0
    for r in range(R):
        have = min(P, -(-max(0, ctx[r] + (0 if assign else max(0, new[r]))) // 64))
        tables[r, :have] = pages[used:used + have]
        used += have
    need = sum(max(0, min(P, -(-(max(0, c) + max(0, n)) // 64)) - min(P, -(-max(0, c) // 64))) for c, n in zip(ctx, new))
    free = pages[used:used + (cut or need + 2)].tolist() if assign else None
    T = sum(max(0, n) for n in new) + pad
    want = _plan_ref(ctx, new, tables.tolist(), free, T)
    t = i32(tables.reshape(R, P))
    cu, kv_len, taken = i32([-7] * (R + 1)), i32([-7] * R), i32([-7] * 2)
    pos, slots = i32([-7] * T), torch.full((T,), -7, dtype=torch.int64, device=DEV)
    z.chunk_plan(i32(ctx), i32(new), t, cu, kv_len, pos, slots, taken, free_pages=None if free is None else i32(free))
    got = [x.cpu().tolist() for x in (t, cu, kv_len, pos, slots, taken)]
    for g, w, what in zip(got, want, ("tables", "cu", "kv_len", "positions", "slots", "taken")):
        assert g == w, (name, what)


def test_plan_with_an_empty_free_list_gives_no_pages():
    t, cu, kv, taken = i32([[-1, -1]]), i32([0, 0]), i32([0]), i32([0, 0])
    pos, slots = i32([0] * 3), torch.zeros(3, dtype=torch.int64, device=DEV)
    z.chunk_plan(i32([0]), i32([3]), t, cu, kv, pos, slots, taken, free_pages=i32([]))
    assert t.tolist() == [[-1, -1]] and slots.tolist() == [-1] * 3 and taken.tolist() == [1, 3] and pos.tolist() == [0, 1, 2]


# ----------------------------------------------------------------- append
def _encode(kind, x16):
    """fp16 rows [..., 128] as the cache's values in 64 bits (zdec_kv_dtype's rules)."""
    if kind == z.KV_F16:
        return x16.double()
    if kind == z.KV_FP8:
        return x16.float().clamp(-448, 448).to(torch.float8_e4m3fn).double()
    b = x16.float().unflatten(-1, (4, 32))
    m = b.abs().amax(-1, keepdim=True)
    d = m / torch.full_like(m, 127.0)     # IEEE division (by a Python number torch multiplies by the reciprocal)
    q = torch.where(d > 0, b / torch.where(d > 0, d, 1.0), 0.0).round().clamp(-127, 127)
    return (q.double() * d.half().double()).flatten(-2)


ODESC = ModelDesc(n_layers=2, hidden=512, n_q_heads=8, n_kv_heads=2, head_dim=128, ffn=512, vocab=100)


def _special_rows(T, heads, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, heads, 128)) * 2).astype(np.float16)
    x[0, 0, :32] = 0.0
    x[0, 0, 32:64] = np.arange(-16, 16) * 0.5
    x[T // 2, 0, :32] = np.arange(32) + 0.5
    x[T // 2, 0, 0] = -127.0
    x[-1, -1, :32] = np.float16(6e-8)
    x[-1, -1, 64:96] = 65504.0
    x[-1, -1, 70] = -1.0
    return x


@pytest.mark.parametrize("types", [(0, 0), (1, 1), (2, 2), (0, 1), (2, 0), (1, 2)])
@pytest.mark.parametrize("start,n", [(0, 1), (5, 200), (64, 64), (61, 8)])
def test_append_encodes_bit_exact_into_a_decoders_cache(types, start, n):
    """Rows appended without rotation (position 0) land exactly where, and with
    the codes that, the decoder's own append gives them (oracle's encoders)."""
    d = ODESC
    dec = z.Decoder(d, cached_model(d, 5), types, max_B=2, max_L=300)
    cache = dec.cache()
    k0, v0 = make_kv_history(d, 3, 0, max(start, 1))
    if start:
        dec.append_kv(1, k0, v0)
    x = _special_rows(n, 4, start + n)                       # 2 key heads, 2 value heads
    dec.extend([1], [n])
    assert dec.seq_len(1) == start + n and dec.seq_len(0) == 0 and cache.lengths.tolist() == [0, start + n]
    cu, kv, taken, pos = i32([0] * 3), i32([0] * 2), i32([0] * 2), i32([0] * n)
    slots = torch.zeros(n, dtype=torch.int64, device=DEV)
    z.chunk_plan(i32([0, start]), i32([0, n]), cache.tables, cu, kv, pos, slots, taken)
    qkv = torch.from_numpy(x.reshape(n, -1)).to(DEV)
    z.chunk_append(cache, 1, qkv, torch.zeros_like(pos), slots, stream=cache.stream)
    dec.sync()
    got = dec.read_kv(1, 1, 0, start + n)
    for codes, scales, kind, src in ((got[0], got[2] if len(got) > 2 else None, types[0], x[:, :2]),
                                     (got[1], got[3] if len(got) > 2 else None, types[1], x[:, 2:])):
        for t in range(n):
            for g in range(2):
                h = src[t, g].view(np.uint16)
                if kind == z.KV_F16:
                    assert np.array_equal(codes[start + t, g], h), (t, g)
                elif kind == z.KV_Q8_0:
                    rs, rq = oracle.q8_0_quantize(h)
                    assert np.array_equal(scales[start + t, g], rs) and np.array_equal(codes[start + t, g], rq), (t, g)
                else:
                    assert np.array_equal(codes[start + t, g], [oracle.e4m3_from_half(int(e)) for e in h]), (t, g)
    # the tokens before, and the other layer, are as they were
    if start:
        ref = z.Decoder(d, cached_model(d, 5), types, max_B=2, max_L=300)
        ref.append_kv(1, k0, v0)
        for layer in range(2):
            a, b = dec.read_kv(1, layer, 0, start), ref.read_kv(1, layer, 0, start)
            for u, v in zip(a, b):
                assert u is None and v is None or np.array_equal(u, v)
        ref.close()
    dec.close()


def _new_pool(n_pages, layers, n_kv, types):
    return z.KVPool(torch.full((n_pages, z.page_bytes(types, layers, n_kv)), 255, dtype=torch.uint8, device=DEV), layers, n_kv, types)


@pytest.mark.parametrize("inp", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("qt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,n_q,n_kv,sections", [(1, 4, 1, (64,)), (67, 6, 3, (16, 24, 24)), (300, 32, 8, (64,)), (130, 1, 1, (1, 0, 63))])
def test_append_rotates(inp, qt, T, n_q, n_kv, sections):
    """Queries and fp16 keys against rotations by 64-bit angles, positions up to
    2^31 - 1 and negative ones; padding rows (slot -1) write no K/V."""
    g = torch.Generator(device=DEV).manual_seed(T)
    wide = torch.randn(T, (n_q + 2 * n_kv) * 128 + 40, generator=g, device=DEV).to(inp)
    qkv = wide[:, 8:8 + (n_q + 2 * n_kv) * 128] if inp != torch.float32 else wide[:, 4:4 + (n_q + 2 * n_kv) * 128]   # strided rows
    axes = len(sections)
    pos = torch.randint(0, 40000, (axes, T), generator=g, device=DEV).int()
    pos[0, 0] = 2 ** 31 - 1
    pos[-1, -1] = -3
    slots = torch.randperm(4 * ((T + 63) // 64) * 64, generator=g, device=DEV)[:T].contiguous()
    slots[T // 2] = -1 if T > 1 else slots[0]
    pool = _new_pool(4 * ((T + 63) // 64), 1, n_kv, (0, 0))
    q_wide = torch.full((T, n_q + 1, 128), 7.0, dtype=qt, device=DEV)
    q = q_wide[:, :n_q]
    z.chunk_append(pool, 0, qkv, pos if axes > 1 else pos[0], slots, q, rope_theta=1e4, sections=sections)
    k, v = (torch.empty(T, n_kv, 128, dtype=torch.float16, device=DEV) for _ in range(2))
    z.chunk_read(pool, 0, slots, k, v)
    x = qkv.double().unflatten(-1, (-1, 128))
    axis = torch.tensor([a for a, s in enumerate(sections) for _ in range(s)], device=DEV)
    ang = pos[axis].double().T * 1e4 ** (-torch.arange(64, dtype=torch.float64, device=DEV) / 64)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x[:, :n_q + n_kv, :64], x[:, :n_q + n_kv, 64:]
    y = torch.cat([a * c - b * s, b * c + a * s], -1)
    # the reference's own angle is off by up to 2^31 * 2^-52 = 2^-21; each of the kernel's products by its cos / sin
    # (2^-24 and their sum's rounding): 2^-22 of |a| + |b| covers the kernel, 2^-20 the reference at far positions
    size = torch.cat([a.abs() + b.abs()] * 2, -1)
    slack = size * torch.where(pos.max() > 2 ** 30, 2.0 ** -20, 2.0 ** -22)
    err = (q.double() - y[:, :n_q]).abs()
    assert (err <= U[qt] * y[:, :n_q].abs() + slack[:, :n_q] * (1 + U[qt]) + TINY[qt]).all()
    assert (q_wide[:, n_q] == 7.0).all()
    there = slots >= 0
    yk = y[there][:, n_q:]
    err = (k[there].double() - yk).abs()
    assert (err <= U[torch.float16] * yk.abs() + slack[there][:, n_q:] * (1 + 2.0 ** -11) + TINY[torch.float16]).all()
    assert torch.equal(v[there], x[there][:, n_q + n_kv:].half())
    assert (k[~there] == 0).all() and (v[~there] == 0).all()
    written = torch.zeros(pool.pages.shape[0] * 64, dtype=torch.bool, device=DEV)
    written[slots[there]] = True
    rest = torch.arange(written.numel(), device=DEV)[~written]
    k, v = (torch.empty(rest.numel(), n_kv, 128, dtype=torch.float16, device=DEV) for _ in range(2))
    z.chunk_read(pool, 0, rest, k, v)
    assert k.isnan().all() and v.isnan().all()       # nothing else was touched


def test_append_without_rotation_is_exact():
    T, pool = 5, _new_pool(1, 1, 1, (0, 0))
    qkv = torch.randn(T, 3 * 128, device=DEV).half()
    q = torch.empty(T, 1, 128, dtype=torch.float16, device=DEV)
    slots = torch.arange(T, device=DEV)
    z.chunk_append(pool, 0, qkv, i32([9, 8, 7, 6, 5]), slots, q, rope_theta=0.0)
    k, v = torch.empty_like(q), torch.empty_like(q)
    z.chunk_read(pool, 0, slots, k, v)
    assert torch.equal(torch.cat([q, k, v], 1).view(T, -1), qkv)


def test_slots_past_the_pool_are_skipped_and_reported():
    pool, status = _new_pool(2, 1, 2, (0, 2)), i32([0])
    slots = torch.tensor([0, 128, -5, 2 ** 40, 127], device=DEV)
    qkv = torch.ones(5, 4 * 128, device=DEV)
    z.chunk_append(pool, 0, qkv, i32([0] * 5), slots, status=status)
    assert status.item() == z.CHUNK_BAD_SLOT
    status.zero_()
    k, v = (torch.empty(5, 2, 128, dtype=torch.float16, device=DEV) for _ in range(2))
    z.chunk_read(pool, 0, slots, k, v, status=status)
    assert status.item() == z.CHUNK_BAD_SLOT
    for r, want in enumerate([1, 0, 0, 0, 1]):
        assert (k[r] == want).all() and (v[r] == want).all()


# ------------------------------------------------------------------- read
@pytest.mark.parametrize("types", [(0, 0), (1, 1), (2, 2), (0, 1), (1, 2), (2, 0)])
@pytest.mark.parametrize("T,n_kv,order", [(1, 1, "run"), (200, 3, "run"), (77, 2, "any"), (129, 8, "holes")])
def test_read_gives_the_cached_values(types, T, n_kv, order):
    g = torch.Generator(device=DEV).manual_seed(T)
    pages = (T + 70) // 64 + 2
    pool = _new_pool(pages, 2, n_kv, types)
    x = (2 * torch.randn(T, 2 * n_kv * 128, generator=g, device=DEV)).half()
    slots = torch.arange(T, device=DEV) + 3 if order == "run" else torch.randperm(pages * 64, generator=g, device=DEV)[:T].contiguous()
    z.chunk_append(pool, 1, x, i32([0] * T), slots, rope_theta=0.0)
    take = torch.where(torch.rand(T, generator=g, device=DEV) < 0.2, -1, slots) if order == "holes" else slots
    k, v = (torch.empty(T, n_kv, 128, dtype=torch.float16, device=DEV) for _ in range(2))
    z.chunk_read(pool, 1, take, k, v)
    rows = x.view(T, 2, n_kv, 128)
    for got, kind, src in ((k, types[0], rows[:, 0]), (v, types[1], rows[:, 1])):
        want = _encode(kind, src).half()       # code * scale is exact in 64 bits: one rounding
        same = got == torch.where((take >= 0)[:, None, None], want, 0)
        assert bool(same.all()), (~same).nonzero()[:5].tolist()


# -------------------------------------------------------------- attention
class Batch:
    """R requests with kv cached tokens and n new ones each, over a pool of pages in random order."""

    def __init__(self, lens, n_q, n_kv, types, io, seed=1, layers=2, spread=1.3, poison=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.n_q, self.n_kv, self.types = lens, n_q, n_kv, types
        n = [-(-kv // 64) for kv, _ in lens]
        order = torch.randperm(sum(n) + 2, generator=g, device=DEV).int()
        self.pool = _new_pool(sum(n) + 2, layers, n_kv, types)
        self.tables = torch.full((len(lens), max(max(n), 1) + 1), -1, dtype=torch.int32, device=DEV)
        self.k, self.v = [], []
        at = 0
        for r, (kv, _) in enumerate(lens):
            self.tables[r, :n[r]] = order[at:at + n[r]]
            x = torch.randn(kv, 2, n_kv, 128, generator=g, device=DEV).half()
            if poison:
                poison(r, x)
            j = torch.arange(kv, device=DEV)
            slots = self.tables[r, j // 64].long() * 64 + j % 64
            z.chunk_append(self.pool, layers - 1, x.flatten(1), torch.zeros(kv, dtype=torch.int32, device=DEV), slots, rope_theta=0.0)
            self.k.append(_encode(types[0], x[:, 0]))
            self.v.append(_encode(types[1], x[:, 1]))
            at += n[r]
        self.T = sum(m for _, m in lens)
        self.cu = i32(np.cumsum([0] + [m for _, m in lens]))
        self.kv_len = i32([kv for kv, _ in lens])
        self.layer = layers - 1
        self.q = (spread * torch.randn(self.T, n_q, 128, generator=g, device=DEV)).to(io)
        self.ws = torch.full((z.chunk_attention_workspace_bytes(n_q, n_kv),), 255, dtype=torch.uint8, device=DEV)

    def run(self, causal=True, window=0, scale=None, q=None, o=None, status=None, stream=None):
        q = self.q if q is None else q
        o = torch.full_like(q, 5.0) if o is None else o
        z.chunk_attention(self.pool, self.layer, q, o, self.cu, self.kv_len, self.tables, self.ws, causal=causal, window=window, scale=scale,
                          status=status, stream=stream)
        return o

    def check(self, o, causal=True, window=0, scale=None, drop=None):
        """Element by element against the formula in 64 bits.  With p the true
        probabilities: scores are off by ds (the fp32 sums over 128 products
        and the scaling, 2^-16 of sum |q k|, and half a step of fp16 on a Q8_0
        key), each p by 2 ds + 2^-11 (its own rounding to fp16), a Q8_0 value
        by 2^-11; the output is rounded once.  Probabilities below 2^-24 of a
        row's running maximum (which lags the final one by at most 2^8) may
        vanish: 2^-16 of the keys' values, weighted 2^-24 each."""
        scale = 128 ** -0.5 if scale is None else scale
        G = self.n_q // self.n_kv
        t0 = 0
        for r, (kv, n) in enumerate(self.lens):
            i, j = torch.arange(n, device=DEV)[:, None] + kv - n, torch.arange(kv, device=DEV)
            see = (j <= i) & ((j > i - window) if window else (j >= 0)) if causal else torch.ones(n, kv, dtype=torch.bool, device=DEV)
            if drop is not None:
                see = see & ~drop(r, j)[None]
            for h in range(self.n_q):
                k, v = self.k[r][:, h // G], self.v[r][:, h // G]
                q = self.q[t0:t0 + n, h].double()
                got = o[t0:t0 + n, h].double()
                some = see.any(1)
                s = (q @ k.T * scale).masked_fill(~see, -torch.inf)
                p = torch.where(some[:, None], s, 0.0).softmax(-1) * see if kv else s
                vs = torch.where(see.any(0)[:, None], v, 0.0)       # values that nothing sees have no influence
                y, pv = p @ vs, p @ vs.abs()
                u_k = 2.0 ** -11 if self.types[0] == z.KV_Q8_0 else 0.0
                u_v = 2.0 ** -11 if self.types[1] == z.KV_Q8_0 else 0.0
                ds = ((2.0 ** -16 + u_k) * scale * (q.abs() @ k.abs().T)).masked_fill(~see, 0)
                ds = ds.amax(1, keepdim=True) if kv else y
                rel = 2 * ds + 2.0 ** -11 + u_v + 2.0 ** -16
                tol = U[self.q.dtype] * y.abs() + 1.05 * rel * pv + 2.0 ** -24 * vs.abs().sum(0) + TINY[self.q.dtype]
                bad = (got - y).abs() > tol
                assert not bad.any() and got.isfinite().all(), (r, h, kv, n, int(bad.sum()), bad.nonzero()[:4].tolist(),
                                                                float(((got - y).abs() / tol).max()))
            t0 += n


PAIRS = [(0, 0), (1, 1), (2, 2), (0, 1), (1, 2), (2, 0)]


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("io", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens", [[(1, 1)], [(65, 1), (700, 1), (64, 1)], [(200, 70), (33, 33), (129, 1)]], ids=["one", "steps", "mixed"])
def test_attention_types(types, io, lens):
    b = Batch(lens, 8, 2, types, io, seed=len(lens))
    b.check(b.run())


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (3, 1), (8, 8), (16, 2), (10, 2), (64, 1)])
@pytest.mark.parametrize("lens", [[(300, 131), (17, 2)]])
def test_attention_head_layouts(n_q, n_kv, lens):
    b = Batch(lens, n_q, n_kv, (0, 0), torch.float16, seed=n_q)
    b.check(b.run())


LENS = {"chunk at the start": [(257, 257)], "empty requests": [(0, 0), (5, 0), (0, 0), (64, 3), (9, 0)], "long step": [(9000, 1)],
        "many": [(1 + (i * 37) % 300, 1 + (i * 5) % 7 if 1 + (i * 37) % 300 >= 7 else 1) for i in range(40)],
        "tiles": [(128, 128), (1000, 129), (640, 127), (64, 64)], "queries before the first key": [(3, 10), (0, 4), (130, 200)]}


@pytest.mark.parametrize("name", LENS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 100)])
def test_attention_lengths_and_masks(name, causal, window):
    b = Batch(LENS[name], 4, 1, (0, 0), torch.float16, seed=7)
    b.check(b.run(causal, window), causal, window)


@pytest.mark.parametrize("types", [(0, 0), (1, 1), (2, 2)])
@pytest.mark.parametrize("lens", [[(5000, 600)], [(30000, 3), (20, 20), (4000, 1)]])
def test_attention_long(types, lens):
    b = Batch(lens, 8, 2, types, torch.bfloat16, seed=11)
    b.check(b.run())
    b.check(b.run(True, 1500), True, 1500)


def test_attention_large_scores_and_a_scale():
    """Scores of hundreds (one key takes all), growing along the keys."""
    b = Batch([(900, 40)], 4, 1, (0, 0), torch.float16, seed=3, spread=30.0)
    b.check(b.run())
    b.check(b.run(scale=0.5), scale=0.5)
    b = Batch([(900, 40)], 4, 1, (0, 0), torch.bfloat16, seed=4, spread=1e4)
    b.check(b.run(scale=1e-5), scale=1e-5)


def test_attention_strided_rows_and_rows_behind_the_last():
    b = Batch([(100, 37), (70, 5)], 6, 2, (2, 2), torch.float16, seed=5)
    wide = torch.full((b.T + 9, 8, 128), 3.0, dtype=torch.float16, device=DEV)
    wide[:b.T, 1:7] = b.q
    out = torch.full((b.T + 9, 7, 128), 3.0, dtype=torch.float16, device=DEV)
    b.run(q=wide[:, 1:7], o=out[:, 1:])
    b.check(out[:b.T, 1:])
    assert (out[b.T:] == 3.0).all() and (out[:, 0] == 3.0).all()


def test_attention_tokens_past_T_are_left_out():
    b = Batch([(100, 37), (70, 20)], 4, 1, (0, 0), torch.float16, seed=6)
    full = b.run()
    short = b.run(q=b.q[:40].contiguous(), o=torch.full_like(b.q, 5.0)[:40])
    assert torch.equal(short, full[:40])


@pytest.mark.parametrize("types", [(0, 0), (2, 2), (1, 0)])
def test_attention_missing_pages_are_left_out(types):
    status = i32([0])
    b = Batch([(500, 90), (300, 1)], 4, 2, types, torch.float16, seed=8)
    assert (b.run(status=status) == b.run()).all() and status.item() == 0
    b.tables[0, 2] = -1
    b.tables[1, 0] = b.pool.pages.shape[0]
    b.tables[1, 4] = 2 ** 31 - 1
    o = b.run(status=status)
    assert status.item() == z.CHUNK_NO_PAGE
    gone = lambda r, j: (j // 64 == 2) if r == 0 else (j // 64 == 0) | (j // 64 == 4)  # noqa: E731
    b.check(o, drop=gone)


@pytest.mark.parametrize("types", [(0, 0), (2, 2), (0, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_non_finite_keys_and_values_stay_with_the_queries_that_see_them(types, bad):
    """A value (and key) that is not finite reaches the queries that see it and
    no other: tokens before it in the chunk (causal) and tokens whose window
    has passed it are as without it."""
    at, kv, n, window = 260, 400, 200, 90

    def poison(r, x):
        x[at, :, :, 17] = bad
        x[kv - 1, 1, :, 3] = bad

    clean = Batch([(kv, n)], 4, 2, types, torch.float16, seed=9)
    dirty = Batch([(kv, n)], 4, 2, types, torch.float16, seed=9, poison=poison)
    if types == (2, 2) and bad == float("inf"):
        pytest.skip("e4m3 saturates: an infinity is 448 there")
    for w in (0, window):
        a, b = clean.run(True, w), dirty.run(True, w)
        i = torch.arange(n, device=DEV) + kv - n
        sees = ((i >= at) & (i < at + w) if w else i >= at) | (i == kv - 1)
        # the same products in fp32, perhaps summed in another order (2^-16 of sum |p v|, at most max |v| < 5), each
        # then rounded to fp16 by half a step
        x, y = a[~sees].double(), b[~sees].double()
        assert y.isfinite().all() and ((x - y).abs() <= 2 * U[torch.float16] * x.abs() + 5 * 2.0 ** -15).all()
        k_bad = types[0] == 0 or bad != bad
        if k_bad:
            assert b[sees & (i < kv - 1)].isnan().any()


def test_attention_is_deterministic_and_captures():
    """The same bits call after call; a graph captured once replays with new
    lengths and queries, two graphs with their own workspaces on two streams."""
    b = Batch([(3000, 1), (800, 300), (64, 64)], 8, 2, (2, 2), torch.bfloat16, seed=10)
    first = b.run()
    for _ in range(3):
        assert torch.equal(b.run(), first)
    s = torch.cuda.Stream()
    o = torch.full_like(b.q, 5.0)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run(o=o)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            b.run(o=o)
    torch.cuda.synchronize()
    o.fill_(1.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, first)
    b.kv_len.copy_(i32([2000, 700, 64]))
    want = b.run()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and not torch.equal(want, first)


# --------------------------------------------------------------- together
@pytest.mark.parametrize("kv_dtype", [0, 1, 2, (1, 0)])
def test_prompts_by_chunks_then_decode_steps(kv_dtype):
    """Two prompts enter a decoder's cache chunk by chunk (extend, plan, append
    with rotation, attention over the pages), as a prefill does layer by layer;
    the cache then equals one filled by append_kv with the same rotated rows,
    bit for bit, the last chunk's attention matches the decoder's own, and a
    decode step gives the same logits."""
    d = ModelDesc(n_layers=2, hidden=512, n_q_heads=8, n_kv_heads=2, head_dim=128, ffn=512, vocab=300)
    w = cached_model(d, 51)
    a = z.Decoder(d, w, kv_dtype, max_B=3, max_L=400)
    b = z.Decoder(d, w, kv_dtype, max_B=3, max_L=400)
    cache = a.cache()
    stream = torch.cuda.ExternalStream(cache.stream)
    gen = torch.Generator(device=DEV).manual_seed(2)
    lens = [0, 0, 0]
    ws = torch.empty(z.chunk_attention_workspace_bytes(8, 2), dtype=torch.uint8, device=DEV)
    with torch.cuda.stream(stream):
        for new in ([70, 0, 33], [1, 0, 64], [100, 0, 1]):
            a.extend([0, 2], [new[0], new[2]])
            T = sum(new)
            ctx, n = i32(lens), i32(new)
            cu, kv, taken, pos = i32([0] * 4), i32([0] * 3), i32([0] * 2), i32([0] * T)
            slots = torch.zeros(T, dtype=torch.int64, device=DEV)
            z.chunk_plan(ctx, n, cache.tables, cu, kv, pos, slots, taken)
            assert torch.equal(kv, cache.lengths)
            rows = []
            for layer in range(2):
                qkv = torch.randn(T, 12 * 128, generator=gen, device=DEV)
                q, o = (torch.empty(T, 8, 128, dtype=torch.float16, device=DEV) for _ in range(2))
                z.chunk_append(cache, layer, qkv, pos, slots, q, rope_theta=d.rope_theta)
                z.chunk_attention(cache, layer, q, o, cu, kv, cache.tables, ws)
                # the same rows, rotated to fp16 on their own, for append_kv
                one = z.KVPool(torch.zeros((T + 63) // 64, z.page_bytes(z.KV_F16, 1, 2), dtype=torch.uint8, device=DEV), 1, 2)
                at = torch.arange(T, device=DEV)
                z.chunk_append(one, 0, qkv, pos, at, q, rope_theta=d.rope_theta)
                k16, v16 = (torch.empty(T, 2, 128, dtype=torch.float16, device=DEV) for _ in range(2))
                z.chunk_read(one, 0, at, k16, v16)
                rows.append((k16, v16, q, o))
            torch.cuda.synchronize()
            for s in (0, 2):
                lo, hi = cu[s].item(), cu[s + 1].item()
                k16 = torch.stack([r[0][lo:hi] for r in rows]).cpu().numpy().view(np.uint16)
                v16 = torch.stack([r[1][lo:hi] for r in rows]).cpu().numpy().view(np.uint16)
                b.append_kv(s, k16, v16)
            lens = [x + y for x, y in zip(lens, new)]
    assert [a.seq_len(i) for i in range(3)] == lens == [b.seq_len(i) for i in range(3)]
    for s in (0, 2):
        for layer in range(2):
            for x, y in zip(a.read_kv(s, layer, 0, lens[s]), b.read_kv(s, layer, 0, lens[s])):
                assert x is None and y is None or np.array_equal(x, y)
    # the last token of slot 0 by the decoder's own attention (rows are slots 0..B-1)
    q, o = rows[1][2], rows[1][3]
    t = cu[1].item() - 1
    ref = b.attention(1, q[t:t + 1].float().cpu().numpy(), [lens[0] - 1])[0]
    u = 2.0 ** -11 * (1 + 1 + 2 + 1)     # output and p rounded, Q8_0 keys (2 ds) and values; max |v| over the cached rows
    assert np.abs(o[t].float().cpu().numpy() - ref).max() <= u * 5.0
    toks = make_tokens(d, 9, 2)
    la, lb = np.empty((2, d.vocab), np.float32), np.empty((2, d.vocab), np.float32)
    pos2 = np.array([lens[0], lens[2]], np.int32)
    _, ia = a.step_host(toks, pos2, la, slots=[0, 2])
    _, ib = b.step_host(toks, pos2, lb, slots=[0, 2])
    assert np.array_equal(la, lb) and np.array_equal(ia, ib)
    a.close()
    b.close()


def test_extend_refuses_and_changes_nothing():
    d = ODESC
    dec = z.Decoder(d, cached_model(d, 5), z.KV_F16, max_B=3, max_L=200, pool_tokens=256)
    free = dec.info()["free_pages"]
    for slots, new, status in (([0, 0], [1, 1], -1), ([3], [1], -1), ([-1], [1], -1), ([0], [-1], -1), ([0], [201], -3),
                               ([0, 1], [200, 100], -3)):
        with pytest.raises(z.ZdecError) as e:
            dec.extend(slots, new)
        assert e.value.status == status, (slots, new)
        assert dec.info()["free_pages"] == free and [dec.seq_len(i) for i in range(3)] == [0, 0, 0]
        assert (dec.block_table(0) < 0).all()
    dec.extend([], [])
    dec.extend([0, 2], [65, 0])
    assert dec.info()["free_pages"] == free - 2 and dec.seq_len(0) == 65 and dec.seq_len(2) == 0
    dec.reset_seq(0)
    assert dec.info()["free_pages"] == free
    dec.close()


def test_wrong_tensors_are_refused():
    b = Batch([(70, 5)], 4, 1, (0, 0), torch.float16)
    o = torch.empty_like(b.q)
    call = lambda **kw: z.chunk_attention(**{**dict(cache=b.pool, layer=0, q=b.q, o=o, cu=b.cu, kv_len=b.kv_len, tables=b.tables,  # noqa: E731
                                                    workspace=b.ws), **kw})
    call()
    for kw in (dict(q=b.q.float()), dict(o=o.bfloat16()), dict(o=o[:3]), dict(cu=b.cu[:1]), dict(cu=b.cu.long()), dict(kv_len=b.kv_len.cpu()),
               dict(tables=b.tables[0]), dict(q=b.q.transpose(0, 1)), dict(q=b.q[:, :, :64]), dict(workspace=b.ws[:100]), dict(layer=2),
               dict(window=3, causal=False), dict(scale=-1.0), dict(tables=b.tables.T)):
        with pytest.raises(z.ZdecError):
            call(**kw)
    with pytest.raises(z.ZdecError):
        z.chunk_append(b.pool, 0, torch.zeros(2, 3 * 128, device=DEV), i32([0, 0]), torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(z.ZdecError):
        z.chunk_append(b.pool, 0, torch.zeros(2, 3 * 128, device=DEV), i32([0, 0]), torch.zeros(2, dtype=torch.int64, device=DEV))


# ------------------------------------- many tokens, many requests, extremes
@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("order", ["run", "any"])
def test_append_and_read_of_whole_tiles(types, order):
    """Enough tokens for CTAs of 64: codes on exact halves, zero blocks, the
    largest values (a Q8_0 product past fp16's top is read as 65504), runs of
    slots that start inside a 16-byte segment."""
    T, n_kv = 1300, 8
    g = torch.Generator(device=DEV).manual_seed(21)
    pages = T // 64 + 3
    pool = _new_pool(pages, 1, n_kv, types)
    x = (2 * torch.randn(T, 2 * n_kv, 128, generator=g, device=DEV)).half()
    half = torch.arange(32, device=DEV).half() - 15.5            # amax 127 / 64: scale 2^-6, every other value a tie
    half[0] = 127.0
    for at, e in ((7, 0), (64, -6), (700, 3), (T - 1, -12)):
        x[at, :, 32:64] = half * 2.0 ** e
        x[at, :, 96:] = -half * 2.0 ** e
    x[9, :, :64] = 0.0
    x[640:643, :, 64:96] = 65504.0
    x[640, :, 70] = -65504.0
    x[641, :, 0:32] = 6e-8
    slots = torch.arange(T, device=DEV) + 5 if order == "run" else torch.randperm(pages * 64, generator=g, device=DEV)[:T].contiguous()
    z.chunk_append(pool, 0, x.flatten(1), i32([0] * T), slots, rope_theta=0.0)
    k, v = (torch.empty(T, n_kv, 128, dtype=torch.float16, device=DEV) for _ in range(2))
    for take in (slots, slots.roll(3), torch.where(torch.arange(T, device=DEV) % 37 == 5, -1, slots)):
        z.chunk_read(pool, 0, take, k, v)
        rows = x.roll(3, 0) if take[0] == slots[-3] else x
        for got, kind, src in ((k, types[0], rows[:, :n_kv]), (v, types[1], rows[:, n_kv:])):
            want = _encode(kind, src).clamp(-65504, 65504).half()
            same = got == torch.where((take >= 0)[:, None, None], want, 0)
            assert bool(same.all()), (~same).nonzero()[:5].tolist()


def test_append_of_many_tokens_is_that_of_its_parts():
    """Thousands of tokens (two per warp) against calls of 700: the same bits."""
    T, n_q, n_kv = 5003, 5, 2
    g = torch.Generator(device=DEV).manual_seed(22)
    x = torch.randn(T, (n_q + 2 * n_kv) * 128, generator=g, device=DEV).bfloat16()
    pos = torch.randint(0, 10 ** 6, (T,), generator=g, device=DEV).int()
    slots = torch.randperm(T + 70, generator=g, device=DEV)[:T].contiguous()
    outs = []
    for step in (T, 700):
        pool = _new_pool((T + 70) // 64 + 1, 1, n_kv, (1, 2))
        q = torch.empty(T, n_q, 128, dtype=torch.bfloat16, device=DEV)
        for a in range(0, T, step):
            part = slice(a, min(a + step, T))
            z.chunk_append(pool, 0, x[part], pos[part].contiguous(), slots[part].contiguous(), q[part], rope_theta=1e6)
        outs.append((q, pool.pages))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("R,n_q,new,types", [(32, 4, 1, (2, 2)), (33, 4, 1, (0, 0)), (512, 2, 1, (1, 1)), (513, 2, 1, (2, 2)), (1100, 2, 1, (0, 0)),
                                             (520, 16, 9, (0, 0)), (530, 16, 9, (1, 2))])
def test_attention_of_many_requests(R, n_q, new, types):
    """Around 32 and 512 requests, where their weights are summed in another
    way; single tokens (row blocks of 128) and several (of 256)."""
    lens = [(new + (i * 37) % 150, 1 + (i * 5) % new if i % 3 else new) for i in range(R)]
    b = Batch(lens, n_q, 1, types, torch.float16, seed=R, layers=1)
    b.check(b.run())


def test_attention_with_a_length_past_the_table():
    """A kv_len above 64 * max_pages counts as that."""
    b = Batch([(128, 5), (100, 30)], 4, 1, (0, 0), torch.float16, seed=23)
    b.tables = b.tables[:, :2].contiguous()
    want = b.run()
    b.kv_len[0] = 5000
    status = i32([0])
    assert torch.equal(b.run(status=status), want) and status.item() == 0
    b.kv_len[0] = 2 ** 31 - 1
    assert torch.equal(b.run(status=status), want) and status.item() == 0


def test_attention_of_bf16_queries_of_any_size():
    """Rows from 2^-130 to 2^120 in one call (the largest brought into fp16's
    range row by row): small ones weigh their keys evenly, large ones as usual."""
    b = Batch([(300, 200), (90, 1), (70, 3)], 4, 2, (0, 1), torch.bfloat16, seed=24, spread=1.0)
    e = torch.tensor([-130, -60, 0, 60, 113, 120], device=DEV)[torch.arange(b.T * 4, device=DEV) % 6].view(b.T, 4, 1)
    b.q = (b.q.double() * 2.0 ** e).bfloat16()
    b.q[17] = 0.0
    b.check(b.run(scale=2.0 ** -120), scale=2.0 ** -120)


def test_attention_graphs_that_replay_together():
    """Two captured calls with their own workspaces, replayed on two streams at
    the same time, between eager calls on a third."""
    bs = [Batch([(3000, 1), (800, 1), (64, 1)], 8, 2, (2, 2), torch.bfloat16, seed=25), Batch([(1500, 300), (64, 64)], 8, 2, (0, 0), torch.float16, seed=26)]
    want = [b.run() for b in bs]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in bs], [], [torch.full_like(b.q, 5.0) for b in bs]
    for b, s, o in zip(bs, streams, outs):
        with torch.cuda.stream(s):
            b.run(o=o)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                b.run(o=o)
        graphs.append(g)
    third = Batch([(700, 40)], 4, 1, (1, 1), torch.float16, seed=27)
    alone = third.run()
    torch.cuda.synchronize()
    for _ in range(10):
        for o in outs:
            o.fill_(1.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = third.run()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, alone)


def test_queries_and_outputs_as_columns_of_one_matrix():
    """qkv, rotated queries and attention outputs side by side: allowed, and
    the same bits as with arrays of their own."""
    b = Batch([(100, 37), (70, 5)], 4, 2, (0, 0), torch.float16, seed=28)
    n = 4 * 128
    wide = torch.full((b.T, 8 * 128 + 2 * n), 3.0, dtype=torch.float16, device=DEV)
    wide[:, :8 * 128] = torch.randn(b.T, 8 * 128, device=DEV)
    pos, none = i32(range(b.T)), torch.full((b.T,), -1, dtype=torch.int64, device=DEV)
    q, o = wide[:, 8 * 128:8 * 128 + n].unflatten(1, (4, 128)), wide[:, 8 * 128 + n:].unflatten(1, (4, 128))
    z.chunk_append(b.pool, b.layer, wide[:, :8 * 128], pos, none, q, rope_theta=1e4)
    b.run(q=q, o=o)
    own = torch.empty(b.T, 4, 128, dtype=torch.float16, device=DEV)
    z.chunk_append(b.pool, b.layer, wide[:, :8 * 128].contiguous(), pos, none, own, rope_theta=1e4)
    assert torch.equal(q, own) and torch.equal(o, b.run(q=own))
