"""CPU checks of the chunk operators' boundary: sizes, and every refusal that
the host makes before it touches a GPU."""
import ctypes

import pytest

import quantized_decode_step_02_gb300 as z

P16 = ctypes.c_void_p(4096)      # an aligned address that no refused call follows
ODD = ctypes.c_void_p(4104)


def _pool(**kw):
    c = dict(base=4096, n_pages=4, n_layers=2, n_kv_heads=2, k_type=0, v_type=0)
    c.update(kw)
    return z._Pool(*(c[f] for f, _ in z._Pool._fields_))


def _msg():
    return z.load_library().zdec_last_global_error().decode()


def test_page_bytes():
    assert z.page_bytes(z.KV_F16, 36, 8) == 36 * 8 * 32768
    assert z.page_bytes((z.KV_Q8_0, z.KV_FP8), 2, 3) == 6 * (8704 + 8192)
    assert z.page_bytes(z.KV_F16, 0, 8) == 0 and z.page_bytes(3, 1, 1) == 0


POOL_FAULTS = [(dict(base=0), "null pool"), (dict(base=4104), "aligned"), (dict(k_type=3), "cache type"), (dict(v_type=-1), "cache type"),
               (dict(n_pages=0), "pool shape"), (dict(n_layers=0), "pool shape"), (dict(n_kv_heads=0), "pool shape")]


@pytest.mark.parametrize("fault,msg", POOL_FAULTS)
def test_bad_pools_are_refused_by_every_call(fault, msg):
    lib, p = z.load_library(), ctypes.byref(_pool(**fault))
    rope = z._Rope(1e6, 1, (ctypes.c_int * 4)(64))
    a = z._ChunkAttn(4, 1, 1, 1, 1, 1, 0, 0.1, 512, 512)
    assert lib.zdec_chunk_append(p, 0, ctypes.byref(rope), 1, 4, P16, 0, 1024, P16, P16, P16, 1, 512, None, None) == -1
    assert msg in _msg()
    assert lib.zdec_chunk_read(p, 0, 1, P16, P16, P16, None, None) == -1
    assert lib.zdec_chunk_attention(p, 0, ctypes.byref(a), P16, P16, P16, P16, P16, P16, 1 << 30, None, None) == -1
    assert msg in _msg()


@pytest.mark.parametrize("layer", [-1, 2])
def test_layers_out_of_range_are_refused(layer):
    lib, p = z.load_library(), ctypes.byref(_pool())
    assert lib.zdec_chunk_read(p, layer, 1, P16, P16, P16, None, None) == -1
    assert "layer" in _msg()


@pytest.mark.parametrize("fault,msg", [
    (dict(R=-1), "R must"), (dict(T=-1), "R must"), (dict(R=(1 << 20) + 1), "R must"), (dict(max_pages=0), "max_pages"),
    (dict(n_free=-1), "n_free"), (dict(ctx=None), "null"), (dict(cu=None), "null"), (dict(slots=None), "null"), (dict(taken=None), "null")])
def test_plan_refusals(fault, msg):
    c = dict(R=1, ctx=P16, new=P16, free=P16, n_free=1, tables=P16, max_pages=2, T=1, cu=P16, kv_len=P16, pos=P16, slots=P16, taken=P16)
    c.update(fault)
    assert z.load_library().zdec_chunk_plan(*c.values(), None) == -1
    assert msg in _msg()


@pytest.mark.parametrize("fault,msg", [
    (dict(theta=-1.0), "theta"), (dict(theta=float("nan")), "theta"), (dict(theta=float("inf")), "theta"), (dict(axes=0), "axes"),
    (dict(axes=5), "axes"), (dict(sections=(32, 31)), "sum"), (dict(sections=(65, -1)), "sections"), (dict(T=-1), "bad T"),
    (dict(in_type=3), "in_type"), (dict(q_type=0), "q_type"), (dict(qkv=None), "null"), (dict(q=None), "null"), (dict(qkv=ODD), "qkv rows"),
    (dict(ld=1023), "qkv rows"), (dict(ld=1028), "qkv rows"), (dict(q=ODD), "q rows"), (dict(q_ld=508), "q rows"), (dict(q_ld=504), "q rows")])
def test_append_refusals(fault, msg):
    c = dict(theta=1e6, axes=2, sections=(32, 32), T=1, nq=4, qkv=P16, in_type=0, ld=1024, q=P16, q_type=1, q_ld=512)
    c.update(fault)
    rope = z._Rope(c["theta"], c["axes"], (ctypes.c_int * 4)(*c["sections"]))
    s = z.load_library().zdec_chunk_append(ctypes.byref(_pool()), 0, ctypes.byref(rope), c["T"], c["nq"], c["qkv"], c["in_type"], c["ld"],
                                           P16, P16, c["q"], c["q_type"], c["q_ld"], None, None)
    assert s == -1 and msg in _msg()


def test_read_refusals():
    lib, p = z.load_library(), ctypes.byref(_pool())
    assert lib.zdec_chunk_read(p, 0, -1, P16, P16, P16, None, None) == -1
    assert lib.zdec_chunk_read(p, 0, 1, None, P16, P16, None, None) == -1 and "null" in _msg()
    assert lib.zdec_chunk_read(p, 0, 1, P16, ODD, P16, None, None) == -1 and "aligned" in _msg()
    assert lib.zdec_chunk_read(p, 0, 0, None, None, None, None, None) == 0      # nothing to do


@pytest.mark.parametrize("fault,status,msg", [
    (dict(n_q=0), -1, "multiple"), (dict(n_q=3), -1, "multiple"), (dict(n_q=130), -5, "heads per kv"), (dict(R=-1), -1, "R must"),
    (dict(T=-1), -1, "R must"), (dict(T=1 << 30), -5, "2^31"), (dict(max_pages=0), -1, "max_pages"), (dict(io=0), -1, "fp16 or bf16"),
    (dict(window=-1), -1, "window"), (dict(window=5, causal=0), -1, "window"), (dict(scale=0.0), -1, "scale"), (dict(scale=-1.0), -1, "scale"),
    (dict(scale=float("nan")), -1, "scale"), (dict(scale=float("inf")), -1, "scale"), (dict(q_ld=504), -1, "rows"), (dict(o_ld=516), -1, "rows"),
    (dict(q=None), -1, "null"), (dict(q=ODD), -1, "rows"), (dict(o=ODD), -1, "rows"), (dict(ws=None), -1, "workspace"),
    (dict(ws=ctypes.c_void_p(4096 + 128)), -1, "workspace"), (dict(ws_bytes=-1), -1, "too small")])
def test_attention_refusals(fault, status, msg):
    need = z.chunk_attention_workspace_bytes(4, 2)
    c = dict(n_q=4, R=1, T=1, max_pages=1, io=1, causal=1, window=0, scale=0.1, q_ld=512, o_ld=512, q=P16, o=P16, ws=P16, ws_bytes=0)
    c.update(fault)
    a = z._ChunkAttn(*(c[k] for k in ("n_q", "R", "T", "max_pages", "io", "causal", "window", "scale", "q_ld", "o_ld")))
    s = z.load_library().zdec_chunk_attention(ctypes.byref(_pool()), 0, ctypes.byref(a), P16, P16, P16, c["q"], c["o"], c["ws"],
                                              need + c["ws_bytes"], None, None)
    assert s == status and msg in _msg()


def test_empty_calls_need_nothing():
    lib, p = z.load_library(), ctypes.byref(_pool())
    a = z._ChunkAttn(4, 0, 0, 1, 1, 1, 0, 0.1, 512, 512)
    assert lib.zdec_chunk_attention(p, 0, ctypes.byref(a), None, None, None, None, None, None, 0, None, None) == 0
    rope = z._Rope(1e6, 1, (ctypes.c_int * 4)(64))
    assert lib.zdec_chunk_append(p, 0, ctypes.byref(rope), 0, 4, None, 0, 1024, None, None, None, 1, 512, None, None) == 0
    assert z.chunk_attention_workspace_bytes(4, 2) > 0
    assert z.chunk_attention_workspace_bytes(5, 2) == 0 and z.chunk_attention_workspace_bytes(0, 2) == 0


def test_context_calls_without_a_context():
    lib = z.load_library()
    assert lib.zdec_get_cache(None, None) == -1
    assert lib.zdec_extend(None, 0, None, None) == -1


def test_host_tensors_are_refused():
    torch = pytest.importorskip("torch")
    pages = torch.zeros(2, z.page_bytes(z.KV_F16, 1, 1), dtype=torch.uint8)
    with pytest.raises(z.ZdecError, match="CUDA tensor"):
        z.KVPool(pages, 1, 1)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(z.ZdecError, match="CUDA tensor"):
        z.chunk_plan(i, i, i[None], torch.zeros(2, dtype=torch.int32), i, i, i.long(), torch.zeros(2, dtype=torch.int32))


def test_overlapping_arrays_are_refused():
    lib, at = z.load_library(), lambda x: ctypes.c_void_p(1 << 20 | x)
    c = dict(R=100, ctx=at(0), new=at(4096), free=None, n_free=0, tables=at(8192), max_pages=2, T=10, cu=at(16384), kv_len=at(20480), pos=at(24576),
             slots=at(28672), taken=at(32768))
    for out, where in (("kv_len", 0), ("kv_len", 396), ("cu", 4096 + 8), ("taken", 4096 + 392), ("pos", 4096 - 4), ("slots", 392)):
        assert lib.zdec_chunk_plan(*{**c, out: at(where)}.values(), None) == -1 and "overlaps" in _msg(), (out, where)
    pool, rope = _pool(), z._Rope(1e6, 1, (ctypes.c_int * 4)(64))
    # (in type, ld, q, q_ld): in place; from the middle; the key columns of the same matrix; another stride
    for typ, ld, q, q_ld in ((1, 1024, 0, 1024), (1, 1024, 512, 1024), (1, 1024, 2 * 512, 1024), (0, 1024, 4 * 1000, 2048), (1, 2048, 2 * 2048 - 16, 512)):
        assert lib.zdec_chunk_append(ctypes.byref(pool), 0, ctypes.byref(rope), 7, 4, at(0), typ, ld, P16, P16, at(q), 1, q_ld, None, None) == -1
        assert "q overlaps qkv" in _msg(), (typ, ld, q, q_ld)
    for q_ld, o, o_ld in ((512, 0, 512), (1024, 1008, 1024), (1024, 2048 - 16, 1024), (1024, 1024, 512)):
        a = z._ChunkAttn(4, 1, 7, 1, 1, 1, 0, 0.1, q_ld, o_ld)
        assert lib.zdec_chunk_attention(ctypes.byref(pool), 0, ctypes.byref(a), P16, P16, P16, at(0), at(o), P16, 1 << 30, None, None) == -1
        assert "o overlaps q" in _msg(), (q_ld, o, o_ld)
