"""Python binding of libzdec, the batched Q4_K decode step for one GB300.

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of ``libzdec.so`` (built from ``csrc/`` for sm_103a).  There is no
CPU or PyTorch fallback; if the library cannot be loaded, every entry point
raises.  PyTorch is used for device buffers and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import numpy as np

from . import _build

__all__ = ["ModelDesc", "Decoder", "ZdecError", "load_library", "q4k_repacked_bytes",
           "q4k_repack", "q4k_gemm", "q4k_gemm_workspace_bytes", "q4k_gemm_static",
           "KVPool", "page_bytes", "chunk_plan", "chunk_append", "chunk_read", "chunk_attention",
           "chunk_attention_workspace_bytes", "CHUNK_BAD_SLOT", "CHUNK_NO_PAGE", "CHUNK_TIMEOUT",
           "Q4K_GEMM_STATIC_MAX_KB", "KV_F16", "KV_Q8_0", "KV_FP8", "PAGE_TOKENS",
           "KERNEL_KINDS", "T_EMBED", "T_WQ", "T_WK", "T_WV", "T_WO", "T_GATE", "T_UP", "T_DOWN"]

KV_F16, KV_Q8_0, KV_FP8 = 0, 1, 2   # per-tensor cache types (zdec_kv_dtype)
PAGE_TOKENS = 64                    # tokens per KV pool page
Q4K_GEMM_STATIC_MAX_KB = 262144   # K*B limit of q4k_gemm_static (ZDEC_Q4K_GEMM_STATIC_MAX_KB)
F32, F16, BF16 = 0, 1, 2            # element types of the chunk operators (zdec_float_type)
CHUNK_BAD_SLOT, CHUNK_NO_PAGE, CHUNK_TIMEOUT = 1, 2, 4   # bits of their status word
STEP_HOST_IO, STEP_EAGER = 1, 2
T_EMBED, T_WQ, T_WK, T_WV, T_WO, T_GATE, T_UP, T_DOWN = range(8)
KERNEL_KINDS = ["embed", "-", "gemm_qkv", "attention", "gemm_o", "gemm_gateup", "gemm_down",
                "gemm_lmhead", "argmax"]
STATUS = {0: "ok", -1: "bad argument", -2: "out of memory", -3: "capacity", -4: "position",
          -5: "unsupported", -6: "cuda error", -7: "timeout", -8: "device check"}

# Every symbol include/zdec.h declares; load_library() checks they are exported.
EXPORTS = ["zdec_create_cache", "zdec_create", "zdec_destroy", "zdec_append_kv", "zdec_decode_step",
           "zdec_decode_step_slots", "zdec_sync", "zdec_reset_seq", "zdec_seq_len", "zdec_last_error",
           "zdec_last_global_error", "zdec_set_gemm_impl", "zdec_set_trace", "zdec_debug_step_trace",
           "zdec_get_info", "zdec_profile_step", "zdec_debug_export_q4k", "zdec_debug_dequant",
           "zdec_debug_read_kv", "zdec_debug_block_table", "zdec_debug_capture_hidden",
           "zdec_debug_attention", "zdec_debug_set_wait_limit", "zdec_q4k_repacked_bytes", "zdec_q4k_repack",
           "zdec_q4k_gemm_workspace_bytes", "zdec_q4k_gemm", "zdec_q4k_gemm_static", "zdec_page_bytes",
           "zdec_get_cache", "zdec_extend", "zdec_chunk_plan", "zdec_chunk_append", "zdec_chunk_read",
           "zdec_chunk_attention", "zdec_chunk_attention_workspace_bytes"]


class ZdecError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"zdec: {STATUS.get(status, status)}: {msg}")
        self.status = status


class _Desc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("hidden", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("vocab", ctypes.c_int), ("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float)]


_PP = ctypes.POINTER(ctypes.c_void_p)


class _Weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("attn_norm", _PP), ("ffn_norm", _PP), ("wq", _PP), ("wk", _PP), ("wv", _PP),
                ("wo", _PP), ("w_gate", _PP), ("w_up", _PP), ("w_down", _PP)]


class _Cache(ctypes.Structure):
    _fields_ = [("k_type", ctypes.c_int), ("v_type", ctypes.c_int), ("max_B", ctypes.c_int),
                ("max_L", ctypes.c_int), ("pool_tokens", ctypes.c_longlong)]


class _Info(ctypes.Structure):
    _fields_ = [("weight_bytes", ctypes.c_size_t), ("arena_bytes", ctypes.c_size_t),
                ("workspace_bytes", ctypes.c_size_t), ("kv_bytes_per_token", ctypes.c_size_t),
                ("kernels_per_step", ctypes.c_int), ("attn_splits", ctypes.c_int),
                ("matvec_max_B", ctypes.c_int), ("attn_segments", ctypes.c_int),
                ("k_type", ctypes.c_int), ("v_type", ctypes.c_int), ("page_tokens", ctypes.c_int),
                ("pool_pages", ctypes.c_int), ("free_pages", ctypes.c_int)]


class _Pool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("n_layers", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("k_type", ctypes.c_int), ("v_type", ctypes.c_int)]


class _CacheView(ctypes.Structure):
    _fields_ = [("pool", _Pool), ("tables", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("max_slots", ctypes.c_int), ("max_pages", ctypes.c_int), ("stream", ctypes.c_void_p)]


class _Rope(ctypes.Structure):
    _fields_ = [("theta", ctypes.c_float), ("axes", ctypes.c_int), ("sections", ctypes.c_int * 4)]


class _ChunkAttn(ctypes.Structure):
    _fields_ = [("n_q", ctypes.c_int), ("R", ctypes.c_int), ("T", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("io_type", ctypes.c_int), ("causal", ctypes.c_int), ("window", ctypes.c_int),
                ("scale", ctypes.c_float), ("q_ld", ctypes.c_longlong), ("o_ld", ctypes.c_longlong)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load_library(build_if_missing: bool = True):
    """Load libzdec.so (building it with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise ImportError(f"libzdec.so not found at {_build.LIB}; run __graft_entry__.build()")
    lib = ctypes.CDLL(_build.LIB)
    for name in EXPORTS:
        if not hasattr(lib, name):
            raise ImportError(f"libzdec.so does not export {name}")
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sigs = {
        "zdec_create": (i, [ctypes.POINTER(_Desc), ctypes.POINTER(_Weights), i, i, i, vp,
                            ctypes.POINTER(vp)]),
        "zdec_create_cache": (i, [ctypes.POINTER(_Desc), ctypes.POINTER(_Weights), ctypes.POINTER(_Cache),
                                  vp, ctypes.POINTER(vp)]),
        "zdec_decode_step_slots": (i, [vp, i, vp, vp, vp, vp, vp, i]),
        "zdec_debug_block_table": (i, [vp, i, vp, i, ctypes.POINTER(i)]),
        "zdec_destroy": (None, [vp]),
        "zdec_append_kv": (i, [vp, i, i, vp, vp, i]),
        "zdec_decode_step": (i, [vp, i, vp, vp, vp, vp, i]),
        "zdec_sync": (i, [vp]),
        "zdec_reset_seq": (i, [vp, i]),
        "zdec_seq_len": (i, [vp, i, ctypes.POINTER(i)]),
        "zdec_last_error": (ctypes.c_char_p, [vp]),
        "zdec_last_global_error": (ctypes.c_char_p, []),
        "zdec_set_gemm_impl": (i, [vp, i]),
        "zdec_get_info": (i, [vp, ctypes.POINTER(_Info)]),
        "zdec_set_trace": (i, [vp, i]),
        "zdec_debug_step_trace": (i, [vp, vp, sz, ctypes.POINTER(sz)]),
        "zdec_profile_step": (i, [vp, i, vp, vp, vp, vp, vp, vp, i, ctypes.POINTER(i)]),
        "zdec_debug_export_q4k": (i, [vp, i, i, i, i, vp]),
        "zdec_debug_dequant": (i, [vp, i, i, i, i, vp]),
        "zdec_debug_read_kv": (i, [vp, i, i, i, i, vp, vp, vp, vp]),
        "zdec_debug_capture_hidden": (i, [vp, vp]),
        "zdec_debug_attention": (i, [vp, i, i, vp, vp, vp]),
        "zdec_debug_set_wait_limit": (i, [vp, ctypes.c_longlong]),
        "zdec_q4k_repacked_bytes": (sz, [i, i]),
        "zdec_q4k_repack": (i, [vp, i, i, vp, vp]),
        "zdec_q4k_gemm_workspace_bytes": (sz, [i, i]),
        "zdec_q4k_gemm": (i, [vp, i, i, vp, i, vp, i, vp, sz, vp]),
        "zdec_q4k_gemm_static": (i, [vp, i, i, vp, i, vp, i, vp]),
    }
    ll = ctypes.c_longlong
    sigs.update({
        "zdec_page_bytes": (sz, [i, i, i, i]),
        "zdec_get_cache": (i, [vp, ctypes.POINTER(_CacheView)]),
        "zdec_extend": (i, [vp, i, vp, vp]),
        "zdec_chunk_plan": (i, [i, vp, vp, vp, i, vp, i, i, vp, vp, vp, vp, vp, vp]),
        "zdec_chunk_append": (i, [ctypes.POINTER(_Pool), i, ctypes.POINTER(_Rope), i, i, vp, i, ll, vp, vp, vp, i, ll,
                                  vp, vp]),
        "zdec_chunk_read": (i, [ctypes.POINTER(_Pool), i, i, vp, vp, vp, vp, vp]),
        "zdec_chunk_attention_workspace_bytes": (sz, [i, i]),
        "zdec_chunk_attention": (i, [ctypes.POINTER(_Pool), i, ctypes.POINTER(_ChunkAttn), vp, vp, vp, vp, vp, vp, sz,
                                     vp, vp]),
    })
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _ptr(x) -> int:
    """Address of a numpy array or torch tensor (must be contiguous)."""
    if x is None:
        return None
    if isinstance(x, np.ndarray):
        assert x.flags["C_CONTIGUOUS"], "array must be C-contiguous"
        return x.ctypes.data
    if hasattr(x, "data_ptr"):
        assert x.is_contiguous(), "tensor must be contiguous"
        return x.data_ptr()
    raise TypeError(type(x))


def _is_cuda(x) -> bool:
    return hasattr(x, "is_cuda") and x.is_cuda


@dataclass(frozen=True)
class ModelDesc:
    n_layers: int = 36
    hidden: int = 4096
    n_q_heads: int = 32
    n_kv_heads: int = 8
    head_dim: int = 128
    ffn: int = 14336
    vocab: int = 151936
    rope_theta: float = 1e6
    rms_eps: float = 1e-6

    @classmethod
    def of(cls, d) -> "ModelDesc":
        return cls(d.n_layers, d.hidden, d.n_q_heads, d.n_kv_heads, d.head_dim, d.ffn, d.vocab,
                   d.rope_theta, d.rms_eps)

    def _c(self) -> _Desc:
        return _Desc(self.n_layers, self.hidden, self.n_q_heads, self.n_kv_heads, self.head_dim,
                     self.ffn, self.vocab, self.rope_theta, self.rms_eps)


class Decoder:
    """One decoder context (weights, paged KV pool, workspace) on the current GPU.

    ``weights`` holds canonical Q4_K matrices as uint8 numpy arrays
    [rows, cols/256*144] (per-layer tensors as lists) and fp32 norm gains;
    the library copies and repacks them at creation.  ``kv_dtype`` is one
    cache type for K and V (KV_F16, KV_Q8_0, KV_FP8) or a (k_type, v_type)
    pair; ``pool_tokens`` sizes the shared page pool (0: max_B * max_L)."""

    def __init__(self, desc, weights: dict, kv_dtype=KV_F16, max_B: int = 1, max_L: int = 2048,
                 stream=None, pool_tokens: int = 0):
        self.lib = load_library()
        self.desc = ModelDesc.of(desc)
        d = self.desc
        L = d.n_layers
        keep = []

        def arr(name):
            want = np.float32 if name.endswith("norm") else np.uint8
            mats = [np.ascontiguousarray(weights[name][l], want) for l in range(L)]
            keep.extend(mats)
            a = (ctypes.c_void_p * L)(*[_ptr(m) for m in mats])
            keep.append(a)
            return ctypes.cast(a, _PP)

        fnorm = np.ascontiguousarray(weights["final_norm"], np.float32)
        embed = np.ascontiguousarray(weights["embed"], np.uint8)
        keep += [fnorm, embed]
        w = _Weights(_ptr(embed), _ptr(fnorm),
                     arr("attn_norm"), arr("ffn_norm"), arr("wq"), arr("wk"), arr("wv"), arr("wo"),
                     arr("w_gate"), arr("w_up"), arr("w_down"))
        kt, vt = (int(kv_dtype), int(kv_dtype)) if np.isscalar(kv_dtype) else (int(kv_dtype[0]), int(kv_dtype[1]))
        self.k_type, self.v_type = kt, vt
        self.kv_dtype = kt if kt == vt else (kt, vt)
        self.max_B, self.max_L = max_B, max_L
        self.stream = stream
        h = ctypes.c_void_p()
        desc_c = d._c()
        cache = _Cache(kt, vt, max_B, max_L, int(pool_tokens))
        s = self.lib.zdec_create_cache(ctypes.byref(desc_c), ctypes.byref(w), ctypes.byref(cache),
                                       ctypes.c_void_p(stream) if stream else None, ctypes.byref(h))
        if s != 0:
            raise ZdecError(s, self.lib.zdec_last_global_error().decode())
        self.h = h

    # ---------------------------------------------------------------- utils
    def _check(self, s: int):
        if s != 0:
            raise ZdecError(s, self.lib.zdec_last_error(self.h).decode())

    def close(self):
        if getattr(self, "h", None):
            self.lib.zdec_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    # ------------------------------------------------------------------ API
    def append_kv(self, seq: int, k16, v16):
        """Append rotated fp16 K/V [n_layers][n][n_kv][hd] (uint16 numpy on the host,
        or a torch float16/int16 CUDA tensor) to sequence `seq`."""
        n = k16.shape[1]
        on_dev = 1 if _is_cuda(k16) else 0
        if not on_dev:
            k16 = np.ascontiguousarray(k16, np.uint16)
            v16 = np.ascontiguousarray(v16, np.uint16)
        self._check(self.lib.zdec_append_kv(self.h, seq, n, _ptr(k16), _ptr(v16), on_dev))

    def _run(self, B, slots, tokens, positions, logits, ids, flags):
        if slots is None:
            self._check(self.lib.zdec_decode_step(self.h, B, _ptr(tokens), _ptr(positions),
                                                  _ptr(logits), _ptr(ids), flags))
        else:
            sl = np.ascontiguousarray(slots, np.int32)
            assert sl.shape == (B,)
            self._check(self.lib.zdec_decode_step_slots(self.h, B, _ptr(sl), _ptr(tokens), _ptr(positions),
                                                        _ptr(logits), _ptr(ids), flags))

    def step(self, tokens, positions, logits=None, ids=None, eager: bool = False, slots=None):
        """Device I/O step: tokens/positions int32 CUDA tensors [B], logits float32
        CUDA [B, vocab] or None, ids int32 CUDA [B]; row b uses cache slot
        slots[b] (host ints; default b).  Asynchronous."""
        B = tokens.shape[0]
        self._run(B, slots, tokens, positions, logits, ids, STEP_EAGER if eager else 0)

    def step_host(self, tokens, positions, logits: np.ndarray | None = None,
                  ids: np.ndarray | None = None, eager: bool = False, slots=None):
        """Host I/O step: numpy int32 tokens/positions; returns (logits, ids) numpy.
        Copies in, runs, copies out and waits.  Row b uses slot slots[b]."""
        tokens = np.ascontiguousarray(tokens, np.int32)
        positions = np.ascontiguousarray(positions, np.int32)
        B = tokens.shape[0]
        if ids is None:
            ids = np.empty(B, np.int32)
        self._run(B, slots, tokens, positions, logits, ids, STEP_HOST_IO | (STEP_EAGER if eager else 0))
        return logits, ids

    def sync(self):
        self._check(self.lib.zdec_sync(self.h))

    def reset_seq(self, seq: int):
        self._check(self.lib.zdec_reset_seq(self.h, seq))

    def seq_len(self, seq: int) -> int:
        n = ctypes.c_int()
        self._check(self.lib.zdec_seq_len(self.h, seq, ctypes.byref(n)))
        return n.value

    def set_gemm_impl(self, impl: int):
        self._check(self.lib.zdec_set_gemm_impl(self.h, impl))

    def set_trace(self, on: bool):
        """Record the launch timeline of the following steps (run eagerly)."""
        self._check(self.lib.zdec_set_trace(self.h, int(bool(on))))

    def step_trace(self) -> np.ndarray:
        """Timeline of the last traced step (see zdec.h): [launches][8] uint64."""
        n = ctypes.c_size_t()
        self._check(self.lib.zdec_debug_step_trace(self.h, None, 0, ctypes.byref(n)))
        if n.value == 0:
            return np.zeros((0, 8), np.uint64)
        out = np.empty(n.value, np.uint64)
        self._check(self.lib.zdec_debug_step_trace(self.h, _ptr(out), n.value, ctypes.byref(n)))
        return out.reshape(-1, 8)

    def info(self) -> dict:
        inf = _Info()
        self._check(self.lib.zdec_get_info(self.h, ctypes.byref(inf)))
        return {f: getattr(inf, f) for f, _ in _Info._fields_}

    def profile_step(self, tokens, positions, logits, ids, cap: int = 4096):
        """One eager step with CUDA events around every launch; returns a list of
        (kind name, milliseconds)."""
        kind = np.zeros(cap, np.int32)
        ms = np.zeros(cap, np.float32)
        n = ctypes.c_int()
        B = tokens.shape[0]
        self._check(self.lib.zdec_profile_step(self.h, B, _ptr(tokens), _ptr(positions), _ptr(logits),
                                               _ptr(ids), _ptr(kind), _ptr(ms), cap, ctypes.byref(n)))
        return [(KERNEL_KINDS[kind[i]], float(ms[i])) for i in range(min(n.value, cap))]

    # --------------------------------------------------------------- chunks
    def cache(self) -> "KVPool":
        """This decoder's own cache for the chunk operators: a KVPool whose
        ``tables`` [max_B, max_L / 64] and ``lengths`` [max_B] are its block
        tables and device lengths (int32 tensors, only to be read) and whose
        ``stream`` is the stream the decoder's calls run on.  Keeps the
        decoder alive; not valid after close()."""
        view = _CacheView()
        self._check(self.lib.zdec_get_cache(self.h, ctypes.byref(view)))
        import torch
        dev = torch.device("cuda", torch.cuda.current_device())
        p = view.pool
        nbytes = page_bytes((p.k_type, p.v_type), p.n_layers, p.n_kv_heads)
        pages = _device_tensor(p.base, (p.n_pages, nbytes), "|u1", self, dev)
        c = KVPool(pages, p.n_layers, p.n_kv_heads, (p.k_type, p.v_type))
        c.tables = _device_tensor(view.tables, (view.max_slots, view.max_pages), "<i4", self, dev)
        c.lengths = _device_tensor(view.lengths, (view.max_slots,), "<i4", self, dev)
        c.stream = view.stream or 0
        return c

    def extend(self, slots, n_new):
        """Take pages for n_new[i] more tokens of slots[i] and advance the
        lengths; the caller writes their K/V in every layer (chunk_append)
        before anything reads them.  Waits for the decoder's stream."""
        sl, nn = np.ascontiguousarray(slots, np.int32), np.ascontiguousarray(n_new, np.int32)
        if sl.ndim != 1 or sl.shape != nn.shape:
            raise ZdecError(-1, "slots and n_new must be vectors of one length")
        self._check(self.lib.zdec_extend(self.h, sl.size, _ptr(sl), _ptr(nn)))

    # ---------------------------------------------------------------- debug
    def set_wait_limit(self, cycles: int):
        """Bound of the projection kernels' stage waits in clock cycles (0: the
        default ~2 s); a wait that runs out makes sync() raise a timeout."""
        self._check(self.lib.zdec_debug_set_wait_limit(self.h, int(cycles)))

    def _cols(self, which: int) -> int:
        d = self.desc
        return {T_WO: d.n_q_heads * d.head_dim, T_DOWN: d.ffn}.get(which, d.hidden)

    def export_q4k(self, which: int, layer: int, row0: int, nrows: int) -> np.ndarray:
        out = np.empty((nrows, self._cols(which) // 256 * 144), np.uint8)
        self._check(self.lib.zdec_debug_export_q4k(self.h, which, layer, row0, nrows, _ptr(out)))
        return out

    def dequant(self, which: int, layer: int, row0: int, nrows: int) -> np.ndarray:
        out = np.empty((nrows, self._cols(which)), np.float32)
        self._check(self.lib.zdec_debug_dequant(self.h, which, layer, row0, nrows, _ptr(out)))
        return out

    def read_kv(self, seq: int, layer: int, t0: int, n: int):
        """Stored K/V of one layer, canonical token-major layout [n][n_kv][hd],
        each tensor in its type: fp16 uint16, Q8_0 int8 codes, FP8 uint8 e4m3
        codes.  Returns (k, v) when neither tensor is Q8_0, else (k, v,
        k_scales, v_scales) with uint16 scales [n][n_kv][hd/32] (None for a
        tensor that is not Q8_0)."""
        d = self.desc
        shape = (n, d.n_kv_heads, d.head_dim)
        dt = {KV_F16: np.uint16, KV_Q8_0: np.int8, KV_FP8: np.uint8}
        k, v = np.empty(shape, dt[self.k_type]), np.empty(shape, dt[self.v_type])
        sshape = (n, d.n_kv_heads, d.head_dim // 32)
        ks = np.empty(sshape, np.uint16) if self.k_type == KV_Q8_0 else None
        vs = np.empty(sshape, np.uint16) if self.v_type == KV_Q8_0 else None
        self._check(self.lib.zdec_debug_read_kv(self.h, seq, layer, t0, n, _ptr(k), _ptr(v), _ptr(ks), _ptr(vs)))
        if ks is None and vs is None:
            return k, v
        return k, v, ks, vs

    def block_table(self, seq: int) -> np.ndarray:
        """Page of each 64 tokens of slot `seq` (-1: none), as the device holds it."""
        n = ctypes.c_int()
        self._check(self.lib.zdec_debug_block_table(self.h, seq, None, 0, ctypes.byref(n)))
        out = np.empty(n.value, np.int32)
        self._check(self.lib.zdec_debug_block_table(self.h, seq, _ptr(out), n.value, ctypes.byref(n)))
        return out

    def step_capture_hidden(self, tokens, positions, logits=None, ids=None):
        """Host I/O step that also returns the fp32 residual after the embedding and
        after every layer: [B, n_layers+1, hidden]."""
        B = len(tokens)
        hid = np.empty((B, self.desc.n_layers + 1, self.desc.hidden), np.float32)
        self._check(self.lib.zdec_debug_capture_hidden(self.h, _ptr(hid)))
        logits, ids = self.step_host(tokens, positions, logits, ids)
        return logits, ids, hid

    def attention(self, layer: int, q: np.ndarray, positions) -> np.ndarray:
        """Attention alone over cached tokens 0..positions[b]: q [B, n_q, hd] fp32
        (already rotated) -> o [B, n_q, hd] fp32."""
        q = np.ascontiguousarray(q, np.float32)
        pos = np.ascontiguousarray(positions, np.int32)
        o = np.empty_like(q)
        self._check(self.lib.zdec_debug_attention(self.h, layer, q.shape[0], _ptr(q), _ptr(pos), _ptr(o)))
        return o


# ------------------------------------------------------------ stateless ops
def _glob_check(s: int):
    if s != 0:
        raise ZdecError(s, load_library().zdec_last_global_error().decode())


def q4k_repacked_bytes(N: int, K: int) -> int:
    return int(load_library().zdec_q4k_repacked_bytes(N, K))


def q4k_repack(canonical_dev, N: int, K: int, repacked_dev, stream=None):
    _glob_check(load_library().zdec_q4k_repack(_ptr(canonical_dev), N, K, _ptr(repacked_dev),
                                               ctypes.c_void_p(stream) if stream else None))


def q4k_gemm_workspace_bytes(K: int, B: int) -> int:
    return int(load_library().zdec_q4k_gemm_workspace_bytes(K, B))


def q4k_gemm(repacked_dev, N: int, K: int, x_dev, y_dev, impl: int, workspace_dev, stream=None):
    B = x_dev.shape[0]
    _glob_check(load_library().zdec_q4k_gemm(_ptr(repacked_dev), N, K, _ptr(x_dev), B, _ptr(y_dev), impl,
                                             _ptr(workspace_dev), workspace_dev.numel() * workspace_dev.element_size(),
                                             ctypes.c_void_p(stream) if stream else None))


def q4k_gemm_static(repacked_dev, N: int, K: int, x_dev, y_dev, impl: int, stream=None):
    """q4k_gemm without a workspace: the library's own per-device scratch
    (K*B <= Q4K_GEMM_STATIC_MAX_KB); calls that may overlap in time race on it."""
    B = x_dev.shape[0]
    _glob_check(load_library().zdec_q4k_gemm_static(_ptr(repacked_dev), N, K, _ptr(x_dev), B, _ptr(y_dev), impl,
                                                    ctypes.c_void_p(stream) if stream else None))


# ------------------------------------------------- chunks of new tokens
class _DeviceArray:
    """Device memory that a decoder owns, as __cuda_array_interface__ (keeps the owner alive)."""

    def __init__(self, ptr, shape, typestr, owner):
        self.owner = owner
        self.__cuda_array_interface__ = {"data": (ptr, False), "shape": shape, "typestr": typestr, "version": 3}


def _device_tensor(ptr, shape, typestr, owner, dev):
    import torch
    return torch.as_tensor(_DeviceArray(ptr, shape, typestr, owner), device=dev)


def page_bytes(kv_dtype, n_layers: int, n_kv_heads: int) -> int:
    """Bytes of one 64-token page of a pool with these cache types (one, or a (K, V) pair)."""
    kt, vt = (int(kv_dtype), int(kv_dtype)) if np.isscalar(kv_dtype) else (int(kv_dtype[0]), int(kv_dtype[1]))
    return int(load_library().zdec_page_bytes(kt, vt, n_layers, n_kv_heads))


class KVPool:
    """A pool of KV pages as the chunk operators take it: ``pages`` is a
    contiguous uint8 CUDA tensor [n_pages, page_bytes(...)] (zeros, or written
    by chunk_append), kept by this object.  Decoder.cache() gives a decoder's
    own pool."""

    def __init__(self, pages, n_layers: int, n_kv_heads: int, kv_dtype=KV_F16):
        kt, vt = (int(kv_dtype), int(kv_dtype)) if np.isscalar(kv_dtype) else (int(kv_dtype[0]), int(kv_dtype[1]))
        nbytes = page_bytes((kt, vt), n_layers, n_kv_heads)
        if nbytes == 0:
            raise ZdecError(-1, "bad cache type or pool shape")
        _tensor(pages, "pages", ("uint8",), (None, nbytes), None)
        self.pages, self.n_layers, self.n_kv_heads, self.k_type, self.v_type = pages, n_layers, n_kv_heads, kt, vt
        self.device, self.index = pages.device, pages.get_device()
        self._c = _Pool(pages.data_ptr(), pages.shape[0], n_layers, n_kv_heads, kt, vt)
        self._ref = ctypes.byref(self._c)


_TYPE_ID = {"float32": F32, "float16": F16, "bfloat16": BF16}


def _tensor(x, name, dtypes, shape, device, strided=False):
    """Check a CUDA tensor's type, shape (None: any) and device; contiguous unless only its first stride is free."""
    if not _is_cuda(x):
        raise ZdecError(-1, f"{name} must be a CUDA tensor")
    if str(x.dtype)[6:] not in dtypes:
        raise ZdecError(-1, f"{name} must be {' or '.join(dtypes)}, not {str(x.dtype)[6:]}")
    if x.dim() != len(shape) or any(w is not None and w != g for w, g in zip(shape, x.shape)):
        raise ZdecError(-1, f"{name} must have shape {shape}, not {tuple(x.shape)}")
    if device is not None and x.device != device:
        raise ZdecError(-1, f"{name} is on {x.device}, the rest on {device}")
    if not (x[:1].is_contiguous() if strided else x.is_contiguous()):
        raise ZdecError(-1, f"{name} must be contiguous" + (" within a row" if strided else ""))


# The calls below are made per layer and step, so their checks come in two
# forms: a quick one, and the one that says what is wrong.
_I32, _I64, _U8, _HALF, _ANY = ("int32",), ("int64",), ("uint8",), ("float16", "bfloat16"), ("float32", "float16", "bfloat16")
_DT = {}   # torch dtypes by name, and torch dtype -> zdec_float_type


def _dtypes():
    if not _DT:
        import torch
        if not torch.cuda.is_available():
            raise ZdecError(-1, "the chunk operators need CUDA tensors")
        _DT.update({n: getattr(torch, n) for n in ("int32", "int64", "uint8", "float16", "bfloat16", "float32")})
        _DT.update({getattr(torch, n): t for n, t in _TYPE_ID.items()})
        _DT["torch"] = torch
        torch.cuda.init()
        # the current stream's handle and the current device without a Stream object in between (1 us less per call)
        _DT["stream"] = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
        _DT["device"] = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _DT


def _rows(x) -> int:
    """Elements from row to row if the rows of x are contiguous within, else 0
    (a single row's own length: its stride says nothing)."""
    if x.is_contiguous():
        return x.stride(0) if x.shape[0] > 1 else x[:1].numel()
    if x.dim() == 3:
        ok = x.stride(2) == 1 and x.stride(1) == x.shape[2]
        return (x.stride(0) if x.shape[0] > 1 else x.shape[1] * x.shape[2]) if ok else 0
    return (x.stride(0) if x.shape[0] > 1 else x.shape[1]) if x.stride(1) == 1 else 0


def _call(index, stream, fn, *args):
    """One stateless call on CUDA device `index`, on `stream` (a cudaStream_t, or None: torch's current stream there)."""
    dt = _DT
    if stream is None:
        stream = dt["stream"](index)
    if dt["device"]() == index:
        s = fn(*args, stream)
    else:
        with dt["torch"].cuda.device(index):
            s = fn(*args, stream)
    if s:
        _glob_check(s)


def _status(x, dev):
    if x is None:
        return None
    _tensor(x, "status", _I32, (1,), dev)
    return x.data_ptr()


def chunk_plan(ctx_len, n_new, tables, cu, kv_len, positions, slots, taken, free_pages=None, stream=None):
    """Offsets, positions, pages and slots of a ragged batch of new tokens, from
    its lengths on the device (zdec_chunk_plan).  int32 CUDA tensors ctx_len,
    n_new [R], tables [R, max_pages] (entries of new pages are set when
    free_pages is given), outputs cu [R + 1], kv_len [R], positions [T], taken
    [2] and int64 slots [T].  Asynchronous."""
    dt = _DT or _dtypes()
    i32, free, n_free = dt["int32"], None, 0
    try:
        R, T, idx, f = ctx_len.numel(), positions.numel(), ctx_len.get_device(), free_pages
        quick = (idx >= 0 and ctx_len.dtype is i32 and n_new.dtype is i32 and tables.dtype is i32 and cu.dtype is i32
                 and kv_len.dtype is i32 and positions.dtype is i32 and taken.dtype is i32 and slots.dtype is dt["int64"]
                 and n_new.get_device() == idx and tables.get_device() == idx and cu.get_device() == idx
                 and kv_len.get_device() == idx and positions.get_device() == idx and taken.get_device() == idx
                 and slots.get_device() == idx and ctx_len.shape == (R,) and n_new.shape == (R,) and kv_len.shape == (R,)
                 and cu.shape == (R + 1,) and tables.dim() == 2 and tables.shape[0] == R and positions.shape == (T,)
                 and slots.shape == (T,) and taken.shape == (2,) and ctx_len.is_contiguous() and n_new.is_contiguous()
                 and tables.is_contiguous() and cu.is_contiguous() and kv_len.is_contiguous() and positions.is_contiguous()
                 and slots.is_contiguous() and taken.is_contiguous()
                 and (f is None or (f.dtype is i32 and f.get_device() == idx and f.dim() == 1 and f.is_contiguous())))
    except AttributeError:
        quick = False
    if not quick:
        _tensor(ctx_len, "ctx_len", _I32, (None,), None)
        dev, R = ctx_len.device, ctx_len.shape[0]
        _tensor(positions, "positions", _I32, (None,), dev)
        T, idx = positions.shape[0], dev.index
        for x, name, shape in ((n_new, "n_new", (R,)), (tables, "tables", (R, None)), (cu, "cu", (R + 1,)), (kv_len, "kv_len", (R,)),
                               (taken, "taken", (2,))):
            _tensor(x, name, _I32, shape, dev)
        _tensor(slots, "slots", _I64, (T,), dev)
        if free_pages is not None:
            _tensor(free_pages, "free_pages", _I32, (None,), dev)
    if free_pages is not None:
        n_free = free_pages.numel()
        free = free_pages.data_ptr() if n_free else taken.data_ptr()   # an empty list: never read, but not "no list"
    _call(idx, stream, load_library().zdec_chunk_plan, R, ctx_len.data_ptr(), n_new.data_ptr(), free, n_free, tables.data_ptr(),
          tables.shape[1], T, cu.data_ptr(), kv_len.data_ptr(), positions.data_ptr(), slots.data_ptr(), taken.data_ptr())


@functools.lru_cache(maxsize=64)
def _rope(theta: float, sections: tuple):
    if not 1 <= len(sections) <= 4:
        raise ZdecError(-1, "sections must have 1 to 4 entries")
    return ctypes.byref(_Rope(theta, len(sections), (ctypes.c_int * 4)(*sections)))


def chunk_append(cache: KVPool, layer: int, qkv, positions, slots, q_out=None, rope_theta: float = 1e6,
                 sections=(64,), status=None, stream=None):
    """Rotate the queries and keys of T new tokens, write the queries to q_out
    and the keys and values, encoded, to the tokens' slots (zdec_chunk_append).
    qkv [T, (n_q + 2 n_kv) * 128] fp32, fp16 or bf16 (rows may be strided),
    positions [axes, T] or [T] int32, slots [T] int64 (negative: no K/V),
    q_out [T, n_q, 128] fp16 or bf16 (or None: qkv holds no queries); sections:
    rotary pairs per position axis (sum 64); rope_theta 0: no rotation;
    status: optional int32 [1].  q_out may not overlap qkv.  Asynchronous."""
    dt, dev, nkv, axes = _DT or _dtypes(), cache.device, cache.n_kv_heads, len(sections)
    rope = _rope(float(rope_theta), tuple(sections))
    idx = cache.index
    quick = False
    if getattr(qkv, "dtype", None) in dt and qkv.dim() == 2 and qkv.get_device() == idx:
        T, width = qkv.shape
        nq = 0 if q_out is None else width // 128 - 2 * nkv
        ld, q_ld = _rows(qkv), 0 if q_out is None else _rows(q_out)
        quick = (width == (nq + 2 * nkv) * 128 and ld > 0 and positions.dtype is dt["int32"] and slots.dtype is dt["int64"]
                 and positions.get_device() == idx and slots.get_device() == idx and positions.is_contiguous()
                 and slots.is_contiguous() and slots.shape == (T,) and (positions.shape == (axes, T) or (axes == 1 and positions.shape == (T,)))
                 and (q_out is None or (q_ld > 0 and q_out.shape == (T, nq, 128) and q_out.get_device() == idx
                                        and (q_out.dtype is dt["float16"] or q_out.dtype is dt["bfloat16"]))))
    if not quick:
        _tensor(qkv, "qkv", _ANY, (None, None), dev, strided=True)
        T, width = qkv.shape
        nq = 0 if q_out is None else q_out.shape[1] if q_out.dim() == 3 else -1
        if width != (nq + 2 * nkv) * 128:
            raise ZdecError(-1, f"qkv rows of {width} elements do not hold {nq} query and 2 * {nkv} K/V heads of 128")
        if q_out is not None:
            _tensor(q_out, "q_out", _HALF, (T, nq, 128), dev, strided=True)
        _tensor(positions, "positions", _I32, (T,) if positions.dim() == 1 and axes == 1 else (axes, T), dev)
        _tensor(slots, "slots", _I64, (T,), dev)
        ld, q_ld = _rows(qkv), 0 if q_out is None else _rows(q_out)
    _call(idx, stream, load_library().zdec_chunk_append, cache._ref, layer, rope, T, nq, qkv.data_ptr(), dt[qkv.dtype], ld,
          positions.data_ptr(), slots.data_ptr(), None if q_out is None else q_out.data_ptr(),
          F16 if q_out is None else dt[q_out.dtype], q_ld, _status(status, dev))


def chunk_read(cache: KVPool, layer: int, slots, k, v, status=None, stream=None):
    """K and V of the given slots [T] int64 as fp16 rows k, v [T, n_kv, 128]
    (zdec_chunk_read); negative slots read as 0.  Asynchronous."""
    dt, dev = _DT or _dtypes(), cache.device
    idx, want = cache.index, (getattr(slots, "shape", (0,))[0], cache.n_kv_heads, 128)
    if not (getattr(slots, "dtype", None) is dt["int64"] and slots.dim() == 1 and slots.get_device() == idx and slots.is_contiguous()
            and k.dtype is dt["float16"] and v.dtype is dt["float16"] and k.shape == want and v.shape == want
            and k.get_device() == idx and v.get_device() == idx and k.is_contiguous() and v.is_contiguous()):
        _tensor(slots, "slots", _I64, (None,), dev)
        _tensor(k, "k", _HALF[:1], want, dev)
        _tensor(v, "v", _HALF[:1], want, dev)
    _call(idx, stream, load_library().zdec_chunk_read, cache._ref, layer, want[0], slots.data_ptr(), k.data_ptr(), v.data_ptr(),
          _status(status, dev))


def chunk_attention_workspace_bytes(n_q: int, n_kv_heads: int) -> int:
    return int(load_library().zdec_chunk_attention_workspace_bytes(n_q, n_kv_heads))


def chunk_attention(cache: KVPool, layer: int, q, o, cu, kv_len, tables, workspace, causal: bool = True,
                    window: int = 0, scale: float | None = None, status=None, stream=None):
    """Attention of the new tokens of R requests over their pages
    (zdec_chunk_attention).  q, o [T, n_q, 128] fp16 or bf16 (rows may be
    strided), int32 cu [R + 1], kv_len [R], tables [R, max_pages]; workspace:
    uint8 CUDA tensor of chunk_attention_workspace_bytes(n_q, n_kv) bytes, one
    per stream of calls; scale: 1 / sqrt(128) if None.  o may not overlap q.
    Asynchronous."""
    dt, dev = _DT or _dtypes(), cache.device
    idx, i32 = cache.index, dt["int32"]
    quick = False
    if (getattr(q, "dtype", None) is dt["float16"] or getattr(q, "dtype", None) is dt["bfloat16"]) and q.dim() == 3 and o.dim() == 3:
        R, q_ld, o_ld = kv_len.numel(), _rows(q), _rows(o)
        quick = (q.get_device() == idx and o.get_device() == idx and o.dtype is q.dtype and o.shape == q.shape and q.shape[2] == 128
                 and q_ld > 0 and o_ld > 0
                 and cu.dtype is i32 and kv_len.dtype is i32 and tables.dtype is i32 and cu.get_device() == idx
                 and kv_len.get_device() == idx and tables.get_device() == idx and cu.is_contiguous() and kv_len.is_contiguous()
                 and tables.is_contiguous()
                 and kv_len.dim() == 1 and cu.shape == (R + 1,) and tables.dim() == 2 and tables.shape[0] == R
                 and workspace.dtype is dt["uint8"] and workspace.get_device() == idx and workspace.is_contiguous())
    if not quick:
        _tensor(q, "q", _HALF, (None, None, 128), dev, strided=True)
        _tensor(o, "o", (str(q.dtype)[6:],), tuple(q.shape), dev, strided=True)
        _tensor(kv_len, "kv_len", _I32, (None,), dev)
        R = kv_len.shape[0]
        _tensor(cu, "cu", _I32, (R + 1,), dev)
        _tensor(tables, "tables", _I32, (R, None), dev)
        _tensor(workspace, "workspace", _U8, (None,), dev)
        q_ld, o_ld = _rows(q), _rows(o)
    T, nq, _ = q.shape
    a = _ChunkAttn(nq, R, T, tables.shape[1], dt[q.dtype], 1 if causal else 0, window, 128 ** -0.5 if scale is None else scale, q_ld, o_ld)
    _call(idx, stream, load_library().zdec_chunk_attention, cache._ref, layer, ctypes.byref(a), cu.data_ptr(), kv_len.data_ptr(),
          tables.data_ptr(), q.data_ptr(), o.data_ptr(), workspace.data_ptr(), workspace.numel(), _status(status, dev))
