"""Python binding of libqmv.so (argument marshalling only).

Every function has the name and argument order of the C entry point declared
in include/qmv.h, include/qmv_step.h or include/qmv_serve.h.  Buffer arguments are torch tensors on the GPU (or raw
device addresses as ints); sizes are ints; ``stream`` is a torch stream (None:
torch's current stream).  A non-zero status raises QmvError.  All compute
happens in the HIP kernels of libqmv.so; there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os

import torch  # loaded first so that libqmv.so binds to torch's HIP runtime

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqmv.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is not built; run `python -m quantized_dequant_matrix_amd.build`")

lib = ctypes.CDLL(_LIB_PATH)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_F = ctypes.c_float

_SIGS = {
    "qmv_status_str": ([ctypes.c_int], ctypes.c_char_p),
    "qmv_q4_0": ([_P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_q8_0": ([_P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_q4_k": ([_P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_q6_k": ([_P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_mxfp4": ([_P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_q4_0_geglu": ([_P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_q4_0_geglu_down": ([_P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_q4_k_geglu_down": ([_P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_q6_k_geglu_down": ([_P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_q4_k_q6_k_qkv": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmm_q4_0_q8act_ws_bytes": ([_I64, _I64, _I64], _SZ),
    "qmm_q4_0_q8act": ([_P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "qmm_q4_0_f32act_ws_bytes": ([_I64, _I64, _I64], _SZ),
    "qmm_q4_0_f32act": ([_P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "logits_topk_ws_bytes": ([_I64, _I64, _I32], _SZ),
    "logits_topk": ([_P, _P, _P, _P, _I64, _I64, _I64, _I32, _F, _P, _SZ, _P], ctypes.c_int),
    "logits_topk_noalloc": ([_P, _P, _P, _P, _I64, _I64, _I64, _I32, _F, _P], ctypes.c_int),
    "logits_sample": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _F, _F, _F, _P, _SZ, _P], ctypes.c_int),
    "qmvdbg_quantize_q8": ([_P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "qmvdbg_qmm_q4_0_q8act_blocksums": ([_P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "qmvdbg_topk_f32": ([_P, _P, _P, _I64, _I64, _I32, _F, _P, _SZ, _P], ctypes.c_int),
    "qmvdbg_sample_f32": ([_P, _P, _P, _P, _P, _I64, _I32, _F, _F, _P], ctypes.c_int),
    "qmvdbg_stream_read": ([_P, _I64, _P, _I32, _P], ctypes.c_int),
}


class _KVCache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("num_pages", _I64), ("kv_heads", _I32),
                ("head_dim", _I32), ("page_size", _I32), ("format", _I32)]


class _KVBatch(ctypes.Structure):
    _fields_ = [("page_table", _P), ("row_start", _P), ("kv_len", _P), ("T", _I64), ("B", _I32), ("max_pages", _I32)]


# include/qmv_step.h
_STEP_SIGS = {
    "kv_write": ([_P, _P, _P, _I64, _P, _I64, _P], ctypes.c_int),
    "kv_read": ([_P, _P, _P, _I64, _P, _I64, _P], ctypes.c_int),
    "attn_paged_ws_bytes": ([_P, _P, _I32], _SZ),
    "attn_paged": ([_P, _P, _P, _I64, _P, _I64, _I32, _F, _I32, _P, _SZ, _P], ctypes.c_int),
    "rmsnorm_add": ([_P, _P, _P, _P, _P, _I64, _I64, _F, _P], ctypes.c_int),
    "rmsnorm_add_q8": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _P], ctypes.c_int),
    "qmm_q4_0_q8_ws_bytes": ([_I64, _I64, _I64], _SZ),
    "qmm_q4_0_q8": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "draft_verify_ws_bytes": ([_I64, _I32, _I64], _SZ),
    "draft_verify": ([_P, _I64, _P, _I64, _P, _P, _P, _P, _P, _I64, _I32, _I64, _F, _F, _P, _SZ, _P], ctypes.c_int),
}

class _KVPool(ctypes.Structure):
    _fields_ = [("page_table", _P), ("free_pages", _P), ("num_pages", _I64), ("B", _I32), ("max_pages", _I32),
                ("page_size", _I32)]


class _Lora(ctypes.Structure):
    _fields_ = [("A", _P), ("Bm", _P), ("rank", _P), ("scale", _P), ("K", _I64), ("N", _I64), ("slots", _I32),
                ("max_rank", _I32), ("format", _I32)]


# include/qmv_serve.h
_EMBED = ([_P, _P, _P, _I64, _I64, _I64, _F, _P], ctypes.c_int)
_SERVE_SIGS = {
    "kv_plan_ws_bytes": ([_P], _SZ),
    "kv_plan": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _SZ, _P], ctypes.c_int),
    "embed_q8_0": _EMBED,
    "embed_q4_0": _EMBED,
    "embed_q4_k": _EMBED,
    "embed_q6_k": _EMBED,
    "lora_add_ws_bytes": ([_P, _I64, _I64], _SZ),
    "lora_add": ([_P, _P, _P, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "logits_draw_ws_bytes": ([_I64, _I64], _SZ),
    "logits_draw": ([_P, _I64, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _F, _P, _SZ, _P], ctypes.c_int),
}
for _name, (_args, _res) in (_SIGS | _STEP_SIGS | _SERVE_SIGS).items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTS = tuple(_SIGS)
STEP_EXPORTS = tuple(_STEP_SIGS)
SERVE_EXPORTS = tuple(_SERVE_SIGS)
KV_Q8, KV_F16 = 0, 1
PLAN_PAGES, PLAN_ROWS, PLAN_LENGTH, PLAN_STACK = 1, 2, 4, 8
LORA_F16, LORA_BF16 = 0, 1

QMV_OK, QMV_ERR_NULL, QMV_ERR_SHAPE, QMV_ERR_ALIGN, QMV_ERR_WORKSPACE, QMV_ERR_LAUNCH, QMV_ERR_ARG = range(7)


# without a GPU: no tensor's device, so that host tensors are refused as such
_device = torch._C._cuda_getDevice if torch.cuda.device_count() else lambda: -2
_raw_stream = torch._C._cuda_getCurrentRawStream


class QmvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


def status_str(status: int) -> str:
    return lib.qmv_status_str(status).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s):
    if s is None:
        return _raw_stream(_device())  # torch's current stream of the current GPU
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _call(name: str, *args) -> None:
    rc = getattr(lib, name)(*args)
    if rc != QMV_OK:
        raise QmvError(rc, name)


def qmv_q4_0(W, x, y, N, K, M=1, stream=None):
    _call("qmv_q4_0", _ptr(W), _ptr(x), _ptr(y), N, K, M, _stream(stream))


def qmv_q8_0(W, x, y, N, K, M=1, stream=None):
    _call("qmv_q8_0", _ptr(W), _ptr(x), _ptr(y), N, K, M, _stream(stream))


def qmv_q4_k(W, x, y, N, K, M=1, stream=None):
    _call("qmv_q4_k", _ptr(W), _ptr(x), _ptr(y), N, K, M, _stream(stream))


def qmv_q6_k(W, x, y, N, K, M=1, stream=None):
    _call("qmv_q6_k", _ptr(W), _ptr(x), _ptr(y), N, K, M, _stream(stream))


def qmv_mxfp4(W_codes, W_scales, x, y, N, K, M=1, stream=None):
    _call("qmv_mxfp4", _ptr(W_codes), _ptr(W_scales), _ptr(x), _ptr(y), N, K, M, _stream(stream))


def qmv_q4_0_geglu(W_gate, W_up, x, h, N, K, M=1, stream=None):
    _call("qmv_q4_0_geglu", _ptr(W_gate), _ptr(W_up), _ptr(x), _ptr(h), N, K, M, _stream(stream))


def qmv_q4_0_geglu_down(W_down, g, u, y, N, K, M=1, stream=None):
    _call("qmv_q4_0_geglu_down", _ptr(W_down), _ptr(g), _ptr(u), _ptr(y), N, K, M, _stream(stream))


def qmv_q4_k_geglu_down(W_down, g, u, y, N, K, M=1, stream=None):
    _call("qmv_q4_k_geglu_down", _ptr(W_down), _ptr(g), _ptr(u), _ptr(y), N, K, M, _stream(stream))


def qmv_q6_k_geglu_down(W_down, g, u, y, N, K, M=1, stream=None):
    _call("qmv_q6_k_geglu_down", _ptr(W_down), _ptr(g), _ptr(u), _ptr(y), N, K, M, _stream(stream))


def qmv_q4_k_q6_k_qkv(Wq, Wk, Wv, x, q, k, v, Nq, Nk, Nv, K, M=1, stream=None):
    _call("qmv_q4_k_q6_k_qkv", _ptr(Wq), _ptr(Wk), _ptr(Wv), _ptr(x), _ptr(q), _ptr(k), _ptr(v), Nq, Nk, Nv, K, M,
          _stream(stream))


def qmm_q4_0_q8act_ws_bytes(N, K, M) -> int:
    return int(lib.qmm_q4_0_q8act_ws_bytes(N, K, M))


def qmm_q4_0_q8act(W, x, y, N, K, M, ws, ws_bytes, stream=None):
    _call("qmm_q4_0_q8act", _ptr(W), _ptr(x), _ptr(y), N, K, M, _ptr(ws), ws_bytes, _stream(stream))


def qmm_q4_0_f32act_ws_bytes(N, K, M) -> int:
    return int(lib.qmm_q4_0_f32act_ws_bytes(N, K, M))


def qmm_q4_0_f32act(W, x, y, N, K, M, ws, ws_bytes, stream=None):
    _call("qmm_q4_0_f32act", _ptr(W), _ptr(x), _ptr(y), N, K, M, _ptr(ws), ws_bytes, _stream(stream))


def logits_topk_ws_bytes(N, M, k) -> int:
    return int(lib.logits_topk_ws_bytes(N, M, k))


def logits_topk(W_q8_0, x, top_val, top_idx, N, K, M, k, softcap, ws, ws_bytes, stream=None):
    _call("logits_topk", _ptr(W_q8_0), _ptr(x), _ptr(top_val), _ptr(top_idx), N, K, M, k, softcap,
          _ptr(ws), ws_bytes, _stream(stream))


def logits_topk_noalloc(W_q8_0, x, top_val, top_idx, N, K, M, k, softcap, stream=None):
    _call("logits_topk_noalloc", _ptr(W_q8_0), _ptr(x), _ptr(top_val), _ptr(top_idx), N, K, M, k, softcap,
          _stream(stream))


def qmvdbg_quantize_q8(x, q, d, K, M, stream=None):
    _call("qmvdbg_quantize_q8", _ptr(x), _ptr(q), _ptr(d), K, M, _stream(stream))


def qmvdbg_qmm_q4_0_q8act_blocksums(W, x, isum, N, K, M, n0, n1, ws, ws_bytes, stream=None):
    _call("qmvdbg_qmm_q4_0_q8act_blocksums", _ptr(W), _ptr(x), _ptr(isum), N, K, M, n0, n1, _ptr(ws), ws_bytes,
          _stream(stream))


def qmvdbg_topk_f32(y, top_val, top_idx, N, M, k, softcap, ws, ws_bytes, stream=None):
    _call("qmvdbg_topk_f32", _ptr(y), _ptr(top_val), _ptr(top_idx), N, M, k, softcap, _ptr(ws), ws_bytes,
          _stream(stream))


def logits_sample(W_q8_0, x, u, token, nucleus, top_val, top_idx, N, K, M, k, softcap, temperature, top_p, ws,
                  ws_bytes, stream=None):
    _call("logits_sample", _ptr(W_q8_0), _ptr(x), _ptr(u), _ptr(token), _ptr(nucleus), _ptr(top_val),
          _ptr(top_idx), N, K, M, k, softcap, temperature, top_p, _ptr(ws), ws_bytes, _stream(stream))


def qmvdbg_sample_f32(top_val, top_idx, u, token, nucleus, M, k, temperature, top_p, stream=None):
    _call("qmvdbg_sample_f32", _ptr(top_val), _ptr(top_idx), _ptr(u), _ptr(token), _ptr(nucleus), M, k,
          temperature, top_p, _stream(stream))


def qmvdbg_stream_read(p, nbytes, out, workgroups, stream=None):
    _call("qmvdbg_stream_read", _ptr(p), nbytes, _ptr(out), workgroups, _stream(stream))


# ---- include/qmv_step.h ----

class KVCache:
    """qmv_kv_cache over torch tensors: k, v [num_pages][kv_heads][page_size][head_dim], int8 with k_scale, v_scale
    float32 [num_pages][kv_heads][page_size] (KV_Q8), or float16 without (KV_F16).  Keeps the tensors alive."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        q8 = k.dtype == torch.int8
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in (torch.int8, torch.float16):
            raise ValueError("k and v: one shape [num_pages][kv_heads][page_size][head_dim], both int8 or both float16")
        scales = (k_scale, v_scale)
        if q8 and any(s is None or s.shape != k.shape[:3] or s.dtype != torch.float32 for s in scales):
            raise ValueError("int8 codes need k_scale and v_scale, float32 [num_pages][kv_heads][page_size]")
        if not q8 and any(s is not None for s in scales):
            raise ValueError("a float16 cache has no scales")
        self.tensors = tensors = tuple(t for t in (k, v, *scales) if t is not None)
        _on_gpu(*tensors)
        self.struct = _KVCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), k.shape[0], k.shape[1], k.shape[3],
                               k.shape[2], KV_Q8 if q8 else KV_F16)
        self.ref = ctypes.addressof(self.struct)
        self.device = tensors[0].get_device()


class KVBatch:
    """qmv_kv_batch over torch tensors: page_table int32 [B][max_pages], row_start int32 [B + 1], kv_len int32 [B];
    T rows in the row buffers.  Keeps the tensors alive."""

    def __init__(self, page_table, row_start, kv_len, T):
        tensors = (page_table, row_start, kv_len)
        if any(t.dtype != torch.int32 for t in tensors) or page_table.dim() != 2:
            raise ValueError("page_table [B][max_pages], row_start [B + 1] and kv_len [B] are int32")
        B = page_table.shape[0]
        if row_start.shape != (B + 1,) or kv_len.shape != (B,):
            raise ValueError("row_start has B + 1 entries and kv_len B")
        _on_gpu(*tensors)
        self.tensors = tensors
        self.struct = _KVBatch(_ptr(page_table), _ptr(row_start), _ptr(kv_len), T, B, page_table.shape[1])
        self.ref = ctypes.addressof(self.struct)
        self.device = tensors[0].get_device()


def _on_gpu(*tensors):
    """The descriptors' tensors are contiguous and on the current GPU."""
    _gpu(_device(), *tensors)
    if not all(t.is_contiguous() for t in tensors):
        raise ValueError("the tensors of a descriptor are contiguous")


def _gpu(d, *tensors):
    """Addresses of tensors that GPU d's kernels can use (a raw address is the caller's word).  The calls below are
    counted in single microseconds, and d is asked for once in each."""
    out = []
    for t in tensors:
        if t is None or isinstance(t, int):
            out.append(t)
        elif t.get_device() == d:  # -1: host memory
            out.append(t.data_ptr())
        else:
            raise ValueError(f"a tensor on {t.device} was given to a kernel of the current GPU")
    return out


def _step(name, d, stream, *args):
    rc = getattr(lib, name)(*args, _raw_stream(d) if stream is None else _stream(stream))
    if rc != QMV_OK:
        raise QmvError(rc, name)


def _desc(cache, batch, d=None):
    """Addresses of the two descriptors, whose tensors are on GPU d (the current one)."""
    d = _device() if d is None else d
    if cache.device != d or batch.device != d:
        raise ValueError("the descriptors' tensors are on another GPU than the current one")
    return cache.ref, batch.ref


def kv_write(cache, batch, k, ldk, v, ldv, stream=None):
    d = _device()
    c, b = _desc(cache, batch, d)
    k, v = _gpu(d, k, v)
    _step("kv_write", d, stream, c, b, k, ldk, v, ldv)


def kv_read(cache, batch, k, ldk, v, ldv, stream=None):
    d = _device()
    c, b = _desc(cache, batch, d)
    k, v = _gpu(d, k, v)
    _step("kv_read", d, stream, c, b, k, ldk, v, ldv)


def attn_paged_ws_bytes(cache, batch, q_heads) -> int:
    return int(lib.attn_paged_ws_bytes(cache.ref, batch.ref, q_heads))


def attn_paged(cache, batch, q, ldq, out, ldo, q_heads, scale, window, ws, ws_bytes, stream=None):
    d = _device()
    c, b = _desc(cache, batch, d)
    q, out, ws = _gpu(d, q, out, ws)
    _step("attn_paged", d, stream, c, b, q, ldq, out, ldo, q_heads, scale, window, ws, ws_bytes)


def rmsnorm_add(x, r, w, z, y, K, M, eps, stream=None):
    d = _device()
    _step("rmsnorm_add", d, stream, *_gpu(d, x, r, w, z, y), K, M, eps)


def rmsnorm_add_q8(x, r, w, z, q, d, K, M, eps, stream=None):
    dev = _device()
    _step("rmsnorm_add_q8", dev, stream, *_gpu(dev, x, r, w, z, q, d), K, M, eps)


def qmm_q4_0_q8_ws_bytes(N, K, M) -> int:
    return int(lib.qmm_q4_0_q8_ws_bytes(N, K, M))


def qmm_q4_0_q8(W, q, d, y, N, K, M, ws, ws_bytes, stream=None):
    dev = _device()
    W, q, d, y, ws = _gpu(dev, W, q, d, y, ws)
    _step("qmm_q4_0_q8", dev, stream, W, q, d, y, N, K, M, ws, ws_bytes)


def draft_verify_ws_bytes(B, G, V) -> int:
    return int(lib.draft_verify_ws_bytes(B, G, V))


def draft_verify(target, ldt, draft, ldd, draft_tokens, n_draft, u, accepted, tokens, B, G, V, temperature, softcap, ws,
                 ws_bytes, stream=None):
    d = _device()
    target, draft, draft_tokens, n_draft, u, accepted, tokens, ws = _gpu(d, target, draft, draft_tokens, n_draft, u,
                                                                         accepted, tokens, ws)
    _step("draft_verify", d, stream, target, ldt, draft, ldd, draft_tokens, n_draft, u, accepted, tokens, B, G, V,
          temperature, softcap, ws, ws_bytes)


# ---- include/qmv_serve.h ----

class KVPool:
    """qmv_kv_pool over torch tensors: page_table int32 [B][max_pages] (the one of KVBatch), free_pages int32
    [num_pages].  Keeps the tensors alive."""

    def __init__(self, page_table, free_pages, page_size):
        if page_table.dtype != torch.int32 or free_pages.dtype != torch.int32 or page_table.dim() != 2 or free_pages.dim() != 1:
            raise ValueError("page_table [B][max_pages] and free_pages [num_pages] are int32")
        _on_gpu(page_table, free_pages)
        self.tensors = page_table, free_pages
        self.struct = _KVPool(_ptr(page_table), _ptr(free_pages), free_pages.shape[0], *page_table.shape, page_size)
        self.ref = ctypes.addressof(self.struct)
        self.device = page_table.get_device()


class Lora:
    """qmv_lora over torch tensors: A [slots][max_rank][K] and Bm [slots][N][max_rank], both float16 or both bfloat16,
    scale float32 [slots], rank int32 [slots] or None.  Keeps the tensors alive."""

    def __init__(self, A, Bm, scale, rank=None):
        if A.dtype != Bm.dtype or A.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError("A and Bm are both float16 or both bfloat16")
        if A.dim() != 3 or Bm.dim() != 3 or A.shape[0] != Bm.shape[0] or A.shape[1] != Bm.shape[2]:
            raise ValueError("A is [slots][max_rank][K] and Bm [slots][N][max_rank]")
        if scale.dtype != torch.float32 or scale.shape != A.shape[:1]:
            raise ValueError("scale is float32 [slots]")
        if rank is not None and (rank.dtype != torch.int32 or rank.shape != A.shape[:1]):
            raise ValueError("rank is int32 [slots]")
        self.tensors = tuple(t for t in (A, Bm, scale, rank) if t is not None)
        _on_gpu(*self.tensors)
        self.struct = _Lora(_ptr(A), _ptr(Bm), _ptr(rank), _ptr(scale), A.shape[2], Bm.shape[1], A.shape[0], A.shape[1],
                            LORA_F16 if A.dtype == torch.float16 else LORA_BF16)
        self.ref = ctypes.addressof(self.struct)
        self.device = A.get_device()


def _own(descriptor, d):
    """Address of a descriptor whose tensors are on GPU d (the current one)."""
    if descriptor.device != d:
        raise ValueError("the descriptor's tensors are on another GPU than the current one")
    return descriptor.ref


def kv_plan_ws_bytes(pool) -> int:
    return int(lib.kv_plan_ws_bytes(pool.ref))


def kv_plan(pool, kv_len, keep, n_new, free_count, new_len, new_count, row_start, position, slot, status, T, ws, ws_bytes,
            stream=None):
    d = _device()
    p = _own(pool, d)
    *args, ws = _gpu(d, kv_len, keep, n_new, free_count, new_len, new_count, row_start, position, slot, status, ws)
    _step("kv_plan", d, stream, p, *args, T, ws, ws_bytes)


def embed_q8_0(W, tokens, y, N, K, M, scale, stream=None):
    d = _device()
    _step("embed_q8_0", d, stream, *_gpu(d, W, tokens, y), N, K, M, scale)


def embed_q4_0(W, tokens, y, N, K, M, scale, stream=None):
    d = _device()
    _step("embed_q4_0", d, stream, *_gpu(d, W, tokens, y), N, K, M, scale)


def embed_q4_k(W, tokens, y, N, K, M, scale, stream=None):
    d = _device()
    _step("embed_q4_k", d, stream, *_gpu(d, W, tokens, y), N, K, M, scale)


def embed_q6_k(W, tokens, y, N, K, M, scale, stream=None):
    d = _device()
    _step("embed_q6_k", d, stream, *_gpu(d, W, tokens, y), N, K, M, scale)


def lora_add_ws_bytes(lora, B, T) -> int:
    return int(lib.lora_add_ws_bytes(lora.ref, B, T))


def lora_add(lora, adapter, row_start, x, ldx, base, ldb, y, ldy, B, T, ws, ws_bytes, stream=None):
    d = _device()
    p = _own(lora, d)
    adapter, row_start, x, base, y, ws = _gpu(d, adapter, row_start, x, base, y, ws)
    _step("lora_add", d, stream, p, adapter, row_start, x, ldx, base, ldb, y, ldy, B, T, ws, ws_bytes)


def logits_draw_ws_bytes(V, M) -> int:
    return int(lib.logits_draw_ws_bytes(V, M))


def logits_draw(logits, ldl, temperature, top_k, top_p, min_p, u, token, kept, V, M, softcap, ws, ws_bytes, stream=None):
    d = _device()
    logits, temperature, top_k, top_p, min_p, u, token, kept, ws = _gpu(d, logits, temperature, top_k, top_p, min_p, u,
                                                                        token, kept, ws)
    _step("logits_draw", d, stream, logits, ldl, temperature, top_k, top_p, min_p, u, token, kept, V, M, softcap, ws, ws_bytes)
