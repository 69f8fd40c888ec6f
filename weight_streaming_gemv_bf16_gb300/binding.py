"""Thin ctypes binding of libwsgemv.so (argument marshalling only).

Every function here has the name of a C entry point without its ``ws_``
prefix and forwards to it; all arithmetic runs in the library's CUDA kernels.
Tensors are torch CUDA tensors (torch supplies device memory and streams);
their data pointers, shapes and the current stream's handle are what cross the
ABI.  A nonzero status raises ``WsError`` carrying the library's message.

If the shared library is missing the import fails loudly: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

C = ctypes
P = C.c_void_p
I32 = C.c_int
SZ = C.c_size_t
F32 = C.c_float
LL = C.c_longlong

DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
PREFETCH_NONE, PREFETCH_L2, PREFETCH_L2_EVICT_LAST, PREFETCH_BULK = 0, 1, 2, 3
BLOCK_QWEN, BLOCK_MLP, BLOCK_HEAD = 1, 2, 3
OP_GEMV, OP_SWIGLU_GEMV, OP_QKV_GEMV, OP_LMHEAD_ARGMAX, OP_ARGMAX_ROWS = 1, 2, 3, 4, 5
PRO_NONE, PRO_RMSNORM, PRO_LAYERNORM = 0, 1, 2
EPI_F32, EPI_BF16, EPI_RESID, EPI_BIAS_GELU, EPI_SWIGLU, EPI_ARGMAX = 0, 1, 2, 3, 4, 5

STATUS = {0: "WS_OK", -1: "WS_ERR_ARG", -2: "WS_ERR_ALIGN", -3: "WS_ERR_SHAPE",
          -4: "WS_ERR_CUDA", -5: "WS_ERR_TIMEOUT", -6: "WS_ERR_NOMEM", -7: "WS_ERR_STATE"}


class WsError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class PrefetchPlan(C.Structure):
    _fields_ = [("blocks", I32), ("threads", I32), ("stride_bytes", I32), ("mode", I32)]


class QwenBlock(C.Structure):
    _fields_ = [(n, P) for n in ("gamma1", "Wq", "Wk", "Wv", "Wo", "gamma2", "Wg", "Wu", "Wd",
                                 "attn", "q", "k", "v", "k_cache", "v_cache")]


class MlpBlock(C.Structure):
    _fields_ = [(n, P) for n in ("gamma", "beta", "W", "bias")]


class HeadBlock(C.Structure):
    _fields_ = [(n, P) for n in ("gamma", "W", "idx", "logits")]


class _BlockUnion(C.Union):
    _fields_ = [("qwen", QwenBlock), ("mlp", MlpBlock), ("head", HeadBlock)]


class BlockDesc(C.Structure):
    _fields_ = [("kind", I32), ("u", _BlockUnion)]


class ChainOpts(C.Structure):
    _fields_ = [("batch", I32), ("hidden", I32), ("kv_dim", I32), ("inter", I32),
                ("vocab", I32), ("eps", F32), ("h_in", P), ("h_out", P), ("x_in", P),
                ("y_out", P), ("h_trace", P), ("use_pdl", I32), ("prefetch", I32),
                ("fixed_plan", PrefetchPlan), ("distance", I32), ("decoy", I32),
                ("tune_pairs", I32), ("tune_min_gain", F32), ("weight_format", I32),
                ("persistent", I32), ("attention", I32), ("s_max", I32), ("pos", P),
                ("mlp_ln", P), ("mlp_pre", P), ("mlp_gelu_grad", P), ("mlp_ln_stats", P)]


class MlpGrads(C.Structure):
    _fields_ = [("dW", P), ("db", P), ("dgamma", P), ("dbeta", P)]


class MlpBackwardOpts(C.Structure):
    _fields_ = [("batch", I32), ("width", I32), ("x_in", P), ("acts", P), ("ln", P),
                ("gelu_grad", P), ("ln_stats", P), ("dz", P), ("dx", P), ("dx_trace", P),
                ("dlin_trace", P), ("dln_trace", P), ("use_pdl", I32), ("prefetch", I32),
                ("fixed_plan", PrefetchPlan), ("distance", I32), ("decoy", I32),
                ("tune_pairs", I32), ("tune_min_gain", F32)]


class Tuning(C.Structure):
    _fields_ = [("ring_bytes", I32), ("grid_cap", I32), ("force_ksplit", I32),
                ("force_rt", I32), ("evict_first", I32), ("piece_bytes", I32),
                ("timeout_ns", C.c_ulonglong), ("l2_ahead", I32),
                ("forms", I32), ("launch_pdl", I32), ("mma", I32), ("ctas_per_sm", I32),
                ("q4_mma", I32)]


class GemvSchedule(C.Structure):
    _fields_ = [(n, I32) for n in ("RT", "S", "KS", "PC", "NP", "NSW", "piece_bytes", "RG",
                                   "grid", "smem_bytes")]


_SIGS = {
    "ws_gemv_bf16": [P, P, P, I32, I32, I32, P, SZ, P],
    "ws_gemv_bf16_noalloc": [P, P, P, I32, I32, I32, P],
    "ws_gemv_residual": [P, P, P, P, I32, I32, I32, P, SZ, P],
    "ws_rmsnorm_gemv": [P, I32, P, P, P, I32, I32, I32, F32, P, SZ, P],
    "ws_qkv_gemv": [P, I32, P, P, P, P, P, P, P, I32, I32, I32, I32, F32, P, SZ, P],
    "ws_swiglu_gemv": [P, I32, P, P, P, P, I32, I32, I32, F32, P, SZ, P],
    "ws_ln_gemv_gelu": [P, P, P, P, P, P, I32, I32, I32, F32, P, SZ, P],
    "ws_lmhead_argmax": [P, I32, P, P, P, P, I32, I32, I32, F32, P, SZ, P],
    "ws_argmax_rows": [P, P, I32, I32, P, SZ, P],
    "ws_decode_attention": [P, P, P, P, P, P, P, P, I32, I32, I32, I32, I32, P, SZ, P],
    "ws_prompt_attention": [P, P, P, I32, P, P, P, I32, I32, I32, I32, I32, LL, LL, LL, P],
    "ws_kv_store_q4": [P, P, I32, P, P, P, P, P, I32, I32, I32, I32, I32, I32, LL, LL, P],
    "ws_kv_load_q4": [P, P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, P],
    "ws_decode_attention_q4": [P, P, P, P, P, P, P, P, I32, I32, I32, I32, I32, P, SZ, P],
    "ws_token_logprobs": [P, I32, LL, P, P, P, P, P, I32, I32, I32, P, SZ, P],
    "ws_quantize_q4": [P, P, I32, I32, P],
    "ws_gemv_q4": [P, P, P, I32, I32, I32, P, SZ, P],
    "ws_rmsnorm": [P, P, P, I32, I32, I32, F32, P],
    "ws_l2_prefetch": [P, SZ, PrefetchPlan, P],
    "ws_chain_create": [P, I32, P, P],
    "ws_chain_tune": [P, P],
    "ws_chain_capture": [P, P],
    "ws_chain_run": [P, P],
    "ws_chain_run_eager": [P, P],
    "ws_chain_step_host": [P, P, P, P, P],
    "ws_chain_plans": [P, P, P, P, I32],
    "ws_chain_op_bytes": [P, P, I32],
    "ws_mlp_backward_create": [P, P, I32, P, P],
    "ws_mlp_backward_tune": [P, P],
    "ws_mlp_backward_capture": [P, P],
    "ws_mlp_backward_run": [P, P],
    "ws_mlp_backward_plan": [P, P, P, P],
    "ws_set_tuning": [P],
    "ws_gemv_plan": [I32, I32, I32, I32, I32, I32, I32, P],
    "ws_read_probe": [P, SZ, I32, P, P],
    "ws_empty_probe": [I32, P, P, P],
    "ws_test_bounded_wait": [C.c_ulonglong, P],
    "ws_test_withhold": [I32, I32],
}
_OTHER = {
    "ws_workspace_bytes": ([I32, I32, I32, I32], SZ),
    "ws_attention_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
    "ws_attention_q4_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
    "ws_logprobs_workspace_bytes": ([I32, I32, I32], SZ),
    "ws_kv_q4_row_bytes": ([I32], SZ),
    "ws_q4_row_bytes": ([I32], SZ),
    "ws_last_error": ([], C.c_char_p),
    "ws_device_error": ([I32], I32),
    "ws_chain_num_ops": ([P], I32),
    "ws_chain_is_persistent": ([P], I32),
    "ws_chain_grid": ([P], I32),
    "ws_chain_debug_stamps": ([P, P, SZ], I32),
    "ws_chain_destroy": ([P], None),
    "ws_mlp_backward_num_launches": ([P], I32),
    "ws_mlp_backward_destroy": ([P], None),
    "ws_get_tuning": ([P], None),
    "ws_debug_gemv_copies": ([I32, I32, I32, I32, I32, I32, P, C.c_long], C.c_long),
    "ws_debug_gemv_copies_q4": ([I32, I32, I32, I32, I32, I32, P, C.c_long, P], C.c_long),
    "ws_debug_kv_places": ([P, P, P, I32, I32, I32, I32, P], C.c_long),
    "ws_version": ([], C.c_char_p),
}

_lib = None


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load libwsgemv.so (built by ``build()``); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: run __graft_entry__.build() (nvcc, sm_103a) first")
    lib = C.CDLL(path)
    for name, args in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = I32
    for name, (args, res) in _OTHER.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise WsError(status, load().ws_last_error().decode(errors="replace"))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle without a Stream object (0.1 us against 3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ws(workspace):
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _dtype_code(t):
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float16:
        return DTYPE_F16
    raise TypeError(f"unsupported dtype {t.dtype}")


# --------------------------------------------------------------------------- ops

def workspace_bytes(op: int, M: int, K: int, B: int) -> int:
    return int(load().ws_workspace_bytes(op, M, K, B))


def new_workspace(op: int, M: int, K: int, B: int, device="cuda"):
    """A zero-filled workspace sized for the op (None when it needs none)."""
    n = workspace_bytes(op, M, K, B)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def gemv_bf16(W, x, y, workspace=None, stream=None):
    M, K = W.shape
    B = x.shape[0]
    wp, wb = _ws(workspace)
    _check(load().ws_gemv_bf16(_ptr(W), _ptr(x), _ptr(y), M, K, B, wp, wb, _stream(stream)))


def gemv_bf16_noalloc(W, x, y, stream=None):
    """ws_gemv_bf16 without a workspace argument and without any allocation:
    split-K scratch comes from the library's fixed device array."""
    M, K = W.shape
    B = x.shape[0]
    _check(load().ws_gemv_bf16_noalloc(_ptr(W), _ptr(x), _ptr(y), M, K, B, _stream(stream)))


def gemv_residual(W, x, h_out, h_in=None, workspace=None, stream=None):
    M, K = W.shape
    B = x.shape[0]
    wp, wb = _ws(workspace)
    _check(load().ws_gemv_residual(_ptr(W), _ptr(x), _ptr(h_in), _ptr(h_out), M, K, B, wp, wb,
                                   _stream(stream)))


def rmsnorm_gemv(x, gamma, W, y, eps, workspace=None, stream=None):
    M, K = W.shape
    B = x.shape[0]
    wp, wb = _ws(workspace)
    _check(load().ws_rmsnorm_gemv(_ptr(x), _dtype_code(x), _ptr(gamma), _ptr(W), _ptr(y), M, K,
                                  B, float(eps), wp, wb, _stream(stream)))


def qkv_gemv(x, gamma, Wq, Wk, Wv, q, k, v, eps, workspace=None, stream=None):
    Mq, K = Wq.shape
    Mkv = Wk.shape[0]
    B = x.shape[0]
    wp, wb = _ws(workspace)
    _check(load().ws_qkv_gemv(_ptr(x), _dtype_code(x), _ptr(gamma), _ptr(Wq), _ptr(Wk),
                              _ptr(Wv), _ptr(q), _ptr(k), _ptr(v), Mq, Mkv, K, B, float(eps),
                              wp, wb, _stream(stream)))


def swiglu_gemv(x, gamma, Wg, Wu, s, eps, workspace=None, stream=None):
    M, K = Wg.shape
    B = x.shape[0]
    wp, wb = _ws(workspace)
    _check(load().ws_swiglu_gemv(_ptr(x), _dtype_code(x), _ptr(gamma), _ptr(Wg), _ptr(Wu),
                                 _ptr(s), M, K, B, float(eps), wp, wb, _stream(stream)))


def ln_gemv_gelu(x, gamma, beta, W, bias, z, eps, workspace=None, stream=None):
    M, K = W.shape
    B = x.shape[0]
    wp, wb = _ws(workspace)
    _check(load().ws_ln_gemv_gelu(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(W), _ptr(bias),
                                  _ptr(z), M, K, B, float(eps), wp, wb, _stream(stream)))


def lmhead_argmax(h, gamma, W, idx, eps, workspace, logits=None, stream=None):
    V, K = W.shape
    B = h.shape[0]
    wp, wb = _ws(workspace)
    _check(load().ws_lmhead_argmax(_ptr(h), _dtype_code(h), _ptr(gamma), _ptr(W), _ptr(idx),
                                   _ptr(logits), V, K, B, float(eps), wp, wb, _stream(stream)))


def argmax_rows(logits, idx, workspace, stream=None):
    rows, cols = logits.shape
    wp, wb = _ws(workspace)
    _check(load().ws_argmax_rows(_ptr(logits), _ptr(idx), rows, cols, wp, wb, _stream(stream)))


def q4_row_bytes(K: int) -> int:
    return int(load().ws_q4_row_bytes(K))


def quantize_q4(W, Wq, stream=None):
    """W bf16 [M, K] -> Wq uint8 [M, q4_row_bytes(K)] (4-bit groups of 128)."""
    M, K = W.shape
    _check(load().ws_quantize_q4(_ptr(W), _ptr(Wq), M, K, _stream(stream)))


def gemv_q4(Wq, x, y, K, workspace=None, stream=None):
    """y [B, M] fp32 = x [B, K] bf16 . W^T for packed 4-bit rows Wq [M, q4_row_bytes(K)]."""
    M = Wq.shape[0]
    B = x.shape[0]
    wp, wb = _ws(workspace)
    _check(load().ws_gemv_q4(_ptr(Wq), _ptr(x), _ptr(y), M, K, B, wp, wb, _stream(stream)))


def attention_workspace_bytes(B, n_heads, n_kv_heads, s_max, head_dim=128) -> int:
    return int(load().ws_attention_workspace_bytes(B, n_heads, n_kv_heads, head_dim, s_max))


def decode_attention(q, k_new, v_new, k_cache, v_cache, pos, workspace, out_f32=None,
                     out_bf16=None, stream=None):
    """q [B, n_heads*128] fp32, k_new/v_new [B, n_kv*128] fp32, caches bf16
    [B, n_kv, s_max, 128] (updated in place at pos), pos int32 [B] on the device."""
    B, n_kv, s_max, d = k_cache.shape
    n_heads = q.shape[1] // d
    wp, wb = _ws(workspace)
    _check(load().ws_decode_attention(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                      _ptr(v_cache), _ptr(pos), _ptr(out_f32), _ptr(out_bf16),
                                      B, n_heads, n_kv, d, s_max, wp, wb, _stream(stream)))


# The serving operators check their tensors here: type, shape, strides and that
# they are on the current device, where the library launches.  Each check hands
# on the pointer (a step's calls are short enough for the host to matter).

_I32, _F32, _U8, _BF16 = torch.int32, torch.float32, torch.uint8, torch.bfloat16
_CODES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
_here = torch.cuda.current_device


def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


def _code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _at(t, dtype, shape, dev: int, what: str):
    """The address of a contiguous tensor of this type and shape; None passes."""
    if t is None:
        return None
    if t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        raise ValueError(f"{what} on {t.device}: expected the current device, cuda:{dev}")
    raise ValueError(f"{what}: expected contiguous {dtype} {tuple(shape)}, "
                     f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")


def _tokens_at(t, dev: int, what: str):
    """[T, heads, d] with each token's heads contiguous -> (shape, token stride, address)."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{what}: expected [tokens, heads, head_dim], got {tuple(shape)}")
    T, n, d = shape
    st, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and n > 1):
        raise ValueError(f"{what}: a token's heads must be contiguous, got strides {t.stride()}")
    if t.get_device() != dev:
        raise ValueError(f"{what} on {t.device}: expected the current device, cuda:{dev}")
    return shape, (st if T > 1 else n * d), t.data_ptr()


def _stream_on(stream, dev: int):
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _space_at(ws, dev: int):
    if ws.get_device() != dev:
        raise ValueError(f"workspace on {ws.device}: expected the current device")
    if not ws.is_contiguous():
        raise ValueError(f"workspace: expected one piece, got strides {ws.stride()}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def prompt_attention(q, k, v, cu_seqlens, out, lse=None, stream=None):
    """Causal attention over packed prompts.  q [T, n_heads, 128], k and v
    [T, n_kv, 128] in bf16 or fp16 (token strides free, so columns of one
    fused projection will do), cu_seqlens int32 [n_seqs + 1] on the device,
    out [T, n_heads * 128] of the same type, lse fp32 [T, n_heads] or None."""
    dev = _here()
    (T, nh, d), qs, qp = _tokens_at(q, dev, "q")
    kshape, ks, kp = _tokens_at(k, dev, "k")
    vshape, vs, vp = _tokens_at(v, dev, "v")
    nkv = kshape[1]
    _need(kshape == vshape and kshape[0] == T and kshape[2] == d, "q, k and v disagree in shape")
    dt = q.dtype
    _need(k.dtype is dt and v.dtype is dt, "q, k and v disagree in type")
    n = cu_seqlens.shape[0]
    _check(load().ws_prompt_attention(
        qp, kp, vp, _code(dt), _at(cu_seqlens, _I32, (n,), dev, "cu_seqlens"),
        _at(out, dt, (T, nh * d), dev, "out"), _at(lse, _F32, (T, nh), dev, "lse"), T,
        n - 1, nh, nkv, d, qs, ks, vs, _stream_on(stream, dev)))


_KV_Q4_ROW = 80  # bytes of a cached row, ws_kv_q4_row_bytes(128)


def kv_q4_row_bytes(head_dim=128) -> int:
    return int(load().ws_kv_q4_row_bytes(head_dim))


def new_kv_cache_q4(n_rows, n_kv_heads, s_max, head_dim=128, device="cuda"):
    """One 4-bit cache (keys or values): uint8 [n_rows, n_kv, s_max, 80]."""
    return torch.zeros((n_rows, n_kv_heads, s_max, kv_q4_row_bytes(head_dim)), dtype=_U8,
                       device=device)


def _kv_q4_args(nkv, k_cache, v_cache, start, cu_seqlens, rows, dev):
    shape = k_cache.shape
    _need(len(shape) == 4 and shape[3] == _KV_Q4_ROW and shape[1] == nkv,
          "k_cache: expected [rows, n_kv, s_max, 80]")
    n = start.shape[0]
    return (_at(cu_seqlens, _I32, (n + 1,), dev, "cu_seqlens"),
            _at(rows, _I32, (n,), dev, "rows"),
            _at(start, _I32, (n,), dev, "start"),
            _at(k_cache, _U8, shape, dev, "k_cache"),
            _at(v_cache, _U8, shape, dev, "v_cache"), n, shape[0], shape[2])


def kv_store_q4(k, v, k_cache, v_cache, start, cu_seqlens=None, rows=None, stream=None):
    """k, v [T, n_kv, 128] (fp32, bf16 or fp16) into the 4-bit caches uint8
    [n_rows, n_kv, s_max, 80] from slot start[i] on of cache row rows[i] (i
    without `rows`) for the tokens cu_seqlens[i] .. cu_seqlens[i + 1] - 1
    (token i alone without `cu_seqlens`)."""
    dev = _here()
    shape, ks, kp = _tokens_at(k, dev, "k")
    vshape, vs, vp = _tokens_at(v, dev, "v")
    dt = k.dtype
    _need(vshape == shape and v.dtype is dt, "k and v disagree")
    T, nkv, d = shape
    cu, rw, st, kc, vc, n, n_rows, s_max = _kv_q4_args(nkv, k_cache, v_cache, start, cu_seqlens,
                                                       rows, dev)
    _check(load().ws_kv_store_q4(kp, vp, _code(dt), cu, rw, st, kc, vc, T, n, n_rows, nkv, d,
                                 s_max, ks, vs, _stream_on(stream, dev)))


def kv_load_q4(k_cache, v_cache, start, k, v, cu_seqlens=None, rows=None, stream=None):
    """The values that cached rows stand for, to k and v [T, n_kv, 128] (fp32,
    bf16 or fp16, contiguous); the other arguments as for kv_store_q4."""
    dev = _here()
    shape, dt = k.shape, k.dtype
    _need(len(shape) == 3, "k: expected [tokens, heads, head_dim]")
    T, nkv, d = shape
    kp = _at(k, dt, shape, dev, "k")
    vp = _at(v, dt, shape, dev, "v")
    cu, rw, st, kc, vc, n, n_rows, s_max = _kv_q4_args(nkv, k_cache, v_cache, start, cu_seqlens,
                                                       rows, dev)
    _check(load().ws_kv_load_q4(kc, vc, cu, rw, st, kp, vp, _code(dt), T, n, n_rows, nkv, d,
                                s_max, _stream_on(stream, dev)))


def attention_q4_workspace_bytes(B, n_heads, n_kv_heads, s_max, head_dim=128) -> int:
    return int(load().ws_attention_q4_workspace_bytes(B, n_heads, n_kv_heads, head_dim, s_max))


def decode_attention_q4(q, k_new, v_new, k_cache, v_cache, pos, workspace, out_f32=None,
                        out_bf16=None, stream=None):
    """decode_attention over the 4-bit caches uint8 [B, n_kv, s_max, 80]: q
    [B, n_heads*128] fp32, k_new/v_new [B, n_kv*128] fp32 (quantised into the
    caches at pos), pos int32 [B] on the device (negative: no sequence)."""
    dev = _here()
    shape = k_cache.shape
    _need(len(shape) == 4 and shape[3] == _KV_Q4_ROW, "k_cache: expected [B, n_kv, s_max, 80]")
    B, nkv, s_max, _ = shape
    d = 128
    nh = q.shape[-1] // d
    new = (B, nkv * d)
    heads = (B, nh * d)
    wp, wb = _space_at(workspace, dev)
    _check(load().ws_decode_attention_q4(
        _at(q, _F32, heads, dev, "q"), _at(k_new, _F32, new, dev, "k_new"),
        _at(v_new, _F32, new, dev, "v_new"), _at(k_cache, _U8, shape, dev, "k_cache"),
        _at(v_cache, _U8, shape, dev, "v_cache"),
        _at(pos, _I32, (B,), dev, "pos"), _at(out_f32, _F32, heads, dev, "out_f32"),
        _at(out_bf16, _BF16, heads, dev, "out_bf16"), B, nh, nkv, d, s_max, wp, wb,
        _stream_on(stream, dev)))


def logprobs_workspace_bytes(rows, V, topk=0) -> int:
    return int(load().ws_logprobs_workspace_bytes(rows, V, topk))


def token_logprobs(logits, workspace, targets=None, logprob=None, entropy=None, top_idx=None,
                   top_logprob=None, stream=None):
    """Log-probabilities over logits [rows, V] (fp32, bf16 or fp16; rows may be
    padded): logprob fp32 [rows] of targets int32 [rows], entropy fp32 [rows],
    top_idx int32 and top_logprob fp32 [rows, topk]; each output may be None."""
    dev = _here()
    rows, V = logits.shape
    st, s1 = logits.stride()
    _need(s1 == 1 or V == 1, "logits: a row's values must be contiguous")
    _need(logits.get_device() == dev, f"logits on {logits.device}: expected the current device")
    top = top_idx if top_idx is not None else top_logprob
    topk = 0 if top is None else top.shape[-1]
    row, alt = (rows,), (rows, topk)
    wp, wb = _space_at(workspace, dev)
    _check(load().ws_token_logprobs(
        logits.data_ptr(), _code(logits.dtype), st if rows > 1 else V,
        _at(targets, _I32, row, dev, "targets"), _at(logprob, _F32, row, dev, "logprob"),
        _at(entropy, _F32, row, dev, "entropy"), _at(top_idx, _I32, alt, dev, "top_idx"),
        _at(top_logprob, _F32, alt, dev, "top_logprob"), rows, V, topk, wp, wb,
        _stream_on(stream, dev)))


def rmsnorm(x, gamma, y, eps, stream=None):
    R, N = x.shape
    _check(load().ws_rmsnorm(_ptr(x), _ptr(gamma), _ptr(y), R, N, _dtype_code(x), float(eps),
                             _stream(stream)))


def l2_prefetch(ptr, nbytes, plan: PrefetchPlan, stream=None):
    _check(load().ws_l2_prefetch(_ptr(ptr), int(nbytes), plan, _stream(stream)))


def read_probe(buf, nbytes, blocks, sink, stream=None):
    _check(load().ws_read_probe(_ptr(buf), int(nbytes), int(blocks), _ptr(sink), _stream(stream)))


def empty_probe(touch, ptr=None, sink=None, stream=None):
    _check(load().ws_empty_probe(int(touch), _ptr(ptr), _ptr(sink), _stream(stream)))


def test_bounded_wait(timeout_ns, stream=None):
    _check(load().ws_test_bounded_wait(int(timeout_ns), _stream(stream)))


def test_withhold(cta, copy=0):
    _check(load().ws_test_withhold(int(cta), int(copy)))


def device_error(reset=False) -> int:
    return int(load().ws_device_error(1 if reset else 0))


def get_tuning() -> Tuning:
    t = Tuning()
    load().ws_get_tuning(C.byref(t))
    return t


def set_tuning(t: Tuning):
    _check(load().ws_set_tuning(C.byref(t)))


def gemv_plan(M, K, B, nmat=1, prologue=PRO_NONE, epilogue=EPI_F32, allow_split=True):
    s = GemvSchedule()
    _check(load().ws_gemv_plan(M, K, B, nmat, prologue, epilogue, 1 if allow_split else 0,
                               C.byref(s)))
    return {n: getattr(s, n) for n, _ in GemvSchedule._fields_}


def debug_gemv_copies_q4(M, K, B, nmat, cta, mma=False):
    """(triples, schedule dict) of CTA `cta` for packed 4-bit rows."""
    lib = load()
    sc = GemvSchedule()
    n = lib.ws_debug_gemv_copies_q4(M, K, B, nmat, cta, int(mma), None, 0, C.byref(sc))
    if n < 0:
        raise WsError(-1, "bad arguments")
    buf = (C.c_longlong * (3 * max(n, 1)))()
    lib.ws_debug_gemv_copies_q4(M, K, B, nmat, cta, int(mma), buf, n, None)
    sched = {f: getattr(sc, f) for f, _ in GemvSchedule._fields_}
    return [(buf[3 * i], buf[3 * i + 1], buf[3 * i + 2]) for i in range(n)], sched


def debug_gemv_copies(M, K, B, nmat, allow_split, cta):
    lib = load()
    n = lib.ws_debug_gemv_copies(M, K, B, nmat, int(allow_split), cta, None, 0)
    if n < 0:
        raise WsError(-1, "bad arguments")
    buf = (C.c_longlong * (3 * max(n, 1)))()
    lib.ws_debug_gemv_copies(M, K, B, nmat, int(allow_split), cta, buf, n)
    return [(buf[3 * i], buf[3 * i + 1], buf[3 * i + 2]) for i in range(n)]


def debug_kv_places(cu_seqlens, rows, start, T, n_rows, s_max):
    """Per token of one head: row * s_max + slot, -1 skipped, -2 flagged (host lists)."""
    def ints(v):
        return None if v is None else (C.c_int32 * len(v))(*v)
    out = (C.c_longlong * T)()
    if load().ws_debug_kv_places(ints(cu_seqlens), ints(rows), ints(start), T, len(start), n_rows,
                                 s_max, out) < 0:
        raise WsError(-1, "bad arguments")
    return list(out)


def version() -> str:
    return load().ws_version().decode()


# --------------------------------------------------------------------------- chain

class Chain:
    """A decode chain: ws_chain_create / tune / capture / run / destroy.

    Keeps the Python objects whose device memory the chain points at alive."""

    def __init__(self, blocks, opts: ChainOpts, keepalive=()):
        arr = (BlockDesc * len(blocks))(*blocks)
        h = P()
        _check(load().ws_chain_create(arr, len(blocks), C.byref(opts), C.byref(h)))
        self.handle = h
        self.opts = opts
        self._keep = list(keepalive)
        self.n_ops = int(load().ws_chain_num_ops(h))
        self.persistent = bool(load().ws_chain_is_persistent(h))

    def tune(self, stream=None):
        _check(load().ws_chain_tune(self.handle, _stream(stream)))

    def capture(self, stream=None):
        _check(load().ws_chain_capture(self.handle, _stream(stream)))

    def run(self, stream=None):
        _check(load().ws_chain_run(self.handle, _stream(stream)))

    def run_eager(self, stream=None):
        _check(load().ws_chain_run_eager(self.handle, _stream(stream)))

    def step_host(self, in_host, attn_host, out_host, stream=None):
        _check(load().ws_chain_step_host(self.handle, _ptr(in_host), _ptr(attn_host),
                                         _ptr(out_host), _stream(stream)))

    def plans(self):
        n = self.n_ops
        pl = (PrefetchPlan * n)()
        lo = (F32 * n)()
        mean = (F32 * n)()
        _check(load().ws_chain_plans(self.handle, pl, lo, mean, n))
        return [((p.mode, p.blocks, p.threads, p.stride_bytes), lo[i], mean[i])
                for i, p in enumerate(pl)]

    def debug_stamps(self, buf):
        """Record per-CTA, per-op timestamps and per-warp wait times into `buf`
        (int64 [grid, ops, 44]) on every later-captured step; None stops.
        Re-capture afterwards."""
        n = 0 if buf is None else buf.numel()
        _check(load().ws_chain_debug_stamps(self.handle, _ptr(buf), n))

    def grid(self) -> int:
        return int(load().ws_chain_grid(self.handle))

    def op_bytes(self):
        n = self.n_ops
        b = (SZ * n)()
        _check(load().ws_chain_op_bytes(self.handle, b, n))
        return list(b)

    def close(self):
        if self.handle:
            load().ws_chain_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MlpBackward:
    """The backward pass of a LayerNorm -> Linear -> GELU chain:
    ws_mlp_backward_create / tune / capture / run / destroy.  Keeps the
    Python objects whose device memory it points at alive."""

    def __init__(self, blocks, grads, opts: MlpBackwardOpts, keepalive=()):
        n = len(blocks)
        barr = (MlpBlock * n)(*blocks)
        garr = (MlpGrads * n)(*grads)
        h = P()
        _check(load().ws_mlp_backward_create(barr, garr, n, C.byref(opts), C.byref(h)))
        self.handle = h
        self.opts = opts
        self._keep = list(keepalive)
        self.n_launches = int(load().ws_mlp_backward_num_launches(h))

    def tune(self, stream=None):
        _check(load().ws_mlp_backward_tune(self.handle, _stream(stream)))

    def capture(self, stream=None):
        _check(load().ws_mlp_backward_capture(self.handle, _stream(stream)))

    def run(self, stream=None):
        _check(load().ws_mlp_backward_run(self.handle, _stream(stream)))

    def plan(self):
        pl = PrefetchPlan()
        lo, mean = F32(), F32()
        _check(load().ws_mlp_backward_plan(self.handle, C.byref(pl), C.byref(lo), C.byref(mean)))
        return (pl.mode, pl.blocks, pl.threads, pl.stride_bytes), lo.value, mean.value

    def close(self):
        if self.handle:
            load().ws_mlp_backward_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def chain_run(chain: Chain, stream=None):
    chain.run(stream)
