"""ctypes binding over libdiffattn.so (include/diffattn.h).

Argument marshalling only: tensors become pointers, shapes and element strides become
the parameter structs, and the current torch CUDA stream becomes the launch stream.
Every step of the operator runs in the library's kernels. There is no fallback: if the
library is missing or a call fails, these functions raise.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libdiffattn.so"

DIFFATTN_F32, DIFFATTN_BF16 = 0, 1
DIFFATTN_V1, DIFFATTN_V2 = 1, 2

STATUS = {
    0: "DIFFATTN_OK",
    -1: "DIFFATTN_ERR_INVALID_ARG",
    -2: "DIFFATTN_ERR_UNSUPPORTED",
    -3: "DIFFATTN_ERR_MISALIGNED",
    -4: "DIFFATTN_ERR_WORKSPACE",
    -5: "DIFFATTN_ERR_CUDA",
    -6: "DIFFATTN_ERR_TIMEOUT",
}

# every symbol include/diffattn.h declares
EXPORTS = (
    "diffattn_version",
    "diffattn_status_string",
    "diffattn_lambda",
    "diffattn_fwd_prefill",
    "diffattn_fwd_prefill_varlen",
    "diffattn_bwd_workspace_size",
    "diffattn_bwd_prefill",
    "diffattn_lambda_bwd",
    "diffattn_fwd_prefill_train",
    "diffattn_bwd_prefill_saved",
    "diffattn_decode_workspace_size",
    "diffattn_fwd_decode",
    "diffattn_fwd_decode_static",
    "diffattn_fwd_decode_v1",
    "diffattn_fwd_decode_paged",
    "diffattn_kv4_write",
    "diffattn_kv4_read",
    "diffattn_decode_kv4_workspace_size",
    "diffattn_fwd_decode_kv4",
    "diffattn_selftest_timeout",
    "diffattn_selftest_exp2",
    "diffattn_debug_bounds_violations",
)


class DiffattnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {status} ({STATUS.get(status, 'unknown')})")


class PrefillParams(ctypes.Structure):
    _fields_ = [
        ("variant", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("batch", ctypes.c_int32),
        ("seqlen", ctypes.c_int32),
        ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("apply_norm", ctypes.c_int32),
        ("norm_eps", ctypes.c_float),
        ("q_strides", ctypes.c_int64 * 3),
        ("k_strides", ctypes.c_int64 * 3),
        ("v_strides", ctypes.c_int64 * 3),
        ("o_strides", ctypes.c_int64 * 3),
        ("kv_seqlen", ctypes.c_int32),
        ("window", ctypes.c_int32),
    ]


class DecodeParams(ctypes.Structure):
    _fields_ = [
        ("variant", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("batch", ctypes.c_int32),
        ("max_kv_len", ctypes.c_int32),
        ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("num_splits", ctypes.c_int32),
        ("q_strides", ctypes.c_int64 * 2),
        ("kv_strides", ctypes.c_int64 * 3),
        ("o_strides", ctypes.c_int64 * 2),
    ]


class Kv4Rows(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("batch", ctypes.c_int32),
        ("n_tokens", ctypes.c_int32),
        ("max_seqlen", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("max_kv_len", ctypes.c_int32),
        ("k_strides", ctypes.c_int64 * 3),
        ("v_strides", ctypes.c_int64 * 3),
        ("cache_strides", ctypes.c_int64 * 3),
    ]


_lib = None


def library_path() -> str:
    return os.environ.get("DIFFATTN_LIBRARY", os.path.join(_HERE, _LIB_NAME))


def load_library():
    """Load libdiffattn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m differential_attention_05_b200.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    vp, i32, f32p = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
    lib.diffattn_version.restype = i32
    lib.diffattn_version.argtypes = []
    lib.diffattn_status_string.restype = ctypes.c_char_p
    lib.diffattn_status_string.argtypes = [i32]
    lib.diffattn_lambda.restype = i32
    lib.diffattn_lambda.argtypes = [f32p, f32p, f32p, f32p, i32, i32, i32, f32p, f32p, vp]
    lib.diffattn_fwd_prefill.restype = i32
    lib.diffattn_fwd_prefill.argtypes = [ctypes.POINTER(PrefillParams), vp, vp, vp, f32p, f32p,
                                         vp, vp, vp]
    lib.diffattn_fwd_prefill_varlen.restype = i32
    lib.diffattn_fwd_prefill_varlen.argtypes = [ctypes.POINTER(PrefillParams), vp, vp, i32, vp, vp,
                                                vp, f32p, f32p, vp, vp, vp]
    lib.diffattn_bwd_workspace_size.restype = i32
    lib.diffattn_bwd_workspace_size.argtypes = [ctypes.POINTER(PrefillParams),
                                                ctypes.POINTER(ctypes.c_size_t)]
    lib.diffattn_bwd_prefill.restype = i32
    lib.diffattn_bwd_prefill.argtypes = [ctypes.POINTER(PrefillParams), vp, vp, vp, f32p, f32p, vp,
                                         vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
    lib.diffattn_fwd_prefill_train.restype = i32
    lib.diffattn_fwd_prefill_train.argtypes = [ctypes.POINTER(PrefillParams), vp, vp, vp, f32p, vp, vp,
                                               f32p, vp, vp]
    lib.diffattn_bwd_prefill_saved.restype = i32
    lib.diffattn_bwd_prefill_saved.argtypes = [ctypes.POINTER(PrefillParams), vp, vp, vp, f32p, vp, vp,
                                               f32p, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
    lib.diffattn_lambda_bwd.restype = i32
    lib.diffattn_lambda_bwd.argtypes = [f32p, f32p, f32p, f32p, i32, i32, f32p, vp, vp, vp, vp, vp]
    lib.diffattn_decode_workspace_size.restype = i32
    lib.diffattn_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeParams),
                                                   ctypes.POINTER(ctypes.c_size_t)]
    lib.diffattn_fwd_decode.restype = i32
    lib.diffattn_fwd_decode.argtypes = [ctypes.POINTER(DecodeParams), vp, vp, vp, vp, f32p, vp,
                                        vp, ctypes.c_size_t, vp, vp]
    lib.diffattn_fwd_decode_static.restype = i32
    lib.diffattn_fwd_decode_static.argtypes = [ctypes.POINTER(DecodeParams), vp, vp, vp, vp, f32p,
                                               vp, vp, vp]
    lib.diffattn_fwd_decode_v1.restype = i32
    lib.diffattn_fwd_decode_v1.argtypes = [ctypes.POINTER(DecodeParams), vp, vp, vp, vp, f32p, f32p,
                                           i32, ctypes.c_float, vp, vp, ctypes.c_size_t, vp, vp]
    lib.diffattn_fwd_decode_paged.restype = i32
    lib.diffattn_fwd_decode_paged.argtypes = [ctypes.POINTER(DecodeParams), ctypes.POINTER(PagedKV),
                                              vp, vp, vp, vp, vp, f32p, f32p, i32, ctypes.c_float,
                                              vp, vp, ctypes.c_size_t, vp, vp]
    lib.diffattn_selftest_timeout.restype = i32
    lib.diffattn_selftest_timeout.argtypes = [vp, i32, vp]
    lib.diffattn_selftest_exp2.restype = i32
    lib.diffattn_selftest_exp2.argtypes = [vp, vp, vp, i32, vp]
    lib.diffattn_debug_bounds_violations.restype = i32
    lib.diffattn_debug_bounds_violations.argtypes = [ctypes.POINTER(ctypes.c_int32)]
    lib.diffattn_kv4_write.restype = i32
    lib.diffattn_kv4_write.argtypes = [ctypes.POINTER(Kv4Rows), vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.diffattn_kv4_read.restype = i32
    lib.diffattn_kv4_read.argtypes = [ctypes.POINTER(Kv4Rows), vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.diffattn_decode_kv4_workspace_size.restype = i32
    lib.diffattn_decode_kv4_workspace_size.argtypes = [ctypes.POINTER(DecodeParams), vp,
                                                       ctypes.POINTER(ctypes.c_size_t)]
    lib.diffattn_fwd_decode_kv4.restype = i32
    lib.diffattn_fwd_decode_kv4.argtypes = [ctypes.POINTER(DecodeParams), vp, vp, vp, vp, vp, f32p, f32p,
                                            i32, ctypes.c_float, vp, vp, ctypes.c_size_t, vp, vp]
    _lib = lib
    return lib


def _check(fn: str, rc: int):
    if rc != 0:
        raise DiffattnError(fn, rc)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return DIFFATTN_BF16
    if t.dtype == torch.float32:
        return DIFFATTN_F32
    raise DiffattnError("dtype", -2)


def diffattn_status_string(status: int) -> str:
    return load_library().diffattn_status_string(int(status)).decode()


def diffattn_lambda(lq1, lk1, lq2, lk2, depth: int, lambda_out=None, lambda_init_out=None,
                    stream=None):
    """lambda[h] = exp(lq1[h].lk1[h]) - exp(lq2[h].lk2[h]) + lambda_init(depth), on device.
    lq*, lk*: float32 CUDA tensors [n_heads, dim]. Returns (lambda_out, lambda_init_out)."""
    import torch
    lib = load_library()
    H, dim = lq1.shape
    if lambda_out is None:
        lambda_out = torch.empty(H, dtype=torch.float32, device=lq1.device)
    if lambda_init_out is None:
        lambda_init_out = torch.empty(1, dtype=torch.float32, device=lq1.device)
    for t in (lq1, lk1, lq2, lk2):
        if not t.is_contiguous():
            raise DiffattnError("diffattn_lambda", -1)
    rc = lib.diffattn_lambda(_ptr(lq1), _ptr(lk1), _ptr(lq2), _ptr(lk2), H, dim, int(depth),
                             _ptr(lambda_out), _ptr(lambda_init_out), _stream(stream))
    _check("diffattn_lambda", rc)
    return lambda_out, lambda_init_out


def prefill_params(q, k, v, out, causal=True, apply_norm=None, norm_eps=1e-5,
                   window=0) -> PrefillParams:
    """Build the prefill parameter struct from tensor shapes and strides.
    V1: q [B,N,H,2,d], k [B,Nk,H,2,d], v [B,Nk,H,2d], out [B,N,H,2d].
    V2: q [B,N,Hq,d], k,v [B,Nk,Hkv,d], out [B,N,Hq/2,d]. Nk >= N: the queries are the last
    N positions (chunked prefill)."""
    p = PrefillParams()
    if q.dim() == 5:
        B, N, H, two, d = q.shape
        p.variant, p.n_q_heads, p.n_kv_heads = DIFFATTN_V1, H, H
        if two != 2:
            raise DiffattnError("diffattn_fwd_prefill", -1)
        p.apply_norm = 1 if apply_norm is None else int(bool(apply_norm))
        qs, ks = q.stride(), k.stride()
        p.q_strides[:] = (qs[0], qs[1], qs[2])
        p.k_strides[:] = (ks[0], ks[1], ks[2])
        if qs[3] != d or ks[3] != d or qs[4] != 1 or ks[4] != 1:
            raise DiffattnError("diffattn_fwd_prefill", -1)
    elif q.dim() == 4:
        B, N, Hq, d = q.shape
        p.variant, p.n_q_heads, p.n_kv_heads = DIFFATTN_V2, Hq, k.shape[2]
        p.apply_norm = 0 if apply_norm is None else int(bool(apply_norm))
        p.q_strides[:] = q.stride()[:3]
        p.k_strides[:] = k.stride()[:3]
        if q.stride(3) != 1 or k.stride(3) != 1:
            raise DiffattnError("diffattn_fwd_prefill", -1)
    else:
        raise DiffattnError("diffattn_fwd_prefill", -1)
    if v.stride(-1) != 1 or out.stride(-1) != 1:
        raise DiffattnError("diffattn_fwd_prefill", -1)
    p.dtype = _dtype_code(q)
    p.batch, p.seqlen, p.head_dim = B, N, d
    p.causal = int(bool(causal))
    p.norm_eps = float(norm_eps)
    if k.shape[1] != v.shape[1]:
        raise DiffattnError("diffattn_fwd_prefill", -1)
    p.kv_seqlen = int(k.shape[1])
    p.window = int(window)
    p.v_strides[:] = v.stride()[:3]
    p.o_strides[:] = out.stride()[:3]
    return p


def diffattn_fwd_prefill(q, k, v, lam, lambda_init=None, out=None, causal=True, apply_norm=None,
                         norm_eps=1e-5, dev_status=None, stream=None, window=0):
    """Fused differential attention prefill (see include/diffattn.h for layouts). k and v
    may hold more positions than q (chunked prefill); window > 0 is a causal sliding window."""
    import torch
    lib = load_library()
    if out is None:
        if q.dim() == 5:
            B, N, H, _, d = q.shape
            out = torch.empty((B, N, H, 2 * d), dtype=q.dtype, device=q.device)
        else:
            B, N, Hq, d = q.shape
            out = torch.empty((B, N, Hq // 2, d), dtype=q.dtype, device=q.device)
    p = prefill_params(q, k, v, out, causal, apply_norm, norm_eps, window)
    rc = lib.diffattn_fwd_prefill(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(lam),
                                  _ptr(lambda_init), _ptr(out), _ptr(dev_status), _stream(stream))
    _check("diffattn_fwd_prefill", rc)
    return out


def diffattn_fwd_prefill_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, lam,
                                lambda_init=None, out=None, causal=True, apply_norm=None,
                                norm_eps=1e-5, window=0, dev_status=None, stream=None):
    """Prefill over packed sequences of different lengths (see include/diffattn.h).
    V1: q [Tq,H,2,d], k [Tk,H,2,d], v [Tk,H,2d] -> out [Tq,H,2d]. V2: q [Tq,Hq,d],
    k,v [Tk,Hkv,d] -> out [Tq,Hq/2,d]. cu_seqlens_q / _k: int32 [S+1] device offsets;
    max_seqlen_q: the longest sequence's query count (host int)."""
    import torch
    lib = load_library()
    if out is None:
        if q.dim() == 4:
            T, H, _, d = q.shape
            out = torch.empty((T, H, 2 * d), dtype=q.dtype, device=q.device)
        else:
            T, Hq, d = q.shape
            out = torch.empty((T, Hq // 2, d), dtype=q.dtype, device=q.device)
    # the packed tensors viewed with a batch axis of one: the fixed-length struct applies
    p = prefill_params(q.unsqueeze(0), k.unsqueeze(0), v.unsqueeze(0), out.unsqueeze(0), causal,
                       apply_norm, norm_eps, window)
    p.batch = int(cu_seqlens_q.numel()) - 1
    if p.batch < 0 or cu_seqlens_k.numel() != cu_seqlens_q.numel():
        raise DiffattnError("diffattn_fwd_prefill_varlen", -1)
    p.seqlen, p.kv_seqlen = int(q.shape[0]), int(k.shape[0])
    for st in (p.q_strides, p.k_strides, p.v_strides, p.o_strides):
        st[0] = 0
    rc = lib.diffattn_fwd_prefill_varlen(ctypes.byref(p), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                         int(max_seqlen_q), _ptr(q), _ptr(k), _ptr(v), _ptr(lam),
                                         _ptr(lambda_init), _ptr(out), _ptr(dev_status),
                                         _stream(stream))
    _check("diffattn_fwd_prefill_varlen", rc)
    return out


def diffattn_bwd_workspace_size(p: PrefillParams) -> int:
    n = ctypes.c_size_t(0)
    _check("diffattn_bwd_workspace_size",
           load_library().diffattn_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def diffattn_bwd_prefill(q, k, v, lam, dout, lambda_init=None, causal=True, apply_norm=None,
                         norm_eps=1e-5, window=0, workspace=None, dev_status=None, stream=None,
                         grads=None):
    """Gradients of diffattn_fwd_prefill (see include/diffattn.h): dout has the forward
    output's layout and dtype. Returns float32 (dq, dk, dv, dlambda) in the shapes of q, k,
    v and lambda (written into `grads` when given: four dense float32 tensors)."""
    import torch
    lib = load_library()
    p = prefill_params(q, k, v, dout, causal, apply_norm, norm_eps, window)
    if grads is None:
        dq = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        dk = torch.empty(k.shape, dtype=torch.float32, device=q.device)
        dv = torch.empty(v.shape, dtype=torch.float32, device=q.device)
        dl = torch.empty(lam.shape, dtype=torch.float32, device=q.device)
    else:
        dq, dk, dv, dl = grads
    need = diffattn_bwd_workspace_size(p)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib.diffattn_bwd_prefill(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(lam),
                                  _ptr(lambda_init), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                                  _ptr(dl), _ptr(workspace), ws_bytes, _ptr(dev_status),
                                  _stream(stream))
    _check("diffattn_bwd_prefill", rc)
    return dq, dk, dv, dl


def diffattn_fwd_prefill_train(q, k, v, lam, out=None, o2=None, lse=None, causal=True, window=0,
                               dev_status=None, stream=None):
    """diffattn_fwd_prefill for training (V2 bf16, d = 128; see include/diffattn.h): returns
    (out, o2, lse) -- the output, the branch-2 output O_2 / l_2 in out's layout, and float32
    [B, Hq/2, N, 2] log2-domain log-sum-exps of both branches."""
    import torch
    lib = load_library()
    B, N, Hq, d = q.shape
    if out is None:
        out = torch.empty((B, N, Hq // 2, d), dtype=q.dtype, device=q.device)
    if o2 is None:
        o2 = torch.empty_like(out)
    if lse is None:
        lse = torch.empty((B, Hq // 2, N, 2), dtype=torch.float32, device=q.device)
    if o2.stride() != out.stride():
        raise ValueError("o2 must have out's layout")
    p = prefill_params(q, k, v, out, causal, None, 1e-5, window)
    rc = lib.diffattn_fwd_prefill_train(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out),
                                        _ptr(o2), _ptr(lse), _ptr(dev_status), _stream(stream))
    _check("diffattn_fwd_prefill_train", rc)
    return out, o2, lse


def diffattn_bwd_prefill_saved(q, k, v, lam, out, o2, lse, dout, causal=True, window=0,
                               workspace=None, dev_status=None, stream=None, grads=None):
    """diffattn_bwd_prefill from diffattn_fwd_prefill_train's (out, o2, lse) (see
    include/diffattn.h): no recompute of the forward. Returns float32 (dq, dk, dv, dlambda)."""
    import torch
    lib = load_library()
    if out.stride() != dout.stride() or o2.stride() != dout.stride():
        raise ValueError("out, o2 and dout must share one layout")
    p = prefill_params(q, k, v, dout, causal, None, 1e-5, window)
    if grads is None:
        grads = (torch.empty(q.shape, dtype=torch.float32, device=q.device),
                 torch.empty(k.shape, dtype=torch.float32, device=q.device),
                 torch.empty(v.shape, dtype=torch.float32, device=q.device),
                 torch.empty(lam.shape, dtype=torch.float32, device=q.device))
    dq, dk, dv, dl = grads
    need = diffattn_bwd_workspace_size(p)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib.diffattn_bwd_prefill_saved(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out),
                                        _ptr(o2), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                                        _ptr(dl), _ptr(workspace), ws_bytes, _ptr(dev_status),
                                        _stream(stream))
    _check("diffattn_bwd_prefill_saved", rc)
    return dq, dk, dv, dl


def diffattn_lambda_bwd(lq1, lk1, lq2, lk2, dlambda, stream=None):
    """Gradients of the four [n_heads, dim] lambda vectors from dL/dlambda [n_heads]."""
    import torch
    lib = load_library()
    H, dim = lq1.shape
    outs = [torch.empty((H, dim), dtype=torch.float32, device=lq1.device) for _ in range(4)]
    rc = lib.diffattn_lambda_bwd(_ptr(lq1), _ptr(lk1), _ptr(lq2), _ptr(lk2), H, dim, _ptr(dlambda),
                                 *[_ptr(o) for o in outs], _stream(stream))
    _check("diffattn_lambda_bwd", rc)
    return tuple(outs)


def decode_params(q, k_cache, v_cache, out, num_splits=0) -> DecodeParams:
    p = DecodeParams()
    B, Hq, d = q.shape
    _, L, Hkv, _ = k_cache.shape
    if tuple(k_cache.stride()) != tuple(v_cache.stride()):
        raise DiffattnError("diffattn_fwd_decode", -1)
    p.variant, p.dtype = DIFFATTN_V2, _dtype_code(q)
    p.batch, p.max_kv_len, p.n_q_heads, p.n_kv_heads, p.head_dim = B, L, Hq, Hkv, d
    p.num_splits = int(num_splits)
    p.q_strides[:] = q.stride()[:2]
    p.kv_strides[:] = k_cache.stride()[:3]
    p.o_strides[:] = out.stride()[:2]
    return p


def decode_params_v1(q, k_cache, v_cache, out, num_splits=0) -> DecodeParams:
    """V1: q [B,H,2,d], k_cache [B,L,H,2,d], v_cache [B,L,H,2d], out [B,H,2d]."""
    p = DecodeParams()
    B, H, two, d = q.shape
    _, L = k_cache.shape[:2]
    if two != 2 or tuple(k_cache.stride()[:3]) != tuple(v_cache.stride()[:3]):
        raise DiffattnError("diffattn_fwd_decode_v1", -1)
    p.variant, p.dtype = DIFFATTN_V1, _dtype_code(q)
    p.batch, p.max_kv_len, p.n_q_heads, p.n_kv_heads, p.head_dim = B, L, H, H, d
    p.num_splits = int(num_splits)
    p.q_strides[:] = q.stride()[:2]
    p.kv_strides[:] = k_cache.stride()[:3]
    p.o_strides[:] = out.stride()[:2]
    return p


def diffattn_decode_workspace_size(p: DecodeParams) -> int:
    n = ctypes.c_size_t(0)
    _check("diffattn_decode_workspace_size",
           load_library().diffattn_decode_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def diffattn_fwd_decode(q, k_cache, v_cache, lam, kv_len=None, out=None, workspace=None,
                        num_splits=0, dev_status=None, stream=None):
    """Split-KV differential decode (V2). q [B,Hq,d], caches [B,L,Hkv,d] -> out [B,Hq/2,d]."""
    import torch
    lib = load_library()
    B, Hq, d = q.shape
    if out is None:
        out = torch.empty((B, Hq // 2, d), dtype=q.dtype, device=q.device)
    p = decode_params(q, k_cache, v_cache, out, num_splits)
    need = diffattn_decode_workspace_size(p)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib.diffattn_fwd_decode(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(kv_len), _ptr(lam), _ptr(out), _ptr(workspace), ws_bytes,
                                 _ptr(dev_status), _stream(stream))
    _check("diffattn_fwd_decode", rc)
    return out


def diffattn_fwd_decode_v1(q, k_cache, v_cache, lam, lambda_init=None, kv_len=None, out=None,
                           apply_norm=True, norm_eps=1e-5, workspace=None, num_splits=0,
                           dev_status=None, stream=None):
    """Split-KV differential decode (V1). q [B,H,2,d], k_cache [B,L,H,2,d],
    v_cache [B,L,H,2d] -> out [B,H,2d], per-head RMSNorm and (1 - lambda_init) scale when
    apply_norm."""
    import torch
    lib = load_library()
    B, H, _, d = q.shape
    if out is None:
        out = torch.empty((B, H, 2 * d), dtype=q.dtype, device=q.device)
    p = decode_params_v1(q, k_cache, v_cache, out, num_splits)
    need = diffattn_decode_workspace_size(p)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib.diffattn_fwd_decode_v1(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(kv_len), _ptr(lam), _ptr(lambda_init), int(bool(apply_norm)),
                                    float(norm_eps), _ptr(out), _ptr(workspace), ws_bytes,
                                    _ptr(dev_status), _stream(stream))
    _check("diffattn_fwd_decode_v1", rc)
    return out


class PagedKV(ctypes.Structure):
    _fields_ = [
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("page_strides", ctypes.c_int64 * 3),
    ]


def paged_kv(k_pages, v_pages, block_table) -> PagedKV:
    """Pool geometry from the page tensors ([P, page_size, heads, ...]) and the block table
    ([B, max_pages_per_seq])."""
    if tuple(k_pages.stride()[:3]) != tuple(v_pages.stride()[:3]) or k_pages.shape[:2] != v_pages.shape[:2]:
        raise DiffattnError("diffattn_fwd_decode_paged", -1)
    pk = PagedKV()
    pk.num_pages, pk.page_size = int(k_pages.shape[0]), int(k_pages.shape[1])
    pk.max_pages_per_seq = int(block_table.shape[1])
    pk.page_strides[:] = k_pages.stride()[:3]
    return pk


def diffattn_fwd_decode_paged(q, k_pages, v_pages, block_table, lam, kv_len=None, lambda_init=None,
                              out=None, apply_norm=None, norm_eps=1e-5, workspace=None,
                              num_splits=0, max_kv_len=None, dev_status=None, stream=None):
    """Split-KV differential decode over a paged cache (block table [B, max_pages_per_seq],
    int32). V2: q [B,Hq,d], pages [P,page,Hkv,d] -> out [B,Hq/2,d]. V1: q [B,H,2,d],
    k_pages [P,page,H,2,d], v_pages [P,page,H,2d] -> out [B,H,2d] (norm and scale when
    apply_norm, default on). max_kv_len defaults to page_size * max_pages_per_seq."""
    import torch
    lib = load_library()
    pk = paged_kv(k_pages, v_pages, block_table)
    p = DecodeParams()
    v1 = q.dim() == 4
    B = q.shape[0]
    if v1:
        _, H, two, d = q.shape
        if two != 2:
            raise DiffattnError("diffattn_fwd_decode_paged", -1)
        p.variant, p.n_q_heads, p.n_kv_heads = DIFFATTN_V1, H, H
        oshape = (B, H, 2 * d)
        norm = True if apply_norm is None else bool(apply_norm)
    else:
        _, Hq, d = q.shape
        p.variant, p.n_q_heads, p.n_kv_heads = DIFFATTN_V2, Hq, int(k_pages.shape[2])
        oshape = (B, Hq // 2, d)
        norm = False if apply_norm is None else bool(apply_norm)
    if out is None:
        out = torch.empty(oshape, dtype=q.dtype, device=q.device)
    p.dtype = _dtype_code(q)
    p.batch, p.head_dim, p.num_splits = B, d, int(num_splits)
    p.max_kv_len = int(max_kv_len if max_kv_len is not None else pk.page_size * pk.max_pages_per_seq)
    p.q_strides[:] = q.stride()[:2]
    p.o_strides[:] = out.stride()[:2]
    need = diffattn_decode_workspace_size(p)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib.diffattn_fwd_decode_paged(ctypes.byref(p), ctypes.byref(pk), _ptr(q), _ptr(k_pages),
                                       _ptr(v_pages), _ptr(block_table), _ptr(kv_len), _ptr(lam),
                                       _ptr(lambda_init), int(norm), float(norm_eps), _ptr(out),
                                       _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))
    _check("diffattn_fwd_decode_paged", rc)
    return out


def diffattn_fwd_decode_static(q, k_cache, v_cache, lam, kv_len=None, out=None, num_splits=0,
                               dev_status=None, stream=None):
    """diffattn_fwd_decode with the partial states in the library's own device array, for
    callers that cannot allocate a workspace (see include/diffattn.h). Calls that overlap
    on the GPU share that array and must be ordered."""
    import torch
    lib = load_library()
    B, Hq, d = q.shape
    if out is None:
        out = torch.empty((B, Hq // 2, d), dtype=q.dtype, device=q.device)
    p = decode_params(q, k_cache, v_cache, out, num_splits)
    rc = lib.diffattn_fwd_decode_static(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(kv_len), _ptr(lam), _ptr(out), _ptr(dev_status),
                                        _stream(stream))
    _check("diffattn_fwd_decode_static", rc)
    return out


KV4_RECORD_BYTES = 144  # DIFFATTN_KV4_RECORD_BYTES


def _kv4_fail(fn, why, status=-1):
    e = DiffattnError(fn, status)
    e.args = (f"{e.args[0]}: {why}",)
    raise e


def _kv4_tensor(fn, name, t, dtype, device, shape=None, dense=True):
    """Refuse an operand of another dtype, device, shape or (where the library takes no
    strides for it) a strided one."""
    if t is None:
        return
    if t.dtype != dtype:
        _kv4_fail(fn, f"{name} is {t.dtype}, not {dtype}", -2)
    if t.device != device:
        _kv4_fail(fn, f"{name} is on {t.device}, the cache on {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        _kv4_fail(fn, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if dense and not t.is_contiguous():
        _kv4_fail(fn, f"{name} must be contiguous")
    if name in ("dev_status", "lambda_init") and t.numel() < 1:
        _kv4_fail(fn, f"{name} is empty")


def _kv4_cache(fn, cache, block_table, max_kv_len, batch):
    """(pool geometry or None, byte strides, positions of an entry) of a cache tensor."""
    import torch
    if cache.dtype != torch.uint8:
        _kv4_fail(fn, f"cache is {cache.dtype}, not torch.uint8", -2)
    if not cache.is_cuda:
        _kv4_fail(fn, "cache is not a CUDA tensor")
    if cache.dim() != 4 or cache.shape[3] != KV4_RECORD_BYTES or cache.stride(3) != 1:
        _kv4_fail(fn, f"cache must be [entries or pages, tokens, heads, {KV4_RECORD_BYTES}] with whole records")
    if block_table is None:
        if cache.shape[0] != batch:
            _kv4_fail(fn, f"cache holds {cache.shape[0]} entries, the batch {batch}")
        room = int(cache.shape[1])
        L = room if max_kv_len is None else int(max_kv_len)
        if L > room:
            _kv4_fail(fn, f"max_kv_len {L} is past the cache's {room} positions")
        return None, cache.stride()[:3], _int32(fn, L)
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        _kv4_fail(fn, f"block_table has shape {tuple(block_table.shape)}, the batch is {batch}")
    _kv4_tensor(fn, "block_table", block_table, torch.int32, cache.device)
    pk = PagedKV()
    pk.num_pages, pk.page_size = int(cache.shape[0]), int(cache.shape[1])
    pk.max_pages_per_seq = int(block_table.shape[1])
    pk.page_strides[:] = cache.stride()[:3]
    L = _int32(fn, pk.page_size * pk.max_pages_per_seq if max_kv_len is None else int(max_kv_len))
    return pk, (0, 0, 0), L


# What a call's checks and parameter structs come to, by the operands' shapes, strides, types
# and devices (not their contents or addresses): a serving loop makes the same calls again and
# again, and the checks cost more than the launch.
_kv4_plans = {}


def _kv4_plan(build, scalars, *tensors):
    key = (build, scalars, *[None if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in tensors])
    plan = _kv4_plans.get(key)
    if plan is None:
        plan = build(scalars, *tensors)
        if len(_kv4_plans) >= 4096:
            _kv4_plans.clear()
        _kv4_plans[key] = plan
    return plan


# the current stream's handle without a Stream object around it (6 us less a call), and the
# current device, where this torch has them
try:
    from torch._C import _cuda_getCurrentRawStream as _raw_stream, _cuda_getDevice as _get_device
except ImportError:  # pragma: no cover
    _raw_stream = _get_device = None


class _Kv4Scope:
    """The launch stream's handle (`raw`), with the cache's device and that stream made current
    until close() where they are not, so that allocations belong to the stream and a call on
    tensors of another device than the current one lands there."""

    __slots__ = ("raw", "stack")

    def __init__(self, device, stream):
        import torch
        if stream is not None and stream.device != device:
            _kv4_fail("stream", f"the stream is on {stream.device}, the cache on {device}")
        self.stack = None
        if stream is not None or torch.cuda.current_device() != device.index:
            import contextlib
            self.stack = contextlib.ExitStack()
            self.stack.enter_context(torch.cuda.device(device))
            if stream is not None:
                self.stack.enter_context(torch.cuda.stream(stream))
        self.raw = (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream

    def close(self):
        if self.stack is not None:
            self.stack.close()


def _kv4_scope(device, stream):
    """(stream handle, scope to close or None): the common case without an object."""
    if stream is None and _raw_stream is not None and _get_device() == device.index:
        return _raw_stream(device.index), None
    scope = _Kv4Scope(device, stream)
    return scope.raw, scope


def _int(x):
    return None if x is None else int(x)


def _int32(fn, x):
    """A count that a parameter struct can hold (ctypes would drop the bits above)."""
    if not -(1 << 31) <= x < 1 << 31:
        _kv4_fail(fn, f"{x} is not an int32")
    return x


def _addr(t):
    return None if t is None else t.data_ptr()


def _kv4_rows_plan(scalars, k, v, cache, pos, cu_seqlens, block_table, dev_status):
    """(parameter struct, pool geometry or None) of a write or a read of rows k and v."""
    fn, max_seqlen, max_kv_len = scalars
    lead = 1 if cu_seqlens is not None else 2
    for name, t in (("k", k), ("v", v)):
        _kv4_tensor(fn, name, t, k.dtype, cache.device, dense=False)
        if t.dim() not in (lead + 2, lead + 3) or t.shape[lead + 1:].numel() != 128:
            _kv4_fail(fn, f"{name} has shape {tuple(t.shape)}: rows of 128 channels behind "
                          + ("[rows, heads]" if lead == 1 else "[batch, rows, heads]"))
        if t.stride(-1) != 1 or (t.dim() == lead + 3 and t.stride(-2) != t.shape[-1]):
            _kv4_fail(fn, f"the 128 channels of {name} must be contiguous")
        if t.shape[:lead + 1] != k.shape[:lead + 1]:
            _kv4_fail(fn, f"k and v differ in rows or heads: {tuple(k.shape)}, {tuple(v.shape)}")
    if cache.dim() == 4 and k.shape[lead] != cache.shape[2]:
        _kv4_fail(fn, f"k has {k.shape[lead]} heads, the cache {cache.shape[2]}")
    return _kv4_rows_params(fn, _dtype_code(k), k.shape[:lead + 1], k.stride()[:lead + 1], v.stride()[:lead + 1],
                            max_seqlen, max_kv_len, cache, pos, cu_seqlens, block_table, dev_status)


def _kv4_rows_params(fn, dtype, shape, k_strides, v_strides, max_seqlen, max_kv_len, cache, pos, cu_seqlens,
                     block_table, dev_status):
    """The same of rows [batch, rows, heads] or packed [rows, heads] by their shape, strides and type."""
    import torch
    packed = cu_seqlens is not None
    if packed:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            _kv4_fail(fn, "cu_seqlens must be [batch + 1]")
        _kv4_tensor(fn, "cu_seqlens", cu_seqlens, torch.int32, cache.device)
        if max_seqlen is None:
            _kv4_fail(fn, "cu_seqlens needs max_seqlen, the most rows of an entry")
    p = Kv4Rows()
    p.dtype = dtype
    p.batch = _int32(fn, cu_seqlens.shape[0] - 1 if packed else shape[0])
    p.n_tokens = _int32(fn, shape[-2])
    p.max_seqlen = _int32(fn, max_seqlen) if packed else 0
    p.n_kv_heads = _int32(fn, shape[-1])
    p.k_strides[:] = (0, *k_strides) if packed else k_strides
    p.v_strides[:] = (0, *v_strides) if packed else v_strides
    pk, p.cache_strides[:], p.max_kv_len = _kv4_cache(fn, cache, block_table, max_kv_len, p.batch)
    _kv4_tensor(fn, "pos", pos, torch.int32, cache.device, (p.batch,))
    _kv4_tensor(fn, "dev_status", dev_status, torch.int32, cache.device)
    return ctypes.pointer(p), None if pk is None else ctypes.cast(ctypes.pointer(pk), ctypes.c_void_p), pk


def _kv4_read_plan(scalars, cache, pos, cu_seqlens, block_table, dev_status):
    """The same of a read into new dense rows, and the shape, strides and type of these."""
    import torch
    fn = "diffattn_kv4_read"
    n_tokens, dtype, max_seqlen, max_kv_len = scalars
    if n_tokens is None or cache.dim() != 4:
        _kv4_fail(fn, "needs n_tokens or k and v, and a cache [., ., H, 144]")
    if n_tokens < 0:
        _kv4_fail(fn, f"n_tokens is {n_tokens}")
    dtype = dtype or torch.bfloat16
    codes = {torch.float32: DIFFATTN_F32, torch.bfloat16: DIFFATTN_BF16}
    if dtype not in codes:
        _kv4_fail(fn, f"rows are bf16 or float32, not {dtype}", -2)
    H = cache.shape[2]
    shape, strides = (n_tokens, H), (H * 128, 128)
    if cu_seqlens is None:
        shape = (cache.shape[0] if block_table is None else block_table.shape[0], *shape)
        strides = (n_tokens * H * 128, *strides)
    plan = _kv4_rows_params(fn, codes[dtype], shape, strides, strides, max_seqlen, max_kv_len, cache, pos, cu_seqlens,
                            block_table, dev_status)
    return *plan, torch.Size((*shape, 128)), (*strides, 1), dtype


def diffattn_kv4_write(k, v, cache, pos=None, cu_seqlens=None, max_seqlen=None, block_table=None,
                       max_kv_len=None, dev_status=None, stream=None):
    """Quantise rows of K and V into a 4-bit cache (see include/diffattn.h): row i of entry b
    becomes the record at position pos[b] + i (pos int32 [B], None = 0). k, v bf16 or float32
    [B,N,H,128] (V1's k [B,N,H,2,64] alike), or packed [rows,H,128] with cu_seqlens int32
    [B+1] and max_seqlen. cache uint8 [B,L,H,144], or a pool [P,page,H,144] with block_table.
    Returns cache."""
    lib = load_library()
    p, pk, _ = _kv4_plan(_kv4_rows_plan, ("diffattn_kv4_write", _int(max_seqlen), _int(max_kv_len)), k, v, cache, pos,
                         cu_seqlens, block_table, dev_status)
    raw, scope = _kv4_scope(cache.device, stream)
    try:
        rc = lib.diffattn_kv4_write(p, pk, k.data_ptr(), v.data_ptr(), _addr(cu_seqlens), _addr(pos),
                                    cache.data_ptr(), _addr(block_table), _addr(dev_status), raw)
    finally:
        if scope is not None:
            scope.close()
    _check("diffattn_kv4_write", rc)
    return cache


def diffattn_kv4_read(cache, n_tokens=None, pos=None, cu_seqlens=None, max_seqlen=None,
                      block_table=None, max_kv_len=None, k=None, v=None, dtype=None,
                      dev_status=None, stream=None):
    """Rows of K and V back from a 4-bit cache (see include/diffattn.h): n_tokens rows of each
    entry from position pos[b] on, or with cu_seqlens n_tokens packed rows in all. Returns
    (k, v), new tensors [B,N,H,128] or [rows,H,128] of `dtype` (default bf16) unless given;
    V1's k is the same rows viewed as [..., H, 2, 64]."""
    import torch
    lib = load_library()
    if (k is None) != (v is None):
        _kv4_fail("diffattn_kv4_read", "give both k and v or neither")
    if not cache.is_cuda:
        _kv4_fail("diffattn_kv4_read", "cache is not a CUDA tensor")
    device = cache.device
    raw, scope = _kv4_scope(device, stream)
    try:
        if k is None:
            p, pk, _, shape, strides, dtype = _kv4_plan(_kv4_read_plan, (_int(n_tokens), dtype, _int(max_seqlen),
                                                                         _int(max_kv_len)), cache, pos, cu_seqlens,
                                                        block_table, dev_status)
            k = torch.empty_strided(shape, strides, dtype=dtype, device=device)
            v = torch.empty_like(k)
        else:
            if (n_tokens is not None and int(n_tokens) != k.shape[0 if cu_seqlens is not None else 1]) or (
                    dtype is not None and dtype != k.dtype):
                _kv4_fail("diffattn_kv4_read", "n_tokens or dtype is not that of the given k")
            p, pk, _ = _kv4_plan(_kv4_rows_plan, ("diffattn_kv4_read", _int(max_seqlen), _int(max_kv_len)), k, v,
                                 cache, pos, cu_seqlens, block_table, dev_status)
        rc = lib.diffattn_kv4_read(p, pk, cache.data_ptr(), _addr(block_table), _addr(cu_seqlens), _addr(pos),
                                   k.data_ptr(), v.data_ptr(), _addr(dev_status), raw)
    finally:
        if scope is not None:
            scope.close()
    _check("diffattn_kv4_read", rc)
    return k, v


def decode_kv4_params(q, cache, out, num_splits=0, block_table=None, max_kv_len=None):
    """(DecodeParams, pool geometry or None) of a decode over a 4-bit cache; `out` may be None
    (its strides are then those of a dense output)."""
    fn = "diffattn_fwd_decode_kv4"
    v1 = q.dim() == 4
    if q.dim() not in (3, 4) or (v1 and q.shape[2] != 2):
        _kv4_fail(fn, f"q has shape {tuple(q.shape)}: V2 [B, Hq, 128], V1 [B, H, 2, 64]")
    if q.stride(-1) != 1 or (v1 and q.stride(2) != q.shape[3]):
        _kv4_fail(fn, "the channels of q must be contiguous")
    p = DecodeParams()
    p.variant = DIFFATTN_V1 if v1 else DIFFATTN_V2
    p.dtype = _dtype_code(q)
    p.batch, p.n_q_heads, p.head_dim = int(q.shape[0]), int(q.shape[1]), int(q.shape[-1])
    p.num_splits = _int32(fn, int(num_splits))
    pk, p.kv_strides[:], p.max_kv_len = _kv4_cache(fn, cache, block_table, max_kv_len, p.batch)
    p.n_kv_heads = int(cache.shape[2])
    p.q_strides[:] = q.stride()[:2]
    units = p.n_q_heads if v1 else p.n_q_heads // 2
    p.o_strides[:] = (units * 128, 128) if out is None else out.stride()[:2]
    return p, pk


def diffattn_decode_kv4_workspace_size(p: DecodeParams, pk=None) -> int:
    n = ctypes.c_size_t(0)
    _check("diffattn_decode_kv4_workspace_size",
           load_library().diffattn_decode_kv4_workspace_size(
               ctypes.byref(p), None if pk is None else ctypes.byref(pk), ctypes.byref(n)))
    return int(n.value)


def _kv4_decode_plan(scalars, q, cache, lam, kv_len, lambda_init, out, block_table, dev_status):
    """(parameter struct, pool geometry or None, workspace bytes, output shape, V1)."""
    import torch
    fn = "diffattn_fwd_decode_kv4"
    num_splits, max_kv_len = scalars
    p, pk = decode_kv4_params(q, cache, out, num_splits, block_table, max_kv_len)
    v1 = p.variant == DIFFATTN_V1
    units = p.n_q_heads if v1 else p.n_q_heads // 2
    device = cache.device
    _kv4_tensor(fn, "q", q, torch.bfloat16, device, dense=False)
    _kv4_tensor(fn, "lam", lam, torch.float32, device, (units,))
    _kv4_tensor(fn, "kv_len", kv_len, torch.int32, device, (p.batch,))
    _kv4_tensor(fn, "lambda_init", lambda_init, torch.float32, device)
    _kv4_tensor(fn, "dev_status", dev_status, torch.int32, device)
    if out is not None:
        _kv4_tensor(fn, "out", out, torch.bfloat16, device, (p.batch, units, 128), dense=False)
        if out.stride(-1) != 1:
            _kv4_fail(fn, "the channels of out must be contiguous")
    need = diffattn_decode_kv4_workspace_size(p, pk)
    return (ctypes.pointer(p), None if pk is None else ctypes.cast(ctypes.pointer(pk), ctypes.c_void_p), need,
            (p.batch, units, 128), v1, pk)


def diffattn_fwd_decode_kv4(q, cache, lam, kv_len=None, lambda_init=None, out=None, apply_norm=None,
                            norm_eps=1e-5, workspace=None, num_splits=0, block_table=None,
                            max_kv_len=None, dev_status=None, stream=None):
    """Split-KV differential decode over a 4-bit cache (see include/diffattn.h): uint8
    [B,L,H,144], or a pool [P,page,H,144] with block_table int32 [B,pages]. V2: q [B,Hq,128] ->
    out [B,Hq/2,128]. V1: q [B,H,2,64] -> out [B,H,128] (norm and scale when apply_norm, default
    on). max_kv_len defaults to the positions the cache or the block table has room for."""
    lib = load_library()
    p, pk, need, shape, v1, _ = _kv4_plan(_kv4_decode_plan, (int(num_splits), _int(max_kv_len)), q, cache, lam, kv_len,
                                          lambda_init, out, block_table, dev_status)
    device = cache.device
    raw, scope = _kv4_scope(device, stream)
    try:
        if out is None:
            out = q.new_empty(shape)
        if workspace is None:
            workspace = cache.new_empty(need) if need else None
            ws_bytes = need
        else:
            if workspace.device != device or not workspace.is_contiguous():
                _kv4_fail("diffattn_fwd_decode_kv4", "workspace must be contiguous and on the cache's device", -4)
            ws_bytes = workspace.numel() * workspace.element_size()
        rc = lib.diffattn_fwd_decode_kv4(
            p, pk, q.data_ptr(), cache.data_ptr(), _addr(block_table), _addr(kv_len), lam.data_ptr(),
            _addr(lambda_init), int(v1 if apply_norm is None else bool(apply_norm)), norm_eps, out.data_ptr(),
            _addr(workspace), ws_bytes, _addr(dev_status), raw)
    finally:
        if scope is not None:
            scope.close()
    _check("diffattn_fwd_decode_kv4", rc)
    return out


def diffattn_selftest_timeout(dev_status, timeout_ms=200, stream=None):
    """Launch the bounded-wait self-test (see include/diffattn.h): a wait that nothing
    completes runs out after `timeout_ms` and DIFFATTN_ERR_TIMEOUT lands in `dev_status`
    (a device int32 tensor) when the block finishes."""
    lib = load_library()
    rc = lib.diffattn_selftest_timeout(_ptr(dev_status), int(timeout_ms), _stream(stream))
    _check("diffattn_selftest_timeout", rc)


def diffattn_selftest_exp2(x, stream=None):
    """Evaluate the V2 prefill's FMA-pipe 2^x and CUDA's exp2f over a device float32 tensor
    `x` (see include/diffattn.h); returns (y, y_ref), device float32 tensors like x."""
    import torch
    lib = load_library()
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 tensor")
    y, y_ref = torch.empty_like(x), torch.empty_like(x)
    rc = lib.diffattn_selftest_exp2(_ptr(x), _ptr(y), _ptr(y_ref), int(x.numel()), _stream(stream))
    _check("diffattn_selftest_exp2", rc)
    return y, y_ref


def diffattn_debug_bounds_violations():
    """The bounds-checked build's count of skipped out-of-range accesses since the last call
    (see include/diffattn.h), or None when the loaded library is the normal build."""
    lib = load_library()
    n = ctypes.c_int32(0)
    rc = lib.diffattn_debug_bounds_violations(ctypes.byref(n))
    if rc == -2:  # DIFFATTN_ERR_UNSUPPORTED: the normal build
        return None
    _check("diffattn_debug_bounds_violations", rc)
    return int(n.value)
