"""Gated delta rule (Gated DeltaNet core) on B200: thin Python binding of libgdn.so.

Every step of the computation runs in the CUDA kernels of ``libgdn.so``; this
module only marshals torch CUDA tensors into the C ABI of ``include/gdn.h``
(pointers, sizes, the current stream) and allocates outputs when the caller
does not pass them.  There is no CPU or PyTorch fallback: if the library is
missing the import fails, and if a call is rejected it raises ``GdnError``.

Functions
---------
chunk_fwd(q, k, v, g, beta, ...)       -> (out, final_state)   prefill, gdn_chunk_fwd
recurrent_step(q, k, v, g, beta, state, ...) -> out            decode, gdn_recurrent_step
chunk_fwd_gated / recurrent_step_gated                         the gate formed in-kernel
chunk_fwd_slots / recurrent_step_slots                         states in a slot-indexed pool
chunk_fwd_ex / recurrent_step_ex                               any of those fusions plus the
                                                               gated RMSNorm epilogue (gdn_ext_t)
gated_rmsnorm(o, z, weight, eps)       -> y                    the epilogue alone, gdn_gated_rmsnorm
qkv_conv_fwd / qkv_conv_update         -> (q, k, v[, state])  causal conv1d + SiLU producing q, k, v

Training:
chunk_bwd(q, k, v, g, beta, dout, ...) -> (dq, dk, dv, dg, dbeta, d_initial_state)   gradients of chunk_fwd
gate_bwd(dg, dbeta, a, b, A_log, dt_bias) -> (da, db, dA_log, ddt_bias)              of the gate
gated_rmsnorm_bwd(dy, o, z, weight)    -> (do, dz, dweight)                           of the epilogue
qkv_conv_bwd(dq, dk, dv, x, weight, ...) -> (dx, dweight, dbias, d_conv_state)        of the conv
act_quantize(x) / act_dequantize       -> (codes, scales) / x   activations kept in 8 bits; the two
                                                               gradients above read them as they are
"""
from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_OK = 0
STATUS_NAMES = {0: "GDN_OK", -1: "GDN_ERR_NULL", -2: "GDN_ERR_SHAPE", -3: "GDN_ERR_ALIGN",
                -4: "GDN_ERR_ALIAS", -5: "GDN_ERR_CUDA", -6: "GDN_ERR_DEVICE",
                -7: "GDN_ERR_DEVICE_TIMEOUT", -8: "GDN_ERR_SEQLENS", -9: "GDN_ERR_GATE"}
KERNELS = {"auto": 0, "simt": 1, "tc": 2}
DTYPE_F32, DTYPE_BF16 = 0, 1


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s" % (what, lib().gdn_status_string(status).decode()))


class GdnParams(ctypes.Structure):
    _fields_ = [("num_qk_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_k_dim", ctypes.c_int32), ("head_v_dim", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("qk_l2norm", ctypes.c_int32),
                ("scale", ctypes.c_float), ("kernel", ctypes.c_int32)]


class GdnExt(ctypes.Structure):
    _fields_ = [("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p), ("slot_ids", ctypes.c_void_p),
                ("num_slots", ctypes.c_int32), ("norm_z", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p),
                ("norm_eps", ctypes.c_float), ("conv_x", ctypes.c_void_p), ("conv_state", ctypes.c_void_p),
                ("conv_weight", ctypes.c_void_p), ("conv_bias", ctypes.c_void_p),
                ("conv_kernel_size", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                "libgdn.so is not built (expected at %s); run "
                "`python -m gated_deltanet_chunk_b200.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, fp, ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
        L.gdn_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, fp, ip, ctypes.c_int32, ctypes.c_int64,
                                    ctypes.c_int32, vp, fp, ctypes.POINTER(GdnParams), vp]
        L.gdn_chunk_fwd.restype = ctypes.c_int
        L.gdn_recurrent_step.argtypes = [vp, vp, vp, fp, fp, fp, vp, ctypes.c_int32,
                                         ctypes.POINTER(GdnParams), vp]
        L.gdn_recurrent_step.restype = ctypes.c_int
        L.gdn_chunk_fwd_gated.argtypes = [vp, vp, vp, fp, fp, fp, fp, fp, ip, ctypes.c_int32,
                                          ctypes.c_int64, ctypes.c_int32, vp, fp,
                                          ctypes.POINTER(GdnParams), vp]
        L.gdn_chunk_fwd_gated.restype = ctypes.c_int
        L.gdn_recurrent_step_gated.argtypes = [vp, vp, vp, fp, fp, fp, fp, fp, vp, ctypes.c_int32,
                                               ctypes.POINTER(GdnParams), vp]
        L.gdn_recurrent_step_gated.restype = ctypes.c_int
        L.gdn_chunk_fwd_slots.argtypes = [vp, vp, vp, fp, fp, fp, ip, ctypes.c_int32, ip, ctypes.c_int32,
                                          ctypes.c_int64, ctypes.c_int32, vp, ctypes.POINTER(GdnParams), vp]
        L.gdn_chunk_fwd_slots.restype = ctypes.c_int
        L.gdn_recurrent_step_slots.argtypes = [vp, vp, vp, fp, fp, fp, ip, ctypes.c_int32, vp, ctypes.c_int32,
                                               ctypes.POINTER(GdnParams), vp]
        L.gdn_recurrent_step_slots.restype = ctypes.c_int
        L.gdn_chunk_fwd_ex.argtypes = [vp, vp, vp, fp, fp, fp, ip, ctypes.c_int32, ctypes.c_int64,
                                       ctypes.c_int32, vp, fp, ctypes.POINTER(GdnParams),
                                       ctypes.POINTER(GdnExt), vp]
        L.gdn_chunk_fwd_ex.restype = ctypes.c_int
        L.gdn_recurrent_step_ex.argtypes = [vp, vp, vp, fp, fp, fp, vp, ctypes.c_int32,
                                            ctypes.POINTER(GdnParams), ctypes.POINTER(GdnExt), vp]
        L.gdn_recurrent_step_ex.restype = ctypes.c_int
        L.gdn_gated_rmsnorm.argtypes = [vp, vp, fp, ctypes.c_float, vp, ctypes.c_int64, ctypes.c_int32,
                                        ctypes.c_int32, vp]
        L.gdn_gated_rmsnorm.restype = ctypes.c_int
        L.gdn_qkv_conv_fwd.argtypes = [vp, fp, fp, vp, ip, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                       vp, vp, vp, vp, ctypes.POINTER(GdnParams), vp]
        L.gdn_qkv_conv_fwd.restype = ctypes.c_int
        L.gdn_qkv_conv_update.argtypes = [vp, fp, fp, vp, ip, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                          vp, vp, vp, ctypes.POINTER(GdnParams), vp]
        L.gdn_qkv_conv_update.restype = ctypes.c_int
        L.gdn_chunk_bwd.argtypes = [vp, vp, vp, fp, fp, fp, fp, fp, vp, fp, ip, ctypes.c_int32, ctypes.c_int64,
                                    vp, vp, vp, vp, vp, fp, vp, ctypes.c_int64, ctypes.POINTER(GdnParams), vp]
        L.gdn_chunk_bwd.restype = ctypes.c_int
        L.gdn_chunk_bwd_workspace.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(GdnParams)]
        L.gdn_chunk_bwd_workspace.restype = ctypes.c_int64
        L.gdn_act_quantize.argtypes = [vp, vp, vp, ctypes.c_int64, ctypes.c_int32, vp]
        L.gdn_act_quantize.restype = ctypes.c_int
        L.gdn_act_dequantize.argtypes = [vp, vp, vp, ctypes.c_int64, ctypes.c_int32, vp]
        L.gdn_act_dequantize.restype = ctypes.c_int
        L.gdn_gated_rmsnorm_bwd.argtypes = [vp, vp, vp, vp, vp, fp, ctypes.c_float, vp, vp, fp, ctypes.c_int64,
                                            ctypes.c_int32, ctypes.c_int32, vp, ctypes.c_int64, vp]
        L.gdn_gated_rmsnorm_bwd.restype = ctypes.c_int
        L.gdn_gated_rmsnorm_bwd_workspace.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]
        L.gdn_gated_rmsnorm_bwd_workspace.restype = ctypes.c_int64
        L.gdn_qkv_conv_bwd.argtypes = [vp, vp, vp, vp, vp, fp, fp, vp, vp, ip, ctypes.c_int32, ctypes.c_int64,
                                       ctypes.c_int32, vp, fp, fp, vp, vp, ctypes.c_int64, ctypes.POINTER(GdnParams), vp]
        L.gdn_qkv_conv_bwd.restype = ctypes.c_int
        L.gdn_qkv_conv_bwd_workspace.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(GdnParams)]
        L.gdn_qkv_conv_bwd_workspace.restype = ctypes.c_int64
        L.gdn_gate_bwd.argtypes = [vp, vp, fp, fp, fp, fp, vp, vp, fp, fp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                   vp, ctypes.c_int64, vp]
        L.gdn_gate_bwd.restype = ctypes.c_int
        L.gdn_gate_bwd_workspace.argtypes = [ctypes.c_int64, ctypes.c_int32]
        L.gdn_gate_bwd_workspace.restype = ctypes.c_int64
        L.gdn_selftest_wait_timeout.argtypes = [ctypes.c_int64, vp]
        L.gdn_selftest_wait_timeout.restype = ctypes.c_int
        L.gdn_device_status.argtypes = [vp]
        L.gdn_device_status.restype = ctypes.c_int
        L.gdn_status_string.argtypes = [ctypes.c_int]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_version.argtypes = []
        L.gdn_version.restype = ctypes.c_int
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    """The raw handle of ``stream``, or of the current device's current stream (read without building a Stream object:
    the small calls are bound by the host)."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def make_params(nqk, nv, dk, dv, io_bf16, qk_l2norm=True, scale=0.0, kernel="auto") -> GdnParams:
    return GdnParams(int(nqk), int(nv), int(dk), int(dv), DTYPE_BF16 if io_bf16 else DTYPE_F32,
                     1 if qk_l2norm else 0, float(scale), KERNELS[kernel])


def _chunk_call(name, gate, q, k, v, initial_state, cu_seqlens, chunk_size, out, final_state,
                output_final_state, num_seqs, qk_l2norm, scale, kernel, stream, check):
    import torch
    T, nqk, dk = q.shape
    nv, dv = v.shape[1], v.shape[2]
    n = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    if out is None:
        out = torch.empty((T, nv, dv), dtype=v.dtype, device=v.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((n, nv, dk, dv), dtype=torch.float32, device=v.device)
    p = make_params(nqk, nv, dk, dv, q.dtype == torch.bfloat16, qk_l2norm, scale, kernel)
    rc = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), *[_ptr(x) for x in gate], _ptr(initial_state),
                              _ptr(cu_seqlens), int(n), int(T), int(chunk_size), _ptr(out),
                              _ptr(final_state), ctypes.byref(p), _stream(stream))
    if check and rc != GDN_OK:
        raise GdnError(rc, name)
    return out, final_state


def chunk_fwd(q, k, v, g, beta, initial_state=None, cu_seqlens=None, chunk_size=64,
              out=None, final_state=None, output_final_state=True, num_seqs=None,
              qk_l2norm=True, scale=0.0, kernel="auto", stream=None, check=True):
    """Chunked gated delta rule over a packed batch (``gdn_chunk_fwd``).

    q, k [T, Nqk, Dk] and v [T, Nv, Dv] (bf16 or fp32, CUDA, contiguous);
    g, beta [T, Nv] fp32; initial_state [N, Nv, Dk, Dv] fp32 or None;
    cu_seqlens [N+1] int32 or None (then ``num_seqs`` equal sequences, default 1).
    Returns ``(out, final_state)``; final_state is None when not requested.
    """
    return _chunk_call("gdn_chunk_fwd", (g, beta), q, k, v, initial_state, cu_seqlens, chunk_size,
                       out, final_state, output_final_state, num_seqs, qk_l2norm, scale, kernel,
                       stream, check)


def chunk_fwd_gated(q, k, v, a, b, A_log, dt_bias, initial_state=None, cu_seqlens=None,
                    chunk_size=64, out=None, final_state=None, output_final_state=True,
                    num_seqs=None, qk_l2norm=True, scale=0.0, kernel="auto", stream=None,
                    check=True):
    """``chunk_fwd`` with the gate formed in-kernel (``gdn_chunk_fwd_gated``).

    a, b [T, Nv] fp32 raw projections; A_log, dt_bias [Nv] fp32:
    beta = sigmoid(b), g = -exp(A_log) * softplus(a + dt_bias).
    """
    return _chunk_call("gdn_chunk_fwd_gated", (a, b, A_log, dt_bias), q, k, v, initial_state,
                       cu_seqlens, chunk_size, out, final_state, output_final_state, num_seqs,
                       qk_l2norm, scale, kernel, stream, check)


def _step_call(name, gate, q, k, v, state, out, qk_l2norm, scale, stream, check):
    import torch
    N, nqk, dk = q.shape
    nv, dv = v.shape[1], v.shape[2]
    if out is None:
        out = torch.empty((N, nv, dv), dtype=v.dtype, device=v.device)
    p = make_params(nqk, nv, dk, dv, q.dtype == torch.bfloat16, qk_l2norm, scale)
    rc = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), *[_ptr(x) for x in gate], _ptr(state),
                              _ptr(out), int(N), ctypes.byref(p), _stream(stream))
    if check and rc != GDN_OK:
        raise GdnError(rc, name)
    return out


def recurrent_step(q, k, v, g, beta, state, out=None, qk_l2norm=True, scale=0.0, stream=None,
                   check=True):
    """One decode token per sequence (``gdn_recurrent_step``); ``state`` is updated in place.

    q, k [N, Nqk, Dk], v [N, Nv, Dv], g, beta [N, Nv], state [N, Nv, Dk, Dv] fp32.
    Returns out [N, Nv, Dv].
    """
    return _step_call("gdn_recurrent_step", (g, beta), q, k, v, state, out, qk_l2norm, scale,
                      stream, check)


def recurrent_step_gated(q, k, v, a, b, A_log, dt_bias, state, out=None, qk_l2norm=True,
                         scale=0.0, stream=None, check=True):
    """``recurrent_step`` with the gate formed in-kernel (``gdn_recurrent_step_gated``).

    a, b [N, Nv] fp32 raw projections; A_log, dt_bias [Nv] fp32.
    """
    return _step_call("gdn_recurrent_step_gated", (a, b, A_log, dt_bias), q, k, v, state, out,
                      qk_l2norm, scale, stream, check)


def selftest_wait_timeout(limit_us=2000, stream=None) -> int:
    """Launch the failure-detection self-test (``gdn_selftest_wait_timeout``); then
    ``device_status()`` reports GDN_ERR_DEVICE_TIMEOUT once."""
    return lib().gdn_selftest_wait_timeout(int(limit_us), _stream(stream))


def device_status(stream=None) -> int:
    """Synchronise the stream and return the library's device status (``gdn_device_status``)."""
    return lib().gdn_device_status(_stream(stream))


def chunk_fwd_slots(q, k, v, g, beta, state_pool, slot_ids, cu_seqlens=None, chunk_size=64, out=None,
                    num_seqs=None, qk_l2norm=True, scale=0.0, kernel="auto", stream=None, check=True):
    """Chunked forward with the states in a slot-indexed pool, updated in place (``gdn_chunk_fwd_slots``).

    state_pool [P, Nv, Dk, Dv] fp32; slot_ids [N] int32 (ids outside [0, P) mark padding
    sequences); cu_seqlens [N+1] or None.  Returns out [T, Nv, Dv].
    """
    import torch
    T, nqk, dk = q.shape
    nv, dv = v.shape[1], v.shape[2]
    n = slot_ids.numel()
    if out is None:
        out = torch.empty((T, nv, dv), dtype=v.dtype, device=v.device)
    p = make_params(nqk, nv, dk, dv, q.dtype == torch.bfloat16, qk_l2norm, scale, kernel)
    rc = lib().gdn_chunk_fwd_slots(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_pool),
                                   _ptr(slot_ids), int(state_pool.shape[0]), _ptr(cu_seqlens), int(n),
                                   int(T), int(chunk_size), _ptr(out), ctypes.byref(p), _stream(stream))
    if check and rc != GDN_OK:
        raise GdnError(rc, "gdn_chunk_fwd_slots")
    return out


def recurrent_step_slots(q, k, v, g, beta, state_pool, slot_ids, out=None, qk_l2norm=True, scale=0.0,
                         stream=None, check=True):
    """One decode token per sequence with slot-indexed states (``gdn_recurrent_step_slots``)."""
    import torch
    N, nqk, dk = q.shape
    nv, dv = v.shape[1], v.shape[2]
    if out is None:
        out = torch.empty((N, nv, dv), dtype=v.dtype, device=v.device)
    p = make_params(nqk, nv, dk, dv, q.dtype == torch.bfloat16, qk_l2norm, scale)
    rc = lib().gdn_recurrent_step_slots(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_pool),
                                        _ptr(slot_ids), int(state_pool.shape[0]), _ptr(out), int(N),
                                        ctypes.byref(p), _stream(stream))
    if check and rc != GDN_OK:
        raise GdnError(rc, "gdn_recurrent_step_slots")
    return out


def make_ext(A_log=None, dt_bias=None, slot_ids=None, num_slots=0, norm_z=None, norm_weight=None,
             norm_eps=1e-6, conv_x=None, conv_state=None, conv_weight=None, conv_bias=None) -> GdnExt:
    """The gdn_ext_t block: fused gate, slot pool, gated RMSNorm epilogue, fused conv (each optional)."""
    p = lambda t: None if t is None else t.data_ptr()
    return GdnExt(p(A_log), p(dt_bias), p(slot_ids), int(num_slots), p(norm_z), p(norm_weight),
                  float(norm_eps), p(conv_x), p(conv_state), p(conv_weight), p(conv_bias),
                  int(conv_weight.shape[1]) if conv_weight is not None else 0)


def chunk_fwd_ex(q, k, v, g, beta, initial_state=None, cu_seqlens=None, chunk_size=64, out=None,
                 final_state=None, output_final_state=True, num_seqs=None, qk_l2norm=True, scale=0.0,
                 kernel="auto", A_log=None, dt_bias=None, slot_ids=None, norm_z=None, norm_weight=None,
                 norm_eps=1e-6, stream=None, check=True):
    """``chunk_fwd`` with any of the fusions of ``gdn_chunk_fwd_ex``.

    A_log, dt_bias: the g, beta arguments are the raw projections a, b.
    slot_ids: ``initial_state`` is a state pool [P, Nv, Dk, Dv], updated in place.
    norm_z [T, Nv, Dv] (dtype of v), norm_weight [Dv] fp32: out holds
    o / sqrt(mean(o^2) + norm_eps) * norm_weight * silu(norm_z) per row.
    Returns ``(out, final_state)``.
    """
    import torch
    T, nqk, dk = q.shape
    nv, dv = v.shape[1], v.shape[2]
    if slot_ids is not None:
        n = slot_ids.numel()
        final_state = initial_state
    else:
        n = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
        if final_state is None and output_final_state:
            final_state = torch.empty((n, nv, dk, dv), dtype=torch.float32, device=v.device)
    if out is None:
        out = torch.empty((T, nv, dv), dtype=v.dtype, device=v.device)
    p = make_params(nqk, nv, dk, dv, q.dtype == torch.bfloat16, qk_l2norm, scale, kernel)
    x = make_ext(A_log, dt_bias, slot_ids, 0 if initial_state is None or slot_ids is None
                 else initial_state.shape[0], norm_z, norm_weight, norm_eps)
    rc = lib().gdn_chunk_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                _ptr(cu_seqlens), int(n), int(T), int(chunk_size), _ptr(out),
                                _ptr(final_state), ctypes.byref(p), ctypes.byref(x), _stream(stream))
    if check and rc != GDN_OK:
        raise GdnError(rc, "gdn_chunk_fwd_ex")
    return out, final_state


def recurrent_step_ex(q, k, v, g, beta, state, out=None, qk_l2norm=True, scale=0.0, A_log=None,
                      dt_bias=None, slot_ids=None, norm_z=None, norm_weight=None, norm_eps=1e-6,
                      conv_x=None, conv_state=None, conv_weight=None, conv_bias=None, shapes=None,
                      stream=None, check=True):
    """``recurrent_step`` with any of the fusions of ``gdn_recurrent_step_ex`` (see chunk_fwd_ex).

    With the conv fused, pass q = k = v = None, ``conv_x`` [N, C], ``conv_state``
    [N or P, C, K] (updated in place), ``conv_weight`` [C, K], ``conv_bias`` and
    ``shapes=(nqk, nv, dk, dv)``.
    """
    import torch
    if conv_x is not None:
        nqk, nv, dk, dv = shapes
        N = conv_x.shape[0]
        io_bf16, dev = conv_x.dtype == torch.bfloat16, conv_x.device
    else:
        N, nqk, dk = q.shape
        nv, dv = v.shape[1], v.shape[2]
        io_bf16, dev = q.dtype == torch.bfloat16, v.device
    if out is None:
        out = torch.empty((N, nv, dv), dtype=torch.bfloat16 if io_bf16 else torch.float32, device=dev)
    p = make_params(nqk, nv, dk, dv, io_bf16, qk_l2norm, scale)
    x = make_ext(A_log, dt_bias, slot_ids, state.shape[0] if slot_ids is not None else 0, norm_z,
                 norm_weight, norm_eps, conv_x, conv_state, conv_weight, conv_bias)
    rc = lib().gdn_recurrent_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(out),
                                     int(N), ctypes.byref(p), ctypes.byref(x), _stream(stream))
    if check and rc != GDN_OK:
        raise GdnError(rc, "gdn_recurrent_step_ex")
    return out


def gated_rmsnorm(o, z, weight, eps=1e-6, out=None, stream=None, check=True):
    """y = o / sqrt(mean(o^2) + eps) * weight * silu(z) over the last axis (``gdn_gated_rmsnorm``).

    o, z [..., D] (bf16 or fp32, same dtype, CUDA, contiguous; D in {64, 128});
    weight [D] fp32.  ``out`` may be ``o`` (in place).
    """
    import torch
    dim = o.shape[-1]
    if out is None:
        out = torch.empty_like(o)
    rc = lib().gdn_gated_rmsnorm(_ptr(o), _ptr(z), _ptr(weight), float(eps), _ptr(out), int(o.numel() // dim),
                                 int(dim), DTYPE_BF16 if o.dtype == torch.bfloat16 else DTYPE_F32,
                                 _stream(stream))
    if check and rc != GDN_OK:
        raise GdnError(rc, "gdn_gated_rmsnorm")
    return out


def _qkv_out(rows, nqk, nv, dk, dv, dtype, device):
    import torch
    return (torch.empty((rows, nqk, dk), dtype=dtype, device=device),
            torch.empty((rows, nqk, dk), dtype=dtype, device=device),
            torch.empty((rows, nv, dv), dtype=dtype, device=device))


def qkv_conv_fwd(mixed_qkv, weight, nqk, nv, dk, dv, bias=None, conv_state=None, cu_seqlens=None,
                 num_seqs=None, output_state=True, state_out=None, stream=None, check=True):
    """Causal depthwise conv1d + SiLU of packed [q | k | v] channels (``gdn_qkv_conv_fwd``).

    mixed_qkv [T, C] (bf16 or fp32), weight [C, K] fp32, bias [C] fp32 or None,
    conv_state [N, C, K] or None (zeros).  Returns ``(q, k, v, state)`` with q, k
    [T, Nqk, Dk], v [T, Nv, Dv] and the new conv_state [N, C, K] (None unless
    requested; ``state_out=conv_state`` updates it in place).
    """
    import torch
    T, C = mixed_qkv.shape
    K = weight.shape[1]
    n = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    q, k, v = _qkv_out(T, nqk, nv, dk, dv, mixed_qkv.dtype, mixed_qkv.device)
    if state_out is None and output_state:
        state_out = torch.empty((n, C, K), dtype=mixed_qkv.dtype, device=mixed_qkv.device)
    p = make_params(nqk, nv, dk, dv, mixed_qkv.dtype == torch.bfloat16)
    rc = lib().gdn_qkv_conv_fwd(_ptr(mixed_qkv), _ptr(weight), _ptr(bias), _ptr(conv_state), _ptr(cu_seqlens),
                                int(n), int(T), int(K), _ptr(q), _ptr(k), _ptr(v), _ptr(state_out),
                                ctypes.byref(p), _stream(stream))
    if check and rc != GDN_OK:
        raise GdnError(rc, "gdn_qkv_conv_fwd")
    return q, k, v, state_out


def qkv_conv_update(mixed_qkv, weight, conv_state, nqk, nv, dk, dv, bias=None, slot_ids=None, out=None,
                    stream=None, check=True):
    """One decode token per sequence through the conv (``gdn_qkv_conv_update``); conv_state in place.

    mixed_qkv [N, C]; conv_state [N, C, K] (or a pool [P, C, K] with slot_ids [N] int32).
    Returns ``(q, k, v)`` with q, k [N, Nqk, Dk] and v [N, Nv, Dv].
    """
    import torch
    N, C = mixed_qkv.shape
    K = weight.shape[1]
    q, k, v = out if out is not None else _qkv_out(N, nqk, nv, dk, dv, mixed_qkv.dtype, mixed_qkv.device)
    p = make_params(nqk, nv, dk, dv, mixed_qkv.dtype == torch.bfloat16)
    rc = lib().gdn_qkv_conv_update(_ptr(mixed_qkv), _ptr(weight), _ptr(bias), _ptr(conv_state), _ptr(slot_ids),
                                   int(conv_state.shape[0]) if slot_ids is not None else 0, int(N), int(K),
                                   _ptr(q), _ptr(k), _ptr(v), ctypes.byref(p), _stream(stream))
    if check and rc != GDN_OK:
        raise GdnError(rc, "gdn_qkv_conv_update")
    return q, k, v


def _checked(what, device, *specs):
    """Raise ``GdnError`` (GDN_ERR_SHAPE) unless every (name, tensor, shape, dtype) given is a contiguous tensor of that
    shape and type on ``device``: gradients often come as views, expanded or in another type."""
    at = -1 if device.index is None else device.index
    for name, t, shape, dtype in specs:
        if t is not None and (t.dtype is not dtype or t.get_device() != at or not t.is_contiguous() or t.shape != shape):
            raise GdnError(-2, "%s (%s is not a contiguous %s tensor of shape %s on %s)"
                           % (what, name, str(dtype).replace("torch.", ""), tuple(shape), device))


def _on_stream(call):
    """With ``stream=`` the whole call, its allocations too, belongs to that stream."""
    @functools.wraps(call)
    def on_stream(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        import torch
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return on_stream


def _run(what, device, check, *args):
    """Call ``what`` on the tensors' device and its current stream."""
    import torch
    if device.type != "cuda":
        raise GdnError(-2, "%s (tensors on %s)" % (what, device))
    if torch._C._cuda_getDevice() != device.index:
        with torch.cuda.device(device):
            return _run(what, device, check, *args)
    rc = getattr(lib(), what)(*args, _stream(None))
    if check and rc != GDN_OK:
        raise GdnError(rc, what)


def chunk_bwd_workspace(q, v, cu_seqlens=None, num_seqs=None, qk_l2norm=True, kernel="auto") -> int:
    """Bytes of workspace that ``chunk_bwd`` needs for these arguments (``gdn_chunk_bwd_workspace``)."""
    import torch
    n = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    p = make_params(q.shape[1], v.shape[1], q.shape[2], v.shape[2], q.dtype == torch.bfloat16, qk_l2norm, kernel=kernel)
    need = lib().gdn_chunk_bwd_workspace(int(n), int(q.shape[0]), ctypes.byref(p))
    if need < 0:
        raise GdnError(need, "gdn_chunk_bwd_workspace")
    return need


@_on_stream
def chunk_bwd(q, k, v, g, beta, dout, initial_state=None, d_final_state=None, cu_seqlens=None, num_seqs=None,
              A_log=None, dt_bias=None, dq=None, dk=None, dv=None, dg=None, dbeta=None, d_initial_state=None,
              output_d_initial_state=None, qk_l2norm=True, scale=0.0, kernel="auto", workspace=None, check=True):
    """Gradients of ``chunk_fwd`` (``gdn_chunk_bwd``); the inputs are those of the forward call.

    dout [T, Nv, Dv] (dtype of v), d_final_state [N, Nv, Dk, Dv] fp32 or None (zeros).
    With A_log, dt_bias the g, beta arguments are the raw projections a, b, and dg,
    dbeta are the gradients of the gate formed from them (then ``gate_bwd``).
    ``workspace``: a CUDA tensor of at least ``chunk_bwd_workspace`` bytes, allocated
    when not given.  Returns ``(dq, dk, dv, dg, dbeta, d_initial_state)``, the token
    gradients in the dtype of q; d_initial_state is None unless an initial state was
    given or it was asked for.

    bf16 tensors with qk_l2norm need g <= 0 and 0 <= beta <= 2 unless ``kernel="simt"``: this
    is not looked at before the launch, a gate outside leaves the results undefined, and
    ``device_status()`` then returns GDN_ERR_GATE.  ``kernel="simt"`` takes any finite gate and
    holds operands in twice as many bits.

    Of this call and the training calls below: tensors of another type, shape or device
    than stated, or that are not contiguous, are refused (``GdnError``, GDN_ERR_SHAPE).
    The call runs on the tensors' device; with ``stream=`` it belongs to that stream as
    if made under ``torch.cuda.stream(stream)``, what it allocates too.
    """
    import torch
    T, nqk, dk_ = q.shape
    nv, dv_ = v.shape[1], v.shape[2]
    n = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    p = make_params(nqk, nv, dk_, dv_, q.dtype == torch.bfloat16, qk_l2norm, scale, kernel)
    io, dev, f32, state = q.dtype, q.device, torch.float32, (n, nv, dk_, dv_)
    _checked("gdn_chunk_bwd", dev, ("q", q, q.shape, torch.bfloat16 if io == torch.bfloat16 else f32), ("k", k, q.shape, io),
             ("v", v, (T, nv, dv_), io), ("g", g, (T, nv), f32), ("beta", beta, (T, nv), f32), ("dout", dout, v.shape, io),
             ("A_log", A_log, (nv,), f32), ("dt_bias", dt_bias, (nv,), f32), ("initial_state", initial_state, state, f32),
             ("d_final_state", d_final_state, state, f32), ("cu_seqlens", cu_seqlens, (n + 1,), torch.int32), ("dq", dq, q.shape, io),
             ("dk", dk, q.shape, io), ("dv", dv, v.shape, io), ("dg", dg, (T, nv), io), ("dbeta", dbeta, (T, nv), io),
             ("d_initial_state", d_initial_state, state, f32))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    dg = torch.empty((T, nv), dtype=q.dtype, device=q.device) if dg is None else dg
    dbeta = torch.empty((T, nv), dtype=q.dtype, device=q.device) if dbeta is None else dbeta
    if d_initial_state is None and (initial_state is not None if output_d_initial_state is None
                                    else output_d_initial_state):
        d_initial_state = torch.empty((n, nv, dk_, dv_), dtype=torch.float32, device=q.device)
    workspace = _workspace(workspace, lib().gdn_chunk_bwd_workspace(int(n), int(T), ctypes.byref(p)), "gdn_chunk_bwd", q.device)
    _run("gdn_chunk_bwd", dev, check, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(A_log), _ptr(dt_bias),
         _ptr(initial_state), _ptr(dout), _ptr(d_final_state), _ptr(cu_seqlens), int(n), int(T), _ptr(dq), _ptr(dk), _ptr(dv),
         _ptr(dg), _ptr(dbeta), _ptr(d_initial_state), _ptr(workspace), _bytes(workspace), ctypes.byref(p))
    return dq, dk, dv, dg, dbeta, d_initial_state


def _kept(x):
    """(tensor, scales) of a saved activation: a tensor, or the pair that ``act_quantize`` returned."""
    return x if isinstance(x, tuple) else (x, None)


def _kept_specs(name, x, scales, shape, io):
    """What ``_checked`` has to see of a saved activation."""
    import torch
    if scales is None:
        return ((name, x, shape, io),)
    return ((name + " codes", x, shape, torch.float8_e4m3fn),
            (name + " scales", scales, (*shape[:-1], shape[-1] // 32), torch.uint8))


def _bytes(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def _workspace(given, need, what, device):
    """The caller's workspace, or one of ``need`` bytes."""
    import torch
    if need < 0:
        raise GdnError(need, what)
    if given is not None:
        _checked(what, device, ("workspace", given, given.shape, given.dtype))
        return given
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


@_on_stream
def act_quantize(x, codes=None, scales=None, check=True):
    """Keep an activation in 8 bits (``gdn_act_quantize``): ``(codes, scales)``.

    x [..., D] (bf16 or fp32, CUDA, contiguous), D a multiple of 32.  codes [..., D]
    float8_e4m3fn; scales [..., D / 32] uint8, one byte e + 127 per 32 values, which
    stand for code * 2^e; 2^e is the least power of two with max |x| <= 448 * 2^e.
    Values that are not finite read back as NaN and do not touch their group's scale.
    """
    import torch
    shape, device, bf16 = x.shape, x.device, x.dtype is torch.bfloat16
    if shape[-1] % 32 != 0:
        raise GdnError(-2, "gdn_act_quantize")
    groups = (*shape[:-1], shape[-1] // 32)
    _checked("gdn_act_quantize", device, ("x", x, shape, torch.bfloat16 if bf16 else torch.float32),
             ("codes", codes, shape, torch.float8_e4m3fn), ("scales", scales, groups, torch.uint8))
    if codes is None:
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=device)
    if scales is None:
        scales = torch.empty(groups, dtype=torch.uint8, device=device)
    _run("gdn_act_quantize", device, check, x.data_ptr(), codes.data_ptr(), scales.data_ptr(), x.numel(),
         DTYPE_BF16 if bf16 else DTYPE_F32)
    return codes, scales


@_on_stream
def act_dequantize(codes, scales, dtype, out=None, check=True):
    """The values that ``act_quantize``'s codes and scales stand for, in ``dtype`` (``gdn_act_dequantize``)."""
    import torch
    shape, device, bf16 = codes.shape, codes.device, dtype is torch.bfloat16
    if shape[-1] % 32 != 0 or not (bf16 or dtype is torch.float32):
        raise GdnError(-2, "gdn_act_dequantize")
    _checked("gdn_act_dequantize", device, ("codes", codes, shape, torch.float8_e4m3fn),
             ("scales", scales, (*shape[:-1], shape[-1] // 32), torch.uint8), ("out", out, shape, dtype))
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    _run("gdn_act_dequantize", device, check, codes.data_ptr(), _ptr(scales), out.data_ptr(), codes.numel(),
         DTYPE_BF16 if bf16 else DTYPE_F32)
    return out


@_on_stream
def gated_rmsnorm_bwd(dy, o, z, weight, eps=1e-6, d_o=None, d_z=None, d_weight=None, workspace=None, check=True):
    """Gradients of ``gated_rmsnorm`` (``gdn_gated_rmsnorm_bwd``): ``(do, dz, dweight)``.

    dy [..., D] (bf16 or fp32; D in {64, 128}).  o and z are the forward call's inputs
    in the dtype of dy, or, each for itself, the pair that ``act_quantize`` returned for
    it.  do, dz have dy's dtype; dweight [D] is fp32.
    """
    import torch
    (o, os_), (z, zs) = _kept(o), _kept(z)
    dim, bf16 = dy.shape[-1], dy.dtype == torch.bfloat16
    rows, io, f32 = int(dy.numel() // dim), DTYPE_BF16 if bf16 else DTYPE_F32, torch.float32
    _checked("gdn_gated_rmsnorm_bwd", dy.device, ("dy", dy, dy.shape, torch.bfloat16 if bf16 else f32),
             *_kept_specs("o", o, os_, dy.shape, dy.dtype), *_kept_specs("z", z, zs, dy.shape, dy.dtype), ("weight", weight, (dim,), f32),
             ("d_o", d_o, dy.shape, dy.dtype), ("d_z", d_z, dy.shape, dy.dtype), ("d_weight", d_weight, (dim,), f32))
    d_o = torch.empty_like(dy) if d_o is None else d_o
    d_z = torch.empty_like(dy) if d_z is None else d_z
    d_weight = torch.empty(dim, dtype=torch.float32, device=dy.device) if d_weight is None else d_weight
    workspace = _workspace(workspace, lib().gdn_gated_rmsnorm_bwd_workspace(rows, int(dim), io), "gdn_gated_rmsnorm_bwd", dy.device)
    _run("gdn_gated_rmsnorm_bwd", dy.device, check, _ptr(dy), _ptr(o), _ptr(os_), _ptr(z), _ptr(zs), _ptr(weight),
         float(eps), _ptr(d_o), _ptr(d_z), _ptr(d_weight), rows, int(dim), io, _ptr(workspace), _bytes(workspace))
    return d_o, d_z, d_weight


@_on_stream
def qkv_conv_bwd(dq, dk, dv, mixed_qkv, weight, bias=None, conv_state=None, cu_seqlens=None, num_seqs=None,
                 d_state_out=None, output_d_state=None, dx=None, d_weight=None, d_bias=None, d_state=None,
                 workspace=None, check=True):
    """Gradients of ``qkv_conv_fwd`` (``gdn_qkv_conv_bwd``): ``(dx, dweight, dbias, d_conv_state)``.

    dq, dk [T, Nqk, Dk], dv [T, Nv, Dv] (bf16 or fp32): the gradients of the call's q, k, v.
    mixed_qkv, weight, bias, conv_state, cu_seqlens: the call's inputs, mixed_qkv also as
    the pair that ``act_quantize`` returned for it.  d_state_out [N, C, K]: the gradient of
    the new conv_state, if there is one.  dx [T, C] and d_conv_state [N, C, K] have dq's
    dtype, dweight [C, K] and dbias [C] are fp32; dbias is None without a bias, and
    d_conv_state unless a conv_state was given or it was asked for.
    """
    import torch
    x, xs = _kept(mixed_qkv)
    T, C = x.shape
    K = weight.shape[1]
    nqk, dkk, nv, dvv = dq.shape[1], dq.shape[2], dv.shape[1], dv.shape[2]
    n = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    if C != 2 * nqk * dkk + nv * dvv:
        raise GdnError(-2, "gdn_qkv_conv_bwd")
    dev, io, f32, state = dq.device, dq.dtype, torch.float32, (n, C, K)
    _checked("gdn_qkv_conv_bwd", dev, ("dq", dq, (T, nqk, dkk), torch.bfloat16 if io == torch.bfloat16 else f32),
             ("dk", dk, dq.shape, io), ("dv", dv, (T, nv, dvv), io), *_kept_specs("mixed_qkv", x, xs, x.shape, io),
             ("weight", weight, (C, K), f32), ("bias", bias, (C,), f32), ("conv_state", conv_state, state, io),
             ("cu_seqlens", cu_seqlens, (n + 1,), torch.int32), ("d_state_out", d_state_out, state, io), ("dx", dx, x.shape, io),
             ("d_weight", d_weight, (C, K), f32), ("d_bias", d_bias, (C,), f32), ("d_state", d_state, state, io))
    dx = torch.empty((T, C), dtype=dq.dtype, device=dev) if dx is None else dx
    d_weight = torch.empty((C, K), dtype=torch.float32, device=dev) if d_weight is None else d_weight
    if d_bias is None and bias is not None:
        d_bias = torch.empty(C, dtype=torch.float32, device=dev)
    if d_state is None and (conv_state is not None if output_d_state is None else output_d_state):
        d_state = torch.empty((n, C, K), dtype=dq.dtype, device=dev)
    p = make_params(nqk, nv, dkk, dvv, dq.dtype == torch.bfloat16)
    workspace = _workspace(workspace, lib().gdn_qkv_conv_bwd_workspace(int(T), int(K), ctypes.byref(p)), "gdn_qkv_conv_bwd", dev)
    _run("gdn_qkv_conv_bwd", dev, check, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(x), _ptr(xs), _ptr(weight), _ptr(bias),
         _ptr(conv_state), _ptr(d_state_out), _ptr(cu_seqlens), int(n), int(T), int(K), _ptr(dx), _ptr(d_weight), _ptr(d_bias),
         _ptr(d_state), _ptr(workspace), _bytes(workspace), ctypes.byref(p))
    return dx, d_weight, d_bias, d_state


@_on_stream
def gate_bwd(dg, dbeta, a, b, A_log, dt_bias, da=None, db=None, dA_log=None, ddt_bias=None, workspace=None, check=True):
    """Gradients of the layer's gate (``gdn_gate_bwd``): ``(da, db, dA_log, ddt_bias)``.

    dg, dbeta [T, Nv] (bf16 or fp32, as ``chunk_bwd`` returns them); a, b [T, Nv] and
    A_log, dt_bias [Nv] fp32, as ``chunk_fwd_gated`` takes them.  da, db have dg's dtype,
    dA_log and ddt_bias [Nv] are fp32.
    """
    import torch
    shape, device, bf16, io, f32 = a.shape, dg.device, dg.dtype is torch.bfloat16, dg.dtype, torch.float32
    T, nv = shape
    head = (nv,)
    _checked("gdn_gate_bwd", device, ("dg", dg, shape, torch.bfloat16 if bf16 else f32), ("dbeta", dbeta, shape, io), ("a", a, shape, f32),
             ("b", b, shape, f32), ("A_log", A_log, head, f32), ("dt_bias", dt_bias, head, f32), ("da", da, shape, io), ("db", db, shape, io),
             ("dA_log", dA_log, head, f32), ("ddt_bias", ddt_bias, head, f32))
    da = torch.empty_like(dg) if da is None else da
    db = torch.empty_like(dg) if db is None else db
    dA_log = torch.empty_like(A_log) if dA_log is None else dA_log
    ddt_bias = torch.empty_like(dt_bias) if ddt_bias is None else ddt_bias
    workspace = _workspace(workspace, lib().gdn_gate_bwd_workspace(T, nv), "gdn_gate_bwd", device)
    _run("gdn_gate_bwd", device, check, _ptr(dg), _ptr(dbeta), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(da), _ptr(db),
         _ptr(dA_log), _ptr(ddt_bias), T, nv, DTYPE_BF16 if bf16 else DTYPE_F32, _ptr(workspace), _bytes(workspace))
    return da, db, dA_log, ddt_bias
