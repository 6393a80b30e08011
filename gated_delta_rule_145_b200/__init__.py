"""B200 (sm_100a) gated delta rule forward pass, the gated linear recurrence with its
gradient, and the trainable steps around them: Python binding of libgdr.so.

The binding only marshals arguments: every step of the computation runs in the CUDA
kernels of ``libgdr.so`` (built in-tree by ``build.py``).  There is no CPU or PyTorch
fallback: importing works without a GPU, but every call needs the library and CUDA
tensors, and fails loudly otherwise.

The functions named ``gdr_*`` mirror the C ABI in ``include/gdr.h`` one to one
(pointer arguments take torch tensors, None or raw integer addresses).  ``prefill``,
``decode_step``, ``linear_recurrence``, ``layer_norm`` and the ``*_backward`` functions are
conveniences that check tensors and allocate the outputs.  None of them is recorded by autograd: the
trainable ones (``linear_recurrence``, ``layer_norm`` and the ``*_backward`` functions) refuse tensors that
require gradients where these are recorded, instead of losing them; call them under
``torch.no_grad()`` or from a ``torch.autograd.Function``.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "GdrError", "library", "gdr_prefill_chunked", "gdr_prefill_chunked_f32",
    "gdr_prefill_recurrent", "gdr_prefill_recurrent_f32", "gdr_decode_step",
    "gdr_decode_step_f32", "gdr_status_string", "gdr_device_status", "prefill", "decode_step", "LIB_PATH",
    "gdr_linear_recurrence", "gdr_linear_recurrence_f32", "gdr_linear_recurrence_backward",
    "gdr_linear_recurrence_backward_f32", "gdr_zero_outer_rows", "gdr_layer_norm", "gdr_layer_norm_f32",
    "gdr_layer_norm_backward", "gdr_layer_norm_backward_f32", "gdr_short_conv_silu_backward",
    "gdr_gated_rmsnorm_backward", "gdr_gated_rmsnorm_backward_f32", "linear_recurrence",
    "linear_recurrence_backward", "layer_norm", "layer_norm_backward",
    "short_conv_silu_backward", "gated_rmsnorm_backward",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgdr.so")

GDR_OK = 0
GDR_ERR_NULL = -1
GDR_ERR_SHAPE = -2
GDR_ERR_UNSUPPORTED = -3
GDR_ERR_ALIGN = -4
GDR_ERR_OOM = -5
GDR_ERR_CUDA = -6
GDR_ERR_TIMEOUT = -7
GDR_ERR_TOO_LARGE = -8


class GdrError(RuntimeError):
    def __init__(self, name, status):
        super().__init__(f"{name} returned {status}: {gdr_status_string(status)}")
        self.status = status


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_F = ctypes.c_float

_SIGS = {
    "gdr_prefill_chunked": [_P] * 11 + [_I] * 7 + [_P],
    "gdr_prefill_chunked_f32": [_P] * 11 + [_I] * 7 + [_P],
    "gdr_prefill_chunked_noalloc": [_P] * 11 + [_I] * 7 + [_P],
    "gdr_prefill_recurrent": [_P] * 11 + [_I] * 6 + [_P],
    "gdr_prefill_recurrent_f32": [_P] * 11 + [_I] * 6 + [_P],
    "gdr_decode_step": [_P] * 9 + [_I] * 5 + [_P],
    "gdr_decode_step_f32": [_P] * 9 + [_I] * 5 + [_P],
    "gdr_gla_prefill_chunked": [_P] * 11 + [_I] * 7 + [_P],
    "gdr_gla_prefill_chunked_f32": [_P] * 11 + [_I] * 7 + [_P],
    "gdr_gla_prefill_recurrent": [_P] * 11 + [_I] * 6 + [_P],
    "gdr_gla_prefill_recurrent_f32": [_P] * 11 + [_I] * 6 + [_P],
    "gdr_gla_decode_step": [_P] * 9 + [_I] * 5 + [_P],
    "gdr_gla_decode_step_f32": [_P] * 9 + [_I] * 5 + [_P],
    "gdr_short_conv_silu": [_P] * 6 + [_I] * 4 + [_P],
    "gdr_gated_rmsnorm": [_P] * 4 + [ctypes.c_longlong, _I, ctypes.c_float, _P],
    "gdr_gated_rmsnorm_f32": [_P] * 4 + [ctypes.c_longlong, _I, ctypes.c_float, _P],
    "gdr_short_conv_silu_backward": [_P] * 10 + [_I] * 4 + [_P],
    "gdr_gated_rmsnorm_backward": [_P] * 7 + [_L, _I, _F, _P],
    "gdr_gated_rmsnorm_backward_f32": [_P] * 7 + [_L, _I, _F, _P],
    "gdr_layer_norm": [_P] * 6 + [_L, _I, _F, _P],
    "gdr_layer_norm_f32": [_P] * 6 + [_L, _I, _F, _P],
    "gdr_layer_norm_backward": [_P] * 8 + [_L, _I, _P],
    "gdr_layer_norm_backward_f32": [_P] * 8 + [_L, _I, _P],
    "gdr_linear_recurrence": [_P] * 9 + [_I] * 3 + [_L, _P],
    "gdr_linear_recurrence_f32": [_P] * 9 + [_I] * 3 + [_L, _P],
    "gdr_linear_recurrence_backward": [_P] * 16 + [_I] * 3 + [_L] * 2 + [_P],
    "gdr_linear_recurrence_backward_f32": [_P] * 16 + [_I] * 3 + [_L] * 2 + [_P],
    "gdr_zero_outer_rows": [_P] * 4 + [_I] * 2 + [_L] * 2 + [_P],
    "gdr_prefill_segment_maps": [_P] * 10 + [_I] * 7 + [_P],
    "gdr_segment_combine": [_P] * 5 + [_I] * 4 + [_P],
    "gdr_prefill_chunked_cp": [_P] * 10 + [_I] * 7 + [_P],
    "gdr_prefill_chunked_host": [_P] * 10 + [_I] * 8 + [_P],
}


def library():
    """The loaded libgdr.so (ctypes).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m gated_delta_rule_145_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = _I
        lib.gdr_device_status.argtypes = [_P]
        lib.gdr_device_status.restype = _I
        lib.gdr_selftest_bounded_wait.argtypes = [_P]
        lib.gdr_selftest_bounded_wait.restype = _I
        lib.gdr_status_string.argtypes = [_I]
        lib.gdr_status_string.restype = ctypes.c_char_p
        lib.gdr_release_workspace.argtypes = []
        lib.gdr_release_workspace.restype = None
        _lib = lib
    return _lib


def gdr_status_string(status: int) -> str:
    return library().gdr_status_string(int(status)).decode()


def gdr_device_status(stream=None) -> int:
    """Synchronise `stream` and return the device-side status (GDR_OK or an error code)."""
    return library().gdr_device_status(_stream(stream))


def gdr_selftest_bounded_wait(stream=None) -> int:
    """Enqueue the failure-detection self-test (see include/gdr.h); gdr_device_status then
    reports GDR_ERR_TIMEOUT once its bounded wait has given up."""
    return library().gdr_selftest_bounded_wait(_stream(stream))


def gdr_release_workspace() -> None:
    """Return the workspace memory cached by earlier calls."""
    library().gdr_release_workspace()


def _stream(s):
    if s is None:
        import torch

        # torch.cuda.current_stream() makes a Stream object (1.3 us) around this integer
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    return s if isinstance(s, int) else s.cuda_stream


_INT_MAX = 0x7fffffff


def _call(name, ptrs, ints, stream, check, longs=()):
    fn = getattr(_lib or library(), name)
    if (max(ints) > _INT_MAX or min(ints) < -_INT_MAX or  # ctypes would drop the upper bits
            longs and max(map(abs, longs)) >= 1 << 62):
        status = GDR_ERR_SHAPE
    else:
        status = fn(*[p if p is None or isinstance(p, int) else p.data_ptr() for p in ptrs],
                    *map(int, ints), *map(int, longs), _stream(stream))
    if check and status != GDR_OK:
        raise GdrError(name, status)
    return status


def gdr_prefill_chunked(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens,
                        B, T, Hk, Hv, dk, dv, chunk, stream=None, check=True):
    return _call("gdr_prefill_chunked",
                 (q, k, v, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens),
                 (B, T, Hk, Hv, dk, dv, chunk), stream, check)


def gdr_prefill_chunked_noalloc(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state,
                                cu_seqlens, B, T, Hk, Hv, dk, dv, chunk, stream=None, check=True):
    """gdr_prefill_chunked on the library's fixed scratch: no device memory is allocated
    (bf16, dk = dv = 128, chunk 32; see include/gdr.h for the size limit)."""
    return _call("gdr_prefill_chunked_noalloc",
                 (q, k, v, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens),
                 (B, T, Hk, Hv, dk, dv, chunk), stream, check)


def gdr_prefill_chunked_host(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state, B,
                             T, Hk, Hv, dk, dv, chunk=32, seg_tokens=0, stream=None,
                             check=True):
    """gdr_prefill_chunked from and to HOST buffers (pinned CPU tensors or raw addresses),
    the copies overlapped with the kernels; complete once `stream` is."""
    return _call("gdr_prefill_chunked_host",
                 (q, k, v, a, b, A_log, dt_bias, init_state, out, final_state),
                 (B, T, Hk, Hv, dk, dv, chunk, seg_tokens), stream, check)


def gdr_prefill_segment_maps(q, k, v, a, b, A_log, dt_bias, phi, nmap, cu_seqlens, B, T, Hk,
                             Hv, dk, dv, chunk, stream=None, check=True):
    """Per-segment state maps S_end = phi S_start + nmap of B segments (include/gdr.h)."""
    return _call("gdr_prefill_segment_maps",
                 (q, k, v, a, b, A_log, dt_bias, phi, nmap, cu_seqlens),
                 (B, T, Hk, Hv, dk, dv, chunk), stream, check)


def gdr_segment_combine(phi, nmap, init_state, seg_init, final_state, G, Hv, dk, dv,
                        stream=None, check=True):
    """Composes G segment maps in order into start states and the final state."""
    return _call("gdr_segment_combine", (phi, nmap, init_state, seg_init, final_state),
                 (G, Hv, dk, dv), stream, check)


def gdr_prefill_chunked_cp(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state, T, Hk,
                           Hv, dk, dv, chunk, nseg, stream=None, check=True):
    """One sequence cut into at most nseg segments processed side by side on this GPU."""
    return _call("gdr_prefill_chunked_cp",
                 (q, k, v, a, b, A_log, dt_bias, init_state, out, final_state),
                 (T, Hk, Hv, dk, dv, chunk, nseg), stream, check)


def gdr_prefill_chunked_f32(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state,
                            cu_seqlens, B, T, Hk, Hv, dk, dv, chunk, stream=None, check=True):
    return _call("gdr_prefill_chunked_f32",
                 (q, k, v, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens),
                 (B, T, Hk, Hv, dk, dv, chunk), stream, check)


def gdr_prefill_recurrent(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state,
                          cu_seqlens, B, T, Hk, Hv, dk, dv, stream=None, check=True):
    return _call("gdr_prefill_recurrent",
                 (q, k, v, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens),
                 (B, T, Hk, Hv, dk, dv), stream, check)


def gdr_prefill_recurrent_f32(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state,
                              cu_seqlens, B, T, Hk, Hv, dk, dv, stream=None, check=True):
    return _call("gdr_prefill_recurrent_f32",
                 (q, k, v, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens),
                 (B, T, Hk, Hv, dk, dv), stream, check)


def gdr_decode_step(q, k, v, a, b, A_log, dt_bias, state, out, B, Hk, Hv, dk, dv, stream=None,
                    check=True):
    return _call("gdr_decode_step", (q, k, v, a, b, A_log, dt_bias, state, out),
                 (B, Hk, Hv, dk, dv), stream, check)


def gdr_decode_step_f32(q, k, v, a, b, A_log, dt_bias, state, out, B, Hk, Hv, dk, dv,
                        stream=None, check=True):
    return _call("gdr_decode_step_f32", (q, k, v, a, b, A_log, dt_bias, state, out),
                 (B, Hk, Hv, dk, dv), stream, check)


# ------------------------------------------------------------------------- conveniences


def _check_tensors(tensors, dtype):
    import torch

    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        want = dtype if name in ("q", "k", "v", "a", "b") else (
            torch.int32 if name == "cu_seqlens" else torch.float32)
        if t.dtype != want:
            raise ValueError(f"{name} must be {want}, got {t.dtype}")


def _gla_wrapper(name, nptr):
    """Mirror of the C entry point `name`: nptr pointer arguments, then the sizes."""
    def fn(*args, stream=None, check=True):
        return _call(name, args[:nptr], args[nptr:], stream, check)
    fn.__name__ = name
    fn.__doc__ = f"{name}: the erase=False (gated linear attention) form; see include/gdr.h."
    return fn


gdr_gla_prefill_chunked = _gla_wrapper("gdr_gla_prefill_chunked", 11)
gdr_gla_prefill_chunked_f32 = _gla_wrapper("gdr_gla_prefill_chunked_f32", 11)
gdr_gla_prefill_recurrent = _gla_wrapper("gdr_gla_prefill_recurrent", 11)
gdr_gla_prefill_recurrent_f32 = _gla_wrapper("gdr_gla_prefill_recurrent_f32", 11)
gdr_gla_decode_step = _gla_wrapper("gdr_gla_decode_step", 9)
gdr_gla_decode_step_f32 = _gla_wrapper("gdr_gla_decode_step_f32", 9)


def gdr_short_conv_silu(x, weight, bias, conv_state_in, conv_state_out, y, B, T, C, width=4,
                        stream=None, check=True):
    """The four-tap causal convolution + SiLU before the rule (see include/gdr.h)."""
    return _call("gdr_short_conv_silu", (x, weight, bias, conv_state_in, conv_state_out, y),
                 (B, T, C, width), stream, check)


def _rows_call(name, ptrs, rows, d, rest, stream, check):
    """A row-wise call: pointers, then rows, d and what follows them (eps)."""
    fn = getattr(_lib or library(), name)
    if not -_INT_MAX <= d <= _INT_MAX or not -1 << 62 < rows < 1 << 62:  # as in _call
        status = GDR_ERR_SHAPE
    else:
        status = fn(*[p if p is None or isinstance(p, int) else p.data_ptr() for p in ptrs],
                    int(rows), int(d), *rest, _stream(stream))
    if check and status != GDR_OK:
        raise GdrError(name, status)
    return status


def _norm_call(name, o, z, weight, y, rows, d, eps, stream, check):
    return _rows_call(name, (o, z, weight, y), rows, d, (float(eps),), stream, check)


def gdr_gated_rmsnorm(o, z, weight, y, rows, d, eps=1e-6, stream=None, check=True):
    """The gated RMS normalisation after the rule, bf16 gate (see include/gdr.h)."""
    return _norm_call("gdr_gated_rmsnorm", o, z, weight, y, rows, d, eps, stream, check)


def gdr_gated_rmsnorm_f32(o, z, weight, y, rows, d, eps=1e-6, stream=None, check=True):
    """The gated RMS normalisation after the rule, fp32 gate (see include/gdr.h)."""
    return _norm_call("gdr_gated_rmsnorm_f32", o, z, weight, y, rows, d, eps, stream, check)


def gdr_short_conv_silu_backward(x, weight, bias, conv_state_in, grad_y, grad_conv_state_out,
                                 grad_x, grad_weight, grad_bias, grad_conv_state_in, B, T, C,
                                 width=4, stream=None, check=True):
    """The gradient of gdr_short_conv_silu (see include/gdr.h)."""
    return _call("gdr_short_conv_silu_backward",
                 (x, weight, bias, conv_state_in, grad_y, grad_conv_state_out, grad_x,
                  grad_weight, grad_bias, grad_conv_state_in), (B, T, C, width), stream, check)


def gdr_gated_rmsnorm_backward(o, z, weight, grad_y, grad_o, grad_z, grad_weight, rows, d,
                               eps=1e-6, stream=None, check=True):
    """The gradient of gdr_gated_rmsnorm, bf16 gate (see include/gdr.h)."""
    return _rows_call("gdr_gated_rmsnorm_backward",
                      (o, z, weight, grad_y, grad_o, grad_z, grad_weight), rows, d,
                      (float(eps),), stream, check)


def gdr_gated_rmsnorm_backward_f32(o, z, weight, grad_y, grad_o, grad_z, grad_weight, rows, d,
                                   eps=1e-6, stream=None, check=True):
    """The gradient of gdr_gated_rmsnorm_f32, fp32 gate (see include/gdr.h)."""
    return _rows_call("gdr_gated_rmsnorm_backward_f32",
                      (o, z, weight, grad_y, grad_o, grad_z, grad_weight), rows, d,
                      (float(eps),), stream, check)


def gdr_layer_norm(x, weight, bias, y, mean, rstd, rows, d, eps=1e-5, stream=None, check=True):
    """Layer normalisation of bf16 rows (see include/gdr.h)."""
    return _rows_call("gdr_layer_norm", (x, weight, bias, y, mean, rstd), rows, d,
                      (float(eps),), stream, check)


def gdr_layer_norm_f32(x, weight, bias, y, mean, rstd, rows, d, eps=1e-5, stream=None,
                       check=True):
    """Layer normalisation of fp32 rows (see include/gdr.h)."""
    return _rows_call("gdr_layer_norm_f32", (x, weight, bias, y, mean, rstd), rows, d,
                      (float(eps),), stream, check)


def gdr_layer_norm_backward(x, weight, mean, rstd, grad_y, grad_x, grad_weight, grad_bias, rows,
                            d, stream=None, check=True):
    """The gradient of gdr_layer_norm (see include/gdr.h)."""
    return _rows_call("gdr_layer_norm_backward",
                      (x, weight, mean, rstd, grad_y, grad_x, grad_weight, grad_bias), rows, d,
                      (), stream, check)


def gdr_layer_norm_backward_f32(x, weight, mean, rstd, grad_y, grad_x, grad_weight, grad_bias,
                                rows, d, stream=None, check=True):
    """The gradient of gdr_layer_norm_f32 (see include/gdr.h)."""
    return _rows_call("gdr_layer_norm_backward_f32",
                      (x, weight, mean, rstd, grad_y, grad_x, grad_weight, grad_bias), rows, d,
                      (), stream, check)


def gdr_linear_recurrence(x, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens, B, T,
                          C, ld, stream=None, check=True):
    """The gated linear recurrence (vector state), bf16 x, a, b (see include/gdr.h)."""
    return _call("gdr_linear_recurrence",
                 (x, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens),
                 (B, T, C, ld), stream, check)


def gdr_linear_recurrence_f32(x, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens,
                              B, T, C, ld, stream=None, check=True):
    """The gated linear recurrence (vector state), fp32 x, a, b (see include/gdr.h)."""
    return _call("gdr_linear_recurrence_f32",
                 (x, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens),
                 (B, T, C, ld), stream, check)


def gdr_linear_recurrence_backward(x, a, b, A_log, dt_bias, init_state, out, grad_out,
                                   grad_final_state, grad_x, grad_a, grad_b, grad_A_log,
                                   grad_dt_bias, grad_init_state, cu_seqlens, B, T, C, ld,
                                   ld_grad, stream=None, check=True):
    """The gradient of gdr_linear_recurrence (see include/gdr.h)."""
    return _call("gdr_linear_recurrence_backward",
                 (x, a, b, A_log, dt_bias, init_state, out, grad_out, grad_final_state, grad_x,
                  grad_a, grad_b, grad_A_log, grad_dt_bias, grad_init_state, cu_seqlens),
                 (B, T, C, ld, ld_grad), stream, check)


def gdr_linear_recurrence_backward_f32(x, a, b, A_log, dt_bias, init_state, out, grad_out,
                                       grad_final_state, grad_x, grad_a, grad_b, grad_A_log,
                                       grad_dt_bias, grad_init_state, cu_seqlens, B, T, C, ld,
                                       ld_grad, stream=None, check=True):
    """The gradient of gdr_linear_recurrence_f32 (see include/gdr.h)."""
    return _call("gdr_linear_recurrence_backward_f32",
                 (x, a, b, A_log, dt_bias, init_state, out, grad_out, grad_final_state, grad_x,
                  grad_a, grad_b, grad_A_log, grad_dt_bias, grad_init_state, cu_seqlens),
                 (B, T, C, ld, ld_grad), stream, check)


def gdr_zero_outer_rows(x, y, z, cu_seqlens, B, T, row_bytes, pitch_bytes, stream=None, check=True):
    """Zeros in the rows of packed tensors that no sequence holds (see include/gdr.h)."""
    return _call("gdr_zero_outer_rows", (x, y, z, cu_seqlens), (B, T), stream, check,
                 (row_bytes, pitch_bytes))


def prefill(q, k, v, a, b, A_log, dt_bias, init_state=None, cu_seqlens=None, chunk=32,
            form="chunked", out=None, final_state=None, stream=None, erase=True):
    """Prefill over q, k [B, T, Hk, dk], v [B, T, Hv, dv], a, b [B, T, Hv] (bf16 or fp32).

    ``form`` is "chunked" (UT transform) or "recurrent".  With ``cu_seqlens`` (int32,
    device, [N + 1]) the tokens are packed along T (B must be 1) into N sequences.
    ``erase=False`` runs gated linear attention (the rule without its erase term).
    Returns (out [B, T, Hv, dv] fp32, final_state [Nseq, Hv, dk, dv] fp32).
    """
    import torch

    dtype = q.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("q, k, v, a, b must be bf16 or fp32")
    _check_tensors(dict(q=q, k=k, v=v, a=a, b=b, A_log=A_log, dt_bias=dt_bias,
                        init_state=init_state, cu_seqlens=cu_seqlens), dtype)
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    nseq = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if cu_seqlens is not None and B != 1:
        raise ValueError("packed sequences need B == 1")
    if out is None:
        out = torch.empty((B, T, Hv, dv), device=q.device, dtype=torch.float32)
    if final_state is None:
        final_state = torch.empty((nseq, Hv, dk, dv), device=q.device, dtype=torch.float32)
    f32 = dtype == torch.float32
    args = (q, k, v, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens,
            nseq, B * T if cu_seqlens is not None else T, Hk, Hv, dk, dv)
    if form == "chunked":
        fn = ((gdr_prefill_chunked_f32 if f32 else gdr_prefill_chunked) if erase else
              (gdr_gla_prefill_chunked_f32 if f32 else gdr_gla_prefill_chunked))
        fn(*args, chunk, stream=stream)
    elif form == "recurrent":
        fn = ((gdr_prefill_recurrent_f32 if f32 else gdr_prefill_recurrent) if erase else
              (gdr_gla_prefill_recurrent_f32 if f32 else gdr_gla_prefill_recurrent))
        fn(*args, stream=stream)
    else:
        raise ValueError(f"unknown form {form!r}")
    return out, final_state


def decode_step(q, k, v, a, b, A_log, dt_bias, state, out=None, stream=None, erase=True):
    """One recurrent step: q, k [B, Hk, dk], v [B, Hv, dv], a, b [B, Hv]; ``state``
    [B, Hv, dk, dv] fp32 is updated in place (``erase=False``: gated linear attention).
    Returns out [B, Hv, dv] fp32."""
    import torch

    dtype = q.dtype
    _check_tensors(dict(q=q, k=k, v=v, a=a, b=b, A_log=A_log, dt_bias=dt_bias, state=state),
                   dtype)
    B, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    if out is None:
        out = torch.empty((B, Hv, dv), device=q.device, dtype=torch.float32)
    f32 = dtype == torch.float32
    fn = ((gdr_decode_step_f32 if f32 else gdr_decode_step) if erase else
          (gdr_gla_decode_step_f32 if f32 else gdr_gla_decode_step))
    fn(q, k, v, a, b, A_log, dt_bias, state, out, B, Hk, Hv, dk, dv, stream=stream)
    return out


def _check(first, *specs):
    """Every (name, tensor, dtype, shape, dense) of `specs` is a CUDA tensor on `first`'s device of
    this type and shape, contiguous if `dense`, and autograd does not expect its gradient; None
    passes."""
    index = first.get_device()  # -1: none; an integer, compared in half of a device's time
    for name, t, dtype, shape, dense in specs:
        if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0 and
                         (not dense or t.is_contiguous()) and not t.requires_grad):
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, not on {first.device}")
        if dense and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        import torch

        if torch.is_grad_enabled():  # autograd would take the result for a constant
            raise ValueError(f"{name} requires a gradient, and this call is not recorded by autograd: "
                             "call it under torch.no_grad() or from a torch.autograd.Function (whose "
                             "backward calls the *_backward functions)")


def _token_stride(tensors, B, T, C):
    """Elements between consecutive tokens of [B, T, C] tensors that share one layout: dense,
    or slices of the last dimension of a wider dense tensor."""
    if B * T * C == 0:
        return max(C, 1)
    if all([t.is_contiguous() for t in tensors]):
        return C
    first = tensors[0].stride()
    ld = first[1] if T > 1 else first[0] if B > 1 else C
    for t in tensors:
        sb, st, sc = t.stride()
        if (C > 1 and sc != 1) or (T > 1 and st != ld) or (B > 1 and sb != T * ld):
            raise ValueError("x, a, b (and their gradients) need one layout, dense or slices of "
                             f"the last dimension of a dense tensor; got strides {t.stride()}")
    return ld


def _input_type(x, name):
    import torch

    if x.dtype is not torch.bfloat16 and x.dtype is not torch.float32:
        raise ValueError(f"{name} must be bf16 or fp32, got {x.dtype}")
    return x.dtype


def _launch(name, t, stream, tensors, sizes, *rest):
    """The C call `name` on `stream` (None: the current one) of t's device, that device current:
    pointers of `tensors` (or None), sizes, `rest`.  As the mirrors above, in less host time."""
    import torch

    index = t.get_device()
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _launch(name, t, stream, tensors, sizes, *rest)
    status = getattr(_lib or library(), name)(
        *[None if v is None else v.data_ptr() for v in tensors], *sizes, *rest, _stream(stream))
    if status != GDR_OK:
        raise GdrError(name, status)


def _empty(t, stream, *specs):
    """Uninitialised tensors of (shape, dtype) on t's device, allocated for use on `stream`: memory
    of the current stream's pool could still be in use by work queued there."""
    import torch

    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=t.device)
        with torch.cuda.stream(stream):
            return _empty(t, None, *specs)
    # of the ways to say it these two take torch the least time: 1.3 and 1.5 us, not 2.6
    like, device = t.dtype if t.is_contiguous() else None, t.device
    return [torch.empty_like(t) if dtype is like and shape == t.shape else
            torch.empty(*shape or ((),), dtype=dtype, device=device) for shape, dtype in specs]


def _recurrence_args(x, a, b, A_log, dt_bias, init_state, cu_seqlens):
    import torch

    dtype = _input_type(x, "x")
    if x.dim() != 3:
        raise ValueError(f"x must be [B, T, C], got shape {tuple(x.shape)}")
    B, T, C = shape = x.shape
    _int_sizes(shape)
    f32 = torch.float32
    nseq = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("packed sequences need B == 1")
        nseq = cu_seqlens.numel() - 1
        _int_sizes((nseq,))
    _check(x, ("x", x, dtype, shape, False), ("a", a, dtype, shape, False),
           ("b", b, dtype, shape, False), ("cu_seqlens", cu_seqlens, torch.int32, (nseq + 1,), True),
           ("A_log", A_log, f32, (C,), True), ("dt_bias", dt_bias, f32, (C,), True),
           ("init_state", init_state, f32, (nseq, C), True))
    return dtype, nseq, T, C, _token_stride((x, a, b), B, T, C)


def linear_recurrence(x, a, b, A_log, dt_bias, init_state=None, cu_seqlens=None, out=None,
                      final_state=None, stream=None):
    """The gated linear recurrence h <- h exp(g) + sigmoid(b) x per channel, with the rule's
    decay g = -exp(A_log) softplus(a + dt_bias): x, a, b [B, T, C] bf16 or fp32, dense or all
    three slices of the last dimension of a dense tensor; A_log, dt_bias [C]; ``init_state``
    [Nseq, C] (zeros if None).  With ``cu_seqlens`` (int32, device, [Nseq + 1]) the tokens are
    packed along T (B must be 1); rows outside them are zero in an ``out`` that the call
    allocates and stay as they were in one that is given.  T = 1 is a decode step;
    ``final_state`` may be ``init_state``.  Returns (out [B, T, C] fp32, final_state [Nseq, C] fp32)."""
    import torch

    dtype, nseq, T, C, ld = _recurrence_args(x, a, b, A_log, dt_bias, init_state, cu_seqlens)
    f32 = torch.float32
    _check(x, ("out", out, f32, x.shape, True),
           ("final_state", final_state, f32, (nseq, C), True))
    fresh = out is None
    if fresh:
        out, = _empty(x, stream, (x.shape, f32))
    if final_state is None:
        final_state, = _empty(x, stream, ((nseq, C), f32))
    _launch("gdr_linear_recurrence_f32" if dtype is f32 else "gdr_linear_recurrence", x, stream,
            (x, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens), (nseq, T, C, ld))
    if fresh and cu_seqlens is not None:
        _launch("gdr_zero_outer_rows", x, stream, (out, None, None, cu_seqlens), (nseq, T, 4 * C, 4 * C))
    return out, final_state


def linear_recurrence_backward(x, a, b, A_log, dt_bias, out, grad_out, grad_final_state=None,
                               init_state=None, cu_seqlens=None, grad_x=None, grad_a=None,
                               grad_b=None, stream=None):
    """The gradient of ``linear_recurrence``: its arguments and its ``out``, with grad_out
    [B, T, C] fp32 and ``grad_final_state`` [Nseq, C] fp32 (zeros if None).  ``grad_x``,
    ``grad_a``, ``grad_b`` may be given, all three, in one layout as x, a, b may have (for
    example slices of one projection's gradient); their rows outside packed sequences stay as
    they were, and are zero where the call allocates them.  Returns (grad_x, grad_a, grad_b,
    grad_A_log [C], grad_dt_bias [C], grad_init_state [Nseq, C])."""
    import torch

    dtype, nseq, T, C, ld = _recurrence_args(x, a, b, A_log, dt_bias, init_state, cu_seqlens)
    f32 = torch.float32
    grads = (grad_x, grad_a, grad_b)
    _check(x, ("out", out, f32, x.shape, True), ("grad_out", grad_out, f32, x.shape, True),
           ("grad_final_state", grad_final_state, f32, (nseq, C), True))
    fresh = grad_x is None
    if grad_x is None or grad_a is None or grad_b is None:
        if any(g is not None for g in grads):
            raise ValueError("give grad_x, grad_a and grad_b together, or none of them")
        grads, ld_grad = _empty(x, stream, *[(x.shape, dtype)] * 3), max(C, 1)
    else:
        _check(x, *[(n, g, dtype, x.shape, False)
                    for n, g in zip(("grad_x", "grad_a", "grad_b"), grads)])
        ld_grad = _token_stride(grads, x.shape[0], T, C)
    grad_A_log, grad_dt_bias, grad_init = _empty(x, stream, ((C,), f32), ((C,), f32),
                                                 ((nseq, C), f32))
    _launch("gdr_linear_recurrence_backward_f32" if dtype is f32 else
            "gdr_linear_recurrence_backward", x, stream,
            (x, a, b, A_log, dt_bias, init_state, out, grad_out, grad_final_state, *grads,
             grad_A_log, grad_dt_bias, grad_init, cu_seqlens), (nseq, T, C, ld, ld_grad))
    if fresh and cu_seqlens is not None:
        row = C * (4 if dtype is f32 else 2)
        _launch("gdr_zero_outer_rows", x, stream, (*grads, cu_seqlens), (nseq, T, row, row))
    return (*grads, grad_A_log, grad_dt_bias, grad_init)


def _int_sizes(shape):
    if max(shape) > _INT_MAX:  # ctypes would drop the upper bits
        raise ValueError(f"sizes have to be below 2^31, got {tuple(shape)}")


def _row_args(x):
    """(rows, d) of x [..., d]."""
    d = x.shape[-1] if x.dim() else 0
    _int_sizes((d,))
    return (x.numel() // d if d else 0), d


def layer_norm(x, weight, bias=None, eps=1e-5, y=None, stream=None):
    """Layer normalisation of x [..., d] (bf16 or fp32) over its last dimension: weight and
    ``bias`` [d] fp32.  ``y`` may be x.  Returns (y, mean [...], rstd [...]); the statistics
    (fp32) are what ``layer_norm_backward`` takes."""
    import torch

    dtype, f32 = _input_type(x, "x"), torch.float32
    rows, d = _row_args(x)
    _check(x, ("x", x, dtype, x.shape, True), ("weight", weight, f32, (d,), True),
           ("bias", bias, f32, (d,), True), ("y", y, dtype, x.shape, True))
    mean, rstd = _empty(x, stream, (x.shape[:-1], f32), (x.shape[:-1], f32))
    if y is None:
        y, = _empty(x, stream, (x.shape, dtype))
    _launch("gdr_layer_norm_f32" if dtype is f32 else "gdr_layer_norm", x, stream,
            (x, weight, bias, y, mean, rstd), (rows, d), float(eps))
    return y, mean, rstd


def layer_norm_backward(x, weight, mean, rstd, grad_y, grad_x=None, stream=None):
    """The gradient of ``layer_norm`` from its x, weight and statistics and grad_y (x's type).
    ``grad_x`` may be grad_y.  Returns (grad_x, grad_weight [d], grad_bias [d])."""
    import torch

    dtype, f32 = _input_type(x, "x"), torch.float32
    rows, d = _row_args(x)
    _check(x, ("x", x, dtype, x.shape, True), ("weight", weight, f32, (d,), True),
           ("mean", mean, f32, x.shape[:-1], True), ("rstd", rstd, f32, x.shape[:-1], True),
           ("grad_y", grad_y, dtype, x.shape, True), ("grad_x", grad_x, dtype, x.shape, True))
    if grad_x is None:
        grad_x, = _empty(x, stream, (x.shape, dtype))
    grad_weight, grad_bias = _empty(x, stream, ((d,), f32), ((d,), f32))
    _launch("gdr_layer_norm_backward_f32" if dtype is f32 else "gdr_layer_norm_backward", x, stream,
            (x, weight, mean, rstd, grad_y, grad_x, grad_weight, grad_bias), (rows, d))
    return grad_x, grad_weight, grad_bias


def short_conv_silu_backward(x, weight, grad_y, bias=None, conv_state_in=None,
                             grad_conv_state_out=None, stream=None):
    """The gradient of gdr_short_conv_silu: x, grad_y [B, T, C] bf16, weight [C, 4], ``bias``
    [C], ``conv_state_in`` and ``grad_conv_state_out`` [B, C, 3] (zeros if None).  Returns
    (grad_x, grad_weight, grad_bias, grad_conv_state_in)."""
    import torch

    f32, bf16 = torch.float32, torch.bfloat16
    if x.dim() != 3:
        raise ValueError(f"x must be [B, T, C], got shape {tuple(x.shape)}")
    B, T, C = x.shape
    _int_sizes(x.shape)
    _check(x, ("x", x, bf16, x.shape, True), ("weight", weight, f32, (C, 4), True),
           ("grad_y", grad_y, bf16, x.shape, True), ("bias", bias, f32, (C,), True),
           ("conv_state_in", conv_state_in, f32, (B, C, 3), True),
           ("grad_conv_state_out", grad_conv_state_out, f32, (B, C, 3), True))
    grad_x, grad_weight, grad_bias, grad_state = _empty(
        x, stream, (x.shape, bf16), ((C, 4), f32), ((C,), f32), ((B, C, 3), f32))
    _launch("gdr_short_conv_silu_backward", x, stream,
            (x, weight, bias, conv_state_in, grad_y, grad_conv_state_out, grad_x, grad_weight,
             grad_bias, grad_state), (B, T, C, 4))
    return grad_x, grad_weight, grad_bias, grad_state


def gated_rmsnorm_backward(o, z, weight, grad_y, eps=1e-6, stream=None):
    """The gradient of gdr_gated_rmsnorm[_f32] over the last dimension d of o [..., d] fp32, z
    bf16 or fp32, weight [d], grad_y fp32.  Returns (grad_o, grad_z, grad_weight [d])."""
    import torch

    f32 = torch.float32
    dtype = _input_type(z, "z")
    rows, d = _row_args(o)
    _check(o, ("o", o, f32, o.shape, True), ("z", z, dtype, o.shape, True),
           ("weight", weight, f32, (d,), True), ("grad_y", grad_y, f32, o.shape, True))
    grad_o, grad_z, grad_weight = _empty(o, stream, (o.shape, f32), (z.shape, dtype), ((d,), f32))
    _launch("gdr_gated_rmsnorm_backward_f32" if dtype is f32 else "gdr_gated_rmsnorm_backward", o,
            stream, (o, z, weight, grad_y, grad_o, grad_z, grad_weight), (rows, d), float(eps))
    return grad_o, grad_z, grad_weight
