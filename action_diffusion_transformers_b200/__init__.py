"""Python binding of the sm_100a quantized-attention library (libsage.so).

The three calls of the C ABI (include/sage.h) keep their names:

    sage_quant_qk(q, k, ...)   K smoothing + INT8 64-token block quantization
    sage_quant_v(v, ...)       V smoothing + per-channel E4M3, transposed
    sage_attn_fwd(...)         INT8 QK^T / FP8 PV attention, FP32 online softmax

and so do the serving calls beside them:

    sage_rope(q, k, ...)       rotary positions (both layouts, partial, scaled)
    sage_kv_write(k, v, ...)   quantized paged KV cache: write, sage_kv_read back
    sage_attn_prompt(...)      causal attention over packed prompts, grouped heads
    sage_attn_token(...)       attention of single tokens over the cache

This module only marshals arguments: torch tensors provide device memory and
the current CUDA stream; every step of the computation runs in the library's
CUDA kernels.  Importing it loads libsage.so and raises ImportError if that has
not been built; a serving call raises it if the extension module that hands
tensors to them does not load (there is no fallback implementation).
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsage.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libsage.so is not built ({LIB_PATH}); run "
                      "`python -m action_diffusion_transformers_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)
try:
    from . import _serve_ext  # built beside the library, for the installed torch and Python
except ImportError as _e:

    class _NoServeExt:
        """The quantized attention needs libsage.so alone; the serving calls raise."""

        def __init__(self, why):
            self.why = why

        def __getattr__(self, name):
            raise ImportError("the serving calls' extension module _serve_ext.so does not load with this torch and "
                              f"Python ({self.why}); run `python -m action_diffusion_transformers_b200.build`")

    _serve_ext = _NoServeExt(str(_e))

SAGE_OK = 0
STATUS_NAMES = {0: "SAGE_OK", 1: "SAGE_ERR_INVALID_ARG", 2: "SAGE_ERR_UNSUPPORTED", 3: "SAGE_ERR_ALIGNMENT",
                4: "SAGE_ERR_CUDA", 5: "SAGE_ERR_DEVICE_TIMEOUT", 6: "SAGE_ERR_WORKSPACE"}
EXPORTED = ("sage_npad", "sage_workspace_bytes", "sage_quant_qk", "sage_quant_v", "sage_attn_fwd",
            "sage_check", "sage_set_wait_timeout_ns", "sage_selftest_wait_timeout", "sage_last_error",
            "sage_quant_qk_static", "sage_quant_qk_normrope", "sage_fp8_quant_rows", "sage_fp8_linear",
            "sage_quant_qkv", "sage_attn_fwd_p_codes", "sage_rope_plan_init", "sage_rope", "sage_kv_write",
            "sage_kv_read", "sage_attn_prompt", "sage_attn_token", "sage_attn_token_workspace_bytes")
QK_STATIC_SCRATCH_BYTES = 8 << 20


GRAN = {"block64": 0, "token": 1, "segment64": 2}   # sage_gran: INT8 scale groups of Q / K
MAX_SEGMENTS = 256


class SageShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
                ("tok_stride", ctypes.c_int64), ("cu_seqlens", ctypes.POINTER(ctypes.c_int32)),
                ("n_seg", ctypes.c_int), ("q_gran", ctypes.c_int), ("k_gran", ctypes.c_int)]


class SageNormRope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("rope_cos", ctypes.c_void_p),
                ("rope_sin", ctypes.c_void_p), ("eps", ctypes.c_float)]


ROPE_MAX_PAIRS = 128
ROPE_SCALING = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3}   # sage_rope_scaling


class SageRows(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p), ("H", ctypes.c_int),
                ("in_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


class SageRopePlan(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("n_axes", ctypes.c_int),
                ("mscale", ctypes.c_float), ("turns", ctypes.c_double * ROPE_MAX_PAIRS),
                ("axis", ctypes.c_ubyte * ROPE_MAX_PAIRS)]


class SageKvCache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("Hk", ctypes.c_int), ("D", ctypes.c_int), ("format", ctypes.c_int)]


class SagePrompt(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int), ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p), ("Hq", ctypes.c_int),
                ("Hk", ctypes.c_int), ("D", ctypes.c_int), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("causal", ctypes.c_int), ("sm_scale", ctypes.c_float)]


class SageToken(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("q_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("dtype", ctypes.c_int), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p), ("max_len", ctypes.c_int),
                ("sm_scale", ctypes.c_float)]


_vp = ctypes.c_void_p
_lib.sage_npad.argtypes = [ctypes.c_int]
_lib.sage_npad.restype = ctypes.c_size_t
_lib.sage_workspace_bytes.argtypes = [SageShape]
_lib.sage_workspace_bytes.restype = ctypes.c_size_t
_lib.sage_quant_qk.argtypes = [_vp, _vp, SageShape, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.sage_quant_qk.restype = ctypes.c_int
_lib.sage_quant_qk_static.argtypes = [_vp, _vp, SageShape, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.sage_quant_qk_static.restype = ctypes.c_int
_lib.sage_quant_qk_normrope.argtypes = [_vp, _vp, SageShape, ctypes.POINTER(SageNormRope), _vp, _vp, _vp, _vp, _vp,
                                        _vp, ctypes.c_size_t, _vp]
_lib.sage_quant_qk_normrope.restype = ctypes.c_int
_lib.sage_quant_qkv.argtypes = [_vp, _vp, _vp, SageShape, ctypes.c_int64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                _vp, ctypes.c_size_t, _vp]
_lib.sage_quant_qkv.restype = ctypes.c_int
_lib.sage_fp8_quant_rows.argtypes = [_vp, ctypes.c_int, ctypes.c_int, ctypes.c_int64, _vp, _vp, _vp]
_lib.sage_fp8_quant_rows.restype = ctypes.c_int
_lib.sage_fp8_linear.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, ctypes.c_int,
                                 _vp]
_lib.sage_fp8_linear.restype = ctypes.c_int
_lib.sage_quant_v.argtypes = [_vp, SageShape, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.sage_quant_v.restype = ctypes.c_int
_lib.sage_attn_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, SageShape, ctypes.c_float, _vp, ctypes.c_int,
                               _vp, _vp]
_lib.sage_attn_fwd.restype = ctypes.c_int
_lib.sage_attn_fwd_p_codes.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, SageShape, ctypes.c_float, _vp,
                                       ctypes.c_int, _vp, _vp, _vp]
_lib.sage_attn_fwd_p_codes.restype = ctypes.c_int
_lib.sage_rope_plan_init.argtypes = [ctypes.POINTER(SageRopePlan), ctypes.c_int, ctypes.c_int, ctypes.c_double,
                                     ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double,
                                     ctypes.c_char_p]
_lib.sage_rope_plan_init.restype = ctypes.c_int
_lib.sage_rope.argtypes = [SageRows, SageRows, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp,
                           ctypes.POINTER(SageRopePlan), ctypes.c_int, _vp]
_lib.sage_rope.restype = ctypes.c_int
_lib.sage_kv_write.argtypes = [_vp, _vp, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, _vp,
                               SageKvCache, _vp]
_lib.sage_kv_write.restype = ctypes.c_int
_lib.sage_kv_read.argtypes = [SageKvCache, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                              _vp]
_lib.sage_kv_read.restype = ctypes.c_int
_lib.sage_attn_prompt.argtypes = [_vp, _vp, _vp, ctypes.POINTER(SagePrompt), _vp, _vp, _vp]
_lib.sage_attn_prompt.restype = ctypes.c_int
_lib.sage_attn_token_workspace_bytes.argtypes = [ctypes.c_int] * 5
_lib.sage_attn_token_workspace_bytes.restype = ctypes.c_size_t
_lib.sage_attn_token.argtypes = [_vp, ctypes.POINTER(SageToken), SageKvCache, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.sage_attn_token.restype = ctypes.c_int
_lib.sage_check.argtypes = [_vp]
_lib.sage_check.restype = ctypes.c_int
_lib.sage_set_wait_timeout_ns.argtypes = [ctypes.c_int64]
_lib.sage_set_wait_timeout_ns.restype = None
_lib.sage_selftest_wait_timeout.argtypes = [ctypes.c_int64, _vp]
_lib.sage_selftest_wait_timeout.restype = ctypes.c_int
_lib.sage_last_error.argtypes = []
_lib.sage_last_error.restype = ctypes.c_char_p


class SageError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.sage_last_error().decode(errors="replace")
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")


def _ok(status: int, where: str) -> None:
    if status != SAGE_OK:
        raise SageError(status, where)


def make_shape(B, N, H, D, tok_stride=0, cu_seqlens=None, q_gran="block64", k_gran="block64") -> SageShape:
    """q_gran / k_gran: a GRAN name (or its integer code) for the Q / K scale groups."""
    s = SageShape(B, N, H, D, int(tok_stride), None, 0, GRAN.get(q_gran, q_gran), GRAN.get(k_gran, k_gran))
    if cu_seqlens is not None:
        arr = (ctypes.c_int32 * len(cu_seqlens))(*[int(x) for x in cu_seqlens])
        s.cu_seqlens = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
        s.n_seg = len(cu_seqlens) - 1
        s._keep = arr  # keep the host array alive with the struct
    return s


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def npad(N: int) -> int:
    return int(_lib.sage_npad(int(N)))


def scale_shape(B: int, H: int, N: int, gran="block64") -> tuple:
    """Shape of a Q or K scale array: one per 64-token block, else one per token."""
    Np = npad(N)
    return (B, H, Np // 64) if GRAN.get(gran, gran) == GRAN["block64"] else (B, H, Np)


def workspace_bytes(shape: SageShape) -> int:
    return int(_lib.sage_workspace_bytes(shape))


def sage_quant_qk(q, k, shape, q_codes, q_scale, k_codes, k_scale, k_mean, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    _ok(_lib.sage_quant_qk(_ptr(q), _ptr(k), shape, _ptr(q_codes), _ptr(q_scale), _ptr(k_codes), _ptr(k_scale),
                           _ptr(k_mean), _ptr(workspace), ws_bytes, _stream(stream)), "sage_quant_qk")


def sage_quant_qk_static(q, k, shape, q_codes, q_scale, k_codes, k_scale, k_mean, stream=None):
    """sage_quant_qk without a workspace: for callers that cannot allocate
    device memory.  Scratch lives in a fixed 8 MiB array inside the library;
    larger shapes raise SageError (SAGE_ERR_WORKSPACE).  Calls that overlap on
    the GPU share that array and race."""
    _ok(_lib.sage_quant_qk_static(_ptr(q), _ptr(k), shape, _ptr(q_codes), _ptr(q_scale), _ptr(k_codes),
                                  _ptr(k_scale), _ptr(k_mean), _stream(stream)), "sage_quant_qk_static")


def sage_quant_qk_normrope(q, k, shape, q_weight, k_weight, rope_cos, rope_sin, eps, q_codes, q_scale, k_codes,
                           k_scale, k_mean, workspace, stream=None):
    """sage_quant_qk on projection outputs: QK RMSNorm (BF16 weights [D], eps)
    and RoPE (float32 cos / sin tables [N, D/2]) applied in the same kernels."""
    nr = SageNormRope(_ptr(q_weight), _ptr(k_weight), _ptr(rope_cos), _ptr(rope_sin), float(eps))
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    _ok(_lib.sage_quant_qk_normrope(_ptr(q), _ptr(k), shape, ctypes.byref(nr), _ptr(q_codes), _ptr(q_scale),
                                    _ptr(k_codes), _ptr(k_scale), _ptr(k_mean), _ptr(workspace), ws_bytes,
                                    _stream(stream)),
        "sage_quant_qk_normrope")


def sage_quant_qkv(q, k, v, shape, v_tok_stride, q_codes, q_scale, k_codes, k_scale, k_mean, v_codes_t, v_scale,
                   v_mean, workspace, stream=None):
    """sage_quant_qk and sage_quant_v in four launches (identical outputs); v may
    have its own token stride (0 means H*D)."""
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    _ok(_lib.sage_quant_qkv(_ptr(q), _ptr(k), _ptr(v), shape, int(v_tok_stride), _ptr(q_codes), _ptr(q_scale),
                            _ptr(k_codes), _ptr(k_scale), _ptr(k_mean), _ptr(v_codes_t), _ptr(v_scale), _ptr(v_mean),
                            _ptr(workspace), ws_bytes, _stream(stream)), "sage_quant_qkv")


def sage_fp8_quant_rows(x, codes, scale, stream=None):
    """Per-row E4M3 codes [R, K] (uint8) and scales [R] (float32) of a BF16 [R, K]
    tensor whose rows may be strided (x.stride(1) must be 1)."""
    R, K = x.shape
    assert x.stride(1) == 1
    _ok(_lib.sage_fp8_quant_rows(_ptr(x), R, K, x.stride(0), _ptr(codes), _ptr(scale), _stream(stream)),
        "sage_fp8_quant_rows")


def sage_fp8_linear(xq, sx, wq, sw, out, stream=None):
    """out [M, N] (BF16 or float32) = row-wise FP8 product of xq [M, K] and wq [N, K]."""
    M, K = xq.shape
    N = wq.shape[0]
    _ok(_lib.sage_fp8_linear(_ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), M, N, K, _ptr(out),
                             1 if out.dtype == torch.float32 else 0, _stream(stream)), "sage_fp8_linear")


def sage_quant_v(v, shape, v_codes_t, v_scale, v_mean, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    _ok(_lib.sage_quant_v(_ptr(v), shape, _ptr(v_codes_t), _ptr(v_scale), _ptr(v_mean), _ptr(workspace),
                          ws_bytes, _stream(stream)), "sage_quant_v")


def sage_attn_fwd(q_codes, q_scale, k_codes, k_scale, v_codes_t, v_scale, v_mean, shape, sm_scale, out,
                  out_fp32, lse=None, stream=None):
    _ok(_lib.sage_attn_fwd(_ptr(q_codes), _ptr(q_scale), _ptr(k_codes), _ptr(k_scale), _ptr(v_codes_t),
                           _ptr(v_scale), _ptr(v_mean), shape, float(sm_scale), _ptr(out), int(bool(out_fp32)),
                           _ptr(lse), _stream(stream)), "sage_attn_fwd")


def sage_attn_fwd_p_codes(q_codes, q_scale, k_codes, k_scale, v_codes_t, v_scale, v_mean, shape, sm_scale, out,
                          out_fp32, p_codes, lse=None, stream=None):
    """sage_attn_fwd plus the E4M3 codes of P in p_codes (uint8 [B*H, N, npad(N)]); a diagnostic."""
    _ok(_lib.sage_attn_fwd_p_codes(_ptr(q_codes), _ptr(q_scale), _ptr(k_codes), _ptr(k_scale), _ptr(v_codes_t),
                                   _ptr(v_scale), _ptr(v_mean), shape, float(sm_scale), _ptr(out),
                                   int(bool(out_fp32)), _ptr(lse), _ptr(p_codes), _stream(stream)),
        "sage_attn_fwd_p_codes")


def sage_check(stream=None) -> None:
    _ok(_lib.sage_check(_stream(stream)), "sage_check")


def sage_check_status(stream=None) -> int:
    return int(_lib.sage_check(_stream(stream)))


def set_wait_timeout_ns(ns: int) -> None:
    _lib.sage_set_wait_timeout_ns(int(ns))


def selftest_wait_timeout(timeout_ns: int, stream=None) -> None:
    _ok(_lib.sage_selftest_wait_timeout(int(timeout_ns), _stream(stream)), "sage_selftest_wait_timeout")


# ------------------------------------------------------------------ serving calls
class RopePlan:
    """Rotation per position of every channel pair (sage_rope_plan).

    rot_dim channels of each head turn; interleaved pairs (2i, 2i+1), else halves (i, i + rot_dim/2).
    scaling: None, "linear", "ntk" or "yarn" for a context `factor` times longer than orig_len.  axis: position
    axis of each pair (positions are then [axes, T]).  inv_freq: radians per position of each pair, in place of
    base and scaling; mscale: factor on cos and sin, in place of the scaling's."""

    def __init__(self, rot_dim, base=10000.0, interleaved=False, scaling=None, factor=1.0, orig_len=0, beta_fast=32.0,
                 beta_slow=1.0, axis=None, inv_freq=None, mscale=None):
        self.struct = SageRopePlan()
        if axis is not None and len(axis) != rot_dim // 2:
            raise ValueError(f"axis must name {rot_dim // 2} pairs (got {len(axis)})")
        if scaling not in ROPE_SCALING:
            raise ValueError(f"scaling must be one of {list(ROPE_SCALING)} (got {scaling!r})")
        _ok(_lib.sage_rope_plan_init(ctypes.byref(self.struct), rot_dim, int(bool(interleaved)), float(base),
                                     ROPE_SCALING[scaling], float(factor), int(orig_len), float(beta_fast),
                                     float(beta_slow), None if axis is None else bytes(int(a) for a in axis)),
            "sage_rope_plan_init")
        if inv_freq is not None:
            if len(inv_freq) != rot_dim // 2:
                raise ValueError(f"inv_freq must hold {rot_dim // 2} values (got {len(inv_freq)})")
            for i, f in enumerate(inv_freq):
                self.struct.turns[i] = float(f) / 6.283185307179586
        if mscale is not None:
            self.struct.mscale = float(mscale)

    # Asked for at each call: a copied or unpickled plan has a struct of its own.
    address = property(lambda self: ctypes.addressof(self.struct))
    n_axes = property(lambda self: self.struct.n_axes)
    rot_dim = property(lambda self: self.struct.rot_dim)


def sage_rope(q, k, positions, plan, q_out=None, k_out=None, transpose=False, stream=None):
    """Rotary positions of q [T, Hq, D] and k [T, Hk, D] (either may be None) in one launch.  positions: int64 [T], or
    [axes, T].  In place without q_out / k_out.  transpose: the gradient of the rotation.  Returns (q_out, k_out)."""
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    status = _serve_ext.rope(q, k, positions, plan.address, q_out, k_out, transpose, stream)
    if status:
        raise SageError(status, "sage_rope")
    return q_out, k_out


# The cache of the calls below: codes [pages, Hk, page_size, D] (int8, or float8_e4m3fn / uint8 for E4M3) and float32
# scales [pages, Hk, page_size], of K and of V.
def sage_kv_write(k, v, slots, k_codes, k_scale, v_codes, v_scale, stream=None):
    """Quantizes the rows of k, v [T, Hk, D] into the cache slots (int64 [T]; page * page_size + offset; a negative
    slot's row is not written)."""
    status = _serve_ext.kv_write(k, v, slots, k_codes, k_scale, v_codes, v_scale, stream)
    if status:
        raise SageError(status, "sage_kv_write")


def sage_kv_read(slots, k_codes, k_scale, v_codes, v_scale, k, v, stream=None):
    """Dequantizes the cache slots (int64 [T]) into k, v [T, Hk, D]; rows of negative slots keep their contents."""
    status = _serve_ext.kv_read(k, v, slots, k_codes, k_scale, v_codes, v_scale, stream)
    if status:
        raise SageError(status, "sage_kv_read")
    return k, v


def sage_attn_prompt(q, k, v, cu_q, cu_k=None, out=None, lse=None, causal=True, sm_scale=0.0, stream=None):
    """Attention over packed sequences: q [Tq, Hq, D], k, v [Tk, Hk, D] BF16 or FP16; cu_q, cu_k host offsets, a list or a
    CPU tensor (cu_k None: cu_q).  causal: query i of a sequence sees keys j <= i + Lk - Lq.  lse: float32 [Hq, Tq] or
    None.  Returns out; without one given it is allocated on the stream of the call."""
    if out is None:
        if stream is None or not q.is_cuda:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            # the memory belongs to the stream that writes it: allocated for the current one, it could be in use there
            # still, or again, while the given one writes
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device=q.device)
            with torch.cuda.stream(stream):
                out = torch.empty_like(q, memory_format=torch.contiguous_format)
    status = _serve_ext.attn_prompt(q, k, v, cu_q, cu_k, out, lse, causal, sm_scale, stream)
    if status:
        raise SageError(status, "sage_attn_prompt")
    return out


def attn_token_workspace_bytes(B, Hq, Hk, D, max_len) -> int:
    return int(_lib.sage_attn_token_workspace_bytes(int(B), int(Hq), int(Hk), int(D), int(max_len)))


def sage_attn_token(q, k_codes, k_scale, v_codes, v_scale, page_table, lens, out, workspace, max_len=None, lse=None,
                    sm_scale=0.0, stream=None):
    """Attention of one token per sequence, q [B, Hq, D] BF16 or FP16, over the cache: page_table int32 [B, pages],
    lens int32 [B] (keys seen).  max_len: upper bound on lens (None: what the table can name).  workspace: at least
    attn_token_workspace_bytes(...) bytes, kept by the caller.  lse: float32 [B, Hq] or None.  Returns out."""
    status = _serve_ext.attn_token(q, k_codes, k_scale, v_codes, v_scale, page_table, lens, out, workspace, max_len, lse,
                                   sm_scale, stream)
    if status:
        raise SageError(status, "sage_attn_token")
    return out


class KVCache:
    """A quantized paged KV cache: int8 or E4M3 codes and a float32 scale per token and KV head."""

    def __init__(self, num_pages, page_size, Hk, D, fmt="int8", device="cuda"):
        dt = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}.get(fmt)
        if dt is None:
            raise ValueError(f"fmt must be 'int8' or 'e4m3' (got {fmt!r})")
        self.num_pages, self.page_size, self.Hk, self.D, self.fmt = num_pages, page_size, Hk, D, fmt
        codes, scales = (num_pages, Hk, page_size, D), (num_pages, Hk, page_size)
        self.k_codes = torch.zeros(codes, dtype=torch.uint8, device=device).view(dt)
        self.v_codes = torch.zeros(codes, dtype=torch.uint8, device=device).view(dt)
        self.k_scale = torch.zeros(scales, dtype=torch.float32, device=device)
        self.v_scale = torch.zeros(scales, dtype=torch.float32, device=device)

    @property
    def tensors(self):
        return self.k_codes, self.k_scale, self.v_codes, self.v_scale

    def write(self, k, v, slots, stream=None):
        sage_kv_write(k, v, slots, *self.tensors, stream=stream)

    def read(self, slots, k, v, stream=None):
        return sage_kv_read(slots, *self.tensors, k, v, stream=stream)

    def attend(self, q, page_table, lens, out, workspace, max_len=None, lse=None, sm_scale=0.0, stream=None):
        return sage_attn_token(q, *self.tensors, page_table, lens, out, workspace, max_len, lse, sm_scale, stream)


class Buffers:
    """Device buffers of one shape for the whole path (torch allocates them)."""

    def __init__(self, B, N, H, D, device="cuda", out_fp32=False, with_lse=False, tok_stride=0,
                 cu_seqlens=None, q_gran="block64", k_gran="block64"):
        self.shape = make_shape(B, N, H, D, tok_stride, cu_seqlens, q_gran, k_gran)
        self.B, self.N, self.H, self.D = B, N, H, D
        Np = npad(N)
        self.Npad = Np
        dev = torch.device(device)
        self.q_codes = torch.empty((B, H, Np, D), dtype=torch.int8, device=dev)
        self.k_codes = torch.empty((B, H, Np, D), dtype=torch.int8, device=dev)
        self.q_scale = torch.empty(scale_shape(B, H, N, q_gran), dtype=torch.float32, device=dev)
        self.k_scale = torch.empty(scale_shape(B, H, N, k_gran), dtype=torch.float32, device=dev)
        self.k_mean = torch.empty((B, H, D), dtype=torch.bfloat16, device=dev)
        self.v_codes_t = torch.empty((B, H, D, Np), dtype=torch.uint8, device=dev)
        self.v_scale = torch.empty((B, H, D), dtype=torch.float32, device=dev)
        self.v_mean = torch.empty((B, H, D), dtype=torch.float32, device=dev)
        self.out = torch.empty((B, N, H, D), dtype=torch.float32 if out_fp32 else torch.bfloat16, device=dev)
        self.out_fp32 = out_fp32
        self.lse = torch.empty((B, H, N), dtype=torch.float32, device=dev) if with_lse else None
        self.workspace = torch.empty(max(256, workspace_bytes(self.shape)), dtype=torch.uint8, device=dev)

    def run(self, q, k, v, sm_scale=0.0, stream=None, v_shape=None, normrope=None):
        """quant_qkv -> attn_fwd; q, k, v are BF16 [B, N, H, D] device tensors
        (v may be a token-strided view; pass v_shape with its tok_stride).  normrope:
        None, or dict(q_w, k_w, cos, sin, eps) of device tensors (and a float): Q and K
        are then projection outputs, normed and rotated inside the quantization."""
        if normrope is None:
            sage_quant_qkv(q, k, v, self.shape, (v_shape or self.shape).tok_stride, self.q_codes, self.q_scale,
                           self.k_codes, self.k_scale, self.k_mean, self.v_codes_t, self.v_scale, self.v_mean,
                           self.workspace, stream)
        else:
            nr = normrope
            sage_quant_qk_normrope(q, k, self.shape, nr["q_w"], nr["k_w"], nr["cos"], nr["sin"], nr["eps"],
                                   self.q_codes, self.q_scale, self.k_codes, self.k_scale, self.k_mean,
                                   self.workspace, stream)
            sage_quant_v(v, v_shape or self.shape, self.v_codes_t, self.v_scale, self.v_mean, self.workspace,
                         stream)
        sage_attn_fwd(self.q_codes, self.q_scale, self.k_codes, self.k_scale, self.v_codes_t, self.v_scale,
                      self.v_mean, self.shape, sm_scale, self.out, self.out_fp32, self.lse, stream)
        return self.out

    def capture(self, q, k, v, sm_scale=0.0, v_shape=None, normrope=None):
        """The launches of run() on these tensors, captured once into a CUDA
        graph; graph.replay() then re-runs them on whatever q, k, v hold, with
        less launch overhead between the kernels.  The calls run once eagerly
        first (on a side stream) so that every one-time setup happens outside
        the capture."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.run(q, k, v, sm_scale, side, v_shape, normrope)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            self.run(q, k, v, sm_scale, side, v_shape, normrope)
        return graph
