"""The norms around a block (include/gdn.h, gdn_gated_norm_* and gdn_residual_norm_*): the
gated norm of a mixer's output, and the step from one block to the next.

Argument marshalling only, by the rules of _layers: x, z and the residual may be slices of a
wider tensor, everything else is contiguous; work is enqueued on `stream`, by default torch's
current stream of the tensors' GPU.
"""
import ctypes

from ._binding import _dtype_code
from ._layers import _call, _fit, _lib, _like, _need, _on, _p, _place, _row_stride, _torch, _workspace


class GatedNormParams(ctypes.Structure):
    """gdn_gated_norm_params_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "H", "D", "dtype", "gate_first")] + [
        ("eps", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("x_stride", "z_stride")]


class ResidualNormParams(ctypes.Structure):
    """gdn_residual_norm_params_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "dtype", "residual_dtype")] + [
        ("eps", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("x_stride", "residual_stride")]


def declare(lib):
    """Argument types of the entry points (called once by load_library)."""
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    G, R = ctypes.POINTER(GatedNormParams), ctypes.POINTER(ResidualNormParams)

    def fn(name, restype, *argtypes):
        f = getattr(lib, name)
        f.restype, f.argtypes = restype, list(argtypes)

    fn("gdn_gated_norm_fwd", ctypes.c_int, G, *[vp] * 5)
    fn("gdn_gated_norm_bwd_workspace_size", sz, G)
    fn("gdn_gated_norm_bwd", ctypes.c_int, G, *[vp] * 8, sz, vp)
    fn("gdn_residual_norm_fwd", ctypes.c_int, R, *[vp] * 8)
    fn("gdn_residual_norm_bwd_workspace_size", sz, R)
    fn("gdn_residual_norm_bwd", ctypes.c_int, R, *[vp] * 13, sz, vp)


def _eps(eps):
    if not eps >= 0:
        raise ValueError("eps must be at least 0, got %r" % (eps,))
    return eps


# ---------------------------------------------------------------------------
# gated norm

def _gated_sizes(x, weight, z, eps, gate_first):
    if x.dim() not in (3, 4):
        raise ValueError("x must be [B, T, H, D] or [B, T, D]")
    B, T, D = x.shape[0], x.shape[1], x.shape[-1]
    _fit((("weight", weight, (D,), _torch().float32), ("z", z, x.shape, x.dtype)))
    p = GatedNormParams(B, T, x.shape[2] if x.dim() == 4 else 1, D, _dtype_code(x.dtype), bool(gate_first), _eps(eps),
                        _row_stride("x", x), 0 if z is None else _row_stride("z", z))
    return ctypes.byref(p)


def gated_norm_fwd(x, weight, z=None, eps=1e-6, gate_first=False, stream=None):
    """Gated RMS norm of a mixer's output through gdn_gated_norm_fwd: x [B,T,H,D] (or
    [B,T,D]) in bf16 or fp32, normed over D, weight [D] fp32, z like x or None.  Returns
    y = r(x) weight silu(z), contiguous; gate_first: r(x silu(z)) weight."""
    p = _gated_sizes(x, weight, z, eps, gate_first)
    index = _place(x, (("z", z),), (("weight", weight),))

    def body(s):
        y = _like(x)
        _lib()
        _call("gdn_gated_norm_fwd", p, x.data_ptr(), weight.data_ptr(), _p(z), y.data_ptr(), s)
        return y
    return _on(index, stream, (x, weight, z), body)


def gated_norm_bwd(x, weight, d_y, z=None, eps=1e-6, gate_first=False, stream=None):
    """Gradients of gated_norm_fwd through gdn_gated_norm_bwd: dict of dx (and dz with z)
    in x's dtype and dweight [D] fp32."""
    p = _gated_sizes(x, weight, z, eps, gate_first)
    _need("d_y", d_y)
    _fit((("d_y", d_y, x.shape, x.dtype),))
    index = _place(x, (("z", z),), (("weight", weight), ("d_y", d_y)))
    ws_bytes = _lib().gdn_gated_norm_bwd_workspace_size(p)

    def body(s):
        g = dict(dx=_like(x), dweight=_like(weight))
        if z is not None:
            g["dz"] = _like(x)
        ws, ws_ptr, ws_size = _workspace(ws_bytes, index)
        _call("gdn_gated_norm_bwd", p, x.data_ptr(), weight.data_ptr(), _p(z), d_y.data_ptr(), g["dx"].data_ptr(),
              _p(g.get("dz")), g["dweight"].data_ptr(), ws_ptr, ws_size, s)
        return g
    return _on(index, stream, (x, weight, z, d_y), body)


# ---------------------------------------------------------------------------
# residual norm

def _residual_sizes(x, residual, weight, post_weight, scale, eps):
    f32 = _torch().float32
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    B, T, C = x.shape
    code = _dtype_code(x.dtype)
    _need("residual", residual)
    _fit((("residual", residual, x.shape, f32 if residual.dtype is f32 else x.dtype), ("weight", weight, (C,), f32),
          ("post_weight", post_weight, (C,), f32), ("scale", scale, (C,), f32)))
    p = ResidualNormParams(B, T, C, code, _dtype_code(residual.dtype), _eps(eps), _row_stride("x", x),
                           _row_stride("residual", residual))
    return ctypes.byref(p)


def residual_norm_fwd(x, residual, weight, post_weight=None, scale=None, eps=1e-6, stream=None):
    """From one block to the next through gdn_residual_norm_fwd: x [B,T,C] (bf16 or fp32),
    the block's output; residual [B,T,C] in x's dtype or fp32; weight, post_weight and scale
    [C] fp32, the latter two or None.  Returns (h, new_residual): new_residual = residual +
    scale r(x) post_weight (x itself without post_weight) in the residual's dtype, and
    h = r(new_residual) weight in x's, of new_residual as it was before it was rounded."""
    p = _residual_sizes(x, residual, weight, post_weight, scale, eps)
    index = _place(x, (("residual", residual),), (("weight", weight), ("post_weight", post_weight), ("scale", scale)))

    def body(s):
        h, new = _like(x), _like(residual)
        _lib()
        _call("gdn_residual_norm_fwd", p, x.data_ptr(), residual.data_ptr(), weight.data_ptr(), _p(post_weight),
              _p(scale), h.data_ptr(), new.data_ptr(), s)
        return h, new
    return _on(index, stream, (x, residual, weight, post_weight, scale), body)


def residual_norm_bwd(x, residual, weight, d_h, d_new_residual=None, post_weight=None, scale=None, eps=1e-6,
                      stream=None):
    """Gradients of residual_norm_fwd through gdn_residual_norm_bwd: dict of dx in x's
    dtype, dresidual in the residual's, and dweight, dpost_weight, dscale [C] fp32 (the
    latter two with their inputs)."""
    p = _residual_sizes(x, residual, weight, post_weight, scale, eps)
    _need("d_h", d_h)
    _fit((("d_h", d_h, x.shape, x.dtype), ("d_new_residual", d_new_residual, x.shape, residual.dtype)))
    index = _place(x, (("residual", residual),),
                   (("weight", weight), ("post_weight", post_weight), ("scale", scale), ("d_h", d_h),
                    ("d_new_residual", d_new_residual)))
    ws_bytes = _lib().gdn_residual_norm_bwd_workspace_size(p)

    def body(s):
        g = dict(dx=_like(x), dresidual=_like(residual), dweight=_like(weight))
        if post_weight is not None:
            g["dpost_weight"] = _like(weight)
        if scale is not None:
            g["dscale"] = _like(weight)
        ws, ws_ptr, ws_size = _workspace(ws_bytes, index)
        _call("gdn_residual_norm_bwd", p, x.data_ptr(), residual.data_ptr(), weight.data_ptr(), _p(post_weight),
              _p(scale), d_h.data_ptr(), _p(d_new_residual), g["dx"].data_ptr(), g["dresidual"].data_ptr(),
              g["dweight"].data_ptr(), _p(g.get("dpost_weight")), _p(g.get("dscale")), ws_ptr, ws_size, s)
        return g
    return _on(index, stream, (x, residual, weight, post_weight, scale, d_h, d_new_residual), body)


# ---------------------------------------------------------------------------
# differentiable forms

_FUNCTIONS = {}


def _gated_function():
    """torch.autograd.Function behind gated_norm (defined on first use, since torch is
    imported lazily)."""
    if "gated" not in _FUNCTIONS:
        torch = _torch()

        class GatedNorm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, weight, z, eps, gate_first):
                ctx.save_for_backward(x, weight, z)
                ctx.eps, ctx.gate_first = eps, gate_first
                return gated_norm_fwd(x, weight, z, eps, gate_first)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, d_y):
                x, weight, z = ctx.saved_tensors
                g = gated_norm_bwd(x, weight, d_y.to(x.dtype).contiguous(), z, ctx.eps, ctx.gate_first)
                return g["dx"], g["dweight"], g.get("dz"), None, None

        _FUNCTIONS["gated"] = GatedNorm
    return _FUNCTIONS["gated"]


def gated_norm(x, weight, z=None, eps=1e-6, gate_first=False):
    """gated_norm_fwd() as a differentiable torch op: gradients reach x, weight and z."""
    return _gated_function().apply(x, weight, z, eps, gate_first)


def _residual_function():
    if "residual" not in _FUNCTIONS:
        torch = _torch()

        class ResidualNorm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, residual, weight, post_weight, scale, eps):
                ctx.set_materialize_grads(False)
                ctx.save_for_backward(x, residual, weight, post_weight, scale)
                ctx.eps = eps
                return residual_norm_fwd(x, residual, weight, post_weight, scale, eps)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, d_h, d_new):
                x, residual, weight, post, scale = ctx.saved_tensors
                d_h = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if d_h is None else d_h.to(x.dtype).contiguous()
                d_new = None if d_new is None else d_new.to(residual.dtype).contiguous()
                g = residual_norm_bwd(x, residual, weight, d_h, d_new, post, scale, ctx.eps)
                return g["dx"], g["dresidual"], g["dweight"], g.get("dpost_weight"), g.get("dscale"), None

        _FUNCTIONS["residual"] = ResidualNorm
    return _FUNCTIONS["residual"]


def residual_norm(x, residual, weight, post_weight=None, scale=None, eps=1e-6):
    """residual_norm_fwd() as a differentiable torch op: returns (h, new_residual); gradients
    reach x, residual, weight, post_weight and scale."""
    return _residual_function().apply(x, residual, weight, post_weight, scale, eps)
