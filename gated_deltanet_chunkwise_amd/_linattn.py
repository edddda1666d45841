"""Linear attention with a decay for each head (include/gdn.h, gdn_linattn_*): prompt,
backward and single-token forms, and the differentiable op.

Argument marshalling only, by the rules of _layers: q, k and v may be slices of a wider
tensor, everything else is contiguous; work is enqueued on `stream`, by default torch's
current stream of the tensors' GPU.
"""
import ctypes

from . import _layers
from ._binding import _dtype_code, _gradient
from ._layers import GDN_ZERO_REST, _call, _fit, _lib, _like, _need, _on, _p, _place, _row_stride, _sequences, _torch, _workspace, _written


class LinattnParams(ctypes.Structure):
    """gdn_linattn_params_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "H", "HV", "K", "V", "num_seqs", "dtype")] + [
        ("scale", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")]


def declare(lib):
    """Argument types of the entry points (called once by load_library)."""
    vp, sz, P = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(LinattnParams)

    def fn(name, restype, *argtypes):
        f = getattr(lib, name)
        f.restype, f.argtypes = restype, list(argtypes)

    fn("gdn_linattn_fwd_workspace_size", sz, P, ctypes.c_int)
    fn("gdn_linattn_fwd", ctypes.c_int, P, *[vp] * 9, sz, vp)
    fn("gdn_linattn_bwd_workspace_size", sz, P, ctypes.c_int)
    fn("gdn_linattn_bwd", ctypes.c_int, P, *[vp] * 13, sz, vp)
    fn("gdn_linattn_decode", ctypes.c_int, P, *[vp] * 8)


def _sizes(q, k, v, log_decay, cu_seqlens, scale):
    """(params, B, T, HV, K, V, sequences)"""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B, T, H, K] and v [B, T, HV, V]")
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    dtype = q.dtype
    _fit((("k", k, q.shape, dtype), ("v", v, (B, T, HV, V), dtype), ("log_decay", log_decay, (HV,), _torch().float32)))
    N = _sequences(cu_seqlens, B)
    code = _dtype_code(dtype)
    p = LinattnParams(B, T, H, HV, K, V, *((0, code) if cu_seqlens is None else (N, code | GDN_ZERO_REST)), scale,
                      _row_stride("q", q), _row_stride("k", k), _row_stride("v", v))
    return ctypes.byref(p), B, T, HV, K, V, N


def linear_attn_fwd(q, k, v, log_decay, cu_seqlens=None, initial_state=None, scale=1.0, output_final_state=True,
                    stream=None):
    """Linear attention with a decay for each head through gdn_linattn_fwd: q, k [B,T,H,K]
    and v [B,T,HV,V] in bf16 or fp32 (K, V 64 or 128; value head hv reads key head
    hv / (HV/H)), log_decay [HV] fp32 (a = exp(log_decay), a constant), initial_state
    [sequences,HV,K,V] fp32 or None.  Returns (o [B,T,HV,V], final_state
    [sequences,HV,K,V] fp32 or None); rows of o behind the last sequence (where cu_seqlens
    end before T) are 0."""
    f32 = _torch().float32
    p, B, T, HV, K, V, N = _sizes(q, k, v, log_decay, cu_seqlens, scale)
    _fit((("initial_state", initial_state, (N, HV, K, V), f32),))
    index = _place(q, (("k", k), ("v", v)),
                   (("log_decay", log_decay), ("cu_seqlens", cu_seqlens), ("initial_state", initial_state)))
    ws_bytes = _lib().gdn_linattn_fwd_workspace_size(p, int(cu_seqlens is not None))

    def body(s):
        o = _like(v)
        fin = _torch().empty((N, HV, K, V), dtype=f32, device=q.device) if output_final_state else None
        ws, ws_ptr, ws_size = _workspace(ws_bytes, index)
        _call("gdn_linattn_fwd", p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _p(cu_seqlens),
              _p(initial_state), o.data_ptr(), _p(fin), ws_ptr, ws_size, s)
        return o, fin
    return _on(index, stream, (q, k, v, log_decay, cu_seqlens, initial_state), body)


def linear_attn_bwd(q, k, v, log_decay, d_o, d_final_state=None, cu_seqlens=None, initial_state=None, scale=1.0,
                    stream=None):
    """Gradients of linear_attn_fwd through gdn_linattn_bwd: dict of dq, dk [B,T,H,K] and
    dv [B,T,HV,V] in q's dtype and dh0 [sequences,HV,K,V] fp32."""
    f32 = _torch().float32
    p, B, T, HV, K, V, N = _sizes(q, k, v, log_decay, cu_seqlens, scale)
    _need("d_o", d_o)
    states = (N, HV, K, V)
    _fit((("d_o", d_o, v.shape, q.dtype), ("d_final_state", d_final_state, states, f32),
          ("initial_state", initial_state, states, f32)))
    index = _place(q, (("k", k), ("v", v)),
                   (("log_decay", log_decay), ("cu_seqlens", cu_seqlens), ("initial_state", initial_state),
                    ("d_o", d_o), ("d_final_state", d_final_state)))
    ws_bytes = _lib().gdn_linattn_bwd_workspace_size(p, int(cu_seqlens is not None))

    def body(s):
        g = dict(dq=_like(q), dk=_like(k), dv=_like(v),
                 dh0=_torch().empty(states, dtype=f32, device=q.device))
        ws, ws_ptr, ws_size = _workspace(ws_bytes, index)
        _call("gdn_linattn_bwd", p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _p(cu_seqlens),
              _p(initial_state), d_o.data_ptr(), _p(d_final_state), g["dq"].data_ptr(), g["dk"].data_ptr(),
              g["dv"].data_ptr(), g["dh0"].data_ptr(), ws_ptr, ws_size, s)
        return g
    return _on(index, stream, (q, k, v, log_decay, cu_seqlens, initial_state, d_o, d_final_state), body)


def _decode_args(q, k, v, log_decay, state, scale, new_state, out):
    f32 = _torch().float32
    p, B, T, HV, K, V, _ = _sizes(q, k, v, log_decay, None, scale)
    _need("state", state)
    shape = (B, HV, K, V)
    _fit((("state", state, shape, f32), ("new_state", new_state, shape, f32), ("out", out, v.shape, q.dtype)))
    index = _place(q, (("k", k), ("v", v)),
                   (("log_decay", log_decay), ("state", state), ("new_state", new_state), ("out", out)))

    def args(s):
        o = _like(v) if out is None else out
        new = state if new_state is None else new_state
        _lib()
        return ((p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state.data_ptr(), new.data_ptr(),
                 o.data_ptr(), s), o, (new,) if out is None else (new, out))
    return index, args


def linear_attn_decode_launcher(q, k, v, log_decay, state, scale=1.0, new_state=None, out=None, stream=None):
    """Check and marshal gdn_linattn_decode's arguments once; returns (launch, o), where
    launch() enqueues the T tokens of q, k and v after `state` [B,HV,K,V], writing the state
    after them to new_state (default: `state` itself).  The stream is as for
    conv_decode_launcher."""
    index, args = _decode_args(q, k, v, log_decay, state, scale, new_state, out)
    keep = (q, k, v, log_decay, state, new_state, out, stream)
    args, o, written = _on(index, stream, keep[:-1], args)
    return _layers._launcher("gdn_linattn_decode", index, args, keep + (o,), written), o


def linear_attn_decode(q, k, v, log_decay, state, scale=1.0, new_state=None, out=None, stream=None):
    """T tokens (1: a decode step) of each of B sequences through gdn_linattn_decode: returns
    o [B,T,HV,V]; the state after them goes to new_state, or updates `state` in place."""
    index, args = _decode_args(q, k, v, log_decay, state, scale, new_state, out)

    def body(s):
        a, o, written = args(s)
        _call("gdn_linattn_decode", *a)
        _written(written)
        return o
    return _on(index, stream, (q, k, v, log_decay, state, new_state, out), body)


_FUNCTION = None


def _function():
    """torch.autograd.Function behind linear_attention (defined on first use, since torch is
    imported lazily)."""
    global _FUNCTION
    if _FUNCTION is None:
        torch = _torch()

        class LinearAttention(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, log_decay, cu_seqlens, initial_state, scale, bits):
                ctx.set_materialize_grads(False)
                o, fin = linear_attn_fwd(q, k, v, log_decay, cu_seqlens, initial_state, scale)
                pairs = [_layers.keep(t, bits)[0] for t in (q, k, v)]
                ctx.save_for_backward(*(t for pair in pairs for t in pair), log_decay, cu_seqlens, initial_state)
                ctx.scale, ctx.dtype = scale, q.dtype
                return o, fin

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, d_o, d_fin):
                qd, qs, kd, ks, vd, vs, log_decay, cu, h0 = ctx.saved_tensors
                q, k, v = (t if sc is None else _layers.unpack8(_layers.Packed8(t, sc, ctx.dtype))
                           for t, sc in ((qd, qs), (kd, ks), (vd, vs)))
                d_o = torch.zeros(v.shape, dtype=ctx.dtype, device=v.device) if d_o is None else _gradient(d_o, ctx.dtype)
                d_fin = None if d_fin is None else _gradient(d_fin, torch.float32)
                g = linear_attn_bwd(q, k, v, log_decay, d_o, d_fin, cu, h0, ctx.scale)
                return (g["dq"], g["dk"], g["dv"], None, None, g["dh0"] if h0 is not None else None, None, None)

        _FUNCTION = LinearAttention
    return _FUNCTION


def linear_attention(q, k, v, log_decay, cu_seqlens=None, initial_state=None, scale=1.0, checkpoint_bits=None):
    """linear_attn_fwd() as a differentiable torch op: returns (o, final_state); gradients
    reach q, k, v and initial_state through gdn_linattn_bwd, which forms the states again.
    log_decay is a constant of the model: one that requires a gradient is refused where gradients
    are recorded.
    checkpoint_bits=8 keeps q, k and v for the backward pass as 8-bit checkpoints (pack8): the
    gradients are then those at the values the checkpoints stand for."""
    if log_decay.requires_grad and _torch().is_grad_enabled():
        raise ValueError("log_decay takes no gradient: pass it detached")
    bits = _layers.kept_bits(checkpoint_bits, q, k, v, initial_state)
    return _function().apply(q, k, v, log_decay, cu_seqlens, initial_state, scale, bits)
