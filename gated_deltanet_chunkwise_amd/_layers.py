"""The layer operators around the gated delta rule: short causal convolution, selective
state space scan and 8-bit activation checkpoints (include/gdn.h, same names).

Argument marshalling only, as in _binding: every step runs in the library's kernels, and
nothing falls back.  Token tensors (x, dt, z, Bm, Cm) may be slices of a wider tensor, as
long as each token's values are contiguous and the tokens evenly spaced; everything else
is contiguous.  All tensors of a call live on one GPU, which need not be torch's current
device.  Work is enqueued on `stream`, by default torch's current stream of that GPU;
outputs and workspaces are allocated for it.
"""
import collections
import contextlib
import ctypes

from . import _binding
from ._binding import GdnError, _check_tensor, _dtype_code, _ptr, _torch

Packed8 = collections.namedtuple("Packed8", ("codes", "scales", "dtype"))
Packed8.__doc__ = """A checkpoint of an activation [..., C] (pack8): codes [..., C] int8, scales
[..., ceil(C / 32)] uint8, and the activation's dtype."""

_ACTIVATIONS = {None: 0, "silu": 1}
PACK_BLOCK = 32  # channels per checkpoint scale


class ConvParams(ctypes.Structure):
    """gdn_conv_params_t."""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "T", "C", "W", "num_seqs", "dtype", "activation")] + [
                    ("x_stride", ctypes.c_int64)]


class ScanParams(ctypes.Structure):
    """gdn_scan_params_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "G", "N", "num_seqs", "dtype")] + [
        (n, ctypes.c_int64) for n in ("x_stride", "dt_stride", "z_stride", "b_stride", "c_stride")]


def declare(lib):
    """Argument types of the entry points (called once by load_library)."""
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
    C, S = ctypes.POINTER(ConvParams), ctypes.POINTER(ScanParams)

    def fn(name, restype, *argtypes):
        f = getattr(lib, name)
        f.restype, f.argtypes = restype, list(argtypes)

    fn("gdn_conv_fwd", ctypes.c_int, C, *[vp] * 8)
    fn("gdn_conv_decode", ctypes.c_int, C, *[vp] * 7)
    fn("gdn_conv_bwd_workspace_size", sz, C, ctypes.c_int)
    fn("gdn_conv_bwd", ctypes.c_int, C, *[vp] * 13, sz, vp)
    fn("gdn_scan_fwd_workspace_size", sz, S, ctypes.c_int)
    fn("gdn_scan_fwd", ctypes.c_int, S, *[vp] * 13, sz, vp)
    fn("gdn_scan_decode", ctypes.c_int, S, *[vp] * 12)
    fn("gdn_scan_bwd_workspace_size", sz, S, ctypes.c_int)
    fn("gdn_scan_bwd", ctypes.c_int, S, *[vp] * 24, sz, vp)
    fn("gdn_pack8", ctypes.c_int, vp, ctypes.c_int, i64, i32, i64, vp, vp, vp)
    fn("gdn_unpack8", ctypes.c_int, vp, vp, i64, i32, vp, ctypes.c_int, vp)


# ---------------------------------------------------------------------------
# checks

def _place(name, t, device):
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must be a GPU tensor on %s, got %s" % (name, device, t.device))


def _dense(named, device):
    """Every given tensor contiguous and on `device` (checked after the shapes)."""
    for name, t in named:
        if t is not None:
            _place(name, t, device)
            if not t.is_contiguous():
                raise ValueError("%s must be contiguous" % name)


def _row_stride(name, t):
    """Elements between the tokens of t [B, T, ...]; raises unless each token's values
    are contiguous and the tokens evenly spaced."""
    B, T = t.shape[0], t.shape[1]
    width = 1
    for size, stride in zip(reversed(t.shape[2:]), reversed(t.stride()[2:])):
        if size != 1 and stride != width:
            raise ValueError("%s: the values of a token must be contiguous" % name)
        width *= size
    if B * T <= 1:
        return width
    ld = t.stride(1) if T > 1 else t.stride(0)
    if ld < width or (T > 1 and B > 1 and t.stride(0) != T * ld):
        raise ValueError("%s: tokens must be evenly spaced and not overlap" % name)
    return ld


def _gpu(name, t):
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor, got %s" % (name, t.device))


@contextlib.contextmanager
def _entered(device, stream, inputs):
    torch = _torch()
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device)
            return
        if stream.device != device:
            raise ValueError("stream belongs to %s, the tensors to %s" % (stream.device, device))
        with torch.cuda.stream(stream):
            yield stream
        for t in inputs:  # not to be reused before the stream is through with them
            if t is not None:
                t.record_stream(stream)


def _on(device, stream, inputs=()):
    """The GPU current and the stream to launch on, in whose order outputs and
    workspaces are allocated."""
    torch = _torch()
    if stream is None and device.index == torch.cuda.current_device():
        return contextlib.nullcontext(torch.cuda.current_stream(device))
    return _entered(device, stream, inputs)


def _call(name, *args):
    st = getattr(_binding.load_library(), name)(*args)
    if st:
        raise GdnError(st, name)


def _stream_arg(stream):
    return ctypes.c_void_p(stream.cuda_stream)


def _workspace(bytes_, device):
    torch = _torch()
    # 256-byte aligned (torch's caching allocator aligns blocks to at least 512)
    return torch.empty(max(int(bytes_), 256), dtype=torch.uint8, device=device)


def _sequences(cu_seqlens, B, device):
    """Number of sequences."""
    if cu_seqlens is None:
        return B
    torch = _torch()
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N+1]")
    if cu_seqlens.dtype != torch.int64:
        raise TypeError("cu_seqlens must be int64, got %s" % cu_seqlens.dtype)
    if B != 1:
        raise ValueError("cu_seqlens needs B == 1, got %d" % B)
    return cu_seqlens.numel() - 1


# ---------------------------------------------------------------------------
# 8-bit activation checkpoints

def pack8(x, stream=None):
    """The 8-bit checkpoint of x [..., C] (fp32 or bf16) through gdn_pack8: a Packed8.
    Rows of C channels may be strided as a slice of a wider tensor is."""
    torch = _torch()
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., C]")
    code = _dtype_code(x.dtype)
    _gpu("x", x)
    C = x.shape[-1]
    rows = x.numel() // C
    ld = C
    if not x.is_contiguous():
        # leading dimensions that merge into evenly spaced rows
        lead = [(n, s) for n, s in zip(x.shape[:-1], x.stride()[:-1]) if n != 1]
        ld = lead[-1][1] if lead else C
        step = ld
        ok = x.stride(-1) == 1 or C == 1
        for n, s in reversed(lead):
            ok = ok and s == step
            step *= n
        if not ok or ld < C:
            raise ValueError("x: rows of contiguous channels must be evenly spaced and not overlap")
    with _on(x.device, stream, (x,)) as s:
        codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        scales = torch.empty(x.shape[:-1] + ((C + PACK_BLOCK - 1) // PACK_BLOCK,), dtype=torch.uint8, device=x.device)
        _call("gdn_pack8", _ptr(x), code, rows, C, ld, _ptr(codes), _ptr(scales), _stream_arg(s))
    return Packed8(codes, scales, x.dtype)


def _check_packed(name, p):
    torch = _torch()
    if p.codes.dim() < 1 or p.codes.shape[-1] < 1:
        raise ValueError("%s.codes must be [..., C]" % name)
    C = p.codes.shape[-1]
    _check_tensor(name + ".codes", p.codes, p.codes.shape, torch.int8)
    _check_tensor(name + ".scales", p.scales, tuple(p.codes.shape[:-1]) + ((C + PACK_BLOCK - 1) // PACK_BLOCK,),
                  torch.uint8)


def unpack8(packed, out=None, stream=None):
    """The activation a Packed8 stands for, in its dtype (gdn_unpack8)."""
    torch = _torch()
    _check_packed("packed", packed)
    code = _dtype_code(packed.dtype)
    _check_tensor("out", out, packed.codes.shape, packed.dtype, required=False)
    _gpu("packed.codes", packed.codes)
    device = packed.codes.device
    _dense([("packed.codes", packed.codes), ("packed.scales", packed.scales), ("out", out)], device)
    C = packed.codes.shape[-1]
    with _on(device, stream, (packed.codes, packed.scales, out)) as s:
        if out is None:
            out = torch.empty(packed.codes.shape, dtype=packed.dtype, device=device)
        _call("gdn_unpack8", _ptr(packed.codes), _ptr(packed.scales), packed.codes.numel() // C, C, _ptr(out), code,
              _stream_arg(s))
    return out


def _maybe_packed(name, t):
    """(tensor, codes or data, scales or None, dtype) of an activation or its checkpoint."""
    if isinstance(t, Packed8):
        _check_packed(name, t)
        return t.codes, t.scales, t.dtype
    return t, None, t.dtype


# ---------------------------------------------------------------------------
# short causal convolution

def _conv_sizes(data, dtype, weight, bias, cu_seqlens, activation):
    torch = _torch()
    if data.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    B, T, C = data.shape
    if weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    _check_tensor("weight", weight, (C, W), torch.float32)
    _check_tensor("bias", bias, (C,), torch.float32, required=False)
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be None or 'silu', got %r" % (activation,))
    N = _sequences(cu_seqlens, B, data.device)
    p = ConvParams(B, T, C, W, 0 if cu_seqlens is None else N, _dtype_code(dtype), _ACTIVATIONS[activation],
                   _row_stride("x", data))
    return p, B, T, C, W, N


def conv_fwd(x, weight, bias=None, cu_seqlens=None, initial_state=None, activation="silu",
             output_final_state=True, stream=None):
    """Short causal depthwise convolution through gdn_conv_fwd: x [B,T,C] (bf16 or fp32),
    weight [C,W] fp32 with W in 2..4, bias [C] fp32 or None, initial_state [N,W-1,C] in
    x's dtype or None, activation "silu" or None.  Returns (y [B,T,C], final_state
    [N,W-1,C] or None)."""
    torch = _torch()
    p, B, T, C, W, N = _conv_sizes(x, x.dtype, weight, bias, cu_seqlens, activation)
    _check_tensor("initial_state", initial_state, (N, W - 1, C), x.dtype, required=False)
    _gpu("x", x)
    _dense([("weight", weight), ("bias", bias), ("cu_seqlens", cu_seqlens), ("initial_state", initial_state)],
           x.device)
    with _on(x.device, stream, (x, weight, bias, cu_seqlens, initial_state)) as s:
        y = torch.empty((B, T, C), dtype=x.dtype, device=x.device)
        fin = torch.empty((N, max(W - 1, 0), C), dtype=x.dtype, device=x.device) if output_final_state else None
        _call("gdn_conv_fwd", ctypes.byref(p), _ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens),
              _ptr(initial_state), _ptr(y), _ptr(fin), _stream_arg(s))
    return y, fin


def conv_bwd(x, weight, bias, d_y, d_final_state=None, cu_seqlens=None, initial_state=None, activation="silu",
             stream=None):
    """Gradients of conv_fwd through gdn_conv_bwd: dict of dx [B,T,C] and dh0 [N,W-1,C]
    in x's dtype, dweight [C,W] and dbias [C] fp32.  x may be its checkpoint (Packed8)."""
    torch = _torch()
    data, scales, dtype = _maybe_packed("x", x)
    p, B, T, C, W, N = _conv_sizes(data, dtype, weight, bias, cu_seqlens, activation)
    _check_tensor("d_y", d_y, (B, T, C), dtype)
    _check_tensor("d_final_state", d_final_state, (N, W - 1, C), dtype, required=False)
    _check_tensor("initial_state", initial_state, (N, W - 1, C), dtype, required=False)
    _gpu("x", data)
    device = data.device
    _dense([("weight", weight), ("bias", bias), ("cu_seqlens", cu_seqlens), ("initial_state", initial_state),
            ("d_y", d_y), ("d_final_state", d_final_state), ("x.scales", scales)], device)
    ws_bytes = int(_binding.load_library().gdn_conv_bwd_workspace_size(ctypes.byref(p), int(cu_seqlens is not None)))
    with _on(device, stream, (data, scales, weight, bias, cu_seqlens, initial_state, d_y, d_final_state)) as s:
        dx = torch.empty((B, T, C), dtype=dtype, device=device)
        dw = torch.empty((C, W), dtype=torch.float32, device=device)
        db = torch.empty((C,), dtype=torch.float32, device=device)
        dh0 = torch.empty((N, max(W - 1, 0), C), dtype=dtype, device=device)
        ws = _workspace(ws_bytes, device)
        _call("gdn_conv_bwd", ctypes.byref(p), _ptr(data), _ptr(scales), _ptr(weight), _ptr(bias),
              _ptr(cu_seqlens), _ptr(initial_state), _ptr(d_y), _ptr(d_final_state), _ptr(dx), _ptr(dw), _ptr(db),
              _ptr(dh0), _ptr(ws), ws.numel(), _stream_arg(s))
    return dict(dx=dx, dweight=dw, dbias=db, dh0=dh0)


def conv_decode_launcher(x, weight, state, bias=None, activation="silu", new_state=None, out=None, stream=None):
    """Check and marshal gdn_conv_decode's arguments once; returns (launch, y), where
    launch() enqueues the convolution of x's T tokens after `state` [B,W-1,C], writing
    the state after them to new_state (default: `state` itself)."""
    torch = _torch()
    p, B, T, C, W, _ = _conv_sizes(x, x.dtype, weight, bias, None, activation)
    _check_tensor("state", state, (B, W - 1, C), x.dtype)
    _check_tensor("new_state", new_state, (B, W - 1, C), x.dtype, required=False)
    _check_tensor("out", out, (B, T, C), x.dtype, required=False)
    _gpu("x", x)
    _dense([("weight", weight), ("bias", bias), ("state", state), ("new_state", new_state), ("out", out)], x.device)
    new = state if new_state is None else new_state
    with _on(x.device, stream, (x, weight, bias, state, new_state, out)) as s:
        if out is None:
            out = torch.empty((B, T, C), dtype=x.dtype, device=x.device)
    args = (ctypes.byref(p), _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(new), _ptr(out), _stream_arg(s))
    return _launcher("gdn_conv_decode", x.device, args, (p, s, x, weight, bias, state, new, out)), out


def _launcher(name, device, args, keep):
    torch = _torch()
    fn = getattr(_binding.load_library(), name)

    def launch():
        keep  # the tensors stay alive as long as the callable
        if torch.cuda.current_device() == device.index:
            st = fn(*args)
        else:
            with torch.cuda.device(device):
                st = fn(*args)
        if st:
            raise GdnError(st, name)
    return launch


def conv_decode(x, weight, state, bias=None, activation="silu", new_state=None, out=None, stream=None):
    """T tokens (1: a decode step) of each of B sequences through gdn_conv_decode: returns
    y [B,T,C]; the state after them goes to new_state, or updates `state` in place."""
    launch, out = conv_decode_launcher(x, weight, state, bias, activation, new_state, out, stream)
    launch()
    return out


# ---------------------------------------------------------------------------
# selective state space scan

def _scan_sizes(x, dtype, dt, A_log, Bm, Cm, skip, z, z_dtype, dt_bias, cu_seqlens):
    torch = _torch()
    f32 = torch.float32
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    if A_log.dim() != 2 or Bm.dim() != 4:
        raise ValueError("A_log must be [D, N] and Bm [B, T, G, N]")
    N, G = A_log.shape[1], Bm.shape[2]
    _check_tensor("dt", dt, (B, T, D), dtype)
    _check_tensor("A_log", A_log, (D, N), f32)
    _check_tensor("Bm", Bm, (B, T, G, N), dtype)
    _check_tensor("Cm", Cm, (B, T, G, N), dtype)
    _check_tensor("skip", skip, (D,), f32, required=False)
    if z is not None:
        if tuple(z.shape) != (B, T, D):
            raise ValueError("z must have shape %s, got %s" % ((B, T, D), tuple(z.shape)))
        if z_dtype != dtype:
            raise TypeError("z must be %s, got %s" % (dtype, z_dtype))
    _check_tensor("dt_bias", dt_bias, (D,), f32, required=False)
    S = _sequences(cu_seqlens, B, x.device)
    p = ScanParams(B, T, D, G, N, 0 if cu_seqlens is None else S, _dtype_code(dtype), _row_stride("x", x),
                   _row_stride("dt", dt), 0 if z is None else _row_stride("z", z), _row_stride("Bm", Bm),
                   _row_stride("Cm", Cm))
    return p, B, T, D, G, N, S


def _scan_place(x, dt, Bm, Cm, z, dense):
    _gpu("x", x)
    for name, t in (("dt", dt), ("Bm", Bm), ("Cm", Cm), ("z", z)):
        if t is not None:
            _place(name, t, x.device)
    _dense(dense, x.device)


def scan_fwd(x, dt, A_log, Bm, Cm, skip=None, z=None, dt_bias=None, cu_seqlens=None, initial_state=None,
             output_final_state=True, stream=None):
    """Selective state space scan through gdn_scan_fwd: x, dt, z [B,T,D] and Bm, Cm
    [B,T,G,N] in bf16 or fp32, A_log [D,N], skip and dt_bias [D] fp32, initial_state
    [sequences,D,N] fp32; skip, z, dt_bias and initial_state may be None.  Returns
    (y [B,T,D], final_state [sequences,D,N] fp32 or None)."""
    torch = _torch()
    p, B, T, D, G, N, S = _scan_sizes(x, x.dtype, dt, A_log, Bm, Cm, skip, z, None if z is None else z.dtype,
                                      dt_bias, cu_seqlens)
    _check_tensor("initial_state", initial_state, (S, D, N), torch.float32, required=False)
    _scan_place(x, dt, Bm, Cm, z, [("A_log", A_log), ("skip", skip), ("dt_bias", dt_bias),
                                   ("cu_seqlens", cu_seqlens), ("initial_state", initial_state)])
    ws_bytes = int(_binding.load_library().gdn_scan_fwd_workspace_size(ctypes.byref(p), int(cu_seqlens is not None)))
    with _on(x.device, stream, (x, dt, A_log, Bm, Cm, skip, z, dt_bias, cu_seqlens, initial_state)) as s:
        y = torch.empty((B, T, D), dtype=x.dtype, device=x.device)
        fin = torch.empty((S, D, N), dtype=torch.float32, device=x.device) if output_final_state else None
        ws = _workspace(ws_bytes, x.device)
        _call("gdn_scan_fwd", ctypes.byref(p), _ptr(x), _ptr(dt), _ptr(A_log), _ptr(Bm), _ptr(Cm), _ptr(skip),
              _ptr(z), _ptr(dt_bias), _ptr(cu_seqlens), _ptr(initial_state), _ptr(y), _ptr(fin), _ptr(ws),
              ws.numel(), _stream_arg(s))
    return y, fin


def scan_bwd(x, dt, A_log, Bm, Cm, d_y, d_final_state=None, skip=None, z=None, dt_bias=None, cu_seqlens=None,
             initial_state=None, stream=None):
    """Gradients of scan_fwd through gdn_scan_bwd: dict of dx, ddt, dBm, dCm (and dz with
    z) in x's dtype, dA_log, dskip, ddt_bias and dh0 in fp32.  x and z may both be their
    checkpoints (Packed8)."""
    torch = _torch()
    f32 = torch.float32
    xd, xs, dtype = _maybe_packed("x", x)
    zd, zs, z_dtype = (None, None, None) if z is None else _maybe_packed("z", z)
    if z is not None and (xs is None) != (zs is None):
        raise ValueError("x and z must both be checkpoints, or neither")
    p, B, T, D, G, N, S = _scan_sizes(xd, dtype, dt, A_log, Bm, Cm, skip, zd, z_dtype, dt_bias, cu_seqlens)
    _check_tensor("d_y", d_y, (B, T, D), dtype)
    _check_tensor("d_final_state", d_final_state, (S, D, N), f32, required=False)
    _check_tensor("initial_state", initial_state, (S, D, N), f32, required=False)
    device = xd.device
    _scan_place(xd, dt, Bm, Cm, zd, [("A_log", A_log), ("skip", skip), ("dt_bias", dt_bias),
                                     ("cu_seqlens", cu_seqlens), ("initial_state", initial_state), ("d_y", d_y),
                                     ("d_final_state", d_final_state), ("x.scales", xs), ("z.scales", zs)])
    ws_bytes = int(_binding.load_library().gdn_scan_bwd_workspace_size(ctypes.byref(p), int(cu_seqlens is not None)))
    with _on(device, stream, (xd, xs, dt, A_log, Bm, Cm, d_y, d_final_state, skip, zd, zs, dt_bias, cu_seqlens,
                              initial_state)) as s:
        new = lambda shape, dt_: torch.empty(shape, dtype=dt_, device=device)  # noqa: E731
        g = dict(dx=new((B, T, D), dtype), ddt=new((B, T, D), dtype), dA_log=new((D, N), f32),
                 dBm=new((B, T, G, N), dtype), dCm=new((B, T, G, N), dtype), dskip=new((D,), f32),
                 ddt_bias=new((D,), f32), dh0=new((S, D, N), f32))
        if z is not None:
            g["dz"] = new((B, T, D), dtype)
        ws = _workspace(ws_bytes, device)
        _call("gdn_scan_bwd", ctypes.byref(p), _ptr(xd), _ptr(xs), _ptr(dt), _ptr(A_log), _ptr(Bm), _ptr(Cm),
              _ptr(skip), _ptr(zd), _ptr(zs), _ptr(dt_bias), _ptr(cu_seqlens), _ptr(initial_state), _ptr(d_y),
              _ptr(d_final_state), _ptr(g["dx"]), _ptr(g["ddt"]), _ptr(g["dA_log"]), _ptr(g["dBm"]),
              _ptr(g["dCm"]), _ptr(g["dskip"]), _ptr(g.get("dz")), _ptr(g["ddt_bias"]), _ptr(g["dh0"]), _ptr(ws),
              ws.numel(), _stream_arg(s))
    return g


def scan_decode_launcher(x, dt, A_log, Bm, Cm, state, skip=None, z=None, dt_bias=None, new_state=None, out=None,
                         stream=None):
    """Check and marshal gdn_scan_decode's arguments once; returns (launch, y), where
    launch() enqueues the scan of x's T tokens after `state` [B,D,N], writing the state
    after them to new_state (default: `state` itself)."""
    torch = _torch()
    p, B, T, D, G, N, _ = _scan_sizes(x, x.dtype, dt, A_log, Bm, Cm, skip, z, None if z is None else z.dtype,
                                      dt_bias, None)
    _check_tensor("state", state, (B, D, N), torch.float32)
    _check_tensor("new_state", new_state, (B, D, N), torch.float32, required=False)
    _check_tensor("out", out, (B, T, D), x.dtype, required=False)
    _scan_place(x, dt, Bm, Cm, z, [("A_log", A_log), ("skip", skip), ("dt_bias", dt_bias), ("state", state),
                                   ("new_state", new_state), ("out", out)])
    new = state if new_state is None else new_state
    with _on(x.device, stream, (x, dt, A_log, Bm, Cm, skip, z, dt_bias, state, new_state, out)) as s:
        if out is None:
            out = torch.empty((B, T, D), dtype=x.dtype, device=x.device)
    args = (ctypes.byref(p), _ptr(x), _ptr(dt), _ptr(A_log), _ptr(Bm), _ptr(Cm), _ptr(skip), _ptr(z), _ptr(dt_bias),
            _ptr(state), _ptr(new), _ptr(out), _stream_arg(s))
    return _launcher("gdn_scan_decode", x.device, args,
                     (p, s, x, dt, A_log, Bm, Cm, skip, z, dt_bias, state, new, out)), out


def scan_decode(x, dt, A_log, Bm, Cm, state, skip=None, z=None, dt_bias=None, new_state=None, out=None,
                stream=None):
    """T tokens (1: a decode step) of each of B sequences through gdn_scan_decode: returns
    y [B,T,D]; the state after them goes to new_state, or updates `state` in place."""
    launch, out = scan_decode_launcher(x, dt, A_log, Bm, Cm, state, skip, z, dt_bias, new_state, out, stream)
    launch()
    return out


# ---------------------------------------------------------------------------
# differentiable forms

def check_bits(bits):
    if bits not in (None, 8):
        raise ValueError("checkpoint_bits must be None or 8, got %r" % (bits,))


def keep(t, bits):
    """What a training step keeps of t for its backward pass: (tensors, dtype)."""
    if bits is None or t is None:
        return (t, None), None
    p = pack8(t.detach())
    return (p.codes, p.scales), p.dtype


def kept(pair, dtype):
    """The other way round: t itself, or its checkpoint."""
    return pair[0] if pair[1] is None else Packed8(pair[0], pair[1], dtype)


_FUNCTIONS = {}


def _conv_function():
    """torch.autograd.Function behind causal_conv (defined on first use, since torch is
    imported lazily)."""
    if "conv" not in _FUNCTIONS:
        torch = _torch()

        class CausalConv(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, weight, bias, cu_seqlens, initial_state, activation, bits):
                ctx.set_materialize_grads(False)
                y, fin = conv_fwd(x, weight, bias, cu_seqlens, initial_state, activation)
                pair, ctx.dtype = keep(x, bits)
                ctx.save_for_backward(*pair, weight, bias, cu_seqlens, initial_state)
                ctx.activation = activation
                return y, fin

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, d_y, d_fin):
                xd, xs, weight, bias, cu, h0 = ctx.saved_tensors
                x = kept((xd, xs), ctx.dtype)
                dtype = ctx.dtype or xd.dtype
                d_y = torch.zeros(xd.shape, dtype=dtype, device=xd.device) if d_y is None else d_y.to(dtype).contiguous()
                d_fin = None if d_fin is None else d_fin.to(dtype).contiguous()
                g = conv_bwd(x, weight, bias, d_y, d_fin, cu, h0, ctx.activation)
                return (g["dx"], g["dweight"], g["dbias"] if bias is not None else None, None,
                        g["dh0"] if h0 is not None else None, None, None)

        _FUNCTIONS["conv"] = CausalConv
    return _FUNCTIONS["conv"]


def causal_conv(x, weight, bias=None, cu_seqlens=None, initial_state=None, activation="silu",
                checkpoint_bits=None):
    """conv_fwd() as a differentiable torch op: returns (y, final_state); gradients reach
    x, weight, bias and initial_state through gdn_conv_bwd.  checkpoint_bits=8 keeps x
    for the backward pass as an 8-bit checkpoint: the gradients are then those at the
    values it stands for."""
    check_bits(checkpoint_bits)
    return _conv_function().apply(x, weight, bias, cu_seqlens, initial_state, activation, checkpoint_bits)


def _scan_function():
    if "scan" not in _FUNCTIONS:
        torch = _torch()

        class SelectiveScan(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, dt, A_log, Bm, Cm, skip, z, dt_bias, cu_seqlens, initial_state, bits):
                ctx.set_materialize_grads(False)
                y, fin = scan_fwd(x, dt, A_log, Bm, Cm, skip, z, dt_bias, cu_seqlens, initial_state)
                xp, ctx.dtype = keep(x, bits)
                zp, _ = keep(z, bits)
                ctx.save_for_backward(*xp, *zp, dt, A_log, Bm, Cm, skip, dt_bias, cu_seqlens, initial_state)
                return y, fin

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, d_y, d_fin):
                xd, xs, zd, zs, dt, A_log, Bm, Cm, skip, dt_bias, cu, h0 = ctx.saved_tensors
                dtype = dt.dtype
                z = None if zd is None else kept((zd, zs), dtype)
                d_y = torch.zeros(dt.shape, dtype=dtype, device=dt.device) if d_y is None else d_y.to(dtype).contiguous()
                d_fin = None if d_fin is None else d_fin.to(torch.float32).contiguous()
                g = scan_bwd(kept((xd, xs), dtype), dt, A_log, Bm, Cm, d_y, d_fin, skip, z, dt_bias, cu, h0)
                return (g["dx"], g["ddt"], g["dA_log"], g["dBm"], g["dCm"],
                        g["dskip"] if skip is not None else None, g.get("dz"),
                        g["ddt_bias"] if dt_bias is not None else None, None,
                        g["dh0"] if h0 is not None else None, None)

        _FUNCTIONS["scan"] = SelectiveScan
    return _FUNCTIONS["scan"]


def selective_scan(x, dt, A_log, Bm, Cm, skip=None, z=None, dt_bias=None, cu_seqlens=None, initial_state=None,
                   checkpoint_bits=None):
    """scan_fwd() as a differentiable torch op: returns (y, final_state); gradients reach
    x, dt, A_log, Bm, Cm, skip, z, dt_bias and initial_state through gdn_scan_bwd, which
    forms the states again.  checkpoint_bits=8 keeps x and z as 8-bit checkpoints (dt, of
    which the decays depend exponentially, and the small Bm and Cm stay as they are): the
    gradients are then those at the values the checkpoints stand for."""
    check_bits(checkpoint_bits)
    return _scan_function().apply(x, dt, A_log, Bm, Cm, skip, z, dt_bias, cu_seqlens, initial_state,
                                  checkpoint_bits)
