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
import ctypes
import functools

from . import _binding
from ._binding import GdnError, _check_tensor, _dtype_code

Packed8 = collections.namedtuple("Packed8", ("codes", "scales", "dtype"))
Packed8.__doc__ = """A checkpoint of an activation [..., C] (pack8): codes [..., C] int8, scales
[..., ceil(C / 32)] uint8, and the activation's dtype."""

GDN_ZERO_REST = 0x100  # include/gdn.h: rows of y behind the last sequence are set to 0
_ACTIVATIONS = {None: 0, "silu": 1}
PACK_BLOCK = 32  # channels per checkpoint scale


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        _TORCH = _binding._torch()
    return _TORCH


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
# checks and launches.  A call of a small problem takes the GPU a few microseconds, so
# these take care to take the host no longer.

_RAW_STREAM = None


def _raw_stream(index):
    """torch's current stream of GPU `index`, as the address the library takes."""
    global _RAW_STREAM
    if _RAW_STREAM is None:
        torch = _torch()
        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _RAW_STREAM(index)


def _lib():
    return _binding._LIB or _binding.load_library()


def _fit(specs):
    """(name, tensor, shape, dtype) each: the tensor, where given, has exactly that shape
    and dtype."""
    for name, t, shape, dtype in specs:
        if t is not None and (t.dtype is not dtype or t.shape != shape):
            _check_tensor(name, t, shape, dtype)


def _need(name, t):
    if t is None:
        raise ValueError("%s is required" % name)


def _place(x, rows, dense):
    """The GPU (its index) that x and every other given tensor live on, `dense` ones
    contiguous; both lists (name, tensor, ...)."""
    index = x.get_device()
    if index < 0:
        raise ValueError("x must be a GPU tensor, got %s" % x.device)
    for spec in rows:
        if spec[1] is not None and spec[1].get_device() != index:
            raise ValueError("%s must be a GPU tensor on %s, got %s" % (spec[0], x.device, spec[1].device))
    for spec in dense:
        t = spec[1]
        if t is not None:
            if t.get_device() != index:
                raise ValueError("%s must be a GPU tensor on %s, got %s" % (spec[0], x.device, t.device))
            if not t.is_contiguous():
                raise ValueError("%s must be contiguous" % spec[0])
    return index


def _row_stride(name, t):
    """Elements between the tokens of t [B, T, ...] (0: dense); raises unless each token's
    values are contiguous and the tokens evenly spaced."""
    if t.is_contiguous():
        return 0
    B, T = t.shape[0], t.shape[1]
    width = 1
    for size, stride in zip(reversed(t.shape[2:]), reversed(t.stride()[2:])):
        if size != 1 and stride != width:
            raise ValueError("%s: the values of a token must be contiguous" % name)
        width *= size
    if B * T <= 1:
        return 0
    ld = t.stride(1) if T > 1 else t.stride(0)
    if ld < width or (T > 1 and B > 1 and t.stride(0) != T * ld):
        raise ValueError("%s: tokens must be evenly spaced and not overlap" % name)
    return ld


def _entered(index, stream, inputs, body):
    torch = _torch()
    with torch.cuda.device(index):
        if stream is None:
            return body(_raw_stream(index))
        if stream.device.index != index:
            raise ValueError("stream belongs to %s, the tensors to GPU %d" % (stream.device, index))
        with torch.cuda.stream(stream):
            out = body(stream.cuda_stream)
        for t in inputs:  # not to be reused before the stream is through with them
            if t is not None:
                t.record_stream(stream)
        return out


def _on(index, stream, inputs, body):
    """body(stream address), with GPU `index` current and outputs and workspaces allocated
    in the order of the stream that it launches on."""
    if stream is None and index == _torch().cuda.current_device():
        return body(_raw_stream(index))
    return _entered(index, stream, inputs, body)


def _call(name, *args):
    """An entry point with its arguments: integers, tensors' addresses (or None) and params."""
    st = getattr(_binding._LIB, name)(*args)
    if st:
        raise GdnError(st, name)


def _p(t):
    return None if t is None else t.data_ptr()


_WRITTEN = None


def _written(tensors):
    """Tells autograd that the call has written to these tensors of the caller's (a tuple),
    as torch's in-place operations do: a backward pass that saved one of them then refuses it."""
    global _WRITTEN
    if _WRITTEN is None:
        torch = _torch()
        _WRITTEN = getattr(torch._C, "_increment_version", torch.autograd.graph.increment_version)
    _WRITTEN(tensors)


_LIKE = None


def _like(t):
    """An uninitialised contiguous tensor of t's shape, dtype and GPU (a third quicker than
    torch.empty with all three spelled out)."""
    global _LIKE
    if _LIKE is None:
        torch = _torch()
        _LIKE = functools.partial(torch.empty_like, memory_format=torch.contiguous_format)
    return _LIKE(t)


def _workspace(bytes_, index):
    """(tensor, address, size); 256-byte aligned (torch's allocator aligns to 512)."""
    if not bytes_:
        return None, None, 0
    torch = _torch()
    t = torch.empty(bytes_, dtype=torch.uint8, device=torch.device("cuda", index))
    return t, t.data_ptr(), bytes_


def _sequences(cu_seqlens, B):
    """Number of sequences."""
    if cu_seqlens is None:
        return B
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N+1]")
    if cu_seqlens.dtype is not _torch().int64:
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
    index = _place(x, (), ())
    C = x.shape[-1]
    ld = 0
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

    def body(s):
        codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        scales = torch.empty(x.shape[:-1] + ((C + PACK_BLOCK - 1) // PACK_BLOCK,), dtype=torch.uint8, device=x.device)
        _lib()
        _call("gdn_pack8", x.data_ptr(), code, x.numel() // C, C, ld, codes.data_ptr(), scales.data_ptr(), s)
        return Packed8(codes, scales, x.dtype)
    return _on(index, stream, (x,), body)


def _check_packed(name, p):
    torch = _torch()
    shape = p.codes.shape
    if not shape or shape[-1] < 1:
        raise ValueError("%s.codes must be [..., C]" % name)
    _fit(((name + ".codes", p.codes, shape, torch.int8),
          (name + ".scales", p.scales, shape[:-1] + ((shape[-1] + PACK_BLOCK - 1) // PACK_BLOCK,), torch.uint8)))


def unpack8(packed, out=None, stream=None):
    """The activation a Packed8 stands for, in its dtype (gdn_unpack8)."""
    torch = _torch()
    codes, scales, dtype = packed
    _check_packed("packed", packed)
    code = _dtype_code(dtype)
    _fit((("out", out, codes.shape, dtype),))
    index = _place(codes, (), (("packed.codes", codes), ("packed.scales", scales), ("out", out)))

    def body(s):
        y = torch.empty(codes.shape, dtype=dtype, device=codes.device) if out is None else out
        C = codes.shape[-1]
        _lib()
        _call("gdn_unpack8", codes.data_ptr(), scales.data_ptr(), codes.numel() // C, C, y.data_ptr(), code, s)
        if out is not None:
            _written((out,))
        return y
    return _on(index, stream, (codes, scales, out), body)


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
    _fit((("weight", weight, (C, W), torch.float32), ("bias", bias, (C,), torch.float32)))
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be None or 'silu', got %r" % (activation,))
    N = _sequences(cu_seqlens, B)
    code = _dtype_code(dtype)
    p = ConvParams(B, T, C, W, *((0, code) if cu_seqlens is None else (N, code | GDN_ZERO_REST)),
                   _ACTIVATIONS[activation], _row_stride("x", data))
    return ctypes.byref(p), B, T, C, W, N


def conv_fwd(x, weight, bias=None, cu_seqlens=None, initial_state=None, activation="silu",
             output_final_state=True, stream=None):
    """Short causal depthwise convolution through gdn_conv_fwd: x [B,T,C] (bf16 or fp32),
    weight [C,W] fp32 with W in 2..4, bias [C] fp32 or None, initial_state [N,W-1,C] in
    x's dtype or None, activation "silu" or None.  Returns (y [B,T,C], final_state
    [N,W-1,C] or None); rows of y behind the last sequence (where cu_seqlens end before
    T) are 0."""
    p, B, T, C, W, N = _conv_sizes(x, x.dtype, weight, bias, cu_seqlens, activation)
    _fit((("initial_state", initial_state, (N, W - 1, C), x.dtype),))
    index = _place(x, (), (("weight", weight), ("bias", bias), ("cu_seqlens", cu_seqlens),
                           ("initial_state", initial_state)))

    def body(s):
        empty = _torch().empty
        y = _like(x)
        fin = empty((N, max(W - 1, 0), C), dtype=x.dtype, device=x.device) if output_final_state else None
        _lib()
        _call("gdn_conv_fwd", p, x.data_ptr(), weight.data_ptr(), _p(bias), _p(cu_seqlens), _p(initial_state),
              y.data_ptr(), _p(fin), s)
        return y, fin
    return _on(index, stream, (x, weight, bias, cu_seqlens, initial_state), body)


def conv_bwd(x, weight, bias, d_y, d_final_state=None, cu_seqlens=None, initial_state=None, activation="silu",
             stream=None):
    """Gradients of conv_fwd through gdn_conv_bwd: dict of dx [B,T,C] and dh0 [N,W-1,C]
    in x's dtype, dweight [C,W] and dbias [C] fp32.  x may be its checkpoint (Packed8)."""
    data, scales, dtype = _maybe_packed("x", x)
    p, B, T, C, W, N = _conv_sizes(data, dtype, weight, bias, cu_seqlens, activation)
    _need("d_y", d_y)
    _fit((("d_y", d_y, (B, T, C), dtype), ("d_final_state", d_final_state, (N, W - 1, C), dtype),
          ("initial_state", initial_state, (N, W - 1, C), dtype)))
    index = _place(data, (), (("weight", weight), ("bias", bias), ("cu_seqlens", cu_seqlens),
                              ("initial_state", initial_state), ("d_y", d_y), ("d_final_state", d_final_state),
                              ("x.scales", scales)))
    ws_bytes = _lib().gdn_conv_bwd_workspace_size(p, int(cu_seqlens is not None))

    def body(s):
        torch = _torch()
        empty, device, f32 = torch.empty, data.device, torch.float32
        g = dict(dx=_like(d_y), dweight=_like(weight),
                 dbias=empty((C,), dtype=f32, device=device),
                 dh0=empty((N, max(W - 1, 0), C), dtype=dtype, device=device))
        ws, ws_ptr, ws_size = _workspace(ws_bytes, index)
        _call("gdn_conv_bwd", p, data.data_ptr(), _p(scales), weight.data_ptr(), _p(bias), _p(cu_seqlens),
              _p(initial_state), d_y.data_ptr(), _p(d_final_state), g["dx"].data_ptr(), g["dweight"].data_ptr(),
              g["dbias"].data_ptr(), g["dh0"].data_ptr(), ws_ptr, ws_size, s)
        return g
    return _on(index, stream, (data, scales, weight, bias, cu_seqlens, initial_state, d_y, d_final_state), body)


def _conv_decode_args(x, weight, state, bias, activation, new_state, out):
    p, B, T, C, W, _ = _conv_sizes(x, x.dtype, weight, bias, None, activation)
    _need("state", state)
    shape = (B, W - 1, C)
    _fit((("state", state, shape, x.dtype), ("new_state", new_state, shape, x.dtype), ("out", out, (B, T, C), x.dtype)))
    index = _place(x, (), (("weight", weight), ("bias", bias), ("state", state), ("new_state", new_state), ("out", out)))

    def args(s):
        y = _like(x) if out is None else out
        new = state if new_state is None else new_state
        _lib()
        return ((p, x.data_ptr(), weight.data_ptr(), _p(bias), state.data_ptr(), new.data_ptr(), y.data_ptr(), s), y,
                (new,) if out is None else (new, out))
    return index, args


def conv_decode_launcher(x, weight, state, bias=None, activation="silu", new_state=None, out=None, stream=None):
    """Check and marshal gdn_conv_decode's arguments once; returns (launch, y), where
    launch() enqueues the convolution of x's T tokens after `state` [B,W-1,C], writing
    the state after them to new_state (default: `state` itself).  Every launch() goes to
    `stream`, or to the stream that was current when the launcher was made, whichever is
    current later: a launcher for a graph is made on the stream that captures it."""
    index, args = _conv_decode_args(x, weight, state, bias, activation, new_state, out)
    keep = (x, weight, state, bias, new_state, out, stream)
    args, y, written = _on(index, stream, keep[:-1], args)
    return _launcher("gdn_conv_decode", index, args, keep + (y,), written), y


def _launcher(name, index, args, keep, written):
    torch = _torch()
    fn = getattr(_lib(), name)

    def launch():
        keep  # the tensors stay alive as long as the callable
        if torch.cuda.current_device() == index:
            st = fn(*args)
        else:
            with torch.cuda.device(index):
                st = fn(*args)
        if st:
            raise GdnError(st, name)
        _written(written)
    return launch


def conv_decode(x, weight, state, bias=None, activation="silu", new_state=None, out=None, stream=None):
    """T tokens (1: a decode step) of each of B sequences through gdn_conv_decode: returns
    y [B,T,C]; the state after them goes to new_state, or updates `state` in place."""
    index, args = _conv_decode_args(x, weight, state, bias, activation, new_state, out)

    def body(s):
        a, y, written = args(s)
        _call("gdn_conv_decode", *a)
        _written(written)
        return y
    return _on(index, stream, (x, weight, state, bias, new_state, out), body)


# ---------------------------------------------------------------------------
# selective state space scan

def _scan_sizes(x, dtype, dt, A_log, Bm, Cm, skip, z, z_dtype, dt_bias, cu_seqlens):
    f32 = _torch().float32
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    shape = x.shape
    B, T, D = shape
    if A_log.dim() != 2 or Bm.dim() != 4:
        raise ValueError("A_log must be [D, N] and Bm [B, T, G, N]")
    N, G = A_log.shape[1], Bm.shape[2]
    rows = (B, T, G, N)
    _fit((("dt", dt, shape, dtype), ("A_log", A_log, (D, N), f32), ("Bm", Bm, rows, dtype), ("Cm", Cm, rows, dtype),
          ("skip", skip, (D,), f32), ("dt_bias", dt_bias, (D,), f32)))
    z_ld = 0
    if z is not None:
        if z.shape != shape:
            raise ValueError("z must have shape %s, got %s" % ((B, T, D), tuple(z.shape)))
        if z_dtype is not dtype:
            raise TypeError("z must be %s, got %s" % (dtype, z_dtype))
        z_ld = _row_stride("z", z)
    S = _sequences(cu_seqlens, B)
    code = _dtype_code(dtype)
    p = ScanParams(B, T, D, G, N, *((0, code) if cu_seqlens is None else (S, code | GDN_ZERO_REST)), _row_stride("x", x),
                   _row_stride("dt", dt), z_ld, _row_stride("Bm", Bm), _row_stride("Cm", Cm))
    return ctypes.byref(p), B, T, D, G, N, S


def scan_fwd(x, dt, A_log, Bm, Cm, skip=None, z=None, dt_bias=None, cu_seqlens=None, initial_state=None,
             output_final_state=True, stream=None):
    """Selective state space scan through gdn_scan_fwd: x, dt, z [B,T,D] and Bm, Cm
    [B,T,G,N] in bf16 or fp32, A_log [D,N], skip and dt_bias [D] fp32, initial_state
    [sequences,D,N] fp32; skip, z, dt_bias and initial_state may be None.  Returns
    (y [B,T,D], final_state [sequences,D,N] fp32 or None); rows of y behind the last
    sequence are 0, as conv_fwd's."""
    f32 = _torch().float32
    p, B, T, D, G, N, S = _scan_sizes(x, x.dtype, dt, A_log, Bm, Cm, skip, z, None if z is None else z.dtype,
                                      dt_bias, cu_seqlens)
    _fit((("initial_state", initial_state, (S, D, N), f32),))
    index = _place(x, (("dt", dt), ("Bm", Bm), ("Cm", Cm), ("z", z)),
                   (("A_log", A_log), ("skip", skip), ("dt_bias", dt_bias), ("cu_seqlens", cu_seqlens),
                    ("initial_state", initial_state)))
    ws_bytes = _lib().gdn_scan_fwd_workspace_size(p, int(cu_seqlens is not None))

    def body(s):
        empty = _torch().empty
        y = _like(x)
        fin = empty((S, D, N), dtype=f32, device=x.device) if output_final_state else None
        ws, ws_ptr, ws_size = _workspace(ws_bytes, index)
        _call("gdn_scan_fwd", p, x.data_ptr(), dt.data_ptr(), A_log.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), _p(skip),
              _p(z), _p(dt_bias), _p(cu_seqlens), _p(initial_state), y.data_ptr(), _p(fin), ws_ptr, ws_size, s)
        return y, fin
    return _on(index, stream, (x, dt, A_log, Bm, Cm, skip, z, dt_bias, cu_seqlens, initial_state), body)


def scan_bwd(x, dt, A_log, Bm, Cm, d_y, d_final_state=None, skip=None, z=None, dt_bias=None, cu_seqlens=None,
             initial_state=None, stream=None):
    """Gradients of scan_fwd through gdn_scan_bwd: dict of dx, ddt, dBm, dCm (and dz with
    z) in x's dtype, dA_log, dskip, ddt_bias and dh0 in fp32.  x and z may both be their
    checkpoints (Packed8)."""
    f32 = _torch().float32
    xd, xs, dtype = _maybe_packed("x", x)
    zd, zs, z_dtype = (None, None, None) if z is None else _maybe_packed("z", z)
    if z is not None and (xs is None) != (zs is None):
        raise ValueError("x and z must both be checkpoints, or neither")
    p, B, T, D, G, N, S = _scan_sizes(xd, dtype, dt, A_log, Bm, Cm, skip, zd, z_dtype, dt_bias, cu_seqlens)
    _need("d_y", d_y)
    _fit((("d_y", d_y, (B, T, D), dtype), ("d_final_state", d_final_state, (S, D, N), f32),
          ("initial_state", initial_state, (S, D, N), f32)))
    index = _place(xd, (("dt", dt), ("Bm", Bm), ("Cm", Cm), ("z", zd)),
                   (("A_log", A_log), ("skip", skip), ("dt_bias", dt_bias), ("cu_seqlens", cu_seqlens),
                    ("initial_state", initial_state), ("d_y", d_y), ("d_final_state", d_final_state),
                    ("x.scales", xs), ("z.scales", zs)))
    ws_bytes = _lib().gdn_scan_bwd_workspace_size(p, int(cu_seqlens is not None))

    def body(s):
        empty, device = _torch().empty, xd.device
        new = lambda shape, dt_: empty(shape, dtype=dt_, device=device)  # noqa: E731
        g = dict(dx=_like(d_y), ddt=_like(d_y), dA_log=_like(A_log), dBm=_like(Bm), dCm=_like(Bm), dskip=new((D,), f32),
                 ddt_bias=new((D,), f32), dh0=new((S, D, N), f32))
        if z is not None:
            g["dz"] = _like(d_y)
        ws, ws_ptr, ws_size = _workspace(ws_bytes, index)
        _call("gdn_scan_bwd", p, xd.data_ptr(), _p(xs), dt.data_ptr(), A_log.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
              _p(skip), _p(zd), _p(zs), _p(dt_bias), _p(cu_seqlens), _p(initial_state), d_y.data_ptr(),
              _p(d_final_state), g["dx"].data_ptr(), g["ddt"].data_ptr(), g["dA_log"].data_ptr(), g["dBm"].data_ptr(),
              g["dCm"].data_ptr(), g["dskip"].data_ptr(), _p(g.get("dz")), g["ddt_bias"].data_ptr(),
              g["dh0"].data_ptr(), ws_ptr, ws_size, s)
        return g
    return _on(index, stream, (xd, xs, dt, A_log, Bm, Cm, d_y, d_final_state, skip, zd, zs, dt_bias, cu_seqlens,
                               initial_state), body)


def _scan_decode_args(x, dt, A_log, Bm, Cm, state, skip, z, dt_bias, new_state, out):
    f32 = _torch().float32
    p, B, T, D, G, N, _ = _scan_sizes(x, x.dtype, dt, A_log, Bm, Cm, skip, z, None if z is None else z.dtype,
                                      dt_bias, None)
    _need("state", state)
    _fit((("state", state, (B, D, N), f32), ("new_state", new_state, (B, D, N), f32), ("out", out, (B, T, D), x.dtype)))
    index = _place(x, (("dt", dt), ("Bm", Bm), ("Cm", Cm), ("z", z)),
                   (("A_log", A_log), ("skip", skip), ("dt_bias", dt_bias), ("state", state), ("new_state", new_state),
                    ("out", out)))

    def args(s):
        y = _like(x) if out is None else out
        new = state if new_state is None else new_state
        _lib()
        return (p, x.data_ptr(), dt.data_ptr(), A_log.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), _p(skip), _p(z),
                _p(dt_bias), state.data_ptr(), new.data_ptr(), y.data_ptr(), s), y, (
                    (new,) if out is None else (new, out))
    return index, args


def scan_decode_launcher(x, dt, A_log, Bm, Cm, state, skip=None, z=None, dt_bias=None, new_state=None, out=None,
                         stream=None):
    """Check and marshal gdn_scan_decode's arguments once; returns (launch, y), where
    launch() enqueues the scan of x's T tokens after `state` [B,D,N], writing the state
    after them to new_state (default: `state` itself).  The stream is as for
    conv_decode_launcher."""
    index, args = _scan_decode_args(x, dt, A_log, Bm, Cm, state, skip, z, dt_bias, new_state, out)
    keep = (x, dt, A_log, Bm, Cm, state, skip, z, dt_bias, new_state, out, stream)
    args, y, written = _on(index, stream, keep[:-1], args)
    return _launcher("gdn_scan_decode", index, args, keep + (y,), written), y


def scan_decode(x, dt, A_log, Bm, Cm, state, skip=None, z=None, dt_bias=None, new_state=None, out=None,
                stream=None):
    """T tokens (1: a decode step) of each of B sequences through gdn_scan_decode: returns
    y [B,T,D]; the state after them goes to new_state, or updates `state` in place."""
    index, args = _scan_decode_args(x, dt, A_log, Bm, Cm, state, skip, z, dt_bias, new_state, out)

    def body(s):
        a, y, written = args(s)
        _call("gdn_scan_decode", *a)
        _written(written)
        return y
    return _on(index, stream, (x, dt, A_log, Bm, Cm, state, skip, z, dt_bias, new_state, out), body)


# ---------------------------------------------------------------------------
# differentiable forms

def kept_bits(bits, *inputs):
    """checkpoint_bits, checked; None where no backward pass can follow, so that nothing is
    packed for one (a Function's forward cannot tell: gradients are off within it)."""
    if bits not in (None, 8):
        raise ValueError("checkpoint_bits must be None or 8, got %r" % (bits,))
    if bits is None:
        return None
    follows = _torch().is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs)
    return bits if follows else None


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
    bits = kept_bits(checkpoint_bits, x, weight, bias, initial_state)
    return _conv_function().apply(x, weight, bias, cu_seqlens, initial_state, activation, bits)


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
    bits = kept_bits(checkpoint_bits, x, dt, A_log, Bm, Cm, skip, z, dt_bias, initial_state)
    return _scan_function().apply(x, dt, A_log, Bm, Cm, skip, z, dt_bias, cu_seqlens, initial_state, bits)
