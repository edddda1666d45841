"""The norms around a block (gated_norm_fwd, gated_norm_bwd, residual_norm_fwd,
residual_norm_bwd and their differentiable forms) against their definitions in 64 bits: widths
off the vectors' and waves' sizes, single rows, gates on either side of the norm, residuals in
either type, missing options, extreme rows."""
import ctypes
import math

import pytest
import torch

import block_oracle as bo
import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
from gated_deltanet_chunkwise_amd._norms import GatedNormParams, ResidualNormParams

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def tol(dtype, n=0):
    """Half a step for the one rounding of the result, and fp32 arithmetic: a row's mean (its
    terms' roundings add in squares, and halve in the root), the exponential, reciprocal and
    root of the hardware (about an ulp each) and a dozen products; the weights' gradients are
    sums over n rows on top, whose roundings add in squares."""
    return (torch.finfo(dtype).eps / 2 if dtype == BF16 else 0) + (24 + math.sqrt(n)) * 2.0 ** -24


# B, T, H, D, dtype
SHAPES = [(1, 1, 1, 1, F32), (2, 3, 2, 7, BF16), (1, 5, 3, 64, BF16), (2, 33, 4, 128, BF16), (1, 17, 2, 128, F32),
          (1, 9, 5, 96, BF16), (1, 9, 5, 100, BF16), (1, 4, 3, 100, F32), (3, 2, 1, 256, BF16), (1, 6, 1, 500, BF16),
          (1, 5, 1, 1001, F32), (1, 3, 1, 2048, BF16), (1, 3, 1, 2050, BF16), (1, 2, 1, 4096, BF16), (1, 2, 1, 4097, BF16),
          (1, 2, 1, 4096, F32), (1, 2, 1, 8192, BF16), (1, 2, 1, 16384, F32), (1, 2, 1, 16384, BF16), (1, 1, 1, 16383, BF16),
          (4, 301, 8, 64, F32), (1, 0, 2, 64, BF16), (0, 3, 2, 64, F32)]
IDS = ["%dx%dx%dx%d-%s" % (*s[:4], str(s[4])[6:]) for s in SHAPES]


def norm(u, eps, held=False):
    """r(u); held: its factor taken for a constant, so that the gradient is c dn alone."""
    c = ((u ** 2).mean(-1, keepdim=True) + eps) ** -0.5
    return u * (c.detach() if held else c)


def gated(x, weight, z=None, *, eps, first, held=False):
    if z is None:
        return (norm(x, eps, held) * weight,)
    gate = z * torch.sigmoid(z)
    return (norm(x * gate, eps, held) * weight if first else norm(x, eps, held) * weight * gate,)


def gated_inputs(B, T, H, D, dtype, gate, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=(3 * r(B, T, H, D)).to(dtype), weight=1 + 0.1 * r(D), z=r(B, T, H, D).to(dtype) if gate != "none" else None)
    return d, r(B, T, H, D).to(dtype)


def check(got, f, d, seeds, rows):
    """The gradients of f.  That of a norm is the difference c dn - c n mean(n dn) of terms that
    fp32 rounds each, and in narrow rows (one channel above all, where n^2 is 1 but for eps) it
    is far smaller than they are: the error counts relative to c dn.  That bounds the other
    term too: |n mean(n dn)| <= |n|^2 |dn| / D <= |dn| over a row, as |n|^2 <= D."""
    leaves = lo.double(d)
    ref = lo.gradients(lambda **k: f(**k), leaves, seeds)
    size = lo.gradients(lambda **k: f(**k, held=True), leaves, seeds)
    assert set(got) == {"d" + k for k in ref}
    for k, t in got.items():
        bo.close(t, ref[k[1:]], tol(t.dtype, rows if t.dim() == 1 else 0), k, each=0.03 if t.dtype == BF16 else None,
                 size=size[k[1:]])


@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gated_norm(shape, gate):
    B, T, H, D, dtype = shape
    d, dy = gated_inputs(*shape, gate)
    c = lo.cuda(d)
    first, eps = gate == "first", 1e-5
    y = gdn.gated_norm_fwd(c["x"], c["weight"], c["z"], eps=eps, gate_first=first)
    f = lambda **k: gated(**k, eps=eps, first=first)  # noqa: E731
    bo.close(y, f(**lo.double(d))[0], tol(dtype), "y")
    got = gdn.gated_norm_bwd(c["x"], c["weight"], dy.cuda(), c["z"], eps=eps, gate_first=first)
    check(got, f, d, (dy.double(),), B * T * H)
    again = gdn.gated_norm_bwd(c["x"], c["weight"], dy.cuda(), c["z"], eps=eps, gate_first=first)
    assert all(torch.equal(got[k], again[k]) for k in got), "the same call gives the same bits"


def residual(x, residual, weight, post_weight=None, scale=None, *, eps, held=False):
    p = x if post_weight is None else norm(x, eps, held) * post_weight
    s = residual + (p if scale is None else scale * p)
    return norm(s, eps, held) * weight, s


def residual_inputs(B, T, C, dtype, res, post, scale, seed=2):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=r(B, T, C).to(dtype), residual=(2 * r(B, T, C)).to(res), weight=1 + 0.1 * r(C),
             post_weight=1 + 0.1 * r(C) if post else None, scale=0.5 + 0.1 * r(C) if scale else None)
    return d, (r(B, T, C).to(dtype), r(B, T, C).to(res))


RESIDUAL = [(s[0], s[1] * s[2], s[3], s[4], res) for s in SHAPES for res in ((BF16, F32) if s[4] == BF16 else (F32,))]


@pytest.mark.parametrize("post,scale", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("shape", RESIDUAL, ids=lambda s: "%dx%dx%d-%s-%s" % (*s[:3], str(s[3])[6:], str(s[4])[6:]))
def test_residual_norm(shape, post, scale):
    B, T, C, dtype, res = shape
    d, seeds = residual_inputs(*shape, post, scale)
    c, eps = lo.cuda(d), 1e-5
    f = lambda **k: residual(**k, eps=eps)  # noqa: E731
    h_ref, s_ref = f(**lo.double(d))
    args = (c["x"], c["residual"], c["weight"])
    opts = dict(post_weight=c["post_weight"], scale=c["scale"], eps=eps)
    h, s = gdn.residual_norm_fwd(*args, **opts)
    assert s.dtype == res
    bo.close(h, h_ref, tol(dtype), "h")
    bo.close(s, s_ref, tol(res), "new residual")
    got = gdn.residual_norm_bwd(*args, seeds[0].cuda(), seeds[1].cuda(), **opts)
    check(got, f, d, [v.double() for v in seeds], B * T)
    again = gdn.residual_norm_bwd(*args, seeds[0].cuda(), seeds[1].cuda(), **opts)
    assert all(torch.equal(got[k], again[k]) for k in got), "the same call gives the same bits"
    # no gradient towards the new residual
    got = gdn.residual_norm_bwd(*args, seeds[0].cuda(), None, **opts)
    check(got, f, d, (seeds[0].double(), None), B * T)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slices_of_wider_tensors(dtype):
    B, T, H, D = 2, 19, 4, 64
    d, dy = gated_inputs(B, T, H, D, dtype, "after")
    c, dy = lo.cuda(d), dy.cuda()
    for off in (0, 8, 3):  # aligned for wide loads, and not
        wide = torch.full((B, T, 2 * H * D + off + 5), float("nan"), dtype=dtype, device="cuda")
        xs, zs = wide[..., off:off + H * D].unflatten(-1, (H, D)), wide[..., off + H * D:off + 2 * H * D].unflatten(-1, (H, D))
        xs.copy_(c["x"])
        zs.copy_(c["z"])
        for first in (False, True):
            y = gdn.gated_norm_fwd(xs, c["weight"], zs, gate_first=first)
            bo.close(y, gated(**lo.double(d), eps=1e-6, first=first)[0], tol(dtype), "y")
            g, g2 = (gdn.gated_norm_bwd(x, c["weight"], dy, z, gate_first=first) for x, z in ((xs, zs), (c["x"], c["z"])))
            for k in g:
                bo.close(g[k], g2[k].cpu().double(), 2 * tol(dtype), k)
    d, seeds = residual_inputs(B, T, 200, dtype, F32, True, True)
    c = lo.cuda(d)
    wide = torch.full((B, T, 500), float("nan"), dtype=dtype, device="cuda")
    res = torch.full((B, T, 333), float("nan"), device="cuda")
    wide[..., 7:207], res[..., 100:300] = c["x"], c["residual"]
    h, s = gdn.residual_norm_fwd(wide[..., 7:207], res[..., 100:300], c["weight"], c["post_weight"], c["scale"])
    ref = residual(**lo.double(d), eps=1e-6)
    bo.close(h, ref[0], tol(dtype), "h")
    bo.close(s, ref[1], tol(F32), "new residual")


def test_three_dimensions_are_one_head():
    d, dy = gated_inputs(2, 5, 1, 200, BF16, "after")
    c = lo.cuda(d)
    flat = {k: v[:, :, 0] if v.dim() == 4 else v for k, v in c.items()}
    assert torch.equal(gdn.gated_norm_fwd(flat["x"], flat["weight"], flat["z"]), gdn.gated_norm_fwd(c["x"], c["weight"], c["z"])[:, :, 0])
    a = gdn.gated_norm_bwd(flat["x"], flat["weight"], dy[:, :, 0].cuda(), flat["z"])
    b = gdn.gated_norm_bwd(c["x"], c["weight"], dy.cuda(), c["z"])
    assert all(torch.equal(a[k].flatten(), b[k].flatten()) for k in a)


def test_rows_do_not_see_each_other():
    for D in (64, 128, 2048, 4096):
        d, dy = gated_inputs(1, 6, 3, D, BF16, "after")
        c = lo.cuda(d)
        y = gdn.gated_norm_fwd(c["x"], c["weight"], c["z"])
        c["x"][0, 2, 1], c["z"][0, 4, 0] = float("nan"), float("inf")
        y2 = gdn.gated_norm_fwd(c["x"], c["weight"], c["z"])
        same = torch.ones(6, 3, dtype=torch.bool)
        same[2, 1] = same[4, 0] = False
        assert torch.equal(y[0][same], y2[0][same]) and y2[0, 2, 1].isnan().all()


def test_rows_of_zeros_and_extreme_gates():
    x = torch.zeros(1, 3, 1, 64, device="cuda")
    x[0, 1] = 1e-30
    w = torch.ones(64, device="cuda")
    z = torch.full_like(x, -200.0)
    z[0, 2] = 200.0
    for first in (False, True):
        y = gdn.gated_norm_fwd(x, w, z, gate_first=first)
        assert (y == 0).sum() >= 128 and y.isfinite().all()
        g = gdn.gated_norm_bwd(x, w, torch.ones_like(x), z, gate_first=first)
        assert all(t.isfinite().all() for t in g.values())


def test_the_residual_in_place():
    """Through the C entry: new_residual may be the residual itself."""
    d, _ = residual_inputs(2, 9, 512, BF16, F32, True, True)
    c = lo.cuda(d)
    h, s = gdn.residual_norm_fwd(c["x"], c["residual"], c["weight"], c["post_weight"], c["scale"])
    r, h2 = c["residual"].clone(), torch.empty_like(c["x"])
    p = ResidualNormParams(2, 9, 512, gdn.GDN_BF16, gdn.GDN_F32, 1e-6, 0, 0)
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = gdn.load_library().gdn_residual_norm_fwd(ctypes.byref(p), P(c["x"]), P(r), P(c["weight"]), P(c["post_weight"]), P(c["scale"]),
                                                  P(h2), P(r), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0 and torch.equal(h, h2) and torch.equal(r, s)


@pytest.mark.parametrize("D", [1, 7, 64, 100, 1001, 2050, 4097])
def test_nothing_is_written_outside(D):
    """Guard bands around every output, a workspace of NaN."""
    lib = gdn.load_library()
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    held = []

    def out(n, dtype):
        t = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
        held.append((t, n))
        return t[256:256 + n]
    d, dy = gated_inputs(1, 5, 3, D, BF16, "after")
    c, dy = lo.cuda(d), dy.cuda()
    p = GatedNormParams(1, 5, 3, D, gdn.GDN_BF16, 0, 1e-6, 0, 0)
    nb = lib.gdn_gated_norm_bwd_workspace_size(ctypes.byref(p))
    ws = torch.full((nb + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    n = 15 * D
    y, dx, dz, dw = out(n, BF16), out(n, BF16), out(n, BF16), out(D, F32)
    assert lib.gdn_gated_norm_fwd(ctypes.byref(p), P(c["x"]), P(c["weight"]), P(c["z"]), P(y), stream) == 0
    assert lib.gdn_gated_norm_bwd(ctypes.byref(p), P(c["x"]), P(c["weight"]), P(c["z"]), P(dy), P(dx), P(dz), P(dw), P(ws), nb, stream) == 0
    assert (ws[nb:] == 0xFF).all()
    g = gdn.gated_norm_bwd(c["x"], c["weight"], dy, c["z"])
    assert torch.equal(dx.view(g["dx"].shape), g["dx"]) and torch.equal(dw, g["dweight"])
    d, seeds = residual_inputs(1, 15, D, BF16, F32, True, True)
    c, seeds = lo.cuda(d), [t.cuda() for t in seeds]
    p = ResidualNormParams(1, 15, D, gdn.GDN_BF16, gdn.GDN_F32, 1e-6, 0, 0)
    nb = lib.gdn_residual_norm_bwd_workspace_size(ctypes.byref(p))
    ws = torch.full((nb + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    h, s, dx, dr = out(n, BF16), out(n, F32), out(n, BF16), out(n, F32)
    dw, dp, ds = out(D, F32), out(D, F32), out(D, F32)
    args = [P(c[k]) for k in ("x", "residual", "weight", "post_weight", "scale")]
    assert lib.gdn_residual_norm_fwd(ctypes.byref(p), *args, P(h), P(s), stream) == 0
    assert lib.gdn_residual_norm_bwd(ctypes.byref(p), *args, P(seeds[0]), P(seeds[1]), P(dx), P(dr), P(dw), P(dp), P(ds), P(ws), nb, stream) == 0
    assert (ws[nb:] == 0xFF).all()
    for t, n in held:
        assert (t[:256] == 7).all() and (t[256 + n:] == 7).all() and t[256:256 + n].isfinite().all()
