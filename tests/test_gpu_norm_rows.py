"""The norms around a block at widths on both sides of every number of lanes and vectors that a
row takes, at addresses of one element's alignment: against the definitions in 64 bits, and
nothing outside the outputs is written (a gate's, a residual's and the weights' gradients, and
the workspace, among them)."""
import ctypes

import pytest
import torch

import block_oracle as bo
import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
from gated_deltanet_chunkwise_amd._norms import GatedNormParams, ResidualNormParams
from test_gpu_layer_runs import Banded, P, run
from test_gpu_norms import BF16, F32, check, gated, gated_inputs, residual, residual_inputs, tol

pytestmark = pytest.mark.gpu
WIDTHS = [3, 4, 5, 8, 9, 31, 33, 63, 65, 127, 129, 255, 257, 511, 513, 1023, 1025, 2047, 2049, 2051, 4095, 4099, 8190, 8193, 16381]
CODE = {BF16: gdn.GDN_BF16, F32: gdn.GDN_F32}


def banded(new, t, dtype=None):
    """t in a banded allocation, one element off the 16 bytes' alignment."""
    dtype = dtype or t.dtype
    return new(t.shape, dtype, torch.empty((), dtype=dtype).element_size()).copy_(t)


def space(new, size, p):
    nb = size(ctypes.byref(p))
    return P(new((nb,), torch.uint8).fill_(0xFF)) if nb else None, nb


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", WIDTHS)
def test_gated_norm_rows(D, dtype):
    T, H, lib, new = 7, 3, gdn.load_library(), Banded()
    d, dy = gated_inputs(1, T, H, D, dtype, "after")
    x, w, z, g = (banded(new, t) for t in (d["x"], d["weight"], d["z"], dy))
    y, dx, dz, dw = (banded(new, torch.zeros_like(t)) for t in (d["x"], d["x"], d["x"], d["weight"]))
    p = GatedNormParams(1, T, H, D, CODE[dtype], 0, 1e-5, 0, 0)
    run("gdn_gated_norm_fwd", ctypes.byref(p), P(x), P(w), P(z), P(y))
    run("gdn_gated_norm_bwd", ctypes.byref(p), P(x), P(w), P(z), P(g), P(dx), P(dz), P(dw),
        *space(new, lib.gdn_gated_norm_bwd_workspace_size, p))
    assert new.untouched()
    f = lambda **k: gated(**k, eps=1e-5, first=False)  # noqa: E731
    bo.close(y, f(**lo.double(d))[0], tol(dtype), "y")
    check(dict(dx=dx, dweight=dw, dz=dz), f, d, (dy.double(),), T * H)


@pytest.mark.parametrize("dtype,res", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("C", WIDTHS)
def test_residual_norm_rows(C, dtype, res):
    T, lib, new = 11, gdn.load_library(), Banded()
    d, seeds = residual_inputs(1, T, C, dtype, res, True, True)
    x, r, w, post, scale = (banded(new, d[n]) for n in ("x", "residual", "weight", "post_weight", "scale"))
    h, dx, s, dr = (banded(new, torch.zeros_like(d[n])) for n in ("x", "x", "residual", "residual"))
    dw, dp, dsc = (banded(new, torch.zeros_like(d["weight"])) for _ in range(3))
    p = ResidualNormParams(1, T, C, CODE[dtype], CODE[res], 1e-5, 0, 0)
    run("gdn_residual_norm_fwd", ctypes.byref(p), P(x), P(r), P(w), P(post), P(scale), P(h), P(s))
    run("gdn_residual_norm_bwd", ctypes.byref(p), P(x), P(r), P(w), P(post), P(scale), P(banded(new, seeds[0])), P(banded(new, seeds[1])),
        P(dx), P(dr), P(dw), P(dp), P(dsc), *space(new, lib.gdn_residual_norm_bwd_workspace_size, p))
    f = lambda **k: residual(**k, eps=1e-5)  # noqa: E731
    h_ref, s_ref = f(**lo.double(d))
    bo.close(h, h_ref, tol(dtype), "h")
    bo.close(s, s_ref, tol(res), "new residual")
    check(dict(dx=dx, dresidual=dr, dweight=dw, dpost_weight=dp, dscale=dsc), f, d, [v.double() for v in seeds], T)
    # in place: the new residual over the old one
    run("gdn_residual_norm_fwd", ctypes.byref(p), P(x), P(r), P(w), P(post), P(scale), P(h), P(r))
    assert torch.equal(r, s) and new.untouched()
