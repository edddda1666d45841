"""The norms' gradients without an eps, and with one below fp32's normal numbers: the rows of a
workgroup behind the last one, which hold nothing, stay out of the weights' gradients."""
import pytest
import torch

import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
from test_gpu_norms import BF16, F32, check, gated, gated_inputs, residual, residual_inputs

pytestmark = pytest.mark.gpu
ROWS, WIDTHS = [1, 15, 17, 33], [2, 64, 65, 128, 512, 1024]


@pytest.mark.parametrize("eps", [0.0, 1e-42])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("rows", ROWS)
def test_gated_norm_without_eps(rows, D, dtype, eps):
    for gate in ("none", "after", "first"):
        d, dy = gated_inputs(1, rows, 1, D, dtype, gate, 5)
        c, first = lo.cuda(d), gate == "first"
        got = gdn.gated_norm_bwd(c["x"], c["weight"], dy.cuda(), c["z"], eps=eps, gate_first=first)
        check(got, lambda **k: gated(**k, eps=eps, first=first), d, (dy.double(),), rows)


@pytest.mark.parametrize("eps", [0.0, 1e-42])
@pytest.mark.parametrize("dtype,res", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("rows", ROWS)
def test_residual_norm_without_eps(rows, C, dtype, res, eps):
    for post, scale in ((True, True), (False, False), (True, False), (False, True)):
        d, seeds = residual_inputs(1, rows, C, dtype, res, post, scale, 6)
        c = lo.cuda(d)
        got = gdn.residual_norm_bwd(c["x"], c["residual"], c["weight"], seeds[0].cuda(), seeds[1].cuda(),
                                    post_weight=c["post_weight"], scale=c["scale"], eps=eps)
        check(got, lambda **k: residual(**k, eps=eps), d, [v.double() for v in seeds], rows)
