"""8-bit activation checkpoints: codes and scales bit for bit against layer_oracle, over
zeros, denormal and largest values, infinities and NaN, odd channel counts and strides;
and their use in gated_delta_rule's backward pass."""
import pytest
import torch

import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
from gated_deltanet_chunkwise_amd.inputs import make_grads, make_inputs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def values(rows, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, C, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g).float())).to(dtype)


def check(x):
    codes, scales = lo.pack(x.cpu())
    p = gdn.pack8(x)
    assert p.dtype == x.dtype
    assert torch.equal(p.codes.cpu(), codes) and torch.equal(p.scales.cpu(), scales)
    back, ref = gdn.unpack8(p), lo.unpack(codes, scales).to(x.dtype)
    assert torch.equal(back.isnan().cpu(), ref.isnan())
    assert torch.equal(back.cpu().nan_to_num(), ref.nan_to_num())
    return p


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,C", [(1, 1), (3, 7), (5, 32), (2, 33), (9, 64), (4, 40), (7, 100), (1, 1000), (33, 128)])
def test_codes_and_scales(rows, C, dtype):
    check(values(rows, C, dtype, rows + C).cuda())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C", [8, 9, 10, 12, 15, 23, 31, 39, 63, 65, 1001])
def test_rows_that_end_inside_a_lane(C, dtype):
    for rows in (1, 2, 300):
        check(values(rows, C, dtype, rows + C).cuda())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_any_address(dtype):
    """Rows, codes and scales at addresses that only their elements are aligned to."""
    wide = values(9, 101, dtype, 3).cuda()
    x = wide[:, 1:42]
    p = gdn.pack8(x)
    q = gdn.pack8(x.contiguous())
    assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    odd = torch.empty(9 * 41 + 1, dtype=torch.int8, device="cuda")[1:].view(9, 41).copy_(p.codes)
    out = torch.empty(9 * 41 + 1, dtype=dtype, device="cuda")[1:].view(9, 41)
    assert torch.equal(gdn.unpack8(gdn.Packed8(odd, p.scales, dtype), out=out), gdn.unpack8(q))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_where_the_scale_changes(dtype):
    # the block's maximum at and next to 127 s, ties between two codes, zeros
    x = torch.zeros(8, 32)
    x[0, 3], x[1, 3], x[2, 3] = 127.0, 127.5, 126.5
    x[3, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])   # ties to even
    x[4, :2] = torch.tensor([-254.0, 1.0])
    x[5, 0], x[6, 0] = 2.0 ** -20, -2.0 ** 20
    check(x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_extreme_values(dtype):
    x = torch.ones(8, 64)
    big = torch.finfo(dtype).max
    x[0, 5], x[1, 5], x[2, 40] = float("inf"), float("nan"), -float("inf")
    x[3, 0], x[4, 0] = big, -big
    x[5] = 2.0 ** -126
    x[6] = 2.0 ** -120
    x[7] = 0
    p = check(x.to(dtype).cuda())
    back = gdn.unpack8(p)
    assert back[0, :32].isnan().all() and not back[0, 32:].isnan().any()
    assert torch.isfinite(back[3:5]).all(), "the largest values stay finite"


def test_strided_rows_and_leading_dimensions():
    wide = values(24, 96, BF16, 3).cuda().view(2, 3, 4, 96)
    for x in (wide[..., 32:96], wide[..., 5:50], wide[:, :, 0], wide[0, :, 1]):
        check_like = x.contiguous()
        a, b = gdn.pack8(x), gdn.pack8(check_like)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    with pytest.raises(ValueError):
        gdn.pack8(wide.transpose(0, 1))
    with pytest.raises(ValueError):
        gdn.pack8(wide.transpose(-1, -2))


def test_empty():
    p = gdn.pack8(torch.empty(0, 64, dtype=BF16, device="cuda"))
    assert p.codes.shape == (0, 64) and gdn.unpack8(p).shape == (0, 64)


def test_rows_further_apart_than_32_bits_reach():
    ld, rows, C = 1 << 26, 40, 64
    big = torch.empty(rows * ld, dtype=BF16, device="cuda")
    x = big.as_strided((rows, C), (ld, 1))
    v = values(rows, C, BF16, 4).cuda()
    x.copy_(v)
    a, b = gdn.pack8(x), gdn.pack8(v)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


def test_graph_replay_and_other_stream():
    x = values(64, 128, BF16, 5).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = gdn.pack8(x, stream=side), gdn.pack8(x)
    side.synchronize()
    assert torch.equal(a.codes, b.codes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdn.unpack8(gdn.pack8(x))
    for i in range(3):
        x.copy_(values(64, 128, BF16, 6 + i))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, gdn.unpack8(gdn.pack8(x)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gated_delta_rule_from_checkpoints(dtype):
    """Its gradients are gdn_bwd's at the values the checkpoints stand for."""
    inp = make_inputs(B=1, T=130, H=2, HV=4, K=64, V=64, dtype=dtype, seed=11, h0=True)
    d_o, d_fin = make_grads(inp, 12)
    d, d_o, d_fin = inp.to("cuda"), d_o.cuda(), d_fin.cuda()
    leaf = [t.detach().clone().requires_grad_() for t in (d.q, d.k, d.v, d.g_raw, d.beta, d.A_log, d.dt_bias, d.h0)]
    o, fin = gdn.gated_delta_rule(*leaf[:7], initial_state=leaf[7], checkpoint_bits=8)
    o2, fin2 = gdn.fwd(d.q, d.k, d.v, d.g_raw, d.beta, d.A_log, d.dt_bias, initial_state=d.h0)
    assert torch.equal(o, o2) and torch.equal(fin, fin2), "the forward pass is at the inputs themselves"
    got = torch.autograd.grad((o, fin), leaf, (d_o, d_fin))
    through = [gdn.unpack8(gdn.pack8(t)) for t in (d.q, d.k, d.v)]
    ref = gdn.bwd(*through, d.g_raw, d.beta, d.A_log, d.dt_bias, d_o, d_fin, initial_state=d.h0)
    # the same kernels on the same values; their LDS atomics may change low bits (gdn.h)
    for name, g, r in zip(("dq", "dk", "dv", "dg_raw", "dbeta", "dA_log", "ddt_bias", "dh0"), got, ref.values()):
        r = r.double()
        assert float((g.double() - r).norm()) <= 1e-3 * float(r.norm()), name
