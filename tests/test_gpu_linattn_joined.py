"""Linear attention in so many segments that their starts are joined by a launch of their own, in
every width and both types, with shared heads: against the 64-bit form, through the C entries with
a workspace of NaN.  Packed, with sequences of one segment and of none among longer ones."""
import ctypes

import pytest
import torch

import block_oracle as bo
import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
from gated_deltanet_chunkwise_amd._linattn import LinattnParams
from test_gpu_layer_runs import Banded, P, run
from test_gpu_linattn import BF16, F32, rows_tol, state_tol

pytestmark = pytest.mark.gpu
MOST = 8  # segments of a sequence that sum their starts themselves
LENGTHS = [5, 0, 64, 1, 700, 3, 0, 0, 65, 64, 20, 420, 0, 7, 128, 0]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_joined_segments(K, V, dtype, packed):
    T, H, HV = 1500, 1, 2
    N = len(LENGTHS) if packed else 1
    cu = lo.offsets(LENGTHS) if packed else None
    used = int(cu[-1]) if packed else T
    d, seeds, ld = bo.linattn_inputs(1, T, H, HV, K, V, dtype, 41, N)
    scale = K ** -0.5

    def form(**x):
        return bo.linattn(log_decay=ld.double(), cu=cu, scale=scale, **x)
    lib, new = gdn.load_library(), Banded()
    code = gdn.GDN_BF16 if dtype == BF16 else gdn.GDN_F32
    p = LinattnParams(1, T, H, HV, K, V, N if packed else 0, code | (0x100 if packed else 0), scale, 0, 0, 0)

    def space(size, kinds, more):
        nb = size(ctypes.byref(p), int(packed))
        least = MOST + 1 + (min(N, MOST + 1) if packed else 0)
        assert nb - more >= kinds * least * HV * K * V * 4, "more segments than sum their own starts"
        return P(new((nb,), torch.uint8, 256 - 4096 % 256).fill_(0xFF)), nb
    g, s, ldc, cuc = lo.cuda(d), lo.cuda(seeds), ld.cuda(), None if cu is None else cu.cuda()
    ins = [P(t) for t in (g["q"], g["k"], g["v"], ldc, cuc, g["h0"])]
    o, fin = new((1, T, HV, V), dtype), new((N, HV, K, V), F32)
    run("gdn_linattn_fwd", ctypes.byref(p), *ins, P(o), P(fin), *space(lib.gdn_linattn_fwd_workspace_size, 1, 0))
    dq, dk = new((1, T, H, K), dtype), new((1, T, H, K), dtype)
    dv, dh0 = new((1, T, HV, V), dtype), new((N, HV, K, V), F32)
    run("gdn_linattn_bwd", ctypes.byref(p), *ins, P(s["d_o"]), P(s["d_fin"]), P(dq), P(dk), P(dv), P(dh0),
        *space(lib.gdn_linattn_bwd_workspace_size, 2, 2 * T * HV * K * 4))
    assert new.untouched()
    o_ref, fin_ref = form(**lo.double(d))
    bo.close(o, o_ref, rows_tol(dtype, T), "o")
    bo.close(fin, fin_ref, state_tol(T), "final state")
    rows = (torch.arange(T) < used).view(1, T, 1, 1)
    ref = lo.gradients(form, lo.double(d), (torch.where(rows, seeds["d_o"].double(), 0.0), seeds["d_fin"].double()))
    for name, t, of in (("dq", dq, "q"), ("dk", dk, "k"), ("dv", dv, "v")):
        bo.close(t, ref[of], rows_tol(dtype, T), name)
    bo.close(dh0, ref["h0"], state_tol(T), "dh0")
    for t in (o, dq, dk, dv):
        assert (t[0, used:] == 0).all()
    for n in (i for i, length in enumerate(LENGTHS) if packed and length == 0):
        assert torch.equal(fin[n], g["h0"][n]) and torch.equal(dh0[n], s["d_fin"][n])


def test_the_same_sequences_alone():
    """Short sequences, packed in one row that is cut into many segments, and each in a call of
    its own (a batch): the same bits, with no segments of several in either."""
    n, T = 300, 64
    d, seeds, ld = bo.linattn_inputs(n, T, 1, 2, 64, 64, BF16, 42)
    g, s, ldc = lo.cuda(d), lo.cuda(seeds), ld.cuda()
    cu = (T * torch.arange(n + 1)).cuda()
    row = lambda t: t.reshape(1, n * T, *t.shape[2:])  # noqa: E731
    a = gdn.linear_attn_fwd(row(g["q"]), row(g["k"]), row(g["v"]), ldc, cu, g["h0"])
    b = gdn.linear_attn_fwd(g["q"], g["k"], g["v"], ldc, None, g["h0"])
    assert torch.equal(a[0], row(b[0])) and torch.equal(a[1], b[1])
    a = gdn.linear_attn_bwd(row(g["q"]), row(g["k"]), row(g["v"]), ldc, row(s["d_o"]), s["d_fin"], cu, g["h0"])
    b = gdn.linear_attn_bwd(g["q"], g["k"], g["v"], ldc, s["d_o"], s["d_fin"], None, g["h0"])
    assert torch.equal(a["dh0"], b["dh0"]) and all(torch.equal(a[k], row(b[k])) for k in ("dq", "dk", "dv"))


@pytest.mark.parametrize("K,V", [(64, 64), (128, 64)])
def test_a_captured_call_under_other_offsets(K, V):
    """Segments, their states' places and which sequences have several follow from the offsets on the
    device: a captured forward and backward pass is replayed under offsets of other lengths."""
    T, N = 1500, 12
    d, seeds, ld = bo.linattn_inputs(1, T, 1, 2, K, V, BF16, 43, N)
    g, s, ldc = lo.cuda(d), lo.cuda(seeds), ld.cuda()

    def passes(cu):
        o, fin = gdn.linear_attn_fwd(g["q"], g["k"], g["v"], ldc, cu, g["h0"])
        return [o, fin, *gdn.linear_attn_bwd(g["q"], g["k"], g["v"], ldc, s["d_o"], s["d_fin"], cu, g["h0"]).values()]
    kinds = [[125] * 12, [1500] + [0] * 11, [0] * 11 + [1500], [64] * 12, [1, 0, 700, 0, 0, 65, 63, 64, 600, 0, 2, 0], [0] * 12]
    cu = lo.offsets(kinds[0]).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        passes(cu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = passes(cu)
    for lengths in kinds + kinds[::-1]:
        cu.copy_(lo.offsets(lengths))
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        want = passes(cu.clone())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), lengths
        assert all(t.isfinite().all() for t in out)
