"""Short causal convolution (conv_fwd, conv_bwd, conv_decode, causal_conv) against the
64-bit form of layer_oracle, at the sizes where it can go wrong: single tokens, sequences
shorter than the window, empty ones, channel counts off the vector width, strided rows,
offsets that end before the batch does."""
import pytest
import torch

import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# B, T, C, W, dtype, silu, lengths, initial state, bias
CASES = [
    (1, 1, 8, 4, BF16, True, None, False, False),
    (3, 2, 72, 4, BF16, True, None, True, True),
    (2, 9, 40, 3, F32, False, None, True, False),
    (2, 65, 64, 2, BF16, False, None, False, True),
    (1, 33, 7, 4, F32, True, None, True, True),
    (1, 300, 1000, 3, BF16, True, None, True, True),
    (2, 130, 520, 4, BF16, True, None, True, True),
    (1, 40, 64, 4, BF16, True, [1, 0, 2, 3, 0, 30, 4], True, True),
    (1, 200, 24, 4, F32, True, [0, 5, 1, 130, 64], True, True),
    (1, 77, 33, 2, BF16, True, [70, 7, 0], False, True),
    (1, 50, 64, 4, BF16, True, [20, 13], True, True),      # ends before T
    (1, 0, 16, 4, F32, True, [0, 0], True, True),          # no tokens at all
]
IDS = ["%dx%dx%d-w%d-%s%s" % (c[0], c[1], c[2], c[3], str(c[4])[6:], "" if c[6] is None else "-packed") for c in CASES]


def make(case, seed=1):
    B, T, C, W, dtype, silu, lengths, h0, bias = case
    cu = None if lengths is None else lo.offsets(lengths)
    S = B if cu is None else len(lengths)
    d, seeds = lo.conv_inputs(B, T, C, W, dtype, seed, S, h0, bias)
    used = B * T if cu is None else int(cu[-1])
    return d, seeds, cu, ("silu" if silu else None), used


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    d, _, cu, act, used = make(case)
    r, g = lo.double(d), lo.cuda(d)
    y_ref, fin_ref = lo.conv(cu=cu, silu=act is not None, **r)
    y, fin = gdn.conv_fwd(g["x"], g["weight"], g["bias"], None if cu is None else cu.cuda(), g["h0"], act)
    T, C = y.shape[1:]
    lo.close(y.view(-1, C)[:used], y_ref.view(-1, C)[:used], case[3], "y")
    assert torch.equal(fin.cpu().to(torch.float64), fin_ref), "the final state is a copy of inputs"


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    d, seeds, cu, act, used = make(case, 2)
    r, g, s = lo.double(d), lo.cuda(d), lo.cuda(seeds)
    if cu is not None:  # rows behind the last sequence have no output
        seeds = dict(seeds, d_y=torch.where(torch.arange(d["x"].shape[1])[:, None] < used, seeds["d_y"], torch.tensor(0., dtype=seeds["d_y"].dtype)))
    ref = lo.gradients(lambda **k: lo.conv(cu=cu, silu=act is not None, **k), r,
                       (seeds["d_y"].double(), seeds["d_fin"].double()))
    got = gdn.conv_bwd(g["x"], g["weight"], g["bias"], s["d_y"], s["d_fin"], None if cu is None else cu.cuda(),
                       g["h0"], act)
    n = case[0] * case[1]
    lo.close(got["dx"], ref["x"], case[3], "dx")
    lo.close(got["dweight"], ref["weight"], n, "dweight")
    if d["bias"] is not None:
        lo.close(got["dbias"], ref["bias"], n, "dbias")
    if d["h0"] is not None:
        lo.close(got["dh0"], ref["h0"], case[3], "dh0")
    again = gdn.conv_bwd(g["x"], g["weight"], g["bias"], s["d_y"], s["d_fin"], None if cu is None else cu.cuda(),
                         g["h0"], act)
    assert all(torch.equal(got[k], again[k]) for k in got), "the same call gives the same bits"


@pytest.mark.parametrize("case", [
    (1, 2600, 4096, 4, BF16, True, [1000, 0, 3, 1590], True, True),
    (2, 800, 4099, 3, F32, True, None, True, True)], ids=["packed", "odd"])
def test_tiles_of_several_groups(case):
    """Enough channels that a lane's tile is longer than one group of loads, in both passes."""
    test_forward(case)
    test_backward(case)


def test_rows_behind_the_last_sequence_stay():
    d, seeds, cu, act, used = make(CASES[10])
    g, s = lo.cuda(d), lo.cuda(seeds)
    lib = gdn.load_library()
    import ctypes
    from gated_deltanet_chunkwise_amd._layers import ConvParams
    B, T, C = g["x"].shape
    y = torch.full((B, T, C), 7.0, dtype=BF16, device="cuda")
    p = ConvParams(B, T, C, 4, 2, gdn.GDN_BF16, 1, 0)
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    c = cu.cuda()
    st = lib.gdn_conv_fwd(ctypes.byref(p), P(g["x"]), P(g["weight"]), P(g["bias"]), P(c), P(g["h0"]), P(y), None,
                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    assert (y[0, used:] == 7).all() and not (y[0, :used] == 7).all()
    got = gdn.conv_bwd(g["x"], g["weight"], g["bias"], s["d_y"], s["d_fin"], c, g["h0"], act)
    assert (got["dx"][0, used:] == 0).all()


@pytest.mark.parametrize("dtype,C,pad", [(BF16, 64, 64), (BF16, 64, 3), (F32, 20, 4), (F32, 20, 1)])
def test_slices_of_a_wider_tensor(dtype, C, pad):
    d, seeds = lo.conv_inputs(2, 37, C, 4, dtype, 3)
    wide = torch.full((2, 37, C + 2 * pad), float("nan"), dtype=dtype, device="cuda")
    x = wide[..., pad:pad + C]
    x.copy_(d["x"])
    g, s = lo.cuda(d), lo.cuda(seeds)
    y, fin = gdn.conv_fwd(x, g["weight"], g["bias"], initial_state=g["h0"])
    y2, fin2 = gdn.conv_fwd(g["x"], g["weight"], g["bias"], initial_state=g["h0"])
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    a = gdn.conv_bwd(x, g["weight"], g["bias"], s["d_y"], s["d_fin"], initial_state=g["h0"])
    b = gdn.conv_bwd(g["x"], g["weight"], g["bias"], s["d_y"], s["d_fin"], initial_state=g["h0"])
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dh0"], b["dh0"])
    for k in ("dweight", "dbias"):  # other tiles, other order of the fp32 sums
        lo.close(a[k], b[k].cpu().double(), 74, k)


def test_rows_further_apart_than_32_bits_reach():
    # 40 tokens 2^26 elements apart: the last starts at element 2.6e9
    ld, T, C = 1 << 26, 40, 16
    big = torch.empty(T * ld, dtype=BF16, device="cuda")
    x = big.as_strided((1, T, C), (T * ld, ld, 1))
    d, _ = lo.conv_inputs(1, T, C, 4, BF16, 4)
    x.copy_(d["x"])
    g = lo.cuda(d)
    y, _ = gdn.conv_fwd(x, g["weight"], g["bias"], initial_state=g["h0"])
    y2, _ = gdn.conv_fwd(g["x"], g["weight"], g["bias"], initial_state=g["h0"])
    assert torch.equal(y, y2)


@pytest.mark.parametrize("B,T,C,W,dtype,inplace", [
    (1, 1, 8, 2, BF16, True), (5, 1, 72, 4, BF16, False), (3, 2, 33, 3, F32, True), (2, 7, 64, 4, F32, False)])
def test_decode_continues_a_prompt(B, T, C, W, dtype, inplace):
    d, _ = lo.conv_inputs(B, 11 + T, C, W, dtype, 5)
    g = lo.cuda(d)
    cut = lambda a, b: g["x"][:, a:b] if b - a == 1 else g["x"][:, a:b].contiguous()  # noqa: E731
    y_all, fin_all = gdn.conv_fwd(g["x"], g["weight"], g["bias"], initial_state=g["h0"])
    _, state = gdn.conv_fwd(cut(0, 11), g["weight"], g["bias"], initial_state=g["h0"])
    keep = state.clone()
    new = None if inplace else torch.full_like(state, float("nan"))
    y = gdn.conv_decode(cut(11, 11 + T), g["weight"], state, g["bias"], new_state=new)
    assert torch.equal(y, y_all[:, 11:]), "the same sums in the same order"
    assert torch.equal(state if inplace else new, fin_all)
    if not inplace:
        assert torch.equal(state, keep)


def test_decode_of_no_tokens_copies_the_state():
    d, _ = lo.conv_inputs(2, 1, 16, 4, BF16, 6)
    g = lo.cuda(d)
    new = torch.full_like(g["h0"], float("nan"))
    gdn.conv_decode(g["x"][:, :0], g["weight"], g["h0"], new_state=new)
    assert torch.equal(new, g["h0"])


def test_a_sequence_does_not_see_its_neighbours():
    d, seeds, cu, act, used = make((1, 40, 64, 4, BF16, True, [10, 20, 10], True, True))
    clean = gdn.conv_fwd(*(t.cuda() for t in (d["x"], d["weight"], d["bias"], cu, d["h0"])))
    x, h0, d_y = d["x"].clone(), d["h0"].clone(), seeds["d_y"].clone()
    x[0, 10:30] = float("nan")
    h0[1] = float("inf")
    d_y[0, 10:30] = float("nan")
    y, fin = gdn.conv_fwd(*(t.cuda() for t in (x, d["weight"], d["bias"], cu, h0)))
    assert torch.equal(y[0, :10], clean[0][0, :10]) and torch.equal(y[0, 30:], clean[0][0, 30:])
    assert torch.equal(fin[[0, 2]], clean[1][[0, 2]])
    a = gdn.conv_bwd(x.cuda(), d["weight"].cuda(), d["bias"].cuda(), d_y.cuda(), None, cu.cuda(), h0.cuda())
    b = gdn.conv_bwd(d["x"].cuda(), d["weight"].cuda(), d["bias"].cuda(), seeds["d_y"].cuda(), None, cu.cuda(), d["h0"].cuda())
    for rows in (slice(0, 10), slice(30, 40)):
        assert torch.equal(a["dx"][0, rows], b["dx"][0, rows])


@pytest.mark.parametrize("dtype,C", [(BF16, 72), (F32, 20), (BF16, 33)])
def test_backward_from_a_checkpoint(dtype, C):
    d, seeds = lo.conv_inputs(2, 70, C, 4, dtype, 7)
    g, s = lo.cuda(d), lo.cuda(seeds)
    p = gdn.pack8(g["x"])
    a = gdn.conv_bwd(p, g["weight"], g["bias"], s["d_y"], s["d_fin"], initial_state=g["h0"])
    b = gdn.conv_bwd(gdn.unpack8(p), g["weight"], g["bias"], s["d_y"], s["d_fin"], initial_state=g["h0"])
    assert all(torch.equal(a[k], b[k]) for k in a), "the checkpoint's values, read in place"


@pytest.mark.parametrize("case", [CASES[7], CASES[8], CASES[9], CASES[10], (1, 2600, 4096, 4, BF16, True, [1000, 0, 3, 1590], True, True)],
                         ids=["short", "fp32", "odd", "ends-early", "several-groups"])
def test_backward_from_a_packed_checkpoint(case):
    d, seeds, cu, act, used = make(case, 11)
    g, s = lo.cuda(d), lo.cuda(seeds)
    p = gdn.pack8(g["x"])
    at = gdn.unpack8(p)
    a, b = (gdn.conv_bwd(x, g["weight"], g["bias"], s["d_y"], s["d_fin"], cu.cuda(), g["h0"], act) for x in (p, at))
    assert all(torch.equal(a[k], b[k]) for k in a)
    live = (torch.arange(case[1]) < used)[:, None]
    ref = lo.gradients(lambda **k: lo.conv(cu=cu, silu=act is not None, **k), dict(lo.double(d), x=at.cpu().double()),
                       (torch.where(live, seeds["d_y"].double(), 0.0), seeds["d_fin"].double()))
    lo.close(a["dx"], ref["x"], case[3], "dx")
    lo.close(a["dweight"], ref["weight"], case[1], "dweight")


@pytest.mark.parametrize("bits", [None, 8])
def test_autograd(bits):
    d, seeds = lo.conv_inputs(2, 50, 64, 4, F32, 8)
    r = lo.double(d)
    at = dict(r)
    if bits:
        codes, scales = lo.pack(d["x"])
        at["x"] = lo.unpack(codes, scales)
    ref = lo.gradients(lo.conv, at, (seeds["d_y"].double(), seeds["d_fin"].double()))
    leaf = {k: v.cuda().requires_grad_() for k, v in d.items()}
    y, fin = gdn.causal_conv(leaf["x"], leaf["weight"], leaf["bias"], initial_state=leaf["h0"], checkpoint_bits=bits)
    y_ref, _ = lo.conv(**r)
    lo.close(y, y_ref, 4, "y")
    ((y * seeds["d_y"].cuda()).sum() + (fin * seeds["d_fin"].cuda()).sum()).backward()
    for k in leaf:
        lo.close(leaf[k].grad, ref[k], 100, "d" + k)


def test_gradient_against_differences():
    d, _ = lo.conv_inputs(1, 12, 8, 3, F32, 9)
    g = lo.cuda(d)
    seed = torch.randn(1, 12, 8, generator=torch.Generator().manual_seed(1)).cuda()
    got = gdn.conv_bwd(g["x"], g["weight"], g["bias"], seed, initial_state=g["h0"])
    # central differences of step e = 2^-6 along a direction: the truncation is e^2 / 6
    # third derivatives (below 1 here: weights of 0.5, silu''' < 1), the fp32 forward's
    # rounding 2^-24 sqrt(96) * |L| / e
    e = 2.0 ** -6
    for name, key in (("x", "dx"), ("weight", "dweight"), ("h0", "dh0")):
        v = torch.randn(g[name].shape, generator=torch.Generator().manual_seed(2)).cuda()
        v /= v.norm()
        L = []
        for sgn in (1, -1):
            h = dict(g)
            h[name] = g[name] + sgn * e * v
            y, _ = gdn.conv_fwd(h["x"], h["weight"], h["bias"], initial_state=h["h0"])
            L.append(float((y.double() * seed.double()).sum()))
        num, ana = (L[0] - L[1]) / (2 * e), float((got[key].double() * v.double()).sum())
        assert abs(num - ana) <= 1e-3 * (1 + abs(ana)), (name, num, ana)


def test_other_stream_and_graph_replay():
    d, seeds = lo.conv_inputs(2, 40, 64, 4, BF16, 10)
    g, s = lo.cuda(d), lo.cuda(seeds)
    ref = gdn.conv_fwd(g["x"], g["weight"], g["bias"], initial_state=g["h0"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdn.conv_fwd(g["x"], g["weight"], g["bias"], initial_state=g["h0"], stream=side)
    side.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    state = g["h0"].clone()

    def work():
        y, fin = gdn.conv_fwd(g["x"], g["weight"], g["bias"], initial_state=g["h0"])
        gr = gdn.conv_bwd(g["x"], g["weight"], g["bias"], s["d_y"], s["d_fin"], initial_state=g["h0"])
        z = gdn.conv_decode(g["x"][:, :1], g["weight"], g["h0"], g["bias"], new_state=state)
        return [y, fin, z, state, *gr.values()]
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(3):
        g["x"].copy_(torch.randn(2, 40, 64, generator=torch.Generator().manual_seed(20 + i)))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for o in outs]
        eager = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager)), i
