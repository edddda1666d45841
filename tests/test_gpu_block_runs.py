"""Linear attention and the norms around it as a block uses them together, with the short
convolution: a training step, a prompt and then single tokens from a captured graph, calls at
once on two streams, launchers, ill-formed and padded offsets, sizes at both ends."""
import ctypes

import pytest
import torch

import block_oracle as bo
import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
from gated_deltanet_chunkwise_amd._linattn import LinattnParams
from test_gpu_layer_runs import Banded, P, run
from test_gpu_linattn import rows_tol, state_tol
from test_gpu_norms import gated, residual

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# ---- a block: norm, projection, convolution, linear attention, gated norm, projection, norm --------

H, HV, K, V, W, C = 1, 2, 64, 64, 4, 96
CQ, CV = H * K, HV * V
PROJ = 2 * CQ + 2 * CV            # q, k, v and the gate
EPS, SCALE = 1e-5, K ** -0.5


def block_inputs(B, T, seed=1, S=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    S = B if S is None else S
    d = dict(x=r(B, T, C), res=2 * r(B, T, C), w1=1 + 0.1 * r(C), post=1 + 0.1 * r(C), scale=0.5 + 0.1 * r(C), w_in=r(PROJ, C) * C ** -0.5,
             conv=r(2 * CQ + CV, W) * 0.5, bias=r(2 * CQ + CV) * 0.1, c0=r(S, W - 1, 2 * CQ + CV), h0=r(S, HV, K, V), wn=1 + 0.1 * r(V),
             w_out=r(C, CV) * CV ** -0.5, w2=1 + 0.1 * r(C))
    return d, (r(B, T, C), r(B, T, C), r(S, HV, K, V) * 0.1), torch.tensor([-0.002, -0.1])


def block(ops, d, ld, cu):
    """(h, residual, final state) with the operators of `ops`."""
    h, res = ops.residual_norm(d["x"], d["res"], d["w1"], d["post"], d["scale"])
    proj = h @ d["w_in"].t()
    qkv, z = proj[..., :2 * CQ + CV], proj[..., 2 * CQ + CV:]
    y = ops.conv(qkv, d["conv"], d["bias"], cu, d["c0"])
    heads = lambda t, n: t.unflatten(-1, (n, -1))  # noqa: E731
    o, fin = ops.attention(heads(y[..., :CQ], H), heads(y[..., CQ:2 * CQ], H), heads(y[..., 2 * CQ:], HV), ld, cu, d["h0"])
    o = ops.gated_norm(o, d["wn"], heads(z, HV))
    h, res = ops.residual_norm(o.flatten(2) @ d["w_out"].t(), res, d["w2"], None, None)
    return h, res, fin


class Own:
    def __init__(self, bits=None):
        self.bits = bits

    def residual_norm(self, x, r, w, post, scale):
        return gdn.residual_norm(x, r, w, post, scale, eps=EPS)

    def conv(self, x, w, b, cu, c0):
        return gdn.causal_conv(x, w, b, cu, c0, checkpoint_bits=self.bits)[0]

    def attention(self, q, k, v, ld, cu, h0):
        return gdn.linear_attention(q, k, v, ld, cu, h0, scale=SCALE, checkpoint_bits=self.bits)

    def gated_norm(self, x, w, z):
        return gdn.gated_norm(x, w, z, eps=EPS)


class Plain:
    def residual_norm(self, x, r, w, post, scale):
        return residual(x, r, w, post, scale, eps=EPS)

    def conv(self, x, w, b, cu, c0):
        return lo.conv(x, w, b, cu, c0)[0]

    def attention(self, q, k, v, ld, cu, h0):
        return bo.linattn(q, k, v, h0, log_decay=ld, cu=cu, scale=SCALE)

    def gated_norm(self, x, w, z):
        return gated(x, w, z, eps=EPS, first=False)[0]


@pytest.mark.parametrize("lengths", [None, [90, 0, 1, 120]])
def test_a_block_trains(lengths):
    B, T = (2, 140) if lengths is None else (1, sum(lengths))
    cu = None if lengths is None else lo.offsets(lengths)
    d, seeds, ld = block_inputs(B, T, S=None if lengths is None else len(lengths))
    r = lo.double(d)
    ref_out = block(Plain(), r, ld.double(), cu)
    ref = lo.gradients(lambda **a: block(Plain(), a, ld.double(), cu), r, [s.double() for s in seeds])
    leaf = {n: t.cuda().requires_grad_() for n, t in d.items()}
    cuc = None if cu is None else cu.cuda()
    out = block(Own(), leaf, ld.cuda(), cuc)
    # every one of some twelve operators on the way there and back adds its own roundings of fp32,
    # which the norms between them may enlarge two or three times
    tol = 12 * 3 * state_tol(T)
    for name, o, want in zip(("h", "residual", "final state"), out, ref_out):
        bo.close(o, want, tol, name)
    sum((o * s.cuda()).sum() for o, s in zip(out, seeds)).backward()
    for n in d:
        bo.close(leaf[n].grad, ref[n], tol, "d" + n)


def test_a_block_trains_from_checkpoints():
    """Gradients of linear attention at its own checkpoints, given the gradient of what follows."""
    d, seeds, ld = bo.linattn_inputs(2, 130, 1, 2, 64, 64, F32, 3)
    g, s, ld = lo.cuda(d), lo.cuda(seeds), ld.cuda()
    leaf = {n: t.clone().requires_grad_() for n, t in g.items()}
    o, fin = gdn.linear_attention(leaf["q"], leaf["k"], leaf["v"], ld, initial_state=leaf["h0"], scale=0.5, checkpoint_bits=8)
    want_o, want_fin = gdn.linear_attn_fwd(g["q"], g["k"], g["v"], ld, initial_state=g["h0"], scale=0.5)
    assert torch.equal(o, want_o) and torch.equal(fin, want_fin)
    got = torch.autograd.grad((o, fin), list(leaf.values()), (s["d_o"], s["d_fin"]))
    at = [gdn.unpack8(gdn.pack8(g[n])) for n in "qkv"]
    ref = gdn.linear_attn_bwd(*at, ld, s["d_o"], s["d_fin"], initial_state=g["h0"], scale=0.5)
    for a, n in zip(got, ("dq", "dk", "dv", "dh0")):
        assert torch.equal(a, ref[n]), n


def test_gradients_that_nobody_asked_for():
    """One output of two used, no initial state, expanded gradients of broadcast sums."""
    d, _, ld = bo.linattn_inputs(1, 70, 1, 2, 64, 64, BF16, 4, h0=False)
    g, ld = lo.cuda(d), ld.cuda()
    ones = torch.ones(1, 70, 2, 64, dtype=BF16, device="cuda")
    leaf = {n: g[n].clone().requires_grad_() for n in "qkv"}
    o, fin = gdn.linear_attention(*leaf.values(), ld)
    ref = gdn.linear_attn_bwd(*leaf.values(), ld, ones)
    for a, n in zip(torch.autograd.grad(o.sum(), list(leaf.values()), retain_graph=True), ("dq", "dk", "dv")):
        assert torch.equal(a, ref[n])
    ref = gdn.linear_attn_bwd(*leaf.values(), ld, torch.zeros_like(ones), torch.ones_like(fin))
    for a, n in zip(torch.autograd.grad(fin.sum(), list(leaf.values())), ("dq", "dk", "dv")):
        assert torch.equal(a, ref[n])
    x, r, w = torch.randn(1, 9, 64, device="cuda"), torch.randn(1, 9, 64, device="cuda"), torch.ones(64, device="cuda")
    leaf = [t.requires_grad_() for t in (x, r, w)]
    h, s = gdn.residual_norm(*leaf)
    a = torch.autograd.grad(s.sum(), leaf, retain_graph=True)
    assert torch.equal(a[0], torch.ones_like(x)) and torch.equal(a[1], torch.ones_like(r)) and (a[2] == 0).all()
    a = torch.autograd.grad(h.sum(), leaf)
    b = gdn.residual_norm_bwd(x, r, w, torch.ones_like(x))
    assert all(torch.equal(p, b[n]) for p, n in zip(a, ("dx", "dresidual", "dweight")))


def test_a_block_answers_from_a_captured_step():
    """A prompt, then single tokens from one captured graph with its states in place; each replay
    against the whole sequence."""
    T, n = 131, 5
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(qkv=r(2, T + n, 2 * CQ + CV), z=r(2, T + n, HV, V), res=r(2, T + n, CV), conv=r(2 * CQ + CV, W) * 0.5, wn=1 + 0.1 * r(V),
             w2=1 + 0.1 * r(CV), c0=r(2, W - 1, 2 * CQ + CV), h0=r(2, HV, K, V))
    ld = torch.tensor([-0.002, -0.1])

    def whole(d):
        y, _ = lo.conv(d["qkv"], d["conv"], None, None, d["c0"])
        o, fin = bo.linattn(y[..., :CQ].unflatten(-1, (H, K)), y[..., CQ:2 * CQ].unflatten(-1, (H, K)), y[..., 2 * CQ:].unflatten(-1, (HV, V)),
                            d["h0"], log_decay=ld.double(), scale=SCALE)
        return residual(gated(o, d["wn"], d["z"], eps=EPS, first=False)[0].flatten(2), d["res"], d["w2"], eps=EPS) + (fin,)
    h_ref, s_ref, fin_ref = whole(lo.double(d))
    c, ldc = lo.cuda(d), ld.cuda()
    heads = lambda y: (y[..., :CQ].unflatten(-1, (H, K)), y[..., CQ:2 * CQ].unflatten(-1, (H, K)), y[..., 2 * CQ:].unflatten(-1, (HV, V)))  # noqa: E731
    y, cs = gdn.conv_fwd(c["qkv"][:, :T].contiguous(), c["conv"], initial_state=c["c0"])
    o, hs = gdn.linear_attn_fwd(*heads(y), ldc, initial_state=c["h0"], scale=SCALE)
    o = gdn.gated_norm_fwd(o, c["wn"], c["z"][:, :T].contiguous(), eps=EPS)
    h, s = gdn.residual_norm_fwd(o.flatten(2), c["res"][:, :T].contiguous(), c["w2"], eps=EPS)
    tol = 12 * state_tol(T + n)
    bo.close(h, h_ref[:, :T], tol, "prompt")
    token = {k: c[k][:, T:T + 1].clone() for k in ("qkv", "z", "res")}
    keep = [cs.clone(), hs.clone()]

    def step():
        y = gdn.conv_decode(token["qkv"], c["conv"], cs)
        o = gdn.linear_attn_decode(*heads(y), ldc, hs, scale=SCALE)
        o = gdn.gated_norm_fwd(o, c["wn"], token["z"], eps=EPS)
        return gdn.residual_norm_fwd(o.flatten(2), token["res"], c["w2"], eps=EPS)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    cs.copy_(keep[0])
    hs.copy_(keep[1])
    for t in range(T, T + n):
        for k in token:
            token[k].copy_(c[k][:, t:t + 1])
        graph.replay()
        torch.cuda.synchronize()
        bo.close(out[0], h_ref[:, t:t + 1], tol, "token %d" % t)
        bo.close(out[1], s_ref[:, t:t + 1], tol, "residual %d" % t)
    bo.close(hs, fin_ref, state_tol(T + n), "state")


@pytest.mark.parametrize("bits", [None, 8])
def test_a_captured_training_step_replays(bits):
    """The block's operators and their gradients in one graph (torch's products left out), its
    workspaces and checkpoints in the graph's own memory; replays against the eager step."""
    T, cu = 300, lo.offsets([170, 1, 100]).cuda()
    d, s, ld = bo.linattn_inputs(1, T, 1, 2, 64, 64, BF16, 6, 3)
    d, s, ld = lo.cuda(d), lo.cuda(s), ld.cuda()
    d.update(wn=torch.ones(64, device="cuda"), z=torch.randn(1, T, 2, 64, device="cuda").to(BF16), res=torch.randn(1, T, 128, device="cuda"),
             w2=torch.ones(128, device="cuda"), post=torch.ones(128, device="cuda"))
    d_h, d_s = torch.randn(1, T, 128, device="cuda").to(BF16), torch.randn(1, T, 128, device="cuda")

    def step():
        leaf = {n: t.detach().requires_grad_() for n, t in d.items()}
        o, fin = gdn.linear_attention(leaf["q"], leaf["k"], leaf["v"], ld, cu, leaf["h0"], scale=0.125, checkpoint_bits=bits)
        o = gdn.gated_norm(o, leaf["wn"], leaf["z"])
        h, r = gdn.residual_norm(o.flatten(2), leaf["res"], leaf["w2"], leaf["post"])
        return [h.detach(), r.detach(), fin.detach(), *torch.autograd.grad((h, r, fin), list(leaf.values()), (d_h, d_s, s["d_fin"]))]
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        step()
    cap.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        outs = step()
    for i in range(3):
        for n in "qkvz":
            d[n].copy_(torch.randn(d[n].shape, generator=torch.Generator().manual_seed(30 + i)))
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for o in outs]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager)), i


# ---- calls at once, streams, launchers -----------------------------------------------------

def test_two_calls_at_once():
    """Passes of different problems on two streams, each with its own workspace, started without
    waiting for one another, against the same calls one after the other."""
    cases = []
    for seed, T in ((7, 700), (8, 450)):
        d, s, ld = bo.linattn_inputs(2, T, 1, 2, 128, 64, BF16, seed)
        cases.append((lo.cuda(d), lo.cuda(s), ld.cuda()))

    def work(case, stream):
        g, s, ld = case
        o, fin = gdn.linear_attn_fwd(g["q"], g["k"], g["v"], ld, initial_state=g["h0"], stream=stream)
        gr = gdn.linear_attn_bwd(g["q"], g["k"], g["v"], ld, s["d_o"], s["d_fin"], initial_state=g["h0"], stream=stream)
        w = torch.ones(64, device="cuda")
        n = gdn.gated_norm_bwd(o, w, s["d_o"], g["v"], stream=stream)
        w = torch.ones(128, device="cuda")
        r = gdn.residual_norm_bwd(o.flatten(2), g["v"].flatten(2), w, s["d_o"].flatten(2), post_weight=w, stream=stream)
        return [o, fin, *gr.values(), *n.values(), *r.values()]
    ref = [work(c, None) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())  # (the weights are made on it)
            got.append(work(c, s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(got, ref) for a, b in zip(x, y))


@pytest.mark.parametrize("dtype,B,T", [(BF16, 3, 1), (F32, 2, 2)])
def test_launchers(dtype, B, T):
    """Repeated launches in place, into other tensors, on a stream of its own and captured,
    against the plain calls bit for bit."""
    d, _, ld = bo.linattn_inputs(B, T, 2, 4, 64, 128, dtype, 9)
    g, ld = lo.cuda(d), ld.cuda()
    a, h0 = (g["q"], g["k"], g["v"], ld), g["h0"]
    ref, state = h0.clone(), h0.clone()
    launch, o = gdn.linear_attn_decode_launcher(*a, state, scale=0.5)
    for i in range(3):
        launch()
        assert torch.equal(o, gdn.linear_attn_decode(*a, ref, scale=0.5)) and torch.equal(state, ref), i
        g["q"].mul_(-0.5)  # the launcher reads the tensors as they are
    new, out = torch.empty_like(h0), torch.empty_like(g["v"])
    launch, o = gdn.linear_attn_decode_launcher(*a, h0, new_state=new, out=out)
    assert o is out
    for i in range(2):  # the same result again: `state` is not written
        new.fill_(float("nan"))
        launch()
        ref.copy_(h0)
        assert torch.equal(out, gdn.linear_attn_decode(*a, ref)) and torch.equal(new, ref), i
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    state = h0.clone()
    torch.cuda.synchronize()
    launch, o = gdn.linear_attn_decode_launcher(*a, state, stream=cap)
    launch()
    cap.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        launch()
    state.copy_(h0)
    ref.copy_(h0)
    for i in range(4):
        g["k"].mul_(-0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, gdn.linear_attn_decode(*a, ref)) and torch.equal(state, ref), i


@pytest.mark.parametrize("launcher", [False, True])
def test_a_state_updated_in_place_is_not_taken_for_the_saved_one(launcher):
    d, _, ld = bo.linattn_inputs(2, 9, 1, 2, 64, 64, F32, 10)
    g, ld = lo.cuda(d), ld.cuda()
    q, one = g["q"].clone().requires_grad_(), [g[n][:, :1].contiguous() for n in "qkv"]

    def decode(s, **k):
        if launcher:
            gdn.linear_attn_decode_launcher(*one, ld, s, **k)[0]()
        else:
            gdn.linear_attn_decode(*one, ld, s, **k)
    o, _ = gdn.linear_attention(q, g["k"], g["v"], ld, initial_state=g["h0"])
    decode(g["h0"], new_state=torch.empty_like(g["h0"]))  # elsewhere: nothing that is saved changes
    o.sum().backward()
    for steps in (lambda: decode(g["h0"]), lambda: decode(g["h0"].clone(), new_state=g["h0"])):
        o, _ = gdn.linear_attention(q, g["k"], g["v"], ld, initial_state=g["h0"])
        steps()
        with pytest.raises(RuntimeError, match="inplace"):
            o.sum().backward()


# ---- offsets -------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,T,lengths", [(BF16, 300, [100, 33]), (F32, 90, [20, 13, 0]), (BF16, 2000, [0, 130, 1]), (F32, 90, [0, 0])])
def test_rows_behind_the_last_sequence_are_zero(dtype, T, lengths):
    """What the operators return there does not depend on what the memory held."""
    cu = lo.offsets(lengths)
    d, seeds, ld = bo.linattn_inputs(1, T, 1, 2, 64, 128, dtype, 11, len(lengths))
    g, s, used = lo.cuda(d), lo.cuda(seeds), int(cu[-1])
    o_ref, _ = bo.linattn(log_decay=ld.double(), cu=cu, **lo.double(d))
    for call, shape in ((lambda: [gdn.linear_attn_fwd(g["q"], g["k"], g["v"], ld.cuda(), cu.cuda(), g["h0"])[0]], [g["v"].shape]),
                        (lambda: [gdn.linear_attn_bwd(g["q"], g["k"], g["v"], ld.cuda(), s["d_o"], s["d_fin"], cu.cuda(), g["h0"])[k]
                                  for k in ("dq", "dk", "dv")], [g["q"].shape, g["k"].shape, g["v"].shape])):
        junk = [torch.full(x, float("nan"), dtype=dtype, device="cuda") for x in shape]
        del junk  # its memory is the next to be given out for tensors of these sizes
        for t in call():
            assert (t[0, used:] == 0).all() and t.isfinite().all()
    bo.close(gdn.linear_attn_fwd(g["q"], g["k"], g["v"], ld.cuda(), cu.cuda(), g["h0"])[0], o_ref, rows_tol(dtype, T), "o")


@pytest.mark.parametrize("T", [12, 300, 3000])
@pytest.mark.parametrize("offsets", [[0, 5, 3, None], [7, 900000, -5, 12], [None, 0, None, 0], [-(1 << 40), 1 << 40, -1, 1 << 62]])
def test_ill_formed_offsets_stay_inside_the_buffers(T, offsets):
    """The results are undefined; nothing outside the outputs and the workspace is written, and
    the calls end."""
    cu = torch.tensor([T if v is None else v for v in offsets], dtype=torch.int64, device="cuda")
    d, seeds, ld = bo.linattn_inputs(1, T, 1, 2, 64, 64, BF16, 12, 3)
    g, s, ld, lib, new = lo.cuda(d), lo.cuda(seeds), ld.cuda(), gdn.load_library(), Banded()
    p = LinattnParams(1, T, 1, 2, 64, 64, 3, gdn.GDN_BF16 | 0x100, 1.0, 0, 0, 0)

    def space(size):
        nb = size(ctypes.byref(p), 1)
        return (P(new((nb,), torch.uint8).fill_(0xFF)) if nb else None), nb
    ins = [P(g["q"]), P(g["k"]), P(g["v"]), P(ld), P(cu), P(g["h0"])]
    o, fin = new((1, T, 2, 64), BF16), new((3, 2, 64, 64), F32)
    run("gdn_linattn_fwd", ctypes.byref(p), *ins, P(o), P(fin), *space(lib.gdn_linattn_fwd_workspace_size))
    outs = [new((1, T, 1, 64), BF16), new((1, T, 1, 64), BF16), new((1, T, 2, 64), BF16), new((3, 2, 64, 64), F32)]
    run("gdn_linattn_bwd", ctypes.byref(p), *ins, P(s["d_o"]), P(s["d_fin"]), *(P(t) for t in outs), *space(lib.gdn_linattn_bwd_workspace_size))
    assert new.untouched()


def test_thousands_of_empty_sequences():
    """Offsets padded to a fixed count, and a run of empty sequences inside: as without the empty
    ones, whose states pass through."""
    lengths = [137, 0, 1] + [0] * 900 + [270, 2] + [0] * 300 + [125] + [0] * 800
    real = [i for i, n in enumerate(lengths) if n]
    T, S = 550, len(lengths)  # 15 tokens behind the last sequence
    cu, few = lo.offsets(lengths).cuda(), lo.offsets([lengths[i] for i in real]).cuda()
    d, s, ld = bo.linattn_inputs(1, T, 1, 2, 64, 64, F32, 13, S)
    d, s, ld = lo.cuda(d), lo.cuda(s), ld.cuda()

    def passes(cu, at):
        h0, df = d["h0"][at].contiguous(), s["d_fin"][at].contiguous()
        o, fin = gdn.linear_attn_fwd(d["q"], d["k"], d["v"], ld, cu, h0)
        g = gdn.linear_attn_bwd(d["q"], d["k"], d["v"], ld, s["d_o"], df, cu, h0)
        return [o, g["dq"], g["dk"], g["dv"]], [fin, g["dh0"]]
    tokens, states = passes(cu, slice(None))
    ref_tokens, ref_states = passes(few, real)
    for x, y in zip(tokens, ref_tokens):  # (segments may be cut elsewhere)
        bo.close(x, y.cpu().double(), 2 * state_tol(T), "rows")
    empty = [i for i in range(S) if i not in real]
    for got, ref, through in zip(states, ref_states, (d["h0"], s["d_fin"])):
        bo.close(got[real], ref.cpu().double(), 2 * state_tol(T), "states")
        assert torch.equal(got[empty], through[empty])


# ---- sizes at both ends ------------------------------------------------------------------------

@pytest.mark.parametrize("packed", [False, True])
def test_many_segments(packed):
    """Segments that are joined by a launch of their own, last ones of a single token, against the
    64-bit form."""
    T = 1500
    lengths = [1409, 0, 64, 27] if packed else None
    cu = None if lengths is None else lo.offsets(lengths)
    d, seeds, ld = bo.linattn_inputs(1, T, 1, 2, 64, 64, BF16, 14, 4 if packed else None)
    g, s, ldc = lo.cuda(d), lo.cuda(seeds), ld.cuda()
    cuc = None if cu is None else cu.cuda()
    o_ref, fin_ref = bo.linattn(log_decay=ld.double(), cu=cu, **lo.double(d))
    o, fin = gdn.linear_attn_fwd(g["q"], g["k"], g["v"], ldc, cuc, g["h0"])
    bo.close(o, o_ref, rows_tol(BF16, T), "o")
    bo.close(fin, fin_ref, state_tol(T), "final state")
    got = gdn.linear_attn_bwd(g["q"], g["k"], g["v"], ldc, s["d_o"], s["d_fin"], cuc, g["h0"])
    # the same gradients of the sequence turned round: q and k exchange their places
    ref = lo.gradients(lambda **x: bo.linattn(log_decay=ld.double(), cu=cu, **x), lo.double(d), [v.double() for v in seeds.values()])
    for k, name in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        bo.close(got[k], ref[name], rows_tol(BF16, T), k)
    bo.close(got["dh0"], ref["h0"], state_tol(T), "dh0")


def test_rows_further_apart_than_32_bits_reach():
    """Tokens 32 MB apart: a chunk's rows within 32-bit offsets, its chunks beyond them."""
    ld_, T = (1 << 24) - 8, 140
    big = torch.empty(T * ld_, dtype=BF16, device="cuda")
    d, s, ld = bo.linattn_inputs(1, T, 1, 1, 64, 64, BF16, 15)
    g, s, ld = lo.cuda(d), lo.cuda(s), ld.cuda()
    view = lambda off, t: big.as_strided((1, T, 1, 64), (T * ld_, ld_, 64, 1), off).copy_(t)  # noqa: E731
    w = dict(g, q=view(0, g["q"]), k=view(1024, g["k"]), v=view(4096, g["v"]))
    a, b = (gdn.linear_attn_fwd(x["q"], x["k"], x["v"], ld, initial_state=x["h0"]) for x in (w, g))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = (gdn.linear_attn_bwd(x["q"], x["k"], x["v"], ld, s["d_o"], s["d_fin"], initial_state=x["h0"]) for x in (w, g))
    assert all(torch.equal(a[n], b[n]) for n in a)
    wide = torch.empty(1, T, ld_ + 8, dtype=BF16, device="cuda")[..., :64].unflatten(-1, (1, 64))
    with pytest.raises(gdn.GdnError) as e:
        gdn.linear_attn_fwd(wide, wide, wide, ld)
    assert e.value.status == 4
    x, r = w["q"][:, :, 0], w["k"][:, :, 0]
    one = torch.ones(64, device="cuda")
    p, q = gdn.residual_norm_fwd(x, r, one), gdn.residual_norm_fwd(x.contiguous(), r.contiguous(), one)
    assert all(torch.equal(a, b) for a, b in zip(p, q))
    del big, w, view, wide, x, r
    torch.cuda.empty_cache()


def test_tensors_beyond_32_bit_offsets():
    """600 thousand tokens of 32 value heads of 128: 2.4e9 elements, 4.9 GB a tensor, and states of
    segments beyond 2 GB.  The last sequence against the same tokens on their own."""
    T, n, H_, HV_ = 600000, 700, 4, 32
    gen = torch.Generator(device="cuda").manual_seed(16)
    r = lambda *s, dtype=BF16: torch.randn(*s, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    q, k, v, d_o = r(1, T, H_, 128), r(1, T, H_, 128), r(1, T, HV_, 128), r(1, T, HV_, 128)
    h0, ld = r(2, HV_, 128, 128, dtype=F32), -torch.rand(HV_, generator=gen, device="cuda")
    cu = torch.tensor([0, T - n, T], device="cuda")
    end = lambda t: t[:, -n:].contiguous()  # noqa: E731
    o, fin = gdn.linear_attn_fwd(q, k, v, ld, cu, h0, scale=0.1)
    o1, fin1 = gdn.linear_attn_fwd(end(q), end(k), end(v), ld, initial_state=h0[1:], scale=0.1)
    bo.close(end(o), o1.cpu().double(), 2 * rows_tol(BF16, n), "o")
    bo.close(fin[1:], fin1.cpu().double(), 2 * state_tol(n), "final state")
    assert o.isfinite().all()
    g = gdn.linear_attn_bwd(q, k, v, ld, d_o, None, cu, h0, scale=0.1)
    g1 = gdn.linear_attn_bwd(end(q), end(k), end(v), ld, end(d_o), initial_state=h0[1:], scale=0.1)
    for name in ("dq", "dk", "dv"):
        bo.close(end(g[name]), g1[name].cpu().double(), 2 * rows_tol(BF16, n), name)
    bo.close(g["dh0"][1:], g1["dh0"].cpu().double(), 2 * state_tol(n), "dh0")
    del g, q, k
    w = torch.ones(128, device="cuda")
    y = gdn.gated_norm_fwd(o, w, v)
    assert torch.equal(end(y), gdn.gated_norm_fwd(end(o), w, end(v)))
    g, g1 = gdn.gated_norm_bwd(o, w, d_o, v), gdn.gated_norm_bwd(end(o), w, end(d_o), end(v))
    assert torch.equal(end(g["dx"]), g1["dx"]) and torch.equal(end(g["dz"]), g1["dz"])
    del g, y
    w = torch.ones(4096, device="cuda")
    h, s = gdn.residual_norm_fwd(o.flatten(2), v.flatten(2), w, w)
    h1, s1 = gdn.residual_norm_fwd(end(o).flatten(2), end(v).flatten(2), w, w)
    assert torch.equal(end(h), h1) and torch.equal(end(s), s1)
    del h, s
    g = gdn.residual_norm_bwd(o.flatten(2), v.flatten(2), w, d_o.flatten(2), post_weight=w)
    g1 = gdn.residual_norm_bwd(end(o).flatten(2), end(v).flatten(2), w, end(d_o).flatten(2), post_weight=w)
    assert torch.equal(end(g["dx"]), g1["dx"]) and torch.equal(end(g["dresidual"]), g1["dresidual"])
    del g, o, v, d_o
    torch.cuda.empty_cache()


@pytest.mark.parametrize("packed", [False, True])
def test_no_sequences_at_all(packed):
    """B = 0, or offsets [0]: empty outputs, and weights' gradients of 0."""
    B, T = (1, 0) if packed else (0, 7)
    d, s, ld = bo.linattn_inputs(B, T, 1, 2, 64, 64, F32, 17, 0)
    d, s, ld = lo.cuda(d), lo.cuda(s), ld.cuda()
    cu = torch.zeros(1, dtype=torch.int64, device="cuda") if packed else None
    o, fin = gdn.linear_attn_fwd(d["q"], d["k"], d["v"], ld, cu, d["h0"])
    g = gdn.linear_attn_bwd(d["q"], d["k"], d["v"], ld, s["d_o"], s["d_fin"], cu, d["h0"])
    assert o.shape == (B, T, 2, 64) and fin.shape == (0, 2, 64, 64) and g["dh0"].shape == (0, 2, 64, 64)
    w = torch.ones(64, device="cuda")
    n = gdn.gated_norm_bwd(o, w, o, o)
    w2 = torch.ones(128, device="cuda")
    r = gdn.residual_norm_bwd(o.flatten(2), o.flatten(2), w2, o.flatten(2), post_weight=w2, scale=w2)
    torch.cuda.synchronize()
    for t in (n["dweight"], r["dweight"], r["dpost_weight"], r["dscale"]):
        assert (t == 0).all()
    if not packed:
        gdn.linear_attn_decode(d["q"], d["k"], d["v"], ld, d["h0"])


def test_a_decode_call_of_no_tokens_passes_the_state_on():
    d, _, ld = bo.linattn_inputs(2, 0, 1, 2, 64, 64, F32, 18)
    g, new = lo.cuda(d), torch.empty(2, 2, 64, 64, device="cuda")
    gdn.linear_attn_decode(g["q"], g["k"], g["v"], ld.cuda(), g["h0"], new_state=new)
    assert torch.equal(new, g["h0"])
