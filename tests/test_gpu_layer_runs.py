"""The layer operators as a layer uses them together: the convolution of a projection's
slices before the gated delta rule and before the selective scan, a prompt and then single
tokens, training steps with and without 8-bit checkpoints; guard bands around everything
they write; calls at once on two streams; replays of captured decode steps."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
import oracle
from gpu_helpers import f64
from gated_deltanet_chunkwise_amd._layers import ConvParams, ScanParams

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ---- convolution, then gated delta rule -------------------------------------------

B, T, H, HV, K, V, W = 2, 70, 1, 2, 64, 64, 4
CQ, CK, CV = H * K, H * K, HV * V
C = CQ + CK + CV


def layer_inputs(seed=1, B=B, T=T):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    # the projection is small so that k, after the convolution, keeps the rule stable
    return dict(proj=r(B, T, C) * 0.3, weight=r(C, W) * 0.5, bias=r(C) * 0.1, g_raw=r(B, T, HV),
                beta=torch.sigmoid(r(B, T, HV)), A_log=r(HV).abs(), dt_bias=r(HV) * 0.1,
                c0=r(B, W - 1, C) * 0.3, h0=r(B, HV, K, V) * 0.1), dict(
                    d_o=r(B, T, HV, V), d_fin=r(B, HV, K, V) * 0.1)


def qkv(y):
    b, t = y.shape[:2]
    return (y[..., :CQ].reshape(b, t, H, K).contiguous(), y[..., CQ:CQ + CK].reshape(b, t, H, K).contiguous(),
            y[..., CQ + CK:].reshape(b, t, HV, V).contiguous())


def oracle_layer(d):
    r = lo.double(d)
    y, c1 = lo.conv(r["proj"], r["weight"], r["bias"], None, r["c0"])
    q, k, v = (t.numpy() for t in qkv(y))
    o, fin = oracle.fwd(q, k, v, *(r[n].numpy() for n in ("g_raw", "beta", "A_log", "dt_bias")), h0=r["h0"].numpy())
    return (q, k, v), o, fin, c1


def close(x, ref, what, tol):
    ref = np.asarray(ref, np.float64)
    x = f64(x) if torch.is_tensor(x) else np.asarray(x)
    rel = np.linalg.norm(x - ref) / np.linalg.norm(ref)
    print("  %-10s rel_l2=%.2e" % (what, rel), flush=True)
    assert np.isfinite(x).all() and rel <= tol, (what, rel)


def test_gated_delta_rule_layer_trains():
    d, seeds = layer_inputs()
    (q, k, v), o_ref, fin_ref, _ = oracle_layer(d)
    r = lo.double(d)
    gr = oracle.bwd(q, k, v, *(r[n].numpy() for n in ("g_raw", "beta", "A_log", "dt_bias")),
                    seeds["d_o"].double().numpy(), seeds["d_fin"].double().numpy(), h0=r["h0"].numpy())
    d_y = torch.cat([torch.from_numpy(np.asarray(gr[n])).reshape(B, T, -1) for n in ("dq", "dk", "dv")], -1)
    ref = lo.gradients(lambda **a: lo.conv(a["x"], a["weight"], a["bias"], None, a["h0"]),
                       dict(x=r["proj"], weight=r["weight"], bias=r["bias"], h0=r["c0"]), (d_y, None))
    leaf = {n: t.cuda().requires_grad_() for n, t in d.items()}
    y, _ = gdn.causal_conv(leaf["proj"], leaf["weight"], leaf["bias"], initial_state=leaf["c0"])
    o, fin = gdn.gated_delta_rule(*qkv(y), leaf["g_raw"], leaf["beta"], leaf["A_log"], leaf["dt_bias"],
                                  initial_state=leaf["h0"])
    # the rule's own bounds for fp32 (tests of gdn_fwd and gdn_bwd), which the
    # convolution's few roundings do not change
    close(o, o_ref, "o", 1e-4)
    close(fin, fin_ref, "final", 1e-4)
    ((o * seeds["d_o"].cuda()).sum() + (fin * seeds["d_fin"].cuda()).sum()).backward()
    for n, g in (("proj", ref["x"]), ("weight", ref["weight"]), ("bias", ref["bias"]), ("c0", ref["h0"]),
                 ("g_raw", gr["dg_raw"]), ("beta", gr["dbeta"]), ("h0", gr["dh0"])):
        close(leaf[n].grad, g, "d" + n, 1e-3)


def test_gated_delta_rule_layer_trains_from_checkpoints():
    """Every operator's gradients are those at its own checkpoint, given the gradient of
    what follows: composed by hand, call by call."""
    d, seeds = layer_inputs(2)
    g = lo.cuda(d)
    leaf = {n: t.clone().requires_grad_() for n, t in g.items()}
    y, _ = gdn.causal_conv(leaf["proj"], leaf["weight"], leaf["bias"], initial_state=leaf["c0"], checkpoint_bits=8)
    o, fin = gdn.gated_delta_rule(*qkv(y), leaf["g_raw"], leaf["beta"], leaf["A_log"], leaf["dt_bias"],
                                  initial_state=leaf["h0"], checkpoint_bits=8)
    ((o * seeds["d_o"].cuda()).sum() + (fin * seeds["d_fin"].cuda()).sum()).backward()
    y2, _ = gdn.conv_fwd(g["proj"], g["weight"], g["bias"], initial_state=g["c0"])
    assert torch.equal(y, y2)
    at = [gdn.unpack8(gdn.pack8(t)) for t in qkv(y2)]
    gr = gdn.bwd(*at, g["g_raw"], g["beta"], g["A_log"], g["dt_bias"], seeds["d_o"].cuda(), seeds["d_fin"].cuda(),
                 initial_state=g["h0"])
    d_y = torch.cat([gr[n].reshape(B, T, -1) for n in ("dq", "dk", "dv")], -1)
    gc = gdn.conv_bwd(gdn.pack8(g["proj"]), g["weight"], g["bias"], d_y, initial_state=g["c0"])
    for n, v in (("proj", gc["dx"]), ("weight", gc["dweight"]), ("bias", gc["dbias"]), ("c0", gc["dh0"]),
                 ("g_raw", gr["dg_raw"]), ("h0", gr["dh0"])):
        close(leaf[n].grad, f64(v), "d" + n, 1e-3)  # gdn_bwd's LDS atomics change low bits


def test_gated_delta_rule_layer_answers():
    """A prompt of 66 tokens, then four single tokens, against the whole."""
    d, _ = layer_inputs(3)
    _, o_ref, fin_ref, c_ref = oracle_layer(d)
    g = lo.cuda(d)
    cut = lambda n, a, b: g[n][:, a:b].contiguous()  # noqa: E731
    y, conv_state = gdn.conv_fwd(cut("proj", 0, 66), g["weight"], g["bias"], initial_state=g["c0"])
    o, state = gdn.fwd(*qkv(y), cut("g_raw", 0, 66), cut("beta", 0, 66), g["A_log"], g["dt_bias"], initial_state=g["h0"])
    outs = [o]
    for t in range(66, 70):
        y = gdn.conv_decode(g["proj"][:, t:t + 1], g["weight"], conv_state, g["bias"])
        outs.append(gdn.decode(*qkv(y), cut("g_raw", t, t + 1), cut("beta", t, t + 1), g["A_log"], state, g["dt_bias"]))
    close(torch.cat(outs, 1), o_ref, "o", 1e-4)
    close(state, fin_ref, "state", 1e-4)
    assert np.array_equal(f64(conv_state), c_ref.numpy())


# ---- convolution, then selective scan ----------------------------------------------

D, N = 70, 16


def scan_layer(seed, S, T, dtype=F32):
    d, _ = lo.scan_inputs(1, T, D, N, 1, dtype, seed, S)
    c, _ = lo.conv_inputs(1, T, D, W, dtype, seed + 1, S)
    return dict(d, proj=c["x"], weight=c["weight"], bias=c["bias"], c0=c["h0"])


def scan_args(d):
    return dict(dt=d["dt"], A_log=d["A_log"], Bm=d["Bm"], Cm=d["Cm"], skip=d["skip"], z=d["z"], dt_bias=d["dt_bias"])


def test_scan_layer_trains_on_packed_sequences():
    lengths = [40, 0, 1, 75]
    cu, T_ = lo.offsets(lengths), sum(lengths)
    d = scan_layer(4, len(lengths), T_)
    seed = torch.randn(1, T_, D, generator=torch.Generator().manual_seed(5))

    def plain(proj, weight, bias, c0, h0, **a):
        y, _ = lo.conv(proj, weight, bias, cu, c0)
        return lo.scan(x=y, cu=cu, h0=h0, **a)
    names = ("proj", "weight", "bias", "c0", "h0", "dt", "A_log", "Bm", "Cm", "skip", "z", "dt_bias")
    r = lo.double(d)
    y_ref, _ = plain(**{n: r[n] for n in names})
    ref = lo.gradients(plain, {n: r[n] for n in names}, (seed.double(), None))
    leaf = {n: d[n].cuda().requires_grad_() for n in names}
    c, _ = gdn.causal_conv(leaf["proj"], leaf["weight"], leaf["bias"], cu.cuda(), leaf["c0"])
    y, _ = gdn.selective_scan(c, **scan_args(leaf), cu_seqlens=cu.cuda(), initial_state=leaf["h0"])
    lo.close(y, y_ref, T_, "y")
    (y * seed.cuda()).sum().backward()
    for n in names:
        lo.close(leaf[n].grad, ref[n], 2 * T_, "d" + n)


def test_scan_layer_answers_from_a_captured_step():
    """A prompt, then single tokens from one captured graph with its states in place: each
    replay continues where the last one ended."""
    T_ = 70
    d = scan_layer(6, 1, T_ + 5)
    r = lo.double(d)
    c_ref, _ = lo.conv(r["proj"], r["weight"], r["bias"], None, r["c0"])
    y_ref, fin_ref = lo.scan(x=c_ref, h0=r["h0"], **scan_args(r))
    g = lo.cuda(d)
    y, cs = gdn.conv_fwd(g["proj"][:, :T_], g["weight"], g["bias"], initial_state=g["c0"])
    y, hs = gdn.scan_fwd(y, *(g[n][:, :T_] if n != "A_log" else g[n] for n in ("dt", "A_log", "Bm", "Cm")), g["skip"],
                         g["z"][:, :T_], g["dt_bias"], initial_state=g["h0"])
    lo.close(y, y_ref[:, :T_], T_, "prompt")
    token = {n: g[n][:, T_:T_ + 1].clone() for n in ("proj", "dt", "Bm", "Cm", "z")}
    keep = [cs.clone(), hs.clone()]

    def step():
        c = gdn.conv_decode(token["proj"], g["weight"], cs, g["bias"])
        return gdn.scan_decode(c, token["dt"], g["A_log"], token["Bm"], token["Cm"], hs, g["skip"], token["z"], g["dt_bias"])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    cs.copy_(keep[0])
    hs.copy_(keep[1])
    got = []
    for t in range(T_, T_ + 5):
        for n in token:
            token[n].copy_(g[n][:, t:t + 1])
        graph.replay()
        torch.cuda.synchronize()
        got.append(out.clone())
    lo.close(torch.cat(got, 1), y_ref[:, T_:], T_ + 5, "tokens")
    lo.close(hs, fin_ref, T_ + 5, "state")


# ---- guard bands -------------------------------------------------------------------

class Banded:
    """Tensors inside larger allocations, 4 KB of a fixed byte on both sides."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype, shift=0):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 8192 + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((buf, 4096 + shift, n))
        return buf[4096 + shift:4096 + shift + n].view(dtype).view(shape)

    def untouched(self):
        torch.cuda.synchronize()
        return all(bool((b[:a] == 0xA5).all()) and bool((b[a + n:] == 0xA5).all()) for b, a, n in self.all)


def P(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def run(name, *args):
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert getattr(gdn.load_library(), name)(*args, s) == 0


@pytest.mark.parametrize("dtype,T,D,N,lengths,shift", [
    (BF16, 70, 64, 16, None, 0), (BF16, 70, 66, 13, None, 2), (F32, 33, 70, 40, [5, 0, 28], 4),
    (BF16, 300, 130, 8, [64, 65, 0, 1, 100], 0)])
def test_nothing_is_written_outside_the_outputs(dtype, T, D, N, lengths, shift):
    code = gdn.GDN_BF16 if dtype == BF16 else gdn.GDN_F32
    new = Banded()
    cu = None if lengths is None else lo.offsets(lengths).cuda()
    S = 1 if cu is None else len(lengths)
    out = lambda *s, dtype=dtype: new(s, dtype, shift if dtype != F32 else (4 if shift else 0))  # noqa: E731
    d, s = lo.conv_inputs(1, T, D, 4, dtype, 7, S)
    g, s = lo.cuda(d), lo.cuda(s)
    p = ConvParams(1, T, D, 4, 0 if cu is None else S, code, 1, 0)
    y, fin = out(1, T, D), out(S, 3, D)
    run("gdn_conv_fwd", ctypes.byref(p), P(g["x"]), P(g["weight"]), P(g["bias"]), P(cu), P(g["h0"]), P(y), P(fin))
    nb = gdn.load_library().gdn_conv_bwd_workspace_size(ctypes.byref(p), int(cu is not None))
    ws = new((nb,), torch.uint8)
    dx, dw, db, dh0 = out(1, T, D), out(D, 4, dtype=F32), out(D, dtype=F32), out(S, 3, D)
    run("gdn_conv_bwd", ctypes.byref(p), P(g["x"]), None, P(g["weight"]), P(g["bias"]), P(cu), P(g["h0"]), P(s["d_y"]),
        P(s["d_fin"]), P(dx), P(dw), P(db), P(dh0), P(ws), nb)
    st, y1 = out(S, 3, D), out(S, 1, D)
    x1 = g["h0"][:, 0].contiguous()
    q = ConvParams(S, 1, D, 4, 0, code, 1, 0)
    run("gdn_conv_decode", ctypes.byref(q), P(x1), P(g["weight"]), P(g["bias"]), P(g["h0"]), P(st), P(y1))
    codes, scales, back = new((T, D), torch.int8, shift), new((T, (D + 31) // 32), torch.uint8, shift), out(T, D)
    run("gdn_pack8", P(g["x"]), code, T, D, 0, P(codes), P(scales))
    run("gdn_unpack8", P(codes), P(scales), T, D, P(back), code)

    d, s = lo.scan_inputs(1, T, D, N, 1, dtype, 8, S)
    g, s = lo.cuda(d), lo.cuda(s)
    p = ScanParams(1, T, D, 1, N, 0 if cu is None else S, code, 0, 0, 0, 0, 0)
    y, fin = out(1, T, D), out(S, D, N, dtype=F32)
    nb = gdn.load_library().gdn_scan_fwd_workspace_size(ctypes.byref(p), int(cu is not None))
    ws = new((nb,), torch.uint8)
    ins = [P(g[n]) for n in ("x", "dt", "A_log", "Bm", "Cm", "skip", "z", "dt_bias")] + [P(cu), P(g["h0"])]
    run("gdn_scan_fwd", ctypes.byref(p), *ins, P(y), P(fin), P(ws), nb)
    nb = gdn.load_library().gdn_scan_bwd_workspace_size(ctypes.byref(p), int(cu is not None))
    ws = new((nb,), torch.uint8)
    o = dict(dx=out(1, T, D), ddt=out(1, T, D), dA=out(D, N, dtype=F32), dB=out(1, T, 1, N), dC=out(1, T, 1, N),
             dskip=out(D, dtype=F32), dz=out(1, T, D), dbias=out(D, dtype=F32), dh0=out(S, D, N, dtype=F32))
    run("gdn_scan_bwd", ctypes.byref(p), ins[0], None, *ins[1:7], None, *ins[7:], P(s["d_y"]), P(s["d_fin"]),
        *(P(t) for t in o.values()), P(ws), nb)
    q = ScanParams(S, 1, D, 1, N, 0, code, 0, 0, 0, 0, 0)
    h1, y1 = out(S, D, N, dtype=F32), out(S, 1, D)
    keep = [g[n][:, :1].expand(S, *g[n][:, :1].shape[1:]).contiguous() for n in ("x", "dt", "Bm", "Cm", "z")]
    x1, dt1, b1, c1, z1 = (P(t) for t in keep)
    run("gdn_scan_decode", ctypes.byref(q), x1, dt1, P(g["A_log"]), b1, c1, P(g["skip"]), z1, P(g["dt_bias"]), P(g["h0"]),
        P(h1), P(y1))
    assert new.untouched()


@pytest.mark.parametrize("T", [12, 100])
def test_ill_formed_offsets_stay_inside_the_buffers(T):
    """A sequence that begins before the one ahead of it ends: what its tokens give is
    undefined, but nothing outside the outputs is written, no tile's state is read that was
    never formed, and the sequence ahead keeps its result."""
    D, N, cu = 64, 16, torch.tensor([0, 5, 3, T], dtype=torch.int64)
    d, s = lo.scan_inputs(1, T, D, N, 1, F32, 11, 3)
    c, cs = lo.conv_inputs(1, T, D, 4, F32, 12, 3)
    g, gc = lo.cuda(d), lo.cuda(c)
    a = [g[n] for n in ("x", "dt", "A_log", "Bm", "Cm")]
    kw = dict(skip=g["skip"], z=g["z"], dt_bias=g["dt_bias"], cu_seqlens=cu.cuda(), initial_state=g["h0"])
    y, fin = gdn.scan_fwd(*a, **kw)
    back = gdn.scan_bwd(*a, s["d_y"].cuda(), s["d_fin"].cuda(), **kw)
    yc, _ = gdn.conv_fwd(gc["x"], gc["weight"], gc["bias"], cu.cuda(), gc["h0"])
    gdn.conv_bwd(gc["x"], gc["weight"], gc["bias"], cs["d_y"].cuda(), cs["d_fin"].cuda(), cu.cuda(), gc["h0"])
    torch.cuda.synchronize()
    ref, _ = lo.scan(cu=torch.tensor([0, 5, T, T]), **{n: v.double() for n, v in d.items()})
    refc, _ = lo.conv(c["x"].double(), c["weight"].double(), c["bias"].double(), torch.tensor([0, 5, T, T]),
                      c["h0"].double())
    lo.close(y[:, :5], ref[:, :5], 5, "y")
    lo.close(yc[:, :5], refc[:, :5], 5, "conv y")
    assert all(t.isfinite().all() for t in (fin[0], back["dx"][:, :5]))


# ---- calls at once ------------------------------------------------------------------

def test_two_calls_at_once():
    """Backward passes of different problems on two streams, each with its own workspace,
    started without waiting for one another, against the same calls one after the other."""
    cases = []
    for seed, T_ in ((9, 500), (10, 333)):
        d, s = lo.scan_inputs(2, T_, 128, 16, 1, BF16, seed)
        c, cs = lo.conv_inputs(2, T_, 128, 4, BF16, seed)
        cases.append((lo.cuda(d), lo.cuda(s), lo.cuda(c), lo.cuda(cs)))

    def work(case, stream):
        g, s, c, cs = case
        a = gdn.scan_bwd(g["x"], g["dt"], g["A_log"], g["Bm"], g["Cm"], s["d_y"], s["d_fin"], g["skip"], g["z"],
                         g["dt_bias"], initial_state=g["h0"], stream=stream)
        b = gdn.conv_bwd(c["x"], c["weight"], c["bias"], cs["d_y"], cs["d_fin"], initial_state=c["h0"], stream=stream)
        return [*a.values(), *b.values(), *gdn.pack8(g["x"], stream=stream)[:2]]
    ref = [work(c, None) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [work(c, s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(got, ref) for a, b in zip(x, y))


# ---- offsets that end before the batch does --------------------------------------------

@pytest.mark.parametrize("dtype,T,D,N,lengths", [
    (BF16, 50, 64, 16, [20, 13]), (F32, 50, 66, 40, [20, 13, 0]), (BF16, 300, 330, 20, [0, 130, 1]), (F32, 90, 24, 8, [0, 0]),
    (BF16, 700, 1056, 16, [63])])
def test_rows_behind_the_last_sequence_are_zero(dtype, T, D, N, lengths):
    """What the operators return there does not depend on what the memory held, so that a
    loss may mask those rows by a product."""
    d, _ = lo.scan_inputs(1, T, D, N, 1, dtype, 15, len(lengths))
    c, _ = lo.conv_inputs(1, T, D, 4, dtype, 16, len(lengths))
    cu, used = lo.offsets(lengths), sum(lengths)
    g, gc, gcu = lo.cuda(d), lo.cuda(c), cu.cuda()
    o = dict(skip=g["skip"], z=g["z"], dt_bias=g["dt_bias"], cu_seqlens=gcu, initial_state=g["h0"])
    y_ref, _ = lo.scan(cu=cu, **lo.double(d))
    c_ref, _ = lo.conv(cu=cu, **lo.double(c))
    for call, ref, steps in (
            (lambda: gdn.conv_fwd(gc["x"], gc["weight"], gc["bias"], gcu, gc["h0"]), c_ref, 4),
            (lambda: gdn.causal_conv(gc["x"], gc["weight"], gc["bias"], gcu, gc["h0"]), c_ref, 4),
            (lambda: gdn.scan_fwd(g["x"], g["dt"], g["A_log"], g["Bm"], g["Cm"], **o), y_ref, T),
            (lambda: gdn.selective_scan(g["x"], g["dt"], g["A_log"], g["Bm"], g["Cm"], **o), y_ref, T)):
        junk = torch.full_like(g["x"], float("nan"))
        del junk  # its memory is the next to be given out for a tensor of this size
        y, _ = call()
        assert (y[0, used:] == 0).all()
        lo.close(y, ref, steps, "y")


# ---- states updated in place ---------------------------------------------------------

@pytest.mark.parametrize("launcher", [False, True])
def test_a_state_updated_in_place_is_not_taken_for_the_saved_one(launcher):
    """A backward pass that needs the initial state refuses one that a decode step has
    overwritten, as torch's own in-place operations have it."""
    d, _ = lo.scan_inputs(2, 9, 64, 16, 1, F32, 17)
    c, _ = lo.conv_inputs(2, 9, 64, 4, F32, 18)
    g, gc = lo.cuda(d), lo.cuda(c)
    w, a = gc["weight"].requires_grad_(), g["A_log"].requires_grad_()
    for state, out, step in (
            (gc["h0"], lambda s: gdn.causal_conv(gc["x"], w, initial_state=s),
             lambda f, s, **k: f(gc["x"][:, :1], gc["weight"].detach(), s, **k)),
            (g["h0"], lambda s: gdn.selective_scan(g["x"], g["dt"], a, g["Bm"], g["Cm"], initial_state=s),
             lambda f, s, **k: f(*(g[n][:, :1] for n in ("x", "dt")), a.detach(), *(g[n][:, :1] for n in ("Bm", "Cm")), s, **k))):
        conv = state is gc["h0"]

        def decode(s, **k):
            if launcher:
                step(gdn.conv_decode_launcher if conv else gdn.scan_decode_launcher, s, **k)[0]()
            else:
                step(gdn.conv_decode if conv else gdn.scan_decode, s, **k)
        y, _ = out(state)
        decode(state, new_state=torch.empty_like(state))  # elsewhere: nothing that is saved changes
        y.sum().backward()
        y, _ = out(state)
        decode(state)
        with pytest.raises(RuntimeError, match="inplace"):
            y.sum().backward()
        y, _ = out(state)
        decode(state.clone(), new_state=state)
        with pytest.raises(RuntimeError, match="inplace"):
            y.sum().backward()


# ---- decode launchers ------------------------------------------------------------------

def decode_step(kind, dtype, Bn, T_, seed):
    """(call on a state and its options, the same through the launcher, the state's inputs,
    the token tensors)."""
    if kind == "conv":
        d, _ = lo.conv_inputs(Bn, T_, 72, 4, dtype, seed)
        g = lo.cuda(d)
        call = lambda f, state, **k: f(g["x"], g["weight"], state, g["bias"], **k)  # noqa: E731
        return call, gdn.conv_decode, gdn.conv_decode_launcher, g["h0"], g["x"]
    d, _ = lo.scan_inputs(Bn, T_, 66, 13, 1, dtype, seed)
    g = lo.cuda(d)
    call = lambda f, state, **k: f(g["x"], g["dt"], g["A_log"], g["Bm"], g["Cm"], state, g["skip"], g["z"],  # noqa: E731
                                   g["dt_bias"], **k)
    return call, gdn.scan_decode, gdn.scan_decode_launcher, g["h0"], g["x"]


@pytest.mark.parametrize("kind", ["conv", "scan"])
@pytest.mark.parametrize("dtype,Bn,T_", [(BF16, 3, 1), (F32, 2, 2)])
def test_launchers(kind, dtype, Bn, T_):
    """Repeated launches in place, into other tensors, and on a stream of its own, against
    the plain calls bit for bit."""
    call, plain, launcher, h0, x = decode_step(kind, dtype, Bn, T_, 19)
    ref, state = h0.clone(), h0.clone()
    launch, y = call(launcher, state)
    for i in range(3):
        launch()
        assert torch.equal(y, call(plain, ref)) and torch.equal(state, ref), i
        x.mul_(-0.5)  # the launcher reads the tensors as they are
    new, out = torch.empty_like(h0), torch.empty_like(x)
    launch, y = call(launcher, h0, new_state=new, out=out)
    assert y is out
    for i in range(2):  # the same result again: `state` is not written
        new.fill_(float("nan"))
        launch()
        ref.copy_(h0)
        assert torch.equal(out, call(plain, ref)) and torch.equal(new, ref), i
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    launch, y = call(launcher, h0, new_state=new, stream=side)
    launch()
    side.synchronize()
    assert torch.equal(y, call(plain, ref.copy_(h0))) and torch.equal(new, ref)


@pytest.mark.parametrize("kind", ["conv", "scan"])
def test_a_captured_launcher_replays(kind):
    call, plain, launcher, h0, x = decode_step(kind, BF16, 2, 1, 20)
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    state, ref = h0.clone(), h0.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(cap):
        launch, y = call(launcher, state)
        launch()
    cap.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        launch()
    state.copy_(h0)
    for i in range(4):
        x.mul_(-0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, call(plain, ref)) and torch.equal(state, ref), i


# ---- ill-formed offsets, every value ----------------------------------------------------

@pytest.mark.parametrize("T", [12, 29, 100, 333])
@pytest.mark.parametrize("dtype,D,N", [(F32, 64, 16), (BF16, 66, 40)])
def test_a_sequence_that_begins_too_early_starts_where_the_one_ahead_ended(T, dtype, D, N):
    """Offsets [0, 5, 3, T] are taken as [0, 5), nothing, [5, T) from the third state: all
    the scan computes, and the convolution but for the last sequence's d_initial, as for
    those; nothing outside the outputs and the workspace is written, and what the
    workspace held (NaN) is not read."""
    bad, good = torch.tensor([0, 5, 3, T], dtype=torch.int64), torch.tensor([0, 5, 5, T], dtype=torch.int64)
    code, lib, new = (gdn.GDN_BF16 if dtype == BF16 else gdn.GDN_F32), gdn.load_library(), Banded()
    out = lambda *s, dtype=dtype: new(s, dtype)  # noqa: E731

    def space(size, p):
        nb = size(ctypes.byref(p), 1)
        return new((nb,), torch.uint8).fill_(0xFF), nb
    cu = bad.cuda()
    d, seeds = lo.scan_inputs(1, T, D, N, 1, dtype, 11, 3)
    g, s = lo.cuda(d), lo.cuda(seeds)
    r = lo.double(d)
    p = ScanParams(1, T, D, 1, N, 3, code, 0, 0, 0, 0, 0)
    y, fin = out(1, T, D), out(3, D, N, dtype=F32)
    ws, nb = space(lib.gdn_scan_fwd_workspace_size, p)
    ins = [P(g[n]) for n in ("x", "dt", "A_log", "Bm", "Cm", "skip", "z", "dt_bias")] + [P(cu), P(g["h0"])]
    run("gdn_scan_fwd", ctypes.byref(p), *ins, P(y), P(fin), P(ws), nb)
    y_ref, fin_ref = lo.scan(cu=good, **r)
    lo.close(y, y_ref, T, "y")
    lo.close(fin, fin_ref, T, "final")
    ws, nb = space(lib.gdn_scan_bwd_workspace_size, p)
    o = dict(x=out(1, T, D), dt=out(1, T, D), A_log=out(D, N, dtype=F32), Bm=out(1, T, 1, N), Cm=out(1, T, 1, N),
             skip=out(D, dtype=F32), z=out(1, T, D), dt_bias=out(D, dtype=F32), h0=out(3, D, N, dtype=F32))
    run("gdn_scan_bwd", ctypes.byref(p), ins[0], None, *ins[1:7], None, *ins[7:], P(s["d_y"]), P(s["d_fin"]),
        *(P(t) for t in o.values()), P(ws), nb)
    ref = lo.gradients(lambda **k: lo.scan(cu=good, **k), r, [t.double() for t in seeds.values()])
    for n, t in o.items():
        lo.close(t, ref[n], 2 * T + D, "d" + n)

    c, cs = lo.conv_inputs(1, T, D, 4, dtype, 12, 3)
    g, s, r = lo.cuda(c), lo.cuda(cs), lo.double(c)
    p = ConvParams(1, T, D, 4, 3, code, 1, 0)
    y, fin = out(1, T, D), out(3, 3, D)
    run("gdn_conv_fwd", ctypes.byref(p), P(g["x"]), P(g["weight"]), P(g["bias"]), P(cu), P(g["h0"]), P(y), P(fin))
    y_ref, fin_ref = lo.conv(cu=good, **r)
    lo.close(y, y_ref, 4, "conv y")
    assert torch.equal(fin.cpu().double(), fin_ref)
    ws, nb = space(lib.gdn_conv_bwd_workspace_size, p)
    o = dict(x=out(1, T, D), weight=out(D, 4, dtype=F32), bias=out(D, dtype=F32), h0=out(3, 3, D))
    run("gdn_conv_bwd", ctypes.byref(p), P(g["x"]), None, P(g["weight"]), P(g["bias"]), P(cu), P(g["h0"]), P(s["d_y"]),
        P(s["d_fin"]), *(P(t) for t in o.values()), P(ws), nb)
    ref = lo.gradients(lambda **k: lo.conv(cu=good, **k), r, [t.double() for t in cs.values()])
    for n, t in o.items():
        if n == "h0":
            t, ref[n] = t[:2], ref[n][:2]
        lo.close(t, ref[n], T, "conv d" + n)
    assert new.untouched()


# ---- a captured training step ------------------------------------------------------------

@pytest.mark.parametrize("bits", [None, 8])
def test_a_captured_training_step_replays(bits):
    """Convolution, scan and their gradients in one graph (gradients returned, not
    accumulated, so that nothing of an earlier eager step is part of it), its workspaces
    and checkpoints in the graph's own memory; replays against the eager step."""
    T_ = 70
    d = lo.cuda(scan_layer(21, 2, T_))
    cu = lo.offsets([50, 13]).cuda()
    seed = torch.randn(1, T_, D, generator=torch.Generator().manual_seed(22)).cuda()
    names = ("proj", "weight", "bias", "c0", "h0", "dt", "A_log", "Bm", "Cm", "skip", "z", "dt_bias")

    def step():
        leaf = {n: d[n].detach().requires_grad_() for n in names}
        c, _ = gdn.causal_conv(leaf["proj"], leaf["weight"], leaf["bias"], cu, leaf["c0"], checkpoint_bits=bits)
        y, fin = gdn.selective_scan(c, **scan_args(leaf), cu_seqlens=cu, initial_state=leaf["h0"], checkpoint_bits=bits)
        return [y.detach(), fin.detach(), *torch.autograd.grad((y, fin), [leaf[n] for n in names], (seed, fin.detach()))]
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        step()
    cap.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        outs = step()
    for i in range(3):
        for n in ("proj", "dt", "z"):
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


# ---- padded offsets ----------------------------------------------------------------------

def test_thousands_of_empty_sequences():
    """Offsets padded to a fixed count, and a run of empty sequences inside a tile: both
    passes as without the empty ones, whose states pass through."""
    lengths = [37, 0, 1] + [0] * 5000 + [70, 2] + [0] * 3000 + [25] + [0] * 7000
    real = [i for i, n in enumerate(lengths) if n]
    T_, C_, N_, S = 150, 40, 5, len(lengths)  # 15 tokens behind the last sequence
    cu, few = lo.offsets(lengths).cuda(), lo.offsets([lengths[i] for i in real]).cuda()
    d, s = lo.scan_inputs(1, T_, C_, N_, 1, F32, 23, S)
    c, cs = lo.conv_inputs(1, T_, C_, 4, F32, 24, S)
    d, s, c, cs = (lo.cuda(t) for t in (d, s, c, cs))
    a, o = [d[n] for n in ("x", "dt", "A_log", "Bm", "Cm")], dict(skip=d["skip"], z=d["z"], dt_bias=d["dt_bias"])

    def passes(cu, at):
        h0, c0, df, cf = (t[at].contiguous() for t in (d["h0"], c["h0"], s["d_fin"], cs["d_fin"]))
        y, fin = gdn.scan_fwd(*a, **o, cu_seqlens=cu, initial_state=h0)
        g = gdn.scan_bwd(*a, s["d_y"], df, **o, cu_seqlens=cu, initial_state=h0)
        cy, cfin = gdn.conv_fwd(c["x"], c["weight"], c["bias"], cu, c0)
        cg = gdn.conv_bwd(c["x"], c["weight"], c["bias"], cs["d_y"], cf, cu, c0)
        return ([y, cy] + [v for k, v in [*g.items(), *cg.items()] if k != "dh0"], [fin, cfin, g["dh0"], cg["dh0"]])
    tokens, states = passes(cu, slice(None))
    ref_tokens, ref_states = passes(few, real)
    assert all(torch.equal(x, y) for x, y in zip(tokens, ref_tokens))
    empty = [i for i in range(S) if i not in real]
    for got, ref, through in zip(states, ref_states, (d["h0"], c["h0"], s["d_fin"], cs["d_fin"])):
        assert torch.equal(got[real], ref) and torch.equal(got[empty], through[empty])


# ---- sizes at both ends ------------------------------------------------------------------

def test_tensors_beyond_32_bit_offsets():
    """1.1 million tokens of 2048 channels: 2.25e9 elements, 4.5 GB a tensor, and workspaces
    of more than 4 GB.  The last sequence against the same tokens on their own."""
    T_, D_, N_, n = 1100000, 2048, 16, 300
    gen = torch.Generator(device="cuda").manual_seed(25)
    r = lambda *s, dtype=BF16: torch.randn(*s, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    x, dt, z, d_y = (r(1, T_, D_) for _ in range(4))
    Bm, Cm, h0, c0 = r(1, T_, 1, N_), r(1, T_, 1, N_), r(2, D_, N_, dtype=F32), r(2, 3, D_)
    w, bias, skip, dt_bias = r(D_, 4, dtype=F32), r(D_, dtype=F32), r(D_, dtype=F32), r(D_, dtype=F32) - 3
    A_log = torch.log(torch.arange(1, N_ + 1, device="cuda").float()).expand(D_, N_).contiguous()
    cu = torch.tensor([0, T_ - n, T_], device="cuda")
    end = lambda t: t[:, -n:].contiguous()  # noqa: E731

    y, fin = gdn.conv_fwd(x, w, bias, cu, c0)
    y1, fin1 = gdn.conv_fwd(end(x), w, bias, initial_state=c0[1:])
    assert torch.equal(end(y), y1) and torch.equal(fin[1:], fin1)
    del y
    g = gdn.conv_bwd(x, w, bias, d_y, None, cu, c0)
    g1 = gdn.conv_bwd(end(x), w, bias, end(d_y), initial_state=c0[1:])
    assert torch.equal(end(g["dx"]), g1["dx"]) and torch.equal(g["dh0"][1:], g1["dh0"])
    del g
    o = dict(skip=skip, dt_bias=dt_bias)
    y, fin = gdn.scan_fwd(x, dt, A_log, Bm, Cm, z=z, **o, cu_seqlens=cu, initial_state=h0)
    last = [end(x), end(dt), A_log, end(Bm), end(Cm)]
    y1, fin1 = gdn.scan_fwd(*last, z=end(z), **o, initial_state=h0[1:])
    lo.close(end(y), y1.cpu().double(), n, "y")
    lo.close(fin[1:], fin1.cpu().double(), n, "final state")
    assert y.isfinite().all()
    del y
    g = gdn.scan_bwd(x, dt, A_log, Bm, Cm, d_y, z=z, **o, cu_seqlens=cu, initial_state=h0)
    g1 = gdn.scan_bwd(*last, end(d_y), z=end(z), **o, initial_state=h0[1:])
    for k in ("dx", "ddt", "dz", "dBm", "dCm"):
        lo.close(end(g[k]), g1[k].cpu().double(), 2 * n + D_, k)
    lo.close(g["dh0"][1:], g1["dh0"].cpu().double(), 2 * n, "dh0")
    del g, x, dt, z, d_y
    rows = torch.randn(T_, D_, generator=gen, device="cuda", dtype=BF16)
    p = gdn.pack8(rows)
    p1 = gdn.pack8(rows[-n:])
    assert torch.equal(p.codes[-n:], p1.codes) and torch.equal(p.scales[-n:], p1.scales)
    assert torch.equal(gdn.unpack8(p)[-n:], gdn.unpack8(p1))
    del rows, p
    torch.cuda.empty_cache()


@pytest.mark.parametrize("packed", [False, True])
def test_no_sequences_at_all(packed):
    """B = 0, or offsets [0]: empty outputs, and parameters' gradients of 0."""
    B_, T_ = (1, 0) if packed else (0, 7)
    d, s = lo.scan_inputs(B_, T_, 40, 5, 1, F32, 26, 0)
    c, cs = lo.conv_inputs(B_, T_, 40, 4, F32, 27, 0)
    d, s, c, cs = (lo.cuda(t) for t in (d, s, c, cs))
    cu = torch.zeros(1, dtype=torch.int64, device="cuda") if packed else None
    a, o = [d[n] for n in ("x", "dt", "A_log", "Bm", "Cm")], dict(skip=d["skip"], z=d["z"], dt_bias=d["dt_bias"], cu_seqlens=cu)
    y, fin = gdn.scan_fwd(*a, **o, initial_state=d["h0"])
    g = gdn.scan_bwd(*a, s["d_y"], s["d_fin"], **o, initial_state=d["h0"])
    cy, cfin = gdn.conv_fwd(c["x"], c["weight"], c["bias"], cu, c["h0"])
    cg = gdn.conv_bwd(c["x"], c["weight"], c["bias"], cs["d_y"], cs["d_fin"], cu, c["h0"])
    assert y.shape == (B_, T_, 40) == cy.shape and fin.shape == (0, 40, 5) and cfin.shape == (0, 3, 40)
    torch.cuda.synchronize()
    for t in (g["dA_log"], g["dskip"], g["ddt_bias"], cg["dweight"], cg["dbias"]):
        assert t.numel() and (t == 0).all()
    if not packed:
        gdn.conv_decode(c["x"][:, :1], c["weight"], c["h0"], c["bias"])
        gdn.scan_decode(*(d[n][:, :1] for n in ("x", "dt")), d["A_log"], *(d[n][:, :1] for n in ("Bm", "Cm")), d["h0"])
