"""Linear attention with a decay for each head (linear_attn_fwd, linear_attn_bwd,
linear_attn_decode, linear_attention) against the 64-bit form of block_oracle: single tokens,
chunks and segments that end early, shared heads, packed sequences with empty ones among them,
decays of zero and of minus infinity, missing states."""
import ctypes
import math

import pytest
import torch

import block_oracle as bo
import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
from gated_deltanet_chunkwise_amd._linattn import LinattnParams

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# B, T, H, HV, K, V, dtype, lengths, initial state
CASES = [
    (1, 1, 1, 1, 64, 64, F32, None, False),
    (2, 1, 2, 4, 128, 128, BF16, None, True),
    (1, 7, 1, 3, 64, 128, BF16, None, True),
    (2, 63, 2, 2, 128, 64, F32, None, True),
    (1, 64, 2, 2, 128, 128, F32, None, True),
    (2, 65, 1, 2, 64, 64, BF16, None, True),
    (1, 128, 2, 2, 64, 128, BF16, None, False),
    (1, 129, 2, 2, 128, 64, BF16, None, True),
    (2, 300, 1, 2, 128, 128, BF16, None, True),
    (1, 330, 2, 2, 64, 64, F32, None, False),
    (1, 451, 1, 4, 64, 64, BF16, None, True),
    (1, 700, 1, 1, 64, 128, F32, None, True),
    (1, 451, 2, 2, 128, 64, BF16, [1, 0, 63, 64, 2, 200, 0, 121], True),
    (1, 450, 1, 3, 64, 64, F32, [128, 192, 130], False),
    (1, 200, 2, 4, 64, 128, BF16, [0, 190, 10, 0], True),
    (1, 300, 2, 2, 64, 64, BF16, [70, 150], True),       # ends before T
    (1, 100, 1, 2, 64, 64, BF16, [20, 30, 0], True),     # the same, in one segment
    (1, 90, 1, 1, 64, 64, F32, [0, 0], True),            # no token belongs to a sequence
    (1, 0, 1, 2, 64, 64, F32, [0, 0], True),             # no tokens at all
    (2, 0, 1, 2, 64, 64, BF16, None, True),
]
IDS = ["%dx%d-h%d-%d-k%d-v%d-%s%s" % (*c[:6], str(c[6])[6:], "" if c[7] is None else "-packed") for c in CASES]


def make(case, seed=1):
    B, T, H, HV, K, V, dtype, lengths, h0 = case
    cu = None if lengths is None else lo.offsets(lengths)
    S = B if cu is None else len(lengths)
    d, seeds, ld = bo.linattn_inputs(B, T, H, HV, K, V, dtype, seed, S, h0)
    return d, seeds, ld, cu, B * T if cu is None else int(cu[-1])


def rows_tol(dtype, T):
    """bf16: the result is rounded once and every term of it once more (the weighted product
    q.k, or the state where it meets q), each by at most half a step.  fp32: as states."""
    return 2 * torch.finfo(dtype).eps / 2 if dtype == BF16 else state_tol(T)


def state_tol(T):
    """Roundings of 2^-24: independent ones of T tokens' products and sums add in squares; of
    each a handful; 32 for the powers of the decay (an exponent x is off by at most x 2^-23,
    on a weight of 2^-x) and the longest sums within a matrix instruction."""
    return (32 + 4 * math.sqrt(T)) * 2.0 ** -24


def fwd(g, ld, cu, scale=1.0, **kw):
    return gdn.linear_attn_fwd(g["q"], g["k"], g["v"], ld.cuda(), None if cu is None else cu.cuda(), g["h0"], scale, **kw)


def bwd(g, s, ld, cu, scale=1.0):
    return gdn.linear_attn_bwd(g["q"], g["k"], g["v"], ld.cuda(), s["d_o"], s["d_fin"], None if cu is None else cu.cuda(),
                               g["h0"], scale)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    d, _, ld, cu, used = make(case)
    scale = case[4] ** -0.5
    o_ref, fin_ref = bo.linattn(log_decay=ld.double(), cu=cu, scale=scale, **lo.double(d))
    o, fin = fwd(lo.cuda(d), ld, cu, scale)
    bo.close(o, o_ref, rows_tol(case[6], case[1]), "o")
    bo.close(fin, fin_ref, state_tol(case[1]), "final state")
    assert (o.view(-1, *o.shape[2:])[used:] == 0).all()
    again = fwd(lo.cuda(d), ld, cu, scale)
    assert torch.equal(o, again[0]) and torch.equal(fin, again[1]), "the same call gives the same bits"


def reference_gradients(case, d, seeds, ld, cu, used, scale):
    rows = (torch.arange(case[0] * case[1]) < used).view(case[0], case[1], 1, 1)
    seed = torch.where(rows, seeds["d_o"].double(), 0.0)
    return lo.gradients(lambda **x: bo.linattn(log_decay=ld.double(), cu=cu, scale=scale, **x), lo.double(d),
                        (seed, seeds["d_fin"].double()))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    d, seeds, ld, cu, used = make(case, 2)
    scale = case[4] ** -0.5
    ref = reference_gradients(case, d, seeds, ld, cu, used, scale)
    g, s = lo.cuda(d), lo.cuda(seeds)
    got = bwd(g, s, ld, cu, scale)
    for k, name in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        bo.close(got[k], ref[name], rows_tol(case[6], case[1]), k)
        assert (got[k].view(-1, *got[k].shape[2:])[used:] == 0).all()
    if d["h0"] is not None:
        bo.close(got["dh0"], ref["h0"], state_tol(case[1]), "dh0")
    again = bwd(g, s, ld, cu, scale)
    assert all(torch.equal(got[k], again[k]) for k in got), "the same call gives the same bits"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,H,HV,K,V", [(1, 1, 1, 1, 64, 64), (3, 1, 2, 4, 128, 128), (2, 5, 3, 3, 64, 128), (5, 2, 1, 2, 128, 64)])
def test_decode(B, T, H, HV, K, V, dtype):
    d, _, ld = bo.linattn_inputs(B, T, H, HV, K, V, dtype, 3)
    o_ref, fin_ref = bo.linattn(log_decay=ld.double(), scale=0.5, **lo.double(d))
    g = lo.cuda(d)
    state, new = g["h0"].clone(), torch.full_like(g["h0"], float("nan"))
    o = gdn.linear_attn_decode(g["q"], g["k"], g["v"], ld.cuda(), state, 0.5, new_state=new)
    # fp32 throughout, bf16 rounded once
    bo.close(o, o_ref, state_tol(T + K) + (torch.finfo(dtype).eps / 2 if dtype == BF16 else 0), "o")
    bo.close(new, fin_ref, state_tol(T), "state")
    assert torch.equal(state, g["h0"]), "the state it starts from stays"
    o2 = gdn.linear_attn_decode(g["q"], g["k"], g["v"], ld.cuda(), state, 0.5)
    assert torch.equal(o2, o) and torch.equal(state, new), "in place"


def test_decode_continues_a_prompt():
    case = (2, 150, 2, 4, 128, 64, BF16, None, True)
    d, _, ld, _, _ = make(case, 4)
    o_ref, fin_ref = bo.linattn(log_decay=ld.double(), **lo.double(d))
    g = lo.cuda(d)
    cut = lambda a, b: {k: v if k == "h0" else v[:, a:b].contiguous() for k, v in g.items()}  # noqa: E731
    head, tail = cut(0, 139), cut(139, 150)
    o1, state = fwd(head, ld, None)
    outs = [o1]
    for t in range(11):
        q, k, v = (tail[n][:, t:t + 1].contiguous() for n in "qkv")
        outs.append(gdn.linear_attn_decode(q, k, v, ld.cuda(), state))
    bo.close(torch.cat(outs, 1), o_ref, rows_tol(BF16, 150), "o")
    bo.close(state, fin_ref, state_tol(150), "state")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [3, 200])
def test_decays_at_the_ends(dtype, T):
    """log_decay of 0 (nothing is forgotten), minus infinity and the lowest value (a token sees
    itself alone), and decays that vanish within a chunk."""
    B, H, K = 1, 4, 64
    d, seeds, _ = bo.linattn_inputs(B, T, H, H, K, K, dtype, 5)
    ld = torch.tensor([0.0, -math.inf, torch.finfo(F32).min, -5.0])
    # (the oracle's exp of the lowest value is 0, as of minus infinity)
    o_ref, fin_ref = bo.linattn(log_decay=ld.double(), **lo.double(d))
    g, s = lo.cuda(d), lo.cuda(seeds)
    o, fin = fwd(g, ld, None)
    for h in range(H):
        bo.close(o[:, :, h], o_ref[:, :, h], rows_tol(dtype, T), "o of head %d" % h)
        bo.close(fin[:, h], fin_ref[:, h], state_tol(T), "state of head %d" % h)
    ref = lo.gradients(lambda **x: bo.linattn(log_decay=ld.double(), **x), lo.double(d), [v.double() for v in seeds.values()])
    got = bwd(g, s, ld, None)
    for h in range(H):
        for k, name in (("dq", "q"), ("dk", "k"), ("dv", "v")):
            bo.close(got[k][:, :, h], ref[name][:, :, h], rows_tol(dtype, T), "%s of head %d" % (k, h))
        bo.close(got["dh0"][:, h], ref["h0"][:, h], state_tol(T), "dh0 of head %d" % h)
    state = g["h0"].clone()
    gdn.linear_attn_decode(g["q"], g["k"], g["v"], ld.cuda(), state)
    for h in range(H):
        bo.close(state[:, h], fin_ref[:, h], state_tol(T), "decode state of head %d" % h)


def test_slices_of_a_wider_projection():
    B, T, H, HV, K, V = 2, 150, 2, 4, 64, 128
    d, seeds, ld = bo.linattn_inputs(B, T, H, HV, K, V, BF16, 6)
    g, s = lo.cuda(d), lo.cuda(seeds)
    wide = torch.cat([g[n].flatten(2) for n in "qkv"] + [torch.full((B, T, 24), float("nan"), dtype=BF16, device="cuda")], -1)
    q, k, v, _ = wide.split([H * K, H * K, HV * V, 24], -1)
    w = dict(g, q=q.unflatten(-1, (H, K)), k=k.unflatten(-1, (H, K)), v=v.unflatten(-1, (HV, V)))
    assert all(torch.equal(a, b) for a, b in zip(fwd(w, ld, None), fwd(g, ld, None)))
    a, b = bwd(w, s, ld, None), bwd(g, s, ld, None)
    assert all(torch.equal(a[n], b[n]) and a[n].is_contiguous() for n in a)
    st = g["h0"].clone(), g["h0"].clone()
    o = [gdn.linear_attn_decode(x["q"], x["k"], x["v"], ld.cuda(), y) for x, y in zip((w, g), st)]
    assert torch.equal(*o) and torch.equal(*st)


def test_rows_off_16_bytes_are_refused():
    d, seeds, ld = bo.linattn_inputs(1, 20, 1, 1, 64, 64, BF16, 6)
    g, s = lo.cuda(d), lo.cuda(seeds)
    wide = torch.zeros(1, 20, 200, dtype=BF16, device="cuda")
    for bad in (wide[..., 4:68].unflatten(-1, (1, 64)), torch.zeros(1, 20, 68, dtype=BF16, device="cuda")[..., :64].unflatten(-1, (1, 64))):
        for call in (lambda w: fwd(w, ld, None), lambda w: bwd(w, s, ld, None),
                     lambda w: gdn.linear_attn_decode(w["q"], w["k"], w["v"], ld.cuda(), w["h0"])):
            for name in "qkv":
                with pytest.raises(gdn.GdnError) as e:
                    call(dict(g, **{name: bad}))
                assert e.value.status == 5


def test_a_sequence_does_not_see_its_neighbours():
    case = (1, 400, 2, 2, 64, 64, BF16, [70, 130, 200], True)
    d, seeds, ld, cu, _ = make(case)
    g, s = lo.cuda(d), lo.cuda(seeds)
    bad, sb = {k: v.clone() for k, v in g.items()}, {k: v.clone() for k, v in s.items()}
    for t in (bad["q"], bad["k"], bad["v"], sb["d_o"]):
        t[0, 70:200] = float("nan")
    bad["h0"][1], sb["d_fin"][1] = float("inf"), float("nan")
    (o, fin), (o2, fin2) = fwd(g, ld, cu), fwd(bad, ld, cu)
    a, b = bwd(g, s, ld, cu), bwd(bad, sb, ld, cu)
    for x, y in ((o, o2), *((a[k], b[k]) for k in ("dq", "dk", "dv"))):
        assert torch.equal(x[0, :70], y[0, :70]) and torch.equal(x[0, 200:], y[0, 200:])
    for x, y in ((fin, fin2), (a["dh0"], b["dh0"])):
        assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2])


def test_a_nan_reaches_what_the_documentation_says():
    d, _, ld = bo.linattn_inputs(1, 200, 1, 2, 64, 64, BF16, 7)
    g = lo.cuda(d)
    o, fin = fwd(g, ld, None)
    q = dict(g, q=g["q"].clone())
    q["q"][0, 90] = float("nan")
    o2, fin2 = fwd(q, ld, None)
    assert torch.equal(fin, fin2) and torch.equal(o[0, :90], o2[0, :90]) and torch.equal(o[0, 91:], o2[0, 91:])
    assert o2[0, 90].isnan().all()
    for name in "kv":
        w = dict(g, **{name: g[name].clone()})
        w[name][0, 90] = float("inf")
        o2, fin2 = fwd(w, ld, None)
        assert torch.equal(o[0, :64], o2[0, :64]) and not fin2.isfinite().any() and not o2[0, 90:].isfinite().any()


def params(case, packed=True):
    B, T, H, HV, K, V, dtype, lengths, _ = case
    return LinattnParams(B, T, H, HV, K, V, len(lengths) if lengths else 0, gdn.GDN_BF16 if dtype == BF16 else gdn.GDN_F32, 1.0, 0, 0, 0)


def test_rows_behind_the_last_sequence_stay_and_nothing_is_written_outside():
    """Through the C entries: without GDN_ZERO_REST rows of o behind the last sequence are left
    as they were; guard bands around every output and a workspace of NaN."""
    case = (1, 300, 2, 4, 64, 128, BF16, [70, 0, 150], True)
    d, seeds, ld, cu, used = make(case)
    g, s, ldc, cuc = lo.cuda(d), lo.cuda(seeds), ld.cuda(), cu.cuda()
    lib, p = gdn.load_library(), params(case)
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    guarded = {}

    def out(name, shape, dtype):
        n = math.prod(shape)
        whole = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
        guarded[name] = whole
        return whole[256:256 + n].view(shape)

    def space(nb):
        return torch.full((nb + 256,), 0xFF, dtype=torch.uint8, device="cuda")

    o, fin = out("o", (1, 300, 4, 128), BF16), out("fin", (3, 4, 64, 128), F32)
    nb = lib.gdn_linattn_fwd_workspace_size(ctypes.byref(p), 1)
    ws = space(nb)
    assert nb > 0 and lib.gdn_linattn_fwd(ctypes.byref(p), P(g["q"]), P(g["k"]), P(g["v"]), P(ldc), P(cuc), P(g["h0"]), P(o),
                                          P(fin), P(ws), nb, stream) == 0
    want, want_fin = fwd(g, ld, cu)
    assert (o[0, used:] == 7).all() and torch.equal(o[0, :used], want[0, :used]) and torch.equal(fin, want_fin)
    assert (ws[nb:] == 0xFF).all()
    dq, dk = out("dq", (1, 300, 2, 64), BF16), out("dk", (1, 300, 2, 64), BF16)
    dv, dh0 = out("dv", (1, 300, 4, 128), BF16), out("dh0", (3, 4, 64, 128), F32)
    nb = lib.gdn_linattn_bwd_workspace_size(ctypes.byref(p), 1)
    ws = space(nb)
    assert lib.gdn_linattn_bwd(ctypes.byref(p), P(g["q"]), P(g["k"]), P(g["v"]), P(ldc), P(cuc), P(g["h0"]), P(s["d_o"]),
                               P(s["d_fin"]), P(dq), P(dk), P(dv), P(dh0), P(ws), nb, stream) == 0
    got = bwd(g, s, ld, cu)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv), ("dh0", dh0)):
        assert torch.equal(t, got[name]), name
    assert (ws[nb:] == 0xFF).all()
    for name, whole in guarded.items():
        assert (whole[:256] == 7).all() and (whole[-256:] == 7).all(), name
