"""Selective state space scan (scan_fwd, scan_bwd, scan_decode, selective_scan) against
the 64-bit form of layer_oracle: state counts and channels off the wave's sizes, groups,
single tokens, tiles that end inside a sequence and sequences that end inside a tile,
empty ones, extreme decays, missing options."""
import ctypes

import pytest
import torch

import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# B, T, D, N, G, dtype, lengths, options present (h0, skip, gate, bias)
ALL = dict(h0=True, skip=True, gate=True, bias=True)
NONE = dict(h0=False, skip=False, gate=False, bias=False)
CASES = [
    (1, 1, 1, 1, 1, F32, None, NONE),
    (2, 1, 64, 16, 1, BF16, None, ALL),
    (1, 7, 70, 5, 1, F32, None, ALL),
    (2, 64, 130, 16, 2, BF16, None, dict(ALL, gate=False)),
    (1, 65, 64, 16, 1, F32, None, ALL),
    (2, 200, 96, 8, 1, BF16, None, dict(ALL, h0=False)),
    (1, 150, 66, 13, 3, BF16, None, dict(ALL, skip=False)),
    (1, 139, 64, 17, 1, F32, None, dict(ALL, bias=False)),
    (2, 70, 64, 32, 2, BF16, None, ALL),
    (1, 100, 64, 33, 1, F32, None, ALL),
    (1, 90, 70, 64, 1, BF16, None, ALL),
    (1, 515, 64, 16, 1, F32, None, ALL),
    (1, 300, 70, 16, 1, BF16, [1, 0, 63, 64, 2, 130, 0, 40], ALL),
    (1, 260, 64, 7, 1, F32, [128, 64, 68], dict(ALL, h0=False, gate=False)),
    (1, 200, 64, 40, 1, F32, [0, 190, 10, 0], ALL),
    (1, 200, 64, 16, 1, BF16, [70, 50], ALL),    # ends before T
    (1, 0, 64, 16, 1, F32, [0, 0], ALL),         # no tokens at all
    (2, 0, 64, 16, 1, BF16, None, ALL),
]
IDS = ["%dx%dx%d-n%d-g%d-%s%s" % (c[0], c[1], c[2], c[3], c[4], str(c[5])[6:], "" if c[6] is None else "-packed") for c in CASES]


def make(case, seed=1):
    B, T, D, N, G, dtype, lengths, opts = case
    cu = None if lengths is None else lo.offsets(lengths)
    S = B if cu is None else len(lengths)
    d, seeds = lo.scan_inputs(B, T, D, N, G, dtype, seed, S, **opts)
    return d, seeds, cu, B * T if cu is None else int(cu[-1])


def fwd(g, cu, **kw):
    return gdn.scan_fwd(g["x"], g["dt"], g["A_log"], g["Bm"], g["Cm"], g["skip"], g["z"], g["dt_bias"],
                        None if cu is None else cu.cuda(), g["h0"], **kw)


def bwd(g, s, cu, x=None, z=None):
    return gdn.scan_bwd(g["x"] if x is None else x, g["dt"], g["A_log"], g["Bm"], g["Cm"], s["d_y"], s["d_fin"],
                        g["skip"], g["z"] if z is None else z, g["dt_bias"], None if cu is None else cu.cuda(), g["h0"])


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    d, _, cu, used = make(case)
    y_ref, fin_ref = lo.scan(cu=cu, **lo.double(d))
    y, fin = fwd(lo.cuda(d), cu)
    D = case[2]
    lo.close(y.view(-1, D)[:used], y_ref.view(-1, D)[:used], case[1], "y")
    lo.close(fin, fin_ref, case[1], "final state")


def check_backward(case, seed=2):
    d, seeds, cu, used = make(case, seed)
    T, D = case[1], case[2]
    rows = (torch.arange(case[0] * T) < used).view(case[0], T, 1)
    ref_seed = torch.where(rows, seeds["d_y"].double(), 0.0)
    ref = lo.gradients(lambda **k: lo.scan(cu=cu, **k), lo.double(d), (ref_seed, seeds["d_fin"].double()))
    g, s = lo.cuda(d), lo.cuda(seeds)
    got = bwd(g, s, cu)
    n = case[0] * T
    for k, name, steps in (("dx", "x", T), ("ddt", "dt", T), ("dBm", "Bm", T + D), ("dCm", "Cm", T + D), ("dz", "z", T),
                           ("dA_log", "A_log", n + T), ("dskip", "skip", n), ("ddt_bias", "dt_bias", n + T), ("dh0", "h0", T)):
        if d[name] is not None:
            lo.close(got[k], ref[name], steps, k)
    assert ("dz" in got) == (d["z"] is not None)
    again = bwd(g, s, cu)
    assert all(torch.equal(got[k], again[k]) for k in got), "the same call gives the same bits"


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    check_backward(case)


def test_many_channels_run_in_one_pass():
    # enough waves that the sequences are not cut into tiles
    case = (4, 150, 16448, 4, 1, BF16, None, ALL)
    d, _, cu, used = make(case)
    y_ref, fin_ref = lo.scan(**lo.double(d))
    y, fin = fwd(lo.cuda(d), cu)
    lo.close(y, y_ref, 150, "y")
    lo.close(fin, fin_ref, 150, "final state")


def test_more_rows_of_bm_and_cm_than_one_grid_sums():
    # 2100 * 64 groups * 2 * 64 states: beyond 2^24 values the sums' workgroups loop
    check_backward((1, 2100, 64, 64, 64, F32, None, ALL))


def forward_workspace(case, length):
    """gdn_scan_fwd_workspace_size() of a case cut into tiles of `length` tokens."""
    B, T, D, N, G = case[:5]
    up = lambda b: -(-b // 256) * 256  # noqa: E731
    np_ = 8 if N <= 8 else 16 * -(-N // 16)
    tiles = -(-T // length) * (1 if case[6] is not None else B)
    return up(up(tiles * np_ * D * 4) + tiles * D * 4) + 2 * up(B * T * G * np_ * 4)


@pytest.mark.parametrize("case,length", [
    ((2, 1030, 2048, 16, 1, BF16, None, ALL), 32),
    ((1, 18500, 2048, 16, 1, BF16, [9000, 0, 77, 9423], ALL), 80),          # rows sent for twice per tile
    ((1, 17001, 2040, 13, 1, F32, [1, 16900, 100], dict(ALL, gate=False)), 72),
    ((1, 2201, 4096, 32, 1, F32, [2100, 101], ALL), 40),                     # two waves per channel, five groups
    ((2, 901, 4100, 40, 2, BF16, None, ALL), 48),                            # three waves, six groups
    ((1, 9000, 4096, 20, 2, BF16, [5000, 3900], ALL), 144)], ids=lambda v: str(v) if isinstance(v, int) else "%dx%dx%d-n%d" % v[:4])
def test_long_tiles(case, length):
    """The tiles of large problems, checked on 64 channels of each group (channels do not
    see each other); the workspace tells their length."""
    from gated_deltanet_chunkwise_amd._layers import ScanParams
    B, T, D, N, G, dtype, lengths, _ = case
    p = ScanParams(B, T, D, G, N, 0 if lengths is None else len(lengths), 0 if dtype == F32 else 1, 0, 0, 0, 0, 0)
    nb = gdn.load_library().gdn_scan_fwd_workspace_size(ctypes.byref(p), int(lengths is not None))
    assert nb == forward_workspace(case, length), "another tile length than this case is for"
    d, _, cu, used = make(case)
    pick = torch.cat([torch.randperm(D // G, generator=torch.Generator().manual_seed(g))[:64].sort()[0] + g * (D // G)
                      for g in range(G)])
    part = {k: v if v is None or k in ("Bm", "Cm") else v[pick] if k in ("A_log", "skip", "dt_bias") else
            v[:, pick] if k == "h0" else v[..., pick] for k, v in d.items()}
    y_ref, fin_ref = lo.scan(cu=cu, **lo.double(part))
    y, fin = fwd(lo.cuda(d), cu)
    steps = T if lengths is None else max(lengths)
    lo.close(y[..., pick.cuda()].view(-1, len(pick))[:used], y_ref.view(-1, len(pick))[:used], steps, "y")
    lo.close(fin[:, pick.cuda()], fin_ref, steps, "final state")
    assert y.isfinite().all() and fin.isfinite().all()


def test_extreme_decays_and_time_steps():
    """States that vanish within a token (A D of about -400, also across whole tiles), that
    never decay (A about -1e-9), and D beyond softplus's threshold and below 1e-9."""
    d, seeds = lo.scan_inputs(1, 200, 64, 8, 1, F32, 3)
    d["A_log"][:, 0], d["A_log"][:, 1], d["A_log"][:, 2] = 3.0, -20.0, -100.0
    d["dt"][0, 50:60] = 30.0
    d["dt"][0, 100:110] = -40.0
    y_ref, fin_ref = lo.scan(**lo.double(d))
    g, s = lo.cuda(d), lo.cuda(seeds)
    y, fin = fwd(g, None)
    lo.close(y, y_ref, 200, "y")
    lo.close(fin, fin_ref, 200, "final state")
    ref = lo.gradients(lo.scan, lo.double(d), (seeds["d_y"].double(), seeds["d_fin"].double()))
    got = bwd(g, s, None)
    for k, name in (("dx", "x"), ("ddt", "dt"), ("dBm", "Bm"), ("dCm", "Cm"), ("dz", "z"), ("dA_log", "A_log"),
                    ("dskip", "skip"), ("ddt_bias", "dt_bias"), ("dh0", "h0")):
        lo.close(got[k], ref[name], 400, k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("low", [-float("inf"), "lowest"])
def test_tokens_masked_by_their_time_step(dtype, low):
    """dt of minus infinity, or the type's lowest value: D = 0, so the token leaves the state
    as it was and takes no gradient of its own; whole tiles of them among others."""
    d, seeds = lo.scan_inputs(1, 130, 64, 16, 1, dtype, 13)
    low = torch.finfo(dtype).min if low == "lowest" else low
    mask = torch.zeros(130, dtype=torch.bool)
    mask[[0, 5, 129]] = True
    mask[40:100] = True
    d["dt"][0, mask] = low
    r = lo.double(d)
    y_ref, fin_ref = lo.scan(**r)
    g, s = lo.cuda(d), lo.cuda(seeds)
    y, fin = fwd(g, None)
    lo.close(y, y_ref, 130, "y")
    lo.close(fin, fin_ref, 130, "final state")
    # (the oracle's own slope at minus infinity is not a number: its inputs at -1000 give the same D)
    at = dict(r, dt=r["dt"].clamp(min=-1000.0))
    ref = lo.gradients(lo.scan, at, (seeds["d_y"].double(), seeds["d_fin"].double()))
    got = bwd(g, s, None)
    assert (got["ddt"][0, mask.cuda()] == 0).all()
    for k, name in (("dx", "x"), ("ddt", "dt"), ("dBm", "Bm"), ("dCm", "Cm"), ("dz", "z"), ("dA_log", "A_log"),
                    ("dskip", "skip"), ("ddt_bias", "dt_bias"), ("dh0", "h0")):
        lo.close(got[k], ref[name], 2 * 130 + 64, k)
    state = g["h0"].clone()
    y1 = gdn.scan_decode(g["x"], g["dt"], g["A_log"], g["Bm"], g["Cm"], state, g["skip"], g["z"], g["dt_bias"])
    lo.close(y1, y_ref, 130, "decode y")
    lo.close(state, fin_ref, 130, "decode state")


def test_rows_behind_the_last_sequence_stay():
    d, seeds, cu, used = make(CASES[15])
    g, s = lo.cuda(d), lo.cuda(seeds)
    from gated_deltanet_chunkwise_amd._layers import ScanParams
    y = torch.full_like(g["x"], 7.0)
    p = ScanParams(1, 200, 64, 1, 16, 2, gdn.GDN_BF16, 0, 0, 0, 0, 0)
    lib = gdn.load_library()
    nb = lib.gdn_scan_fwd_workspace_size(ctypes.byref(p), 1)
    ws, c = torch.empty(nb, dtype=torch.uint8, device="cuda"), cu.cuda()
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = lib.gdn_scan_fwd(ctypes.byref(p), P(g["x"]), P(g["dt"]), P(g["A_log"]), P(g["Bm"]), P(g["Cm"]), None, None,
                          None, P(c), None, P(y), None, P(ws), nb,
                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    assert (y[0, used:] == 7).all() and not (y[0, :used] == 7).all()
    got = bwd(g, s, cu)
    for k in ("dx", "ddt", "dz", "dBm", "dCm"):
        assert (got[k][0, used:] == 0).all(), k


def test_slices_of_wider_tensors():
    d, seeds = lo.scan_inputs(2, 70, 64, 16, 2, BF16, 4)
    g, s = lo.cuda(d), lo.cuda(seeds)
    xz = torch.cat([g["x"], g["z"], g["dt"]], -1)
    bc = torch.full((2, 70, 80), float("nan"), dtype=BF16, device="cuda")
    bc[..., 8:40], bc[..., 41:73] = g["Bm"].flatten(2), g["Cm"].flatten(2)  # Cm off 4 bytes
    w = dict(g, x=xz[..., :64], z=xz[..., 64:128], dt=xz[..., 128:], Bm=bc[..., 8:40].unflatten(-1, (2, 16)),
             Cm=bc[..., 41:73].unflatten(-1, (2, 16)))
    assert all(torch.equal(a, b) for a, b in zip(fwd(w, None), fwd(g, None)))
    a, b = bwd(w, s, None), bwd(g, s, None)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_rows_further_apart_than_32_bits_reach():
    ld, T, D = 1 << 26, 40, 64
    big = torch.empty(T * ld, dtype=BF16, device="cuda")
    d, _ = lo.scan_inputs(1, T, D, 16, 1, BF16, 5)
    g = lo.cuda(d)
    view = lambda off, t: big.as_strided((1, T, D), (T * ld, ld, 1), off).copy_(t)  # noqa: E731
    w = dict(g, x=view(0, g["x"]), z=view(1000, g["z"]), dt=view(5000, g["dt"]))
    assert all(torch.equal(a, b) for a, b in zip(fwd(w, None), fwd(g, None)))


def test_a_sequence_does_not_see_its_neighbours():
    case = (1, 300, 64, 16, 1, BF16, [70, 130, 100], ALL)
    d, seeds, cu, _ = make(case)
    g, s = lo.cuda(d), lo.cuda(seeds)
    bad = {k: None if v is None else v.clone() for k, v in g.items()}
    sb = {k: v.clone() for k, v in s.items()}
    for k in ("x", "dt", "Bm", "Cm", "z"):
        bad[k][0, 70:200] = float("nan")
    bad["h0"][1] = float("inf")
    sb["d_y"][0, 70:200] = float("nan")
    sb["d_fin"][1] = float("nan")
    (y, fin), (y2, fin2) = fwd(g, cu), fwd(bad, cu)
    a, b = bwd(g, s, cu), bwd(bad, sb, cu)
    for rows in (slice(0, 70), slice(200, 300)):
        assert torch.equal(y[0, rows], y2[0, rows])
        assert all(torch.equal(a[k][0, rows], b[k][0, rows]) for k in ("dx", "ddt", "dz", "dBm", "dCm"))
    assert torch.equal(fin[[0, 2]], fin2[[0, 2]]) and torch.equal(a["dh0"][[0, 2]], b["dh0"][[0, 2]])


@pytest.mark.parametrize("B,T,D,N,G,dtype,inplace,opts", [
    (1, 1, 64, 16, 1, BF16, True, ALL), (5, 1, 70, 13, 1, F32, False, ALL), (3, 2, 66, 4, 3, BF16, True, NONE),
    (2, 3, 33, 64, 1, F32, False, dict(ALL, gate=False)), (7, 1, 40, 1, 2, BF16, False, ALL), (2, 1, 64, 20, 1, F32, True, ALL)])
def test_decode(B, T, D, N, G, dtype, inplace, opts):
    d, _ = lo.scan_inputs(B, T, D, N, G, dtype, 6, **dict(opts, h0=True))
    y_ref, fin_ref = lo.scan(**lo.double(d))
    g = lo.cuda(d)
    state = g["h0"].clone()
    new = None if inplace else torch.full_like(state, float("nan"))
    y = gdn.scan_decode(g["x"], g["dt"], g["A_log"], g["Bm"], g["Cm"], state, g["skip"], g["z"], g["dt_bias"], new)
    lo.close(y, y_ref, T, "y")
    lo.close(state if inplace else new, fin_ref, T, "state")
    if not inplace:
        assert torch.equal(state, g["h0"])


@pytest.mark.parametrize("dtype,D", [(BF16, 72), (F32, 33)])
def test_backward_from_checkpoints(dtype, D):
    d, seeds = lo.scan_inputs(2, 70, D, 16, 1, dtype, 7)
    g, s = lo.cuda(d), lo.cuda(seeds)
    px, pz = gdn.pack8(g["x"]), gdn.pack8(g["z"])
    a = bwd(g, s, None, px, pz)
    b = bwd(dict(g, x=gdn.unpack8(px), z=gdn.unpack8(pz)), s, None)
    assert all(torch.equal(a[k], b[k]) for k in a), "the checkpoints' values, read in place"


@pytest.mark.parametrize("case", [
    (1, 300, 70, 16, 1, BF16, [1, 0, 63, 64, 2, 130, 0, 40], ALL),
    (1, 200, 66, 33, 1, F32, [0, 120, 50], ALL),            # ends before T
    (2, 90, 130, 64, 2, BF16, None, ALL),
    (1, 150, 64, 20, 1, F32, [150], dict(ALL, gate=False))], ids=["packed", "n33", "n64", "n20"])
def test_backward_from_checkpoints_packed_and_with_many_states(case):
    d, seeds, cu, used = make(case, 12)
    g, s = lo.cuda(d), lo.cuda(seeds)
    px = gdn.pack8(g["x"])
    pz = None if g["z"] is None else gdn.pack8(g["z"])
    at = dict(g, x=gdn.unpack8(px), z=None if pz is None else gdn.unpack8(pz))
    a, b = bwd(g, s, cu, px, pz), bwd(at, s, cu)
    assert a.keys() == b.keys() and all(torch.equal(a[k], b[k]) for k in a)
    live = (torch.arange(case[1]) < used)[:, None] | torch.tensor(cu is None)
    ref = lo.gradients(lambda **k: lo.scan(cu=cu, **k), lo.double({k: None if v is None else v.cpu() for k, v in at.items()}),
                       (torch.where(live, seeds["d_y"].double(), 0.0), seeds["d_fin"].double()))
    n = case[0] * case[1]
    for k, name in (("dx", "x"), ("ddt", "dt"), ("dBm", "Bm"), ("dCm", "Cm"), ("dz", "z"), ("dA_log", "A_log"),
                    ("dskip", "skip"), ("ddt_bias", "dt_bias"), ("dh0", "h0")):
        if d[name] is not None:
            lo.close(a[k], ref[name], 2 * n + case[2], k)


@pytest.mark.parametrize("bits", [None, 8])
def test_autograd(bits):
    d, seeds = lo.scan_inputs(2, 40, 64, 8, 1, F32, 8)
    r = lo.double(d)
    at = dict(r)
    if bits:
        for k in ("x", "z"):
            at[k] = lo.unpack(*lo.pack(d[k]))
    ref = lo.gradients(lo.scan, at, (seeds["d_y"].double(), seeds["d_fin"].double()))
    leaf = {k: v.cuda().requires_grad_() for k, v in d.items()}
    y, fin = gdn.selective_scan(leaf["x"], leaf["dt"], leaf["A_log"], leaf["Bm"], leaf["Cm"], leaf["skip"], leaf["z"],
                                leaf["dt_bias"], initial_state=leaf["h0"], checkpoint_bits=bits)
    lo.close(y, lo.scan(**r)[0], 40, "y")
    ((y * seeds["d_y"].cuda()).sum() + (fin * seeds["d_fin"].cuda()).sum()).backward()
    for k in leaf:
        lo.close(leaf[k].grad, ref[k], 150, "d" + k)


def test_autograd_of_the_final_state_alone():
    d, seeds = lo.scan_inputs(1, 20, 64, 8, 1, F32, 9)
    ref = lo.gradients(lo.scan, lo.double(d), (None, seeds["d_fin"].double()))
    leaf = {k: v.cuda().requires_grad_() for k, v in d.items()}
    _, fin = gdn.selective_scan(leaf["x"], leaf["dt"], leaf["A_log"], leaf["Bm"], leaf["Cm"], leaf["skip"], leaf["z"],
                                leaf["dt_bias"], initial_state=leaf["h0"])
    (fin * seeds["d_fin"].cuda()).sum().backward()
    for k in ("x", "dt", "Bm", "A_log", "h0"):
        lo.close(leaf[k].grad, ref[k], 64, "d" + k)
    assert (leaf["z"].grad == 0).all()


def test_gradient_against_differences():
    d, _ = lo.scan_inputs(1, 12, 8, 4, 1, F32, 10)
    g = lo.cuda(d)
    seed = torch.randn(1, 12, 8, generator=torch.Generator().manual_seed(1)).cuda()
    got = bwd(g, dict(d_y=seed, d_fin=None), None)
    # central differences of step 2^-6 along unit directions: e^2 / 6 = 4e-5 of third
    # derivatives of order 1 to 10, and the fp32 forward's rounding 2^-24 * 10 / e = 4e-5
    e = 2.0 ** -6
    for name, key in (("x", "dx"), ("dt", "ddt"), ("Bm", "dBm"), ("Cm", "dCm"), ("z", "dz"), ("A_log", "dA_log"),
                      ("skip", "dskip"), ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        v = torch.randn(g[name].shape, generator=torch.Generator().manual_seed(2)).cuda()
        v /= v.norm()
        L = []
        for sgn in (1, -1):
            y, _ = fwd(dict(g, **{name: g[name] + sgn * e * v}), None)
            L.append(float((y.double() * seed.double()).sum()))
        num, ana = (L[0] - L[1]) / (2 * e), float((got[key].double() * v.double()).sum())
        assert abs(num - ana) <= 1e-3 * (1 + abs(ana)), (name, num, ana)


def test_other_stream_and_graph_replay():
    d, seeds = lo.scan_inputs(1, 200, 64, 16, 1, BF16, 11)
    g, s = lo.cuda(d), lo.cuda(seeds)
    ref = fwd(g, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fwd(g, None, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    state = g["h0"].clone()

    def work():
        y, fin = fwd(g, None)
        gr = bwd(g, s, None)
        z = gdn.scan_decode(g["x"][:, :1], g["dt"][:, :1], g["A_log"], g["Bm"][:, :1], g["Cm"][:, :1], g["h0"],
                            g["skip"], g["z"][:, :1], g["dt_bias"], new_state=state)
        return [y, fin, z, state, *gr.values()]
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(3):
        g["x"].copy_(torch.randn(1, 200, 64, generator=torch.Generator().manual_seed(20 + i)))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for o in outs]
        eager = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager)), i
