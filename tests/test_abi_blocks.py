"""The C entries of linear attention and of the norms around a block on the CPU: sizes,
pointers, alignment and workspaces are validated before anything is enqueued (no address is
ever read; without a GPU a call that gets as far as enqueuing answers GDN_ERR_LAUNCH)."""
import ctypes

import pytest

import gated_deltanet_chunkwise_amd as gdn
from gated_deltanet_chunkwise_amd._linattn import LinattnParams
from gated_deltanet_chunkwise_amd._norms import GatedNormParams, ResidualNormParams

OK, ENULL, ESHAPE, EDTYPE, EUNSUP, EALIGN, EWS, ELAUNCH = range(8)
BIG = 1 << 46


def made(cls, defaults, kw):
    d = dict(defaults, **kw)
    return cls(*(d[n] for n, _ in cls._fields_))


def LP(**kw):
    return made(LinattnParams, dict(B=2, T=700, H=2, HV=4, K=64, V=128, num_seqs=0, dtype=gdn.GDN_BF16, scale=1.0, q_stride=0,
                                    k_stride=0, v_stride=0), kw)


def GP(**kw):
    return made(GatedNormParams, dict(B=2, T=20, H=4, D=64, dtype=gdn.GDN_BF16, gate_first=0, eps=1e-6, x_stride=0, z_stride=0), kw)


def RP(**kw):
    return made(ResidualNormParams, dict(B=2, T=20, C=64, dtype=gdn.GDN_BF16, residual_dtype=gdn.GDN_F32, eps=1e-6, x_stride=0,
                                         residual_stride=0), kw)


def entry(name, names, sized=False):
    """The entry with fake, aligned addresses by name; keywords replace some."""
    def call(p, ws_bytes=BIG, **given):
        base = {n: 0x100000 * (i + 1) for i, n in enumerate(names.split())}
        if "cu" in base:
            base["cu"] = None
        base.update(given)
        args = list(base.values()) + ([ws_bytes] if sized else [])
        return getattr(gdn.load_library(), name)(p and ctypes.byref(p), *args, None)
    return call


fwd = entry("gdn_linattn_fwd", "q k v log_decay cu h0 o fin ws", True)
bwd = entry("gdn_linattn_bwd", "q k v log_decay cu h0 d_o d_fin dq dk dv dh0 ws", True)
decode = entry("gdn_linattn_decode", "q k v log_decay state new o")
gfwd = entry("gdn_gated_norm_fwd", "x weight z y")
gbwd = entry("gdn_gated_norm_bwd", "x weight z d_y dx dz dweight ws", True)
rfwd = entry("gdn_residual_norm_fwd", "x residual weight post scale h new")
rbwd = entry("gdn_residual_norm_bwd", "x residual weight post scale d_h d_new dx dres dweight dpost dscale ws", True)


def size(name, p, *packed):
    return getattr(gdn.load_library(), name)(p and ctypes.byref(p), *packed)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), EDTYPE), (dict(dtype=gdn.GDN_F16), EDTYPE), (dict(dtype=gdn.GDN_BF16 | 0x200), EDTYPE), (dict(H=0), ESHAPE),
    (dict(HV=0), ESHAPE), (dict(HV=3), ESHAPE), (dict(HV=1), ESHAPE), (dict(K=32), EUNSUP), (dict(V=96), EUNSUP), (dict(K=256), EUNSUP),
    (dict(B=-1), ESHAPE), (dict(T=-1), ESHAPE), (dict(q_stride=127), ESHAPE), (dict(k_stride=-128), ESHAPE), (dict(v_stride=511), ESHAPE),
    (dict(B=2, T=(1 << 30) - 100), EUNSUP), (dict(B=1 << 16, T=1 << 15), EUNSUP),
    (dict(q_stride=1 << 24), EUNSUP), (dict(v_stride=1 << 40), EUNSUP), (dict(H=1 << 20, HV=1 << 20, T=1), EUNSUP),
    (dict(H=(1 << 31) - 1, HV=(1 << 31) - 1), EUNSUP)])
def test_linattn_sizes(kw, status):
    p = LP(**kw)
    assert fwd(p) == status and bwd(p) == status and decode(p) == status
    for name in ("gdn_linattn_fwd_workspace_size", "gdn_linattn_bwd_workspace_size"):
        assert size(name, p, 0) == 0


def test_linattn_packed_rules():
    cu = 0x9000000
    for call in (fwd, bwd):
        assert call(LP(B=2, num_seqs=3), cu=cu) == ESHAPE      # one row of tokens
        assert call(LP(B=1, num_seqs=-1), cu=cu) == ESHAPE
        assert call(LP(B=1, num_seqs=0), cu=cu) == ESHAPE      # tokens of no sequence
        assert call(LP(B=1, num_seqs=2), cu=cu + 4) == EALIGN
        assert call(None) == ENULL
    assert decode(LP(B=1, num_seqs=2)) == ESHAPE and decode(None) == ENULL


@pytest.mark.parametrize("call,P_,required,optional,small", [
    (fwd, LP, "q k v o log_decay ws", "h0 fin", "log_decay"),
    (bwd, LP, "q k v d_o dq dk dv log_decay ws", "h0 d_fin dh0", "log_decay"),
    (decode, LP, "q k v o state new log_decay", "", "log_decay"),
    (gfwd, GP, "x weight y", "z", ""), (gbwd, GP, "x weight d_y dx dz dweight ws", "z", ""),
    (rfwd, RP, "x residual weight h new", "post scale", ""),
    (rbwd, RP, "x residual weight d_h dx dres dweight ws", "post scale d_new dpost dscale", "")])
def test_pointers(call, P_, required, optional, small):
    for n in required.split():
        assert call(P_(), **{n: None}) == ENULL, n
    for n in required.split() + optional.split():
        assert call(P_(), **{n: 0x100001}) == EALIGN, n
    if P_ is LP:  # rows and states: 16 bytes
        for n in required.split() + optional.split():
            if n not in ("ws", "log_decay"):
                assert call(P_(), **{n: 0x100008}) == EALIGN, n
    # what may be missing is not asked for: a later check answers
    for n in optional.split():
        assert call(P_(), **{n: None}, **{required.split()[0]: 0x100001}) == EALIGN, n


def test_linattn_rows_are_whole_vectors():
    for kw in (dict(q_stride=132), dict(k_stride=130), dict(v_stride=513)):
        assert fwd(LP(**kw)) == EALIGN and bwd(LP(**kw)) == EALIGN and decode(LP(**kw)) == EALIGN
    assert fwd(LP(dtype=gdn.GDN_F32, q_stride=130)) == EALIGN


def test_workspaces():
    for p, name, call in ((LP(), "gdn_linattn_fwd_workspace_size", fwd), (LP(), "gdn_linattn_bwd_workspace_size", bwd)):
        need = size(name, p, 0)
        assert need > 0 and need % 256 == 0 and call(p, ws_bytes=need - 1) == EWS
        assert call(p, ws=0x100080) == EALIGN and size(name, None, 0) == 0
    for p, name, call in ((GP(), "gdn_gated_norm_bwd_workspace_size", gbwd), (RP(), "gdn_residual_norm_bwd_workspace_size", rbwd)):
        need = size(name, p)
        assert need > 0 and need % 256 == 0 and call(p, ws_bytes=need - 1) == EWS
        assert call(p, ws=0x100080) == EALIGN and size(name, None) == 0


def test_linattn_workspace_sizes():
    """States of the segments (twice backward), and the gradients of shared key heads; none of
    the former where a sequence is one segment."""
    f = lambda **kw: size("gdn_linattn_fwd_workspace_size", LP(**kw), int("num_seqs" in kw))  # noqa: E731
    b = lambda **kw: size("gdn_linattn_bwd_workspace_size", LP(**kw), int("num_seqs" in kw))  # noqa: E731
    assert f(T=0) == 0 and f(B=0) == 0 and b(T=0) == 0
    assert f(T=64) == 0 and f(T=128) == 0 and b(T=128, HV=2) == 0
    assert b(T=128) == 2 * 2 * 128 * 4 * 64 * 4                       # dq and dk of four value heads
    state = 64 * 128 * 4
    assert f(B=1, T=640, H=1, HV=1) == 5 * state                      # segments of two chunks
    assert b(B=1, T=640, H=1, HV=1) == 2 * 5 * state
    assert f(B=1, T=640, H=1, HV=1, num_seqs=3) == (5 + 3) * state
    assert f(B=256, T=4096, H=1, HV=1) == 0                           # the sequences alone fill the device


def test_linattn_launches_beyond_the_grid():
    assert fwd(LP(B=1 << 23, T=1, H=1, HV=1), ws_bytes=1 << 60) == EUNSUP
    assert bwd(LP(B=1 << 22, T=1, H=1, HV=1), ws_bytes=1 << 60) == EUNSUP
    assert decode(LP(B=1 << 22, T=1, H=1, HV=1)) == EUNSUP
    assert fwd(LP(B=1, T=64, H=1, HV=1, num_seqs=1 << 24), cu=0x9000000, ws_bytes=1 << 60) == EUNSUP


def test_nothing_to_do():
    assert decode(LP(B=0)) == OK and decode(LP(T=0), new=0x500000) == OK  # `new` is `state` (the fifth address)
    assert fwd(LP(T=0), fin=None) == OK and fwd(LP(B=0)) == OK and bwd(LP(T=0), dh0=None) == OK and bwd(LP(B=0)) == OK
    assert gfwd(GP(B=0)) == OK and gfwd(GP(T=0)) == OK and rfwd(RP(T=0)) == OK
    # no token pointer is asked for
    assert fwd(LP(T=0), q=None, k=None, v=None, o=None, fin=None) == OK
    assert gfwd(GP(T=0), x=None, z=None, y=None) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), EDTYPE), (dict(dtype=gdn.GDN_F16), EDTYPE), (dict(B=-1), ESHAPE), (dict(T=-1), ESHAPE), (dict(D=0), ESHAPE),
    (dict(H=0), ESHAPE), (dict(eps=-1.0), ESHAPE), (dict(eps=float("nan")), ESHAPE), (dict(gate_first=2), ESHAPE), (dict(D=16385), EUNSUP),
    (dict(x_stride=255), ESHAPE), (dict(z_stride=-1), ESHAPE), (dict(B=1 << 15, T=1 << 15), EUNSUP), (dict(H=(1 << 31) - 1), EUNSUP)])
def test_gated_norm_sizes(kw, status):
    p = GP(**kw)
    assert gfwd(p) == status and gbwd(p) == status and size("gdn_gated_norm_bwd_workspace_size", p) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), EDTYPE), (dict(residual_dtype=gdn.GDN_F16), EDTYPE), (dict(dtype=gdn.GDN_F32, residual_dtype=gdn.GDN_BF16), EDTYPE),
    (dict(T=-1), ESHAPE), (dict(C=0), ESHAPE), (dict(C=16385), EUNSUP), (dict(eps=-1e-9), ESHAPE), (dict(x_stride=63), ESHAPE),
    (dict(residual_stride=63), ESHAPE), (dict(B=1 << 16, T=1 << 15), EUNSUP)])
def test_residual_norm_sizes(kw, status):
    p = RP(**kw)
    assert rfwd(p) == status and rbwd(p) == status and size("gdn_residual_norm_bwd_workspace_size", p) == 0


def test_gated_norm_without_a_gate_needs_no_gradient_of_it():
    assert gbwd(GP(), z=None, dz=None, x=0x100001) == EALIGN  # a later check answers
