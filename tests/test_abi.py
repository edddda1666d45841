"""The C ABI boundary on the CPU: the library loads, exports every entry point
include/gdn.h declares, and validates arguments without touching a GPU (no
device pointer is ever dereferenced by these calls)."""
import ctypes
import os
import re

import pytest

import gated_deltanet_chunkwise_amd as gdn
from gated_deltanet_chunkwise_amd import _binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn.h")

OK, ENULL, ESHAPE, EDTYPE, EUNSUP, EALIGN, EWS, ELAUNCH, ESCRATCH = range(9)


def declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gdn_\w+)\s*\(", text)))


def test_header_declares_expected_entry_points():
    assert declared_functions() == sorted(_binding.SYMBOLS)


def test_library_exports_every_declared_symbol():
    lib = ctypes.CDLL(gdn.lib_path())
    for name in declared_functions():
        assert hasattr(lib, name), name


def test_status_strings():
    seen = set()
    for s in range(9):
        msg = gdn.status_string(s)
        assert msg and msg not in seen
        seen.add(msg)
    assert gdn.status_string(99) == "unknown status"


def P(**kw):
    d = dict(B=2, T=200, H=4, HV=8, K=128, V=64, dtype=gdn.GDN_BF16, num_seqs=0, scale=1.0)
    d.update(kw)
    return gdn.make_params(**d)


def ptrs(**over):
    """12 fake, aligned, never-dereferenced addresses in gdn_fwd's order."""
    names = ["q", "k", "v", "g_raw", "beta", "A_log", "dt_bias", "cu_seqlens",
             "initial_state", "o", "final_state", "workspace"]
    base = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
    base["cu_seqlens"] = None
    base.update(over)
    return [base[n] for n in names]


def test_valid_call_checks_ok():
    p = P()
    ws = gdn.workspace_size(p)
    assert gdn.check(p, ptrs(), ws) == OK
    assert gdn.check(p, ptrs(initial_state=None, final_state=None, dt_bias=None), ws) == OK


@pytest.mark.parametrize("name", ["q", "k", "v", "g_raw", "beta", "A_log", "o", "workspace"])
def test_required_pointer_null(name):
    p = P()
    assert gdn.check(p, ptrs(**{name: None}), gdn.workspace_size(p)) == ENULL


@pytest.mark.parametrize("name,addr", [("q", 0x10008), ("o", 0x10004), ("v", 0x10002),
                                       ("g_raw", 0x10002), ("beta", 0x10001),
                                       ("A_log", 0x10003), ("initial_state", 0x10002),
                                       ("final_state", 0x10001), ("workspace", 0x10080)])
def test_misaligned(name, addr):
    p = P()
    assert gdn.check(p, ptrs(**{name: addr}), gdn.workspace_size(p)) == EALIGN


def test_workspace_too_small():
    p = P()
    assert gdn.check(p, ptrs(), gdn.workspace_size(p) - 1) == EWS


@pytest.mark.parametrize("kw,status", [
    (dict(HV=6), ESHAPE),            # HV % H != 0
    (dict(H=0), ESHAPE),
    (dict(T=-1), ESHAPE),
    (dict(B=-2), ESHAPE),
    (dict(K=96), EUNSUP),
    (dict(V=256), EUNSUP),
    (dict(K=32), EUNSUP),
    (dict(dtype=7), EDTYPE),
])
def test_bad_shapes(kw, status):
    p = P(**kw)
    assert gdn.check(p, ptrs(), 1 << 40) == status
    assert gdn.workspace_size(p) == 0


def test_packed_rules():
    # cu_seqlens needs B == 1
    assert gdn.check(P(num_seqs=3), ptrs(cu_seqlens=0x90000), 1 << 40) == ESHAPE
    p = P(B=1, T=1000, num_seqs=3)
    ws = gdn.workspace_size(p, packed=True)
    assert gdn.check(p, ptrs(cu_seqlens=0x90000), ws) == OK
    assert gdn.check(p, ptrs(cu_seqlens=0x90004), ws) == EALIGN
    assert gdn.check(p, ptrs(cu_seqlens=0x90000), ws - 256) == EWS


def test_stage_mask_outside_the_stages_is_rejected():
    """gdn_fwd_stages validates like gdn_fwd, then refuses unknown stage bits
    before anything is enqueued (the fake pointers are never used)."""
    lib = gdn.load_library()
    p = P()
    ws = gdn.workspace_size(p)
    vp = [ctypes.c_void_p(a) for a in ptrs()]
    for mask in (gdn.STAGE_ALL + 1, 1 << 31):
        assert lib.gdn_fwd_stages(ctypes.byref(p), *vp, ws, mask, None) == EUNSUP
    # argument errors come first, as in gdn_fwd
    vp_null = [ctypes.c_void_p(a) if a else None for a in ptrs(q=None)]
    assert lib.gdn_fwd_stages(ctypes.byref(p), *vp_null, ws, 1, None) == ENULL
    assert gdn.STAGE_ALL == 15 and gdn.STAGE_BITS["chain"] == 4


def test_empty_token_batch_needs_no_token_pointers():
    p = P(T=0)
    null = dict(q=None, k=None, v=None, g_raw=None, beta=None, A_log=None, o=None)
    assert gdn.check(p, ptrs(**null), gdn.workspace_size(p)) == OK


def test_workspace_layout():
    for dtype, esz in ((gdn.GDN_BF16, 2), (gdn.GDN_F32, 4)):
        for packed in (False, True):
            B = 1 if packed else 3
            p = P(B=B, T=1000, dtype=dtype, num_seqs=5 if packed else 0)
            lay = gdn.workspace_layout(p, packed)
            slots = 1000 // 64 + 5 if packed else B * ((1000 + 63) // 64)
            assert lay.num_slots == slots
            HV, K, V = 8, 128, 64
            hsl = HV * slots
            offs = [lay.gamma, lay.beta, lay.w, lay.kt, lay.u, lay.hc, lay.vn, lay.pm,
                    lay.chunk_map, lay.seq_slot, lay.seq_order, lay.total]
            assert all(o % 256 == 0 for o in offs)
            assert offs == sorted(offs)
            assert lay.beta - lay.gamma >= hsl * 64 * 4
            assert lay.kt - lay.w >= hsl * 64 * K * esz
            assert lay.u - lay.kt >= hsl * 64 * K * esz
            assert lay.hc - lay.u >= hsl * 64 * V * esz
            assert lay.vn - lay.hc >= hsl * K * V * esz
            assert lay.pm - lay.vn >= hsl * 64 * V * esz
            # P^T fragments: [it 4][jb 2][lane 64] of 8 elements per chunk and head
            assert lay.chunk_map - lay.pm >= hsl * 4 * 2 * 64 * 8 * esz
            if packed:
                assert lay.seq_slot - lay.chunk_map >= slots * 16
                assert lay.seq_order - lay.seq_slot >= (5 + 1) * 4
                assert lay.total - lay.seq_order >= 5 * 4
            assert lay.total == gdn.workspace_size(p, packed)


def test_missing_library_fails_loudly(monkeypatch):
    monkeypatch.setattr(_binding, "_LIB", None)
    monkeypatch.setattr(_binding, "_LIB_PATH", "/nonexistent/libgdn.so")
    with pytest.raises(OSError):
        _binding.load_library()


def test_kda_gate_validation():
    """gdn_kda_gate rejects bad arguments before enqueuing anything."""
    lib = gdn.load_library()
    F32, BF16, F16 = gdn.GDN_F32, gdn.GDN_BF16, gdn.GDN_F16
    g, A, b, y = (ctypes.c_void_p(0x10000 * i) for i in (1, 2, 3, 4))

    def call(g=g, gt=BF16, A=A, b=b, y=y, yt=F32, T=8, H=4, D=64):
        return lib.gdn_kda_gate(g, gt, A, b, y, yt, T, H, D, None)
    assert call(T=-1) == ESHAPE
    assert call(H=0) == ESHAPE
    assert call(D=0) == ESHAPE
    assert call(T=1 << 62, H=4, D=64) == ESHAPE            # T*H*D beyond int64
    assert call(gt=7) == EDTYPE
    assert call(yt=-1) == EDTYPE
    assert call(g=None) == ENULL
    assert call(A=None) == ENULL
    assert call(y=None) == ENULL
    assert call(g=ctypes.c_void_p(0x10001)) == EALIGN       # bf16 needs 2 bytes
    assert call(y=ctypes.c_void_p(0x10002)) == EALIGN       # fp32 needs 4
    assert call(b=ctypes.c_void_p(0x30002)) == EALIGN
    # nothing to do: no pointer is needed and nothing is enqueued
    assert call(g=None, A=None, b=None, y=None, T=0) == OK
    assert F16 == 2


def test_decode_validation():
    """gdn_decode: gdn_fwd's size rules, fixed-length sequences only, a state is
    required, and nothing is enqueued when there are no tokens."""
    lib = gdn.load_library()
    vp = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(9)]   # q k v g beta A dt state o

    def call(p, ptrs=vp):
        return lib.gdn_decode(ctypes.byref(p), *ptrs, None)
    assert call(P(num_seqs=2, B=1)) == ESHAPE
    assert call(P(K=96)) == EUNSUP
    assert call(P(dtype=gdn.GDN_F16)) == EDTYPE
    assert call(P(HV=6)) == ESHAPE
    assert call(P(), vp[:7] + [None] + vp[8:]) == ENULL               # state
    assert call(P(), [None] + vp[1:]) == ENULL                         # q
    assert call(P(), vp[:3] + [ctypes.c_void_p(0x40002)] + vp[4:]) == EALIGN
    # no tokens: only the state is needed, and nothing is launched
    none = [None] * 7 + [vp[7], None]
    assert call(P(T=0), none) == OK
    assert call(P(B=0), none) == OK


def test_segment_layout():
    """seg_chunks > 0 adds the segment tables and buffers."""
    p0 = P(B=2, T=700, H=2, HV=4, K=128, V=64)
    p2 = P(B=2, T=700, H=2, HV=4, K=128, V=64, seg_chunks=3)
    l0, l2 = gdn.workspace_layout(p0), gdn.workspace_layout(p2)
    assert l0.num_segs == 0 and l0.seg_m == 0
    assert l2.num_segs == 2 * 4                      # 11 chunks per sequence -> 4 segments
    per = l2.num_segs * 4 * 128
    assert l2.seg_e - l2.seq_seg >= (2 + 1) * 4
    assert l2.seg_m - l2.seg_e >= per * 64 * 4
    assert l2.seg_h - l2.seg_m >= per * 128 * 4
    assert l2.total - l2.seg_h >= per * 64 * 4
    assert gdn.workspace_size(p2) == l2.total > gdn.workspace_size(p0)
    # packed: an upper bound of slots / L + N segments
    lp = gdn.workspace_layout(P(B=1, T=1000, num_seqs=3, seg_chunks=2), packed=True)
    assert lp.num_segs == (1000 // 64 + 3) // 2 + 3
    # negative values other than GDN_SEG_AUTO (-1) are errors
    assert gdn.check(P(seg_chunks=-3), ptrs(), 1 << 40) == ESHAPE


def _bwd_call(lib, p, ws_bytes, **over):
    """gdn_bwd with fake, aligned device addresses (never dereferenced: every
    case below fails validation, or has no work)."""
    names = ("q", "k", "v", "g_raw", "beta", "A_log", "dt_bias", "cu_seqlens", "h0", "d_o",
             "dht", "dq", "dk", "dv", "dg_raw", "dbeta", "dA_log", "ddt_bias", "dh0", "ws")
    addr = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    addr.update(cu_seqlens=0, h0=0, dht=0)
    addr.update(over)
    vp = [ctypes.c_void_p(addr[n]) if addr[n] else None for n in names[:-1]]
    ws = ctypes.c_void_p(addr["ws"]) if addr["ws"] else None
    return lib.gdn_bwd(ctypes.byref(p), *vp, ws, ws_bytes, None)


def test_bwd_validation():
    lib = gdn.load_library()
    p = P()
    ws = lib.gdn_bwd_workspace_size(ctypes.byref(p), 0)
    assert ws > gdn.workspace_size(p)  # the forward layout plus the backward's buffers
    for name in ("q", "k", "v", "g_raw", "beta", "A_log", "d_o", "dq", "dk", "dv", "dg_raw",
                 "dbeta", "dA_log", "ws"):
        assert _bwd_call(lib, p, ws, **{name: 0}) == ENULL, name
    for name, addr in (("q", 0x100008), ("d_o", 0x100004), ("dq", 0x100002),
                       ("dv", 0x100008), ("dg_raw", 0x100002), ("dh0", 0x100001),
                       ("ddt_bias", 0x100003), ("ws", 0x100080)):
        assert _bwd_call(lib, p, ws, **{name: addr}) == EALIGN, name
    assert _bwd_call(lib, p, ws - 256) == EWS
    bad = P(K=96)
    assert lib.gdn_bwd_workspace_size(ctypes.byref(bad), 0) == 0
    assert _bwd_call(lib, bad, ws) == EUNSUP
    assert _bwd_call(lib, P(HV=3, H=2), ws) == ESHAPE
    # the WY backward's 32-bit row offsets: 64 HV V beyond int32 is rejected
    # by the backward only (the forward takes it)
    wide = P(B=1, T=64, H=1, HV=262144, K=128, V=128)
    assert gdn.workspace_size(wide) > 0
    assert lib.gdn_bwd_workspace_size(ctypes.byref(wide), 0) == 0
    assert _bwd_call(lib, wide, ws) == EUNSUP
    assert _bwd_call(lib, P(num_seqs=2), ws, cu_seqlens=0x90000) == ESHAPE  # packed needs B == 1
    # no tokens: token pointers may be NULL (dA_log is still required)
    e = P(T=0)
    null = dict(q=0, k=0, v=0, g_raw=0, beta=0, d_o=0, dq=0, dk=0, dv=0, dg_raw=0, dbeta=0)
    assert _bwd_call(lib, e, lib.gdn_bwd_workspace_size(ctypes.byref(e), 0),
                     **dict(null, dA_log=0)) == ENULL


def test_bwd_workspace_grows_with_the_problem():
    lib = gdn.load_library()
    sizes = [lib.gdn_bwd_workspace_size(ctypes.byref(P(T=t)), 0) for t in (64, 128, 1000)]
    assert sizes[0] < sizes[1] < sizes[2]
    pk = P(B=1, T=1000, num_seqs=5)
    assert lib.gdn_bwd_workspace_size(ctypes.byref(pk), 1) > gdn.workspace_size(pk, packed=True)


def test_packed_call_without_sequences():
    """A packed call with no sequence but tokens is rejected before anything is
    enqueued, forward and backward (every per-chunk launch would otherwise read
    a chunk map nothing wrote); no sequence and no token is a valid no-op."""
    lib = gdn.load_library()
    bad = P(B=1, T=64, num_seqs=0)
    assert gdn.workspace_size(bad, packed=True) == 0
    assert gdn.check(bad, ptrs(cu_seqlens=0x90000), 1 << 40) == ESHAPE
    assert lib.gdn_bwd_workspace_size(ctypes.byref(bad), 1) == 0
    assert _bwd_call(lib, bad, 1 << 40, cu_seqlens=0x90000) == ESHAPE
    empty = P(B=1, T=0, num_seqs=0)
    ws = gdn.workspace_size(empty, packed=True)
    null = dict(q=None, k=None, v=None, g_raw=None, beta=None, A_log=None, o=None)
    assert gdn.check(empty, ptrs(cu_seqlens=0x90000, **null), ws) == OK
    # the same sizes without cu_seqlens are a fixed-length call (N = B = 1)
    assert gdn.check(bad, ptrs(), 1 << 40) == OK


def test_noalloc_rejects_problems_beyond_the_scratch():
    """gdn_fwd_noalloc checks its arguments, and that the problem's workspace
    fits GDN_SCRATCH_BYTES, before it looks up the scratch address or enqueues
    anything (so these calls never touch a GPU)."""
    lib = gdn.load_library()
    vp = lambda **kw: [ctypes.c_void_p(a) if a else None for a in ptrs(**kw)[:11]]  # noqa: E731
    # B=4, T=8192, H=HV=16, K=V=128 bf16: 836 MiB of workspace
    big = P(B=4, T=8192, H=16, HV=16, K=128, V=128)
    assert gdn.workspace_size(big) > gdn.GDN_SCRATCH_BYTES
    assert lib.gdn_fwd_noalloc(ctypes.byref(big), *vp(), None) == ESCRATCH
    # argument errors are reported like gdn_fwd's
    small = P(B=2, T=2048, H=8, HV=8, K=128, V=128)
    assert gdn.workspace_size(small) <= gdn.GDN_SCRATCH_BYTES
    assert lib.gdn_fwd_noalloc(ctypes.byref(small), *vp(q=None), None) == ENULL
    assert lib.gdn_fwd_noalloc(ctypes.byref(small), *vp(o=0x10004), None) == EALIGN
    assert lib.gdn_fwd_noalloc(ctypes.byref(P(K=96)), *vp(), None) == EUNSUP
    assert lib.gdn_fwd_noalloc(None, *vp(), None) == ENULL
    assert "scratch" in gdn.status_string(ESCRATCH)


def test_automatic_segments_layout():
    """seg_chunks = GDN_SEG_AUTO: the workspace holds the shortest segments the
    choice may take (16 chunks) for fixed-length input; packed input keeps the
    plain pass (no segment buffers).  Other negative values are rejected."""
    auto = P(B=1, T=65536, H=2, HV=2, K=128, V=128, seg_chunks=gdn.GDN_SEG_AUTO)
    assert gdn.workspace_size(auto) == gdn.workspace_size(
        P(B=1, T=65536, H=2, HV=2, K=128, V=128, seg_chunks=16))
    assert gdn.workspace_layout(auto).num_segs == 65536 // 64 // 16
    packed = P(B=1, T=65536, H=2, HV=2, K=128, V=128, num_seqs=3, seg_chunks=gdn.GDN_SEG_AUTO)
    assert gdn.workspace_size(packed, packed=True) == gdn.workspace_size(
        P(B=1, T=65536, H=2, HV=2, K=128, V=128, num_seqs=3), packed=True)
    assert gdn.workspace_size(P(seg_chunks=-2)) == 0
    assert gdn.check(P(seg_chunks=-2), ptrs(), 1 << 40) == ESHAPE
    # an explicit length is reported as given (no device query needed)
    assert gdn.seg_chunks(P(seg_chunks=5)) == 5 and gdn.seg_chunks(P()) == 0


# ---- the layer operators (convolution, scan, checkpoints) --------------------------

def CP(**kw):
    from gated_deltanet_chunkwise_amd._layers import ConvParams
    d = dict(B=2, T=20, C=64, W=4, num_seqs=0, dtype=gdn.GDN_BF16, activation=1, x_stride=0)
    d.update(kw)
    return ConvParams(*(d[n] for n, _ in ConvParams._fields_))


def SP(**kw):
    from gated_deltanet_chunkwise_amd._layers import ScanParams
    d = dict(B=2, T=20, D=64, G=2, N=16, num_seqs=0, dtype=gdn.GDN_BF16, x_stride=0, dt_stride=0,
             z_stride=0, b_stride=0, c_stride=0)
    d.update(kw)
    return ScanParams(*(d[n] for n, _ in ScanParams._fields_))


def addresses(names, given):
    """Fake, aligned, never-dereferenced addresses by name; `given` replaces some."""
    base = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    for n in ("cu", "x_scales", "z_scales"):
        if n in base:
            base[n] = None
    base.update(given)
    return [base[n] for n in names]


def conv_fwd(p, **given):
    names = ("x", "weight", "bias", "cu", "h0", "y", "fin")
    return gdn.load_library().gdn_conv_fwd(p and ctypes.byref(p), *addresses(names, given), None)


def conv_decode(p, **given):
    names = ("x", "weight", "bias", "state", "new", "y")
    return gdn.load_library().gdn_conv_decode(p and ctypes.byref(p), *addresses(names, given), None)


def conv_bwd(p, ws_bytes=1 << 40, **given):
    names = ("x", "x_scales", "weight", "bias", "cu", "h0", "d_y", "d_fin", "dx", "dw", "db", "dh0", "ws")
    return gdn.load_library().gdn_conv_bwd(p and ctypes.byref(p), *addresses(names, given), ws_bytes, None)


def scan_fwd(p, ws_bytes=1 << 40, **given):
    names = ("x", "dt", "A_log", "Bm", "Cm", "skip", "z", "dt_bias", "cu", "h0", "y", "fin", "ws")
    return gdn.load_library().gdn_scan_fwd(p and ctypes.byref(p), *addresses(names, given), ws_bytes, None)


def scan_decode(p, **given):
    names = ("x", "dt", "A_log", "Bm", "Cm", "skip", "z", "dt_bias", "state", "new", "y")
    return gdn.load_library().gdn_scan_decode(p and ctypes.byref(p), *addresses(names, given), None)


def scan_bwd(p, ws_bytes=1 << 40, **given):
    names = ("x", "x_scales", "dt", "A_log", "Bm", "Cm", "skip", "z", "z_scales", "dt_bias", "cu", "h0", "d_y",
             "d_fin", "dx", "ddt", "dA_log", "dBm", "dCm", "dskip", "dz", "ddt_bias", "dh0", "ws")
    return gdn.load_library().gdn_scan_bwd(p and ctypes.byref(p), *addresses(names, given), ws_bytes, None)


CONV_BAD = [(dict(dtype=7), EDTYPE), (dict(dtype=gdn.GDN_F16), EDTYPE), (dict(C=0), ESHAPE), (dict(W=0), ESHAPE),
            (dict(W=1), EUNSUP), (dict(W=5), EUNSUP), (dict(activation=2), ESHAPE), (dict(B=-1), ESHAPE),
            (dict(T=-1), ESHAPE), (dict(x_stride=63), ESHAPE), (dict(x_stride=-64), ESHAPE),
            (dict(B=1 << 16, T=1 << 15), EUNSUP), (dict(B=2, T=(1 << 30) - 100), EUNSUP)]


@pytest.mark.parametrize("kw,status", CONV_BAD)
def test_conv_refuses_sizes(kw, status):
    p = CP(**kw)
    assert conv_fwd(p) == status and conv_bwd(p) == status and conv_decode(p) == status
    assert gdn.load_library().gdn_conv_bwd_workspace_size(ctypes.byref(p), 0) == 0


SCAN_BAD = [(dict(dtype=7), EDTYPE), (dict(dtype=gdn.GDN_F16), EDTYPE), (dict(D=0), ESHAPE), (dict(G=0), ESHAPE),
            (dict(N=0), ESHAPE), (dict(G=3), ESHAPE), (dict(N=65), EUNSUP), (dict(B=-1), ESHAPE),
            (dict(x_stride=63), ESHAPE), (dict(dt_stride=1), ESHAPE), (dict(z_stride=-1), ESHAPE),
            (dict(b_stride=31), ESHAPE), (dict(c_stride=31), ESHAPE), (dict(B=65536, T=1), EUNSUP),
            (dict(B=2, T=(1 << 30) - 100), EUNSUP), (dict(D=1 << 26, G=1), EUNSUP)]


@pytest.mark.parametrize("kw,status", SCAN_BAD)
def test_scan_refuses_sizes(kw, status):
    p = SP(**kw)
    assert scan_fwd(p) == status and scan_bwd(p) == status and scan_decode(p) == status
    for f in ("gdn_scan_fwd_workspace_size", "gdn_scan_bwd_workspace_size"):
        assert getattr(gdn.load_library(), f)(ctypes.byref(p), 0) == 0


@pytest.mark.parametrize("call,P_", [(conv_fwd, CP), (conv_bwd, CP), (scan_fwd, SP), (scan_bwd, SP)])
def test_layer_packed_rules(call, P_):
    cu = 0x9000000
    assert call(P_(B=2, num_seqs=3), cu=cu) == ESHAPE      # one row of tokens
    assert call(P_(B=1, num_seqs=-1), cu=cu) == ESHAPE
    assert call(P_(B=1, num_seqs=0), cu=cu) == ESHAPE      # tokens of no sequence
    assert call(P_(B=1, num_seqs=2), cu=cu + 4) == EALIGN
    assert call(None) == ENULL


@pytest.mark.parametrize("call,P_", [(conv_decode, CP), (scan_decode, SP)])
def test_layer_decode_is_for_sequences_of_one_length(call, P_):
    assert call(P_(B=1, num_seqs=2)) == ESHAPE
    assert call(None) == ENULL


@pytest.mark.parametrize("call,P_,required,optional", [
    (conv_fwd, CP, "x weight y", "bias h0 fin"),
    (conv_decode, CP, "x weight y state new", "bias"),
    (conv_bwd, CP, "x weight d_y dx dw ws", "bias h0 d_fin db dh0"),
    (scan_fwd, SP, "x dt A_log Bm Cm y", "skip z dt_bias h0 fin"),
    (scan_decode, SP, "x dt A_log Bm Cm y state new", "skip z dt_bias"),
    (scan_bwd, SP, "x dt A_log Bm Cm d_y dx ddt dA_log dBm dCm dz ws", "skip dt_bias h0 d_fin dskip ddt_bias dh0")])
def test_layer_pointers(call, P_, required, optional):
    for n in required.split():
        assert call(P_(), **{n: None}) == ENULL, n
    for n in required.split() + optional.split():
        assert call(P_(), **{n: 0x100001}) == EALIGN, n
    # what may be missing is not asked for: a later check answers
    later = dict(x=0x100001)
    for n in optional.split():
        assert call(P_(), **{n: None}, **later) == EALIGN, n


def test_layer_workspaces():
    lib = gdn.load_library()
    need = lib.gdn_conv_bwd_workspace_size(ctypes.byref(CP()), 0)
    assert need > 0 and conv_bwd(CP(), ws_bytes=need - 1) == EWS
    p = SP(T=500)
    for size, call in ((lib.gdn_scan_fwd_workspace_size, scan_fwd), (lib.gdn_scan_bwd_workspace_size, scan_bwd)):
        need = size(ctypes.byref(p), 0)
        assert need > 0 and need % 256 == 0 and call(p, ws_bytes=need - 1) == EWS
        assert call(p, ws=0x100080) == EALIGN and call(p, ws=None) == ENULL
        assert size(None, 0) == 0
    # a short call with whole rows of Bm and Cm forms nothing in between
    assert lib.gdn_scan_fwd_workspace_size(ctypes.byref(SP(T=1, dtype=gdn.GDN_F32)), 0) >= 0


def test_checkpoints_are_dense():
    assert conv_bwd(CP(x_stride=128), x_scales=0x9000000) == ESHAPE
    assert scan_bwd(SP(x_stride=128), x_scales=0x9000000, z_scales=0x9100000) == ESHAPE
    assert scan_bwd(SP(z_stride=128), x_scales=0x9000000, z_scales=0x9100000) == ESHAPE
    assert scan_bwd(SP(), x_scales=0x9000000) == ESHAPE    # one of x and z alone
    assert scan_bwd(SP(), z_scales=0x9000000) == ESHAPE


def test_pack8_validation():
    lib = gdn.load_library()
    A, B_, C_ = 0x100000, 0x200000, 0x300000
    pack = lambda x=A, dt=gdn.GDN_BF16, rows=4, C=64, ld=0, codes=B_, scales=C_: lib.gdn_pack8(  # noqa: E731
        x, dt, rows, C, ld, codes, scales, None)
    unpack = lambda codes=A, scales=B_, rows=4, C=64, y=C_, dt=gdn.GDN_BF16: lib.gdn_unpack8(  # noqa: E731
        codes, scales, rows, C, y, dt, None)
    for f in (pack, unpack):
        assert f(dt=gdn.GDN_F16) == EDTYPE and f(dt=9) == EDTYPE
        assert f(rows=-1) == ESHAPE and f(C=0) == ESHAPE and f(rows=1 << 60) == ESHAPE
        assert f(codes=None) == ENULL and f(scales=None) == ENULL
        assert f(rows=0) == OK
    assert pack(ld=63) == ESHAPE and pack(x=None) == ENULL and pack(x=A + 1) == EALIGN
    assert pack(x=A + 2, dt=gdn.GDN_F32) == EALIGN
    assert unpack(y=None) == ENULL and unpack(y=C_ + 1) == EALIGN


def test_layer_calls_with_nothing_to_do_enqueue_nothing():
    assert conv_decode(CP(B=0)) == OK and scan_decode(SP(B=0)) == OK
    assert conv_decode(CP(T=0), new=0x400000) == OK        # `new` is `state` (the fourth address)
    assert conv_fwd(CP(T=0), fin=None) == OK and scan_fwd(SP(T=0), fin=None) == OK


# A launch holds less than 2^32 threads per dimension of its grid; sizes beyond that are
# refused before the first of a call's kernels is enqueued (without a GPU a call that gets
# as far as enqueuing answers GDN_ERR_LAUNCH).
GRID = [
    (conv_decode, CP(B=1 << 20, T=1, C=(1 << 13) + 1)),              # a lane per sequence and channel
    (lambda p: conv_fwd(p, x=0x100004), CP(B=1 << 22, T=1, C=256, dtype=gdn.GDN_F32)),  # exactly 2^32
    (conv_bwd, CP(B=1, T=20, C=1 << 26)),                            # the sums over tiles
    (conv_bwd, CP(B=1 << 23, T=0, C=513)),                           # initial states
    (scan_decode, SP(B=1 << 15, T=1, D=1 << 16, N=8)),
    (scan_fwd, SP(B=65535, T=1, D=1 << 17, G=1 << 17, N=1)),         # a wave per sequence and group
    (lambda p: scan_bwd(p, ws_bytes=1 << 50), SP(B=65535, T=1, D=1 << 17, G=1 << 17, N=1)),
    (scan_bwd, SP(B=1, T=20, D=1 << 24, G=1, N=64)),                 # the sums over tiles
]


@pytest.mark.parametrize("call,p", GRID)
def test_layer_launches_beyond_the_grid(call, p):
    assert call(p) == EUNSUP


@pytest.mark.parametrize("call", [scan_fwd, scan_bwd])
def test_empty_sequences_beyond_the_grid(call):
    # a workgroup copies each empty sequence's state
    assert call(SP(B=1, T=0, num_seqs=1 << 25), cu=0x9000000) == EUNSUP


# Sizes whose products pass 64 bits (or that no memory holds) are refused, and their
# workspaces asked for as 0: a size that wrapped round would let the call through.
@pytest.mark.parametrize("call,p,cu", [
    (conv_fwd, CP(B=(1 << 31) - 1, T=0, C=(1 << 31) - 1), None),     # B 3 C
    (conv_decode, CP(B=(1 << 31) - 1, T=0, C=(1 << 31) - 1), None),
    (conv_fwd, CP(B=1, T=0, C=(1 << 31) - 1, num_seqs=(1 << 31) - 1), 0x9000000),
    (conv_bwd, CP(B=(1 << 31) - 1, T=0, C=(1 << 31) - 1), None)])
def test_conv_sizes_beyond_64_bits(call, p, cu):
    assert (call(p, cu=cu) if cu else call(p)) == EUNSUP


def test_scan_sizes_beyond_64_bits():
    p = SP(B=1, T=(1 << 31) - 5000, D=1 << 24, G=1 << 24, N=63)
    assert scan_fwd(p) == EUNSUP and scan_bwd(p) == EUNSUP and scan_decode(p) == EUNSUP
    for f in ("gdn_scan_fwd_workspace_size", "gdn_scan_bwd_workspace_size"):
        assert getattr(gdn.load_library(), f)(ctypes.byref(p), 0) == 0


@pytest.mark.parametrize("call,P_", [(conv_fwd, CP), (conv_bwd, CP), (conv_decode, CP), (scan_fwd, SP), (scan_bwd, SP),
                                     (scan_decode, SP)])
def test_zero_rest_is_a_bit_of_the_dtype(call, P_):
    for code in (gdn.GDN_F32, gdn.GDN_BF16):
        assert call(P_(dtype=code | 0x100), x=0x100001) == EALIGN  # a later check answers
    for code in (gdn.GDN_F16 | 0x100, 7 | 0x100, gdn.GDN_BF16 | 0x200):
        assert call(P_(dtype=code)) == EDTYPE


def test_layer_workspace_sizes():
    """What the forward scan's workspace holds: nothing of tiles where a row is one tile (32
    tokens or fewer), the two fp32 copies of Bm and Cm (for calls that cannot read them in
    place) always; nothing without tokens."""
    size = lambda **kw: gdn.load_library().gdn_scan_fwd_workspace_size(ctypes.byref(SP(**kw)), 0)  # noqa: E731
    up = lambda b: -(-b // 256) * 256  # noqa: E731
    for T in (1, 20, 32):
        for N, np_ in ((16, 16), (5, 8), (33, 48)):
            assert size(T=T, N=N) == 2 * up(2 * T * 2 * np_ * 4)
    tiles = 2 * 3  # of 16 tokens
    assert size(T=33) == up(up(tiles * 16 * 64 * 4) + tiles * 64 * 4) + 2 * up(2 * 33 * 2 * 16 * 4)
    assert size(T=0) == 0 and size(B=0) == 0
