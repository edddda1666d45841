"""The layer operators' wrappers on the CPU: every tensor's shape and dtype is checked
before anything reaches the library, and tensors that are not on a GPU are refused; the
64-bit forms that the GPU tests compare with are held to differences and to each other."""
import pytest
import torch

import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
from gated_deltanet_chunkwise_amd import _binding, _layers

BF16, F32 = torch.bfloat16, torch.float32


class _NoCalls:
    def __getattr__(self, name):
        raise AssertionError("library call %s reached" % name)


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(_binding, "_LIB", _NoCalls())


def conv_case():
    return dict(x=torch.zeros(2, 9, 64, dtype=BF16), weight=torch.zeros(64, 4), bias=torch.zeros(64),
                h0=torch.zeros(2, 3, 64, dtype=BF16), d_y=torch.zeros(2, 9, 64, dtype=BF16),
                d_fin=torch.zeros(2, 3, 64, dtype=BF16), cu=None)


def conv_calls(d):
    return [lambda: gdn.conv_fwd(d["x"], d["weight"], d["bias"], d["cu"], d["h0"]),
            lambda: gdn.conv_bwd(d["x"], d["weight"], d["bias"], d["d_y"], d["d_fin"], d["cu"], d["h0"]),
            lambda: gdn.causal_conv(d["x"], d["weight"], d["bias"], d["cu"], d["h0"]),
            lambda: gdn.conv_decode(d["x"], d["weight"], d["h0"], d["bias"])]


CONV = [("x", torch.zeros(9, 64, dtype=BF16), ValueError), ("x", torch.zeros(2, 9, 64, dtype=torch.float16), TypeError),
        ("weight", torch.zeros(63, 4), ValueError), ("weight", torch.zeros(64, 4, dtype=BF16), TypeError),
        ("weight", torch.zeros(64), ValueError), ("bias", torch.zeros(1, 64), ValueError),
        ("bias", torch.zeros(64, dtype=torch.float64), TypeError), ("h0", torch.zeros(2, 4, 64, dtype=BF16), ValueError),
        ("h0", torch.zeros(2, 3, 64), TypeError)]


@pytest.mark.parametrize("name,bad,error", CONV)
def test_conv_refuses(name, bad, error):
    d = dict(conv_case(), **{name: bad})
    for call in conv_calls(d):
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("name,bad,error", [
    ("d_y", torch.zeros(2, 8, 64, dtype=BF16), ValueError), ("d_y", torch.zeros(2, 9, 64), TypeError), ("d_y", None, ValueError),
    ("d_fin", torch.zeros(1, 3, 64, dtype=BF16), ValueError), ("cu", torch.zeros(3, dtype=torch.int32), TypeError),
    ("cu", torch.zeros(3, dtype=torch.int64), ValueError), ("cu", torch.zeros(1, 3, dtype=torch.int64), ValueError),
    ("cu", torch.zeros(0, dtype=torch.int64), ValueError)])
def test_conv_backward_refuses(name, bad, error):
    d = dict(conv_case(), **{name: bad})
    with pytest.raises(error):
        conv_calls(d)[1]()


def test_host_tensors_are_refused():
    for call in conv_calls(conv_case()) + scan_calls(scan_case()):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="GPU tensor"):
        gdn.pack8(torch.zeros(2, 64))
    with pytest.raises(ValueError, match="GPU tensor"):
        gdn.unpack8(gdn.Packed8(torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 2, dtype=torch.uint8), F32))


def test_unknown_activation_and_bits():
    d = conv_case()
    with pytest.raises(ValueError, match="activation"):
        gdn.conv_fwd(d["x"], d["weight"], activation="relu")
    for f in (lambda: gdn.causal_conv(d["x"], d["weight"], checkpoint_bits=4),
              lambda: gdn.selective_scan(*[None] * 5, checkpoint_bits=16),
              lambda: gdn.gated_delta_rule(*[None] * 6, checkpoint_bits=True + 6)):
        with pytest.raises(ValueError, match="checkpoint_bits"):
            f()


def scan_case():
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(x=z(2, 9, 64), dt=z(2, 9, 64), A_log=z(64, 16, dtype=F32), Bm=z(2, 9, 2, 16), Cm=z(2, 9, 2, 16),
                skip=z(64, dtype=F32), z=z(2, 9, 64), dt_bias=z(64, dtype=F32), h0=z(2, 64, 16, dtype=F32),
                d_y=z(2, 9, 64), d_fin=z(2, 64, 16, dtype=F32))


def scan_calls(d):
    a = (d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"])
    o = dict(skip=d["skip"], z=d["z"], dt_bias=d["dt_bias"])
    return [lambda: gdn.scan_fwd(*a, **o, initial_state=d["h0"]),
            lambda: gdn.scan_bwd(*a, d["d_y"], d["d_fin"], **o, initial_state=d["h0"]),
            lambda: gdn.selective_scan(*a, **o, initial_state=d["h0"]),
            lambda: gdn.scan_decode(*a, d["h0"], **o)]


@pytest.mark.parametrize("name,bad,error", [
    ("x", torch.zeros(2, 64, dtype=BF16), ValueError), ("x", torch.zeros(2, 9, 64), TypeError),
    ("dt", torch.zeros(2, 9, 32, dtype=BF16), ValueError), ("dt", torch.zeros(2, 9, 64), TypeError),
    ("A_log", torch.zeros(64), ValueError), ("A_log", torch.zeros(63, 16), ValueError),
    ("A_log", torch.zeros(64, 16, dtype=BF16), TypeError), ("Bm", torch.zeros(2, 9, 32, dtype=BF16), ValueError),
    ("Bm", torch.zeros(2, 9, 2, 8, dtype=BF16), ValueError), ("Cm", torch.zeros(2, 9, 1, 16, dtype=BF16), ValueError),
    ("Cm", torch.zeros(2, 9, 2, 16), TypeError), ("skip", torch.zeros(1), ValueError),
    ("z", torch.zeros(2, 9, 63, dtype=BF16), ValueError), ("z", torch.zeros(2, 9, 64), TypeError),
    ("dt_bias", torch.zeros(64, dtype=BF16), TypeError), ("h0", torch.zeros(1, 64, 16), ValueError),
    ("h0", torch.zeros(2, 64, 16, dtype=BF16), TypeError)])
def test_scan_refuses(name, bad, error):
    d = dict(scan_case(), **{name: bad})
    for call in scan_calls(d):
        with pytest.raises(error):
            call()


def packed(*shape, scales=None, dtype=BF16):
    c = torch.zeros(*shape, dtype=torch.int8)
    return gdn.Packed8(c, torch.zeros(*(scales or shape[:-1] + ((shape[-1] + 31) // 32,)), dtype=torch.uint8), dtype)


def test_scan_backward_refuses():
    d = scan_case()
    for k, v in (("d_y", None), ("d_y", torch.zeros(2, 9, 63, dtype=BF16)), ("d_fin", torch.zeros(2, 64, 8)),
                 ("x", packed(2, 9, 64)), ("z", packed(2, 9, 64))):  # one checkpoint of two
        with pytest.raises(ValueError):
            scan_calls(dict(d, **{k: v}))[1]()
    both = dict(d, x=packed(2, 9, 64), z=packed(2, 9, 64, dtype=F32))
    with pytest.raises(TypeError):
        scan_calls(both)[1]()


def test_checkpoint_refuses():
    with pytest.raises(TypeError):
        gdn.pack8(torch.zeros(2, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        gdn.pack8(torch.zeros(()))
    with pytest.raises(ValueError):
        gdn.unpack8(packed(2, 64, scales=(2, 3)))
    bad = packed(2, 64)
    with pytest.raises(TypeError):
        gdn.unpack8(bad._replace(codes=bad.codes.to(torch.uint8)))
    with pytest.raises(TypeError):
        gdn.unpack8(bad._replace(dtype=torch.float16))
    with pytest.raises(ValueError):
        gdn.unpack8(bad, out=torch.zeros(2, 32, dtype=BF16))


@pytest.mark.parametrize("t,want", [
    (torch.zeros(2, 9, 64), 0), (torch.zeros(2, 9, 96)[..., 16:80], 96), (torch.zeros(2, 1, 96)[..., :64], 96),
    (torch.zeros(1, 9, 64)[:, 2:5], 0), (torch.zeros(2, 9, 64)[:, 3:4], 576), (torch.zeros(1, 1, 96)[..., :64], 0),
    (torch.zeros(1, 18, 64)[:, ::2], 128), (torch.zeros(2, 9, 3, 80)[..., 0, 16:48].unflatten(-1, (2, 16)), 240)])
def test_row_strides(t, want):
    assert _layers._row_stride("t", t) == want


@pytest.mark.parametrize("t", [torch.zeros(2, 9, 64)[:, :8], torch.zeros(2, 64, 9).transpose(1, 2),
                               torch.zeros(1, 1, 64).expand(2, 9, 64), torch.zeros(9, 2, 64).transpose(0, 1),
                               torch.zeros(2, 9, 128)[..., ::2], torch.zeros(2, 9, 2, 32)[..., :16]])
def test_rows_that_are_not_evenly_spaced(t):
    with pytest.raises(ValueError):
        _layers._row_stride("t", t)


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("wanted", ["nothing", "a weight", "x"])
def test_checkpoints_are_formed_only_for_a_backward_pass(monkeypatch, grad, wanted):
    packs = []
    monkeypatch.setattr(_layers, "pack8", lambda t: packs.append(t.shape) or packed(*t.shape, dtype=t.dtype))
    monkeypatch.setattr(_layers, "conv_fwd", lambda x, *a: (x.clone(), x.clone()))
    monkeypatch.setattr(_layers, "scan_fwd", lambda x, *a: (x.clone(), x.clone()))
    monkeypatch.setattr(_binding, "fwd", lambda q, k, v, *a, **kw: (v.clone(), v.clone()))
    d, c = scan_case(), conv_case()
    d["A_log"].requires_grad_(wanted == "a weight")
    c["weight"].requires_grad_(wanted == "a weight")
    for t in (d["x"], c["x"]):
        t.requires_grad_(wanted == "x")
    q = torch.zeros(1, 5, 2, 64, requires_grad=wanted == "x")
    w = torch.zeros(2, requires_grad=wanted == "a weight")
    g = torch.zeros(1, 5, 2)
    with torch.set_grad_enabled(grad):
        outs = (gdn.causal_conv(c["x"], c["weight"], checkpoint_bits=8),
                gdn.selective_scan(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], z=d["z"], checkpoint_bits=8),
                gdn.gated_delta_rule(q, q, q, g, g, w, checkpoint_bits=8))
    follows = grad and wanted != "nothing"
    assert all(t.requires_grad == follows for o in outs for t in o)
    assert len(packs) == (6 if follows else 0)  # x; x and z; q, k and v


# ---- the forms the GPU tests compare with ----------------------------------------

@pytest.mark.parametrize("lengths", [None, [0, 4, 1, 0, 5]])
def test_oracle_gradients_are_differences(lengths):
    cu = None if lengths is None else lo.offsets(lengths)
    S = 1 if cu is None else len(lengths)
    for f, (d, seeds) in ((lo.conv, lo.conv_inputs(1, 10, 6, 3, F32, 1, S)),
                          (lo.scan, lo.scan_inputs(1, 10, 6, 3, 2, F32, 1, S))):
        d, seeds = lo.double(d), [v.double() for v in seeds.values()]
        grads = lo.gradients(lambda **k: f(cu=cu, **k), d, seeds)
        for name, g in grads.items():
            v = torch.randn(g.shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
            e = 1e-5  # central differences: e^2 of third derivatives, 2^-53 / e of rounding
            L = [sum((s * o).sum() for s, o in zip(seeds, f(cu=cu, **dict(d, **{name: d[name] + q * e * v}))))
                 for q in (1, -1)]
            assert abs(float((L[0] - L[1]) / (2 * e) - (g * v).sum())) < 1e-6, name


def test_oracle_continues_from_its_final_states():
    d, _ = lo.scan_inputs(1, 12, 6, 3, 2, F32, 2)
    d = lo.double(d)
    cut = lambda a, b: {k: v[:, a:b] if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in d.items()}  # noqa: E731
    y, fin = lo.scan(**d)
    y1, mid = lo.scan(**cut(0, 5))
    y2, fin2 = lo.scan(**dict(cut(5, 12), h0=mid))
    assert torch.allclose(torch.cat([y1, y2], 1), y, rtol=1e-13) and torch.allclose(fin2, fin, rtol=1e-13)
    c, _ = lo.conv_inputs(1, 12, 6, 4, F32, 2)
    c = lo.double(c)
    y, fin = lo.conv(**c)
    y1, mid = lo.conv(**dict(c, x=c["x"][:, :2]))  # shorter than the window
    y2, fin2 = lo.conv(**dict(c, x=c["x"][:, 2:], h0=mid))
    # torch's sigmoid differs by its last bit between vector and scalar code
    assert torch.allclose(torch.cat([y1, y2], 1), y, rtol=1e-14, atol=0) and torch.equal(fin2, fin)


def test_oracle_checkpoint_by_hand():
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, 0.49] + [0.0] * 27 + [1.0, float("inf")]])
    codes, scales = lo.pack(x)
    assert codes[0, :5].tolist() == [127, 0, 2, -2, 0] and scales[0].tolist() == [127, 255]
    codes, scales = lo.pack(torch.tensor([[127.5, 1.0]]))
    assert codes.tolist() == [[64, 0]] and scales.tolist() == [[128]]
    assert lo.unpack(codes, scales).tolist() == [[128.0, 0.0]]
