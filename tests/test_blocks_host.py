"""Linear attention's and the norms' wrappers on the CPU: every tensor's shape and dtype is
checked before anything reaches the library, and tensors that are not on a GPU are refused; the
64-bit form of linear attention is held to differences and to itself."""
import pytest
import torch

import block_oracle as bo
import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo
from gated_deltanet_chunkwise_amd import _binding

BF16, F32 = torch.bfloat16, torch.float32


class _NoCalls:
    def __getattr__(self, name):
        raise AssertionError("library call %s reached" % name)


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(_binding, "_LIB", _NoCalls())


def attn_case():
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(q=z(2, 9, 2, 64), k=z(2, 9, 2, 64), v=z(2, 9, 4, 128), ld=z(4, dtype=F32), h0=z(2, 4, 64, 128, dtype=F32),
                d_o=z(2, 9, 4, 128), d_fin=z(2, 4, 64, 128, dtype=F32), cu=None)


def attn_calls(d):
    a = (d["q"], d["k"], d["v"], d["ld"])
    return [lambda: gdn.linear_attn_fwd(*a, d["cu"], d["h0"]), lambda: gdn.linear_attn_bwd(*a, d["d_o"], d["d_fin"], d["cu"], d["h0"]),
            lambda: gdn.linear_attention(*a, d["cu"], d["h0"]), lambda: gdn.linear_attn_decode(*a, d["h0"]),
            lambda: gdn.linear_attn_decode_launcher(*a, d["h0"])]


@pytest.mark.parametrize("name,bad,error", [
    ("q", torch.zeros(9, 2, 64, dtype=BF16), ValueError), ("q", torch.zeros(2, 9, 2, 64), TypeError),
    ("q", torch.zeros(2, 9, 2, 64, dtype=torch.float16), TypeError), ("k", torch.zeros(2, 9, 1, 64, dtype=BF16), ValueError),
    ("k", torch.zeros(2, 9, 2, 64), TypeError), ("v", torch.zeros(2, 8, 4, 128, dtype=BF16), ValueError),
    ("v", torch.zeros(2, 9, 512, dtype=BF16), ValueError), ("v", torch.zeros(2, 9, 4, 128), TypeError),
    ("ld", torch.zeros(2), ValueError), ("ld", torch.zeros(4, dtype=BF16), TypeError), ("ld", torch.zeros(4, 1), ValueError),
    ("h0", torch.zeros(2, 4, 128, 64), ValueError), ("h0", torch.zeros(2, 4, 64, 128, dtype=BF16), TypeError)])
def test_linear_attention_refuses(name, bad, error):
    for call in attn_calls(dict(attn_case(), **{name: bad})):
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("name,bad,error", [
    ("d_o", None, ValueError), ("d_o", torch.zeros(2, 9, 4, 64, dtype=BF16), ValueError), ("d_o", torch.zeros(2, 9, 4, 128), TypeError),
    ("d_fin", torch.zeros(1, 4, 64, 128), ValueError), ("d_fin", torch.zeros(2, 4, 64, 128, dtype=BF16), TypeError),
    ("cu", torch.zeros(3, dtype=torch.int32), TypeError), ("cu", torch.zeros(3, dtype=torch.int64), ValueError)])
def test_linear_attention_backward_refuses(name, bad, error):
    with pytest.raises(error):
        attn_calls(dict(attn_case(), **{name: bad}))[1]()


def test_the_decay_is_a_constant():
    d = attn_case()
    d["ld"].requires_grad_()
    with pytest.raises(ValueError, match="log_decay"):
        attn_calls(d)[2]()
    with pytest.raises(ValueError, match="checkpoint_bits"):
        gdn.linear_attention(d["q"], d["k"], d["v"], d["ld"].detach(), checkpoint_bits=4)


def test_a_decode_step_needs_a_state():
    d = attn_case()
    for f in (gdn.linear_attn_decode, gdn.linear_attn_decode_launcher):
        with pytest.raises(ValueError, match="state"):
            f(d["q"], d["k"], d["v"], d["ld"], None)
        with pytest.raises(ValueError):
            f(d["q"], d["k"], d["v"], d["ld"], d["h0"], out=torch.zeros(2, 9, 4, 64, dtype=BF16))
        with pytest.raises(TypeError):
            f(d["q"], d["k"], d["v"], d["ld"], d["h0"], new_state=d["h0"].to(BF16))


def norm_case():
    return dict(x=torch.zeros(2, 9, 4, 64, dtype=BF16), w=torch.zeros(64), z=torch.zeros(2, 9, 4, 64, dtype=BF16),
                d_y=torch.zeros(2, 9, 4, 64, dtype=BF16))


def norm_calls(d):
    return [lambda: gdn.gated_norm_fwd(d["x"], d["w"], d["z"]), lambda: gdn.gated_norm_bwd(d["x"], d["w"], d["d_y"], d["z"]),
            lambda: gdn.gated_norm(d["x"], d["w"], d["z"])]


@pytest.mark.parametrize("name,bad,error", [
    ("x", torch.zeros(9, 64, dtype=BF16), ValueError), ("x", torch.zeros(2, 9, 4, 64, dtype=torch.float16), TypeError),
    ("w", torch.zeros(4, 64), ValueError), ("w", torch.zeros(64, dtype=BF16), TypeError), ("z", torch.zeros(2, 9, 256, dtype=BF16), ValueError),
    ("z", torch.zeros(2, 9, 4, 64), TypeError)])
def test_gated_norm_refuses(name, bad, error):
    for call in norm_calls(dict(norm_case(), **{name: bad})):
        with pytest.raises(error):
            call()


def test_gated_norm_refuses_more():
    d = norm_case()
    for bad, error in ((None, ValueError), (torch.zeros(2, 9, 4, 64), TypeError), (torch.zeros(2, 9, 2, 64, dtype=BF16), ValueError)):
        with pytest.raises(error):
            norm_calls(dict(d, d_y=bad))[1]()
    for eps in (-1e-6, float("nan")):
        with pytest.raises(ValueError, match="eps"):
            gdn.gated_norm_fwd(d["x"], d["w"], d["z"], eps=eps)


def res_case():
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(x=z(2, 9, 64), r=z(2, 9, 64, dtype=F32), w=z(64, dtype=F32), post=z(64, dtype=F32), scale=z(64, dtype=F32), d_h=z(2, 9, 64),
                d_r=z(2, 9, 64, dtype=F32))


def res_calls(d):
    o = dict(post_weight=d["post"], scale=d["scale"])
    return [lambda: gdn.residual_norm_fwd(d["x"], d["r"], d["w"], **o), lambda: gdn.residual_norm_bwd(d["x"], d["r"], d["w"], d["d_h"], d["d_r"], **o),
            lambda: gdn.residual_norm(d["x"], d["r"], d["w"], **o)]


@pytest.mark.parametrize("name,bad,error", [
    ("x", torch.zeros(9, 64, dtype=BF16), ValueError), ("x", torch.zeros(2, 9, 64, dtype=torch.float16), TypeError),
    ("r", None, ValueError), ("r", torch.zeros(2, 9, 64, dtype=torch.float16), TypeError), ("r", torch.zeros(2, 8, 64), ValueError),
    ("w", torch.zeros(63), ValueError), ("w", torch.zeros(64, dtype=BF16), TypeError), ("post", torch.zeros(1, 64), ValueError),
    ("scale", torch.zeros(1), ValueError), ("scale", torch.zeros(64, dtype=torch.float64), TypeError)])
def test_residual_norm_refuses(name, bad, error):
    for call in res_calls(dict(res_case(), **{name: bad})):
        with pytest.raises(error):
            call()


def test_residual_norm_refuses_more():
    d = res_case()
    with pytest.raises(TypeError):  # a residual of fewer bits than the block's output
        res_calls(dict(d, x=d["x"].float(), r=d["r"].to(BF16), d_h=d["d_h"].float()))[0]()
    for k, bad, error in (("d_h", None, ValueError), ("d_h", torch.zeros(2, 9, 64), TypeError), ("d_r", torch.zeros(2, 9, 64, dtype=BF16), TypeError)):
        with pytest.raises(error):
            res_calls(dict(d, **{k: bad}))[1]()


def test_host_tensors_are_refused():
    for call in attn_calls(attn_case()) + norm_calls(norm_case()) + res_calls(res_case()):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


def test_rows_that_are_not_evenly_spaced():
    d = attn_case()
    for bad in (torch.zeros(2, 9, 64, 2, dtype=BF16).transpose(2, 3), torch.zeros(2, 12, 2, 64, dtype=BF16)[:, :9],
                torch.zeros(2, 9, 2, 128, dtype=BF16)[..., :64]):
        with pytest.raises(ValueError, match="q"):
            attn_calls(dict(d, q=bad))[0]()
    with pytest.raises(ValueError, match="z"):
        norm_calls(dict(norm_case(), z=torch.zeros(2, 4, 9, 64, dtype=BF16).transpose(1, 2)))[0]()


# ---- the form the GPU tests compare with ---------------------------------------------

@pytest.mark.parametrize("lengths", [None, [0, 4, 1, 0, 5]])
def test_oracle_gradients_are_differences(lengths):
    cu = None if lengths is None else lo.offsets(lengths)
    S = 1 if cu is None else len(lengths)
    d, seeds, ld = bo.linattn_inputs(1, 10, 1, 2, 3, 4, F32, 1, S)
    d, seeds = lo.double(d), [v.double() for v in seeds.values()]
    f = lambda **k: bo.linattn(log_decay=ld.double(), cu=cu, scale=0.7, **k)  # noqa: E731
    for name, g in lo.gradients(f, d, seeds).items():
        v = torch.randn(g.shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
        e = 1e-5  # central differences: e^2 of third derivatives, 2^-53 / e of rounding
        L = [sum((s * o).sum() for s, o in zip(seeds, f(**dict(d, **{name: d[name] + q * e * v})))) for q in (1, -1)]
        assert abs(float((L[0] - L[1]) / (2 * e) - (g * v).sum())) < 1e-6, name


def test_oracle_continues_from_its_final_states():
    d, _, ld = bo.linattn_inputs(1, 12, 2, 4, 3, 4, F32, 2)
    d = lo.double(d)
    cut = lambda a, b: {k: v if k == "h0" else v[:, a:b] for k, v in d.items()}  # noqa: E731
    o, fin = bo.linattn(log_decay=ld.double(), **d)
    o1, mid = bo.linattn(log_decay=ld.double(), **cut(0, 5))
    o2, fin2 = bo.linattn(log_decay=ld.double(), **dict(cut(5, 12), h0=mid))
    assert torch.allclose(torch.cat([o1, o2], 1), o, rtol=1e-13) and torch.allclose(fin2, fin, rtol=1e-13)


def test_oracle_by_hand():
    one = lambda *v: torch.tensor(v, dtype=torch.float64).view(1, -1, 1, 1)  # noqa: E731
    o, fin = bo.linattn(one(1, 2, 3), one(1, 1, 2), one(4, 5, 6), torch.full((1, 1, 1, 1), 8.0, dtype=torch.float64),
                        log_decay=torch.log(torch.tensor([0.5], dtype=torch.float64)), scale=2.0)
    # H: 8 -> 4 + 4 -> 4 + 5 -> 4.5 + 12
    assert o.flatten().tolist() == pytest.approx([16.0, 36.0, 99.0]) and float(fin) == pytest.approx(16.5)
