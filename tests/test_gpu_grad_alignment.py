"""Gradients that reach a differentiable op as autograd makes them: parts of a longer tensor (the
backward pass of a concatenation), off 16 bytes."""
import pytest
import torch

import gated_deltanet_chunkwise_amd as gdn

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_attention_takes_gradients_at_any_address(dtype):
    gen = torch.Generator().manual_seed(71)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    B, T, H, K = 2, 70, 2, 64
    leaves = [r(B, T, H, K).to(dtype).requires_grad_() for _ in range(3)] + [r(B, H, K, K).requires_grad_()]
    ld, w, wf = torch.tensor([-0.1, -1.0], device="cuda"), r(B * T * H * K).to(dtype), r(B * H * K * K)

    def gradients(loss):
        for t in leaves:
            t.grad = None
        o, fin = gdn.linear_attention(*leaves[:3], ld, None, leaves[3])
        loss(o.flatten(), fin.flatten()).backward()
        return [t.grad for t in leaves]
    one = lambda t: t.new_zeros(1)  # noqa: E731
    whole = gradients(lambda o, fin: (o * w).sum() + (fin * wf).sum())
    parts = gradients(lambda o, fin: (torch.cat([one(o), o]) * torch.cat([one(o), w])).sum() +
                      (torch.cat([one(fin), fin]) * torch.cat([one(fin), wf])).sum())
    assert all(torch.equal(a, b) for a, b in zip(whole, parts))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_gated_delta_rule_takes_gradients_at_any_address(dtype):
    gen = torch.Generator().manual_seed(72)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    B, T, H, K = 2, 70, 2, 64
    q, k, v = (torch.nn.functional.normalize(r(B, T, H, K), dim=-1).to(dtype).requires_grad_() for _ in range(3))
    g, beta, A_log = r(B, T, H).requires_grad_(), torch.sigmoid(r(B, T, H)).requires_grad_(), r(H).abs().requires_grad_()
    leaves = [q, k, v, g, beta, A_log]
    w, wf = r(B * T * H * K).to(dtype), r(B * H * K * K)

    def gradients(loss):
        for t in leaves:
            t.grad = None
        o, fin = gdn.gated_delta_rule(q, k, v, g, beta, A_log)
        loss(o.flatten(), fin.flatten()).backward()
        return [t.grad for t in leaves]
    one = lambda t: t.new_zeros(1)  # noqa: E731
    whole = gradients(lambda o, fin: (o * w).sum() + (fin * wf).sum())
    parts = gradients(lambda o, fin: (torch.cat([one(o), o]) * torch.cat([one(o), w])).sum() +
                      (torch.cat([one(fin), fin]) * torch.cat([one(fin), wf])).sum())
    # dq, dk and dv repeat exactly; the gates' gradients are sums by LDS atomics, whose order (and so
    # their low bits) include/gdn.h leaves open
    assert all(torch.equal(a, b) for a, b in zip(whole[:3], parts[:3]))
    assert all(t.isfinite().all() for t in parts)
