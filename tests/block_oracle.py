"""Plain 64-bit forms of linear attention and of the norms around a block (torch on the CPU,
one token at a time; the gradients by automatic differentiation), and the inputs and
comparisons of their tests."""
import torch

import layer_oracle as lo

F64 = torch.float64


def linattn(q, k, v, h0=None, *, log_decay, cu=None, scale=1.0):
    """o (0 behind the last sequence) and the final states; all tensors fp64."""
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    q, k = (t.repeat_interleave(HV // H, 2).reshape(B * T, HV, K) for t in (q, k))
    v = v.reshape(B * T, HV, V)
    a = torch.exp(log_decay)[:, None, None]
    outs, fins, done = [], [], 0
    for n, s in enumerate(lo.spans(B, T, cu)):
        h = torch.zeros(HV, K, V, dtype=F64) if h0 is None else h0[n]
        for t in range(s.start, s.stop):
            h = a * h + k[t][:, :, None] * v[t][:, None, :]
            outs.append(scale * (h * q[t][:, :, None]).sum(1))
        fins.append(h)
        done = s.stop
    o = torch.stack(outs) if outs else torch.zeros(0, HV, V, dtype=F64)
    o = torch.cat([o, torch.zeros(B * T - done, HV, V, dtype=F64)])
    return o.view(B, T, HV, V), torch.stack(fins) if fins else torch.zeros(0, HV, K, V, dtype=F64)


def linattn_inputs(B, T, H, HV, K, V, dtype, seed, S=None, h0=True):
    """Heads that forget within a few tokens to heads that hold all."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    S = B if S is None else S
    d = dict(q=r(B, T, H, K).to(dtype), k=r(B, T, H, K).to(dtype), v=r(B, T, HV, V).to(dtype),
             h0=r(S, HV, K, V) if h0 else None)
    ld = -torch.exp2(torch.linspace(-11.0, 1.0, HV)) if HV > 1 else torch.tensor([-0.02])
    return d, dict(d_o=r(B, T, HV, V).to(dtype), d_fin=r(S, HV, K, V) * 0.3), ld


def close(got, ref, tol, what, each=None, size=None):
    """Relative 2-norm within `tol`, and every element within `each` (16 tol unless given)
    of the larger of its own value and the tensor's root mean square; both relative to
    `size` where that is given."""
    got = got.detach().cpu().to(F64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not ref.numel():
        return
    assert torch.isfinite(got).all(), what + ": not finite"
    size = ref if size is None else size
    err, rms = (got - ref).abs(), float(size.norm()) / ref.numel() ** 0.5
    rel = float(err.norm() / size.norm()) if rms else float(err.norm())
    worst = float((err / size.abs().clamp(min=rms)).max()) if rms else float(err.max())
    print("  %-24s rel_l2=%.2e (%.2e) worst=%.2e" % (what, rel, tol, worst), flush=True)
    assert rel <= tol, (what, rel, tol)
    assert worst <= (16 * tol if each is None else each), (what, worst)
