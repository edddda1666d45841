"""Plain 64-bit forms of the layer operators (torch on the CPU, one token at a time; the
gradients by automatic differentiation), and the inputs and comparisons of their tests."""
import math

import torch

F64 = torch.float64


def spans(B, T, cu):
    """(row slice of the flattened tokens) of every sequence."""
    if cu is None:
        return [slice(b * T, (b + 1) * T) for b in range(B)]
    off = cu.tolist()
    return [slice(off[n], off[n + 1]) for n in range(len(off) - 1)]


def conv(x, weight, bias=None, cu=None, h0=None, silu=True):
    """y (0 behind the last sequence) and the final state; all tensors fp64."""
    B, T, C = x.shape
    W = weight.shape[1]
    rows = x.reshape(B * T, C)
    ys, fins = [], []
    done = 0
    for n, s in enumerate(spans(B, T, cu)):
        before = torch.zeros(W - 1, C, dtype=F64) if h0 is None else h0[n]
        line = torch.cat([before, rows[s]])
        pre = sum(line[j:j + s.stop - s.start] * weight[:, j] for j in range(W))
        pre = pre + (0 if bias is None else bias)
        ys.append(pre * torch.sigmoid(pre) if silu else pre)
        fins.append(line[line.shape[0] - (W - 1):])
        done = s.stop
    ys.append(torch.zeros(B * T - done, C, dtype=F64))
    return torch.cat(ys).view(B, T, C), torch.stack(fins) if fins else torch.zeros(0, W - 1, C, dtype=F64)


def softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def scan(x, dt, A_log, Bm, Cm, skip=None, z=None, dt_bias=None, cu=None, h0=None):
    """y (0 behind the last sequence) and the final states; all tensors fp64."""
    B, T, D = x.shape
    G, N = Bm.shape[2:]
    A = -torch.exp(A_log)
    wide = lambda t: t.reshape(B * T, G, 1, N).expand(-1, G, D // G, N).reshape(B * T, D, N)  # noqa: E731
    delta = softplus(dt if dt_bias is None else dt + dt_bias).reshape(B * T, D)
    xr, Br, Cr = x.reshape(B * T, D), wide(Bm), wide(Cm)
    ys, fins, done = [], [], 0
    for n, s in enumerate(spans(B, T, cu)):
        h = torch.zeros(D, N, dtype=F64) if h0 is None else h0[n]
        for t in range(s.start, s.stop):
            h = torch.exp(delta[t][:, None] * A) * h + (delta[t] * xr[t])[:, None] * Br[t]
            ys.append((h * Cr[t]).sum(1))
        fins.append(h)
        done = s.stop
    y = torch.stack(ys) if ys else torch.zeros(0, D, dtype=F64)
    if skip is not None:
        y = y + skip * xr[:done]
    if z is not None:
        zr = z.reshape(B * T, D)[:done]
        y = y * zr * torch.sigmoid(zr)
    y = torch.cat([y, torch.zeros(B * T - done, D, dtype=F64)])
    return y.view(B, T, D), torch.stack(fins) if fins else torch.zeros(0, D, N, dtype=F64)


def gradients(f, inputs, seeds):
    """d/d(inputs) of sum <seed, output> for f(**inputs) -> outputs; a dict by name (a
    zero tensor where nothing depends on the input)."""
    leaf = {k: v.clone().requires_grad_() for k, v in inputs.items() if v is not None}
    outs = f(**{k: leaf.get(k) for k in inputs})
    total = sum((s * o).sum() for s, o in zip(seeds, outs) if s is not None)
    got = torch.autograd.grad(total, list(leaf.values()), allow_unused=True)
    return {k: torch.zeros_like(v) if g is None else g for (k, v), g in zip(leaf.items(), got)}


def pack(x):
    """(codes, scale bytes) of a checkpoint, block by block in Python's own arithmetic
    (math.frexp and round are exact; round takes ties to even)."""
    rows = x.reshape(-1, x.shape[-1]).double()
    C = rows.shape[1]
    nblk = (C + 31) // 32
    codes = torch.zeros(rows.shape, dtype=torch.int8)
    scales = torch.zeros(rows.shape[0], nblk, dtype=torch.uint8)
    for r in range(rows.shape[0]):
        for b in range(nblk):
            v = rows[r, 32 * b:32 * b + 32].tolist()
            if not all(math.isfinite(a) for a in v):
                scales[r, b] = 255
                continue
            m, e = math.frexp(max(abs(a) for a in v))  # m 2^e, m in [1/2, 1), or 0
            e = e - 7 if m <= 127 / 128 else e - 6
            e = -126 if m == 0 else min(max(e, -126), 121)
            scales[r, b] = e + 127
            for i, a in enumerate(v):
                codes[r, 32 * b + i] = max(-127, min(127, round(a / 2.0 ** e)))
    return codes.view(x.shape), scales.view(*x.shape[:-1], nblk)


def unpack(codes, scales):
    """The values a checkpoint stands for, fp64 (NaN where the byte is 255)."""
    C = codes.shape[-1]
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return codes.double() * s.repeat_interleave(32, -1)[..., :C]


# ---- inputs and comparisons ------------------------------------------------------

def offsets(lengths):
    return torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)) if lengths else [0], dtype=torch.int64)


def conv_inputs(B, T, C, W, dtype, seed, S=None, h0=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    S = B if S is None else S
    return dict(x=r(B, T, C).to(dtype), weight=r(C, W) * 0.5, bias=r(C) * 0.2 if bias else None,
                h0=r(S, W - 1, C).to(dtype) if h0 else None), dict(
                    d_y=r(B, T, C).to(dtype), d_fin=r(S, W - 1, C).to(dtype))


def scan_inputs(B, T, D, N, G, dtype, seed, S=None, h0=True, skip=True, gate=True, bias=True):
    """Decay rates and time steps as such layers have them: exp(-A D) from about 0.2 to
    0.999 per token."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    S = B if S is None else S
    d = dict(x=r(B, T, D).to(dtype), dt=(r(B, T, D) * 0.5 + (0 if bias else -3)).to(dtype),
             A_log=torch.log(torch.arange(1, N + 1).float()).expand(D, N) + 0.1 * r(D, N),
             Bm=r(B, T, G, N).to(dtype), Cm=r(B, T, G, N).to(dtype), skip=1 + 0.1 * r(D) if skip else None,
             z=r(B, T, D).to(dtype) if gate else None, dt_bias=r(D) - 3 if bias else None,
             h0=r(S, D, N) * 0.5 if h0 else None)
    return d, dict(d_y=r(B, T, D).to(dtype), d_fin=r(S, D, N) * 0.2)


def double(d):
    return {k: None if v is None else v.to(F64) for k, v in d.items()}


def cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def close(got, ref, steps, what):
    """Relative 2-norm and every element.  The kernels compute in fp32 and round once:
    half a step of the result's type (finfo.eps / 2 relative), and of each of `steps`
    dependent steps at most 8 roundings of 2^-24 (the exponent's argument, its
    exponential, two products, a sum, softplus's three), whose errors at worst add up."""
    half = torch.finfo(got.dtype).eps / 2
    tol = 8 * (steps + 16) * 2.0 ** -24
    got = got.detach().cpu().to(F64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not ref.numel():
        return
    assert torch.isfinite(got).all(), what + ": not finite"
    err = (got - ref).abs()
    rel = float(err.norm() / ref.norm()) if float(ref.norm()) else float(err.norm())
    print("  %-24s rel_l2=%.2e (%.2e) max=%.2e" % (what, rel, half + tol, float(err.max())), flush=True)
    assert rel <= half + tol, (what, rel, half + tol)
    worst = (err - half * ref.abs()).max()
    assert float(worst) <= tol * float(ref.abs().max()) + half * 2.0 ** -126, (what, float(worst))
