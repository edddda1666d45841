"""Linear attention with a decay for each head, and the norms around such a block, as they
are measured, in training, prompt and single-token form: `linear_attention`, the gated norm
of its output (`gated_norm`) and the step from one block to the next (`residual_norm`).

`own` false: the plain form, elementary torch operations in 32 bits, rounded once at the
end.  `own` true: the library's entry points.  `exact` is the definition in 64 bits, token
by token.

    linear attention  a = exp(log_decay[hv]);  H_t = a H_{t-1} + k_t v_t^T;  o_t = scale H_t^T q_t
                      (value head hv reads query and key head hv / (HV/H))
    gated norm        r(u) = u / sqrt(mean(u^2) + eps);  y = r(x) weight silu(z),
                      or y = r(x silu(z)) weight (gate first);  silu(z) = z / (1 + e^-z)
    residual norm     p = r(x) post_weight, or x;  s = residual + scale p;  h = r(s) weight
"""
import math

import torch

import gated_deltanet_chunkwise_amd as gdn

own = False

BF16, FP32 = "bf16", "fp32"
DT = {BF16: torch.bfloat16, FP32: torch.float32}
EPS = 1e-6
PIECE = 64  # tokens that the plain form of linear attention treats as one matrix


def listed():
    return [
        # one token for each of 64 decoding sequences, 16 heads of 128
        dict(name="attn_step", op="attn_step", B=64, T=1, H=16, HV=16, K=128, V=128, dtype=BF16),
        # the prompts of two sequences of 2048 tokens; q, k and v are slices of one projection
        dict(name="attn_prompt", op="attn", B=2, T=2048, H=16, HV=16, K=128, V=128, dtype=BF16, seqs=0, wide=True),
        # twelve packed prompts of 32768 tokens in all, four value heads per key head: the longest call
        dict(name="attn_packed_long", op="attn", B=1, T=32768, H=4, HV=16, K=128, V=128, dtype=BF16, seqs=12, wide=False),
        # full precision, odd numbers of tokens and heads, keys and values of two widths
        dict(name="attn_fp32_odd", op="attn", B=3, T=777, H=5, HV=5, K=64, V=128, dtype=FP32, seqs=0, wide=False),
        # the backward pass of a training step
        dict(name="attn_backward", op="attn_bwd", B=2, T=2048, H=16, HV=16, K=128, V=128, dtype=BF16, seqs=0),
        # the backward pass of ragged packed sequences, four value heads per key head
        dict(name="attn_backward_packed", op="attn_bwd", B=1, T=5003, H=2, HV=8, K=128, V=64, dtype=BF16, seqs=7),
        # the gated norm of one token's 16 heads for each of 64 sequences: the smallest call
        dict(name="gated_norm_step", op="gnorm", B=64, T=1, H=16, D=128, dtype=BF16, gate="after", wide=False),
        # the same of a wide training batch; the gate is a slice of a projection
        dict(name="gated_norm_batch", op="gnorm", B=4, T=8192, H=16, D=128, dtype=BF16, gate="after", wide=True),
        # its backward pass
        dict(name="gated_norm_backward", op="gnorm_bwd", B=2, T=2048, H=16, D=128, dtype=BF16, gate="after"),
        # between two blocks, one token of 64 sequences, the residual in full precision
        dict(name="residual_norm_step", op="rnorm", B=64, T=1, C=2048, dtype=BF16, res=FP32, post=True, scale=True),
        # between two blocks of a prompt, full precision, odd sizes, no norm behind the block
        dict(name="residual_norm_fp32_odd", op="rnorm", B=1, T=5003, C=1000, dtype=FP32, res=FP32, post=False, scale=True),
        # the backward pass of a training step
        dict(name="residual_norm_backward", op="rnorm_bwd", B=4, T=4096, C=2048, dtype=BF16, res=BF16, post=True, scale=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_step", "attn", "attn", "attn_bwd", "attn_bwd", "gnorm", "gnorm_bwd", "rnorm", "rnorm_bwd"])
    dtype = rng.choice([BF16, BF16, FP32])
    if op.startswith("attn"):
        H, G = rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([1, 1, 2, 4])
        c = dict(op=op, H=H, HV=H * G, K=rng.choice([64, 128]), V=rng.choice([64, 128]), dtype=dtype)
        if op == "attn_step":
            return dict(c, B=_log(rng, 1, 1024 // (H * G)), T=rng.choice([1, 1, 2, 4]))
        seqs = rng.choice([0, 0, 3, 9])
        B = 1 if seqs else rng.choice([1, 2, 3, 8])
        most = 1 << (18 if op == "attn" else 15)                   # tokens times value heads
        c = dict(c, B=B, T=max(1, min(_log(rng, 1, 32768), most // (B * H * G))), seqs=seqs)
        return dict(c, wide=rng.random() < 0.5) if op == "attn" else c
    if op.startswith("gnorm"):
        H = rng.choice([1, 4, 16, 5])
        D = _log(rng, 64, 8192) if H == 1 else rng.choice([64, 128, 128, 96, 100, 256])
        B, most = rng.choice([1, 2, 64]), 1 << (25 if op == "gnorm" else 23)
        c = dict(op=op, B=B, T=max(1, min(_log(rng, 1, 16384), most // (B * H * D))), H=H, D=D, dtype=dtype,
                 gate=rng.choice(["after", "after", "first", "none"]))
        return dict(c, wide=rng.random() < 0.5) if op == "gnorm" else c
    C, B = _log(rng, 64, 8192), rng.choice([1, 2, 64])
    return dict(op=op, B=B, T=max(1, min(_log(rng, 1, 16384), (1 << 25) // (B * C))), C=C, dtype=dtype,
                res=rng.choice([dtype, FP32]), post=rng.random() < 0.5, scale=rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------


def _offsets(case):
    """The packed sequences' first tokens and the end, some of them empty or a single
    token where there is room; None for sequences of one length."""
    n, T = case.get("seqs", 0), case["T"]
    if not n:
        return None
    g = torch.Generator().manual_seed(1000 * n + T)
    cuts = sorted(int(v) for v in torch.randint(0, T + 1, (n - 1,), generator=g))
    return [0] + cuts + [T]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], DT[case["dtype"]]
    B, T = case["B"], case["T"]

    def normal(*shape, scale=1.0, shift=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)

    s = dict(case=case, dtype=dt)
    if op.startswith("attn"):
        H, HV, K, V = case["H"], case["HV"], case["K"], case["V"]
        off = _offsets(case)
        s["cu"] = None if off is None else torch.tensor(off, dtype=torch.int64, device="cuda")
        S = B if off is None else len(off) - 1
        if case.get("wide"):
            qkv = normal(B, T, 2 * H * K + HV * V, dtype=dt)
            q, k, v = qkv.split([H * K, H * K, HV * V], -1)
            s["q"], s["k"], s["v"] = q.unflatten(-1, (H, K)), k.unflatten(-1, (H, K)), v.unflatten(-1, (HV, V))
        else:
            s["q"], s["k"], s["v"] = normal(B, T, H, K, dtype=dt), normal(B, T, H, K, dtype=dt), normal(B, T, HV, V, dtype=dt)
        # heads that forget within a few tokens to heads that hold thousands
        s["log_decay"] = -torch.exp(torch.rand(HV, generator=g, device="cuda") * math.log(2.0 ** 11) - math.log(2.0 ** 12))
        s["h0"] = normal(S, HV, K, V)
        s["scale"] = K ** -0.5
        if op == "attn_step":
            s["new"] = torch.empty_like(s["h0"])
        if op == "attn_bwd":
            s["d_o"] = normal(B, T, HV, V, dtype=dt)
            s["d_fin"] = normal(S, HV, K, V, scale=0.1)
        return s
    if op.startswith("gnorm"):
        H, D = case["H"], case["D"]
        s["x"] = normal(B, T, H, D, scale=3.0, dtype=dt)
        s["weight"] = normal(D, scale=0.1, shift=1.0)
        s["z"] = None
        if case["gate"] != "none":
            s["z"] = normal(B, T, 2 * H * D, dtype=dt)[..., H * D:].unflatten(-1, (H, D)) if case.get("wide") else normal(B, T, H, D, dtype=dt)
        if op == "gnorm_bwd":
            s["d_y"] = normal(B, T, H, D, dtype=dt)
        return s
    C, rdt = case["C"], DT[case["res"]]
    s["x"], s["residual"] = normal(B, T, C, dtype=dt), normal(B, T, C, scale=4.0, dtype=rdt)
    s["weight"] = normal(C, scale=0.1, shift=1.0)
    s["post"] = normal(C, scale=0.1, shift=1.0) if case["post"] else None
    s["scale"] = normal(C, scale=0.1, shift=0.5) if case["scale"] else None
    if op == "rnorm_bwd":
        s["d_h"], s["d_res"] = normal(B, T, C, dtype=dt), normal(B, T, C, dtype=rdt)
    return s


# ---- plain forms -------------------------------------------------------------


def _pieces(s):
    """Sequences in pieces of PIECE tokens from their first on.  Of every token (flattened):
    its piece and its place there.  Of every piece: its sequence, its number there and its
    length.  Of every sequence: its length.  (Pieces that hold no token have length 0.)"""
    B, T = s["case"]["B"], s["case"]["T"]
    first = torch.arange(B, device="cuda") * T if s["cu"] is None else s["cu"][:-1]
    end = first + T if s["cu"] is None else s["cu"][1:]
    N = first.numel()
    base = first // PIECE + torch.arange(N, device="cuda")          # pieces of two sequences never meet
    tok = torch.arange(B * T, device="cuda")
    seq = torch.searchsorted(end, tok, right=True)
    pos = tok - first[seq]
    piece = torch.arange(B * T // PIECE + N, device="cuda")
    pseq = torch.searchsorted(base, piece, right=True) - 1
    num = piece - base[pseq]
    plen = ((end - first)[pseq] - num * PIECE).clamp(0, PIECE)
    return base[seq] + pos // PIECE, pos % PIECE, pseq, num, plen, end - first


def _cut(t, at, pieces):
    """[heads, pieces, PIECE, width] in 32 bits, 0 where a piece ends early, of t [B, T, heads, width]."""
    out = torch.zeros(pieces, PIECE, *t.shape[2:], device="cuda")
    out[at] = t.float().flatten(0, 1)
    return out.permute(2, 0, 1, 3).contiguous()


def _joined(t, at, shape):
    return t.permute(1, 2, 0, 3)[at].reshape(shape)


def _power(log_decay, n):
    """exp(n log_decay), [heads, ...] for n [...] of whole numbers."""
    return torch.exp(log_decay.view(-1, *[1] * n.dim()) * n.float())


def _attn_parts(s, back):
    c = s["case"]
    H, HV, K, V = c["H"], c["HV"], c["K"], c["V"]
    at0, at1, pseq, num, plen, length = _pieces(s)
    at, P, ld = (at0, at1), pseq.numel(), s["log_decay"]
    q, k = (_cut(s[n], at, P).repeat_interleave(HV // H, 0) for n in ("q", "k"))
    v = _cut(s["v"], at, P)
    i = torch.arange(PIECE, device="cuda")
    gap = i[:, None] - i
    decay = torch.where(gap >= 0, _power(ld, gap.clamp(min=0)), 0.0)[:, None]         # [HV, 1, t, s]
    after = _power(ld, (plen[:, None] - 1 - i).clamp(min=0))[..., None]               # from s to the piece's end
    upto = _power(ld, i + 1)[:, None, :, None]                                        # from the piece's start through t
    add = torch.matmul((k * after).transpose(2, 3).contiguous(), v).flatten(2)        # [HV, P, K V]
    # states ahead of the pieces: what earlier pieces of the same sequence left, and its start
    first = num * PIECE
    mine = pseq[:, None] == pseq
    gap = (first[:, None] - (first + plen)).clamp(min=0)
    link = torch.where(mine & (num[:, None] > num), _power(ld, gap), 0.0)             # [HV, P, P]
    h0 = s["h0"].transpose(0, 1).flatten(2)                                           # [HV, N, K V]
    H_ = (torch.matmul(link, add) + _power(ld, first)[..., None] * h0[:, pseq]).view(HV, P, K, V)
    left = (length[pseq] - first - plen).clamp(min=0)                                 # tokens behind a piece
    of_seq = pseq == torch.arange(length.numel(), device="cuda")[:, None]               # [N, P]
    fin = torch.matmul(torch.where(of_seq, _power(ld, left)[:, None], 0.0), add) + _power(ld, length)[..., None] * h0
    fin = fin.view(HV, -1, K, V).transpose(0, 1)
    if not back:
        o = torch.matmul(torch.matmul(q, k.transpose(2, 3).contiguous()) * decay, v) + upto * torch.matmul(q, H_)
        return (s["scale"] * _joined(o, at, s["v"].shape)).to(s["dtype"]), fin.contiguous()
    d_o = _cut(s["d_o"], at, P) * s["scale"]
    got = torch.matmul((q * upto).transpose(2, 3).contiguous(), d_o).flatten(2)
    # the states' gradients behind the pieces: what later pieces ask for, and the end's
    back_link = torch.where(mine & (num[:, None] < num), _power(ld, (first - (first + plen)[:, None]).clamp(min=0)), 0.0)
    d_fin = s["d_fin"].transpose(0, 1).flatten(2)
    dH = (torch.matmul(back_link, got) + _power(ld, left)[..., None] * d_fin[:, pseq]).view(HV, P, K, V)
    dh0 = torch.matmul(torch.where(of_seq, _power(ld, first)[:, None], 0.0), got) + _power(ld, length)[..., None] * d_fin
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * decay
    d_score = torch.matmul(d_o, v.transpose(2, 3).contiguous()) * decay
    dq = torch.matmul(d_score, k) + upto * torch.matmul(d_o, H_.transpose(2, 3).contiguous())
    dk = torch.matmul(d_score.transpose(2, 3).contiguous(), q) + after * torch.matmul(v, dH.transpose(2, 3).contiguous())
    dv = torch.matmul(score.transpose(2, 3).contiguous(), d_o) + after * torch.matmul(k, dH)
    dq, dk = (t.view(H, HV // H, *t.shape[1:]).sum(1) for t in (dq, dk))
    out = dict(dq=_joined(dq, at, s["q"].shape), dk=_joined(dk, at, s["k"].shape), dv=_joined(dv, at, s["v"].shape))
    return dict({n: t.to(s["dtype"]) for n, t in out.items()}, dh0=dh0.view(HV, -1, K, V).transpose(0, 1).contiguous())


def _step(s):
    """A few tokens of every sequence: the sum over them written out, no pieces."""
    c = s["case"]
    G, T = c["HV"] // c["H"], c["T"]
    q, k = (s[n].float().repeat_interleave(G, 2).transpose(1, 2) for n in ("q", "k"))  # [B, HV, T, K]
    v, h0, ld = s["v"].float().transpose(1, 2), s["h0"], s["log_decay"]
    i = torch.arange(T, device="cuda")
    gap = i[:, None] - i
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * torch.where(gap >= 0, _power(ld, gap.clamp(min=0)), 0.0)
    o = torch.matmul(score, v) + _power(ld, i + 1)[..., None] * torch.matmul(q, h0)
    kw = (k * _power(ld, T - 1 - i)[..., None]).transpose(2, 3).contiguous()
    new = torch.exp(ld * T)[:, None, None] * h0 + torch.matmul(kw, v)
    return dict(o=(s["scale"] * o.transpose(1, 2)).to(s["dtype"]), state=new)


def _rstd(u):
    return torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)


def _norm_back(u, r, du):
    """Through u r: r (du - u r mean(u r du)) for the gradient du towards u r."""
    n = u * r
    return r * (du - n * (n * du).mean(-1, keepdim=True))


def _gnorm(s):
    x, w, z = s["x"].float(), s["weight"], None if s["z"] is None else s["z"].float()
    if z is None:
        y = x * _rstd(x) * w
    elif s["case"]["gate"] == "first":
        u = x * z * torch.sigmoid(z)
        y = u * _rstd(u) * w
    else:
        y = x * _rstd(x) * w * z * torch.sigmoid(z)
    return y.to(s["dtype"])


def _gnorm_bwd(s):
    x, w, dy = s["x"].float(), s["weight"], s["d_y"].float()
    if s["z"] is None:
        r = _rstd(x)
        return dict(dx=_norm_back(x, r, dy * w).to(s["dtype"]), dweight=(dy * x * r).sum((0, 1, 2)))
    z = s["z"].float()
    g = torch.sigmoid(z)
    silu, slope = z * g, g + z * g * (1 - g)
    if s["case"]["gate"] == "first":
        u = x * silu
        r = _rstd(u)
        du = _norm_back(u, r, dy * w)
        dx, dz, dw = du * silu, du * x * slope, dy * u * r
    else:
        r = _rstd(x)
        n = x * r
        dx, dz, dw = _norm_back(x, r, dy * w * silu), dy * n * w * slope, dy * silu * n
    return dict(dx=dx.to(s["dtype"]), dz=dz.to(s["dtype"]), dweight=dw.sum((0, 1, 2)))


def _rnorm(s):
    x, scale = s["x"].float(), 1.0 if s["scale"] is None else s["scale"]
    p = x if s["post"] is None else x * _rstd(x) * s["post"]
    new = s["residual"].float() + scale * p
    return dict(h=(new * _rstd(new) * s["weight"]).to(s["dtype"]), residual=new.to(s["residual"].dtype))


def _rnorm_bwd(s):
    x, scale, dh = s["x"].float(), 1.0 if s["scale"] is None else s["scale"], s["d_h"].float()
    rx = _rstd(x)
    p = x if s["post"] is None else x * rx * s["post"]
    new = s["residual"].float() + scale * p
    r = _rstd(new)
    d = s["d_res"].float() + _norm_back(new, r, dh * s["weight"])
    dp = d * scale
    dx = dp if s["post"] is None else _norm_back(x, rx, dp * s["post"])
    out = dict(dx=dx.to(s["dtype"]), dresidual=d.to(s["residual"].dtype), dweight=(dh * new * r).sum((0, 1)))
    if s["post"] is not None:
        out["dpost_weight"] = (dp * x * rx).sum((0, 1))
    if s["scale"] is not None:
        out["dscale"] = (d * p).sum((0, 1))
    return out


def run(s):
    op = s["case"]["op"]
    if op == "attn":
        if own:
            o, fin = gdn.linear_attn_fwd(s["q"], s["k"], s["v"], s["log_decay"], cu_seqlens=s["cu"], initial_state=s["h0"], scale=s["scale"])
        else:
            o, fin = _attn_parts(s, False)
        return dict(o=o, final_state=fin)
    if op == "attn_step":
        if own:
            o = gdn.linear_attn_decode(s["q"], s["k"], s["v"], s["log_decay"], s["h0"], scale=s["scale"], new_state=s["new"])
            return dict(o=o, state=s["new"])
        return _step(s)
    if op == "attn_bwd":
        if own:
            return gdn.linear_attn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["d_o"], s["d_fin"], cu_seqlens=s["cu"], initial_state=s["h0"], scale=s["scale"])
        return _attn_parts(s, True)
    first = s["case"].get("gate") == "first"
    if op == "gnorm":
        return gdn.gated_norm_fwd(s["x"], s["weight"], s["z"], eps=EPS, gate_first=first) if own else _gnorm(s)
    if op == "gnorm_bwd":
        return gdn.gated_norm_bwd(s["x"], s["weight"], s["d_y"], s["z"], eps=EPS, gate_first=first) if own else _gnorm_bwd(s)
    if op == "rnorm":
        if own:
            h, new = gdn.residual_norm_fwd(s["x"], s["residual"], s["weight"], post_weight=s["post"], scale=s["scale"], eps=EPS)
            return dict(h=h, residual=new)
        return _rnorm(s)
    if own:
        return gdn.residual_norm_bwd(s["x"], s["residual"], s["weight"], s["d_h"], s["d_res"], post_weight=s["post"], scale=s["scale"], eps=EPS)
    return _rnorm_bwd(s)


def work(case):
    op, e = case["op"], 2 if case["dtype"] == BF16 else 4
    tok = case["B"] * case["T"]
    if op.startswith("attn"):
        H, HV, K, V = case["H"], case["HV"], case["K"], case["V"]
        state = (case.get("seqs", 0) or case["B"]) * HV * K * V * 4
        qk, v = tok * H * K * e, tok * HV * V * e
        kv = tok * HV * K * V
        if op == "attn_bwd":
            # q, k, v, d_o and the states at both ends in, dq, dk, dv and one state out; the states
            # formed again, the three gradients, the states' own
            return dict(bytes=4 * qk + 3 * v + 3 * state, flops=10 * kv)
        return dict(bytes=2 * qk + 2 * v + 2 * state, flops=4 * kv)
    if op.startswith("gnorm"):
        n, gated = tok * case["H"] * case["D"], case["gate"] != "none"
        if op == "gnorm":
            return dict(bytes=(3 if gated else 2) * n * e + case["D"] * 4, flops=(9 if gated else 4) * n)
        return dict(bytes=(5 if gated else 3) * n * e + 2 * case["D"] * 4, flops=(22 if gated else 10) * n)
    n, C, f = tok * case["C"], case["C"], 4 if case["res"] == FP32 else 2
    vecs = 1 + case["post"] + case["scale"]
    if op == "rnorm":
        return dict(bytes=2 * n * e + 2 * n * f + vecs * C * 4, flops=10 * n)
    return dict(bytes=3 * n * e + 3 * n * f + 2 * vecs * C * 4, flops=25 * n)


# ---- the definitions, token by token, in 64 bits --------------------------------


def _exact_attn(s, back):
    """One token of all sequences at a time; a shorter one is padded at its end with steps
    that leave its state alone."""
    c = s["case"]
    B, T, G, HV, K, V = c["B"], c["T"], c["HV"] // c["H"], c["HV"], c["K"], c["V"]
    off = _offsets(c) or [b * T for b in range(B + 1)]
    spans = [(n, off[n], off[n + 1]) for n in range(len(off) - 1)]
    L = max(b - a for _, a, b in spans)

    def side(t):
        t = t.double().flatten(0, 1)
        if t.shape[1] != HV:
            t = t.repeat_interleave(G, 1)
        out = torch.zeros(L, len(spans), *t.shape[1:], dtype=torch.float64, device="cuda")
        for n, a, b in spans:
            out[:b - a, n] = t[a:b]
        return out

    def flat(t, shape):
        out = torch.empty(B * T, *t.shape[2:], dtype=torch.float64, device="cuda")
        for n, a, b in spans:
            out[a:b] = t[:b - a, n]
        if out.shape[1] != shape[2]:
            out = out.view(B * T, shape[2], G, -1).sum(2)
        return out.view(shape)

    q, k, v = side(s["q"]), side(s["k"]), side(s["v"])
    a = torch.exp(s["log_decay"].double())
    long_ = torch.tensor([y - x for _, x, y in spans], device="cuda")
    step = lambda t: torch.where((t < long_)[:, None], a, 1.0)[..., None, None]  # noqa: E731
    d_o = side(s["d_o"]) * s["scale"] if back else None
    h, out = s["h0"].double(), []
    for t in range(L):
        h = step(t) * h + k[t][..., None] * v[t][..., None, :]
        out.append((h * d_o[t][..., None, :]).sum(-1) if back else s["scale"] * (h * q[t][..., None]).sum(-2))
    out = torch.stack(out)
    if not back:
        return flat(out, s["v"].shape), h
    dh, dk, dv = s["d_fin"].double(), torch.empty_like(k), torch.empty_like(v)
    for t in range(L - 1, -1, -1):
        dh = dh + q[t][..., None] * d_o[t][..., None, :]
        dk[t], dv[t] = (dh * v[t][..., None, :]).sum(-1), (dh * k[t][..., None]).sum(-2)
        dh = step(t) * dh
    return dict(dq=flat(out, s["q"].shape), dk=flat(dk, s["k"].shape), dv=flat(dv, s["v"].shape), dh0=dh)


def _graded(f, leaves, seeds):
    """The gradients of sum <seed, output> by automatic differentiation of the definition."""
    leaves = {n: t.double().requires_grad_() for n, t in leaves.items() if t is not None}
    total = sum((o * d.double()).sum() for o, d in zip(f(leaves), seeds))
    return dict(zip(("d" + n for n in leaves), torch.autograd.grad(total, list(leaves.values()))))


def _exact_norm(u):
    return u / ((u ** 2).sum(-1, keepdim=True) / u.shape[-1] + EPS).sqrt()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("attn", "attn_step"):
        o, fin = _exact_attn(s, False)
        return dict(o=o, final_state=fin) if op == "attn" else dict(o=o, state=fin)
    if op == "attn_bwd":
        return _exact_attn(s, True)
    if op.startswith("gnorm"):
        def f(t):
            if "z" not in t:
                return (_exact_norm(t["x"]) * t["weight"],)
            gate = t["z"] / (1 + torch.exp(-t["z"]))
            return (_exact_norm(t["x"] * gate) * t["weight"] if case["gate"] == "first" else _exact_norm(t["x"]) * t["weight"] * gate,)
        leaves = dict(x=s["x"], z=s["z"], weight=s["weight"])
        if op == "gnorm":
            return f({n: t.double() for n, t in leaves.items() if t is not None})[0]
        return _graded(f, leaves, (s["d_y"],))

    def f(t):
        p = _exact_norm(t["x"]) * t["post_weight"] if "post_weight" in t else t["x"]
        new = t["residual"] + (p * t["scale"] if "scale" in t else p)
        return _exact_norm(new) * t["weight"], new
    leaves = dict(x=s["x"], residual=s["residual"], weight=s["weight"], post_weight=s["post"], scale=s["scale"])
    if op == "rnorm":
        return dict(zip(("h", "residual"), f({n: t.double() for n, t in leaves.items() if t is not None})))
    return _graded(f, leaves, (s["d_h"], s["d_res"]))
