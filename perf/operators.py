"""The layer operators around the gated delta rule, as they are measured: the short
causal convolution, the selective state space scan and the 8-bit activation
checkpoints, in training, prompt and single-token form.

`own` false: the plain form, elementary torch operations in 32 bits, rounded once at
the end.  `own` true: the library's entry points.  `exact` is the definition in 64
bits, token by token.

    convolution  y[t,c] = act(bias[c] + sum_j weight[c,j] x[t-W+1+j,c]),  act(s) = s/(1+e^-s) or s
    scan         D = softplus(dt + dt_bias),  A = -exp(A_log)
                 h[t,d,n] = exp(D[t,d] A[d,n]) h[t-1,d,n] + D[t,d] Bm[t,n] x[t,d]
                 y[t,d]   = (sum_n Cm[t,n] h[t,d,n] + skip[d] x[t,d]) silu(z[t,d])
    checkpoint   blocks of 32 channels: s = the least power of two with max|x| <= 127 s
                 (at least 2^-126), code = round(x/s) to the nearest, ties to even
"""
import math

import torch

import gated_deltanet_chunkwise_amd as gdn

own = False

BF16, FP32 = "bf16", "fp32"
DT = {BF16: torch.bfloat16, FP32: torch.float32}
BLOCK = 32  # channels that share one checkpoint scale


def listed():
    return [
        # one token for each of 64 decoding sequences through the convolution of one
        # projection of 16 heads of 128: the smallest call, where latency counts
        dict(name="conv_step", op="conv_step", B=64, T=1, C=2048, W=4, dtype=BF16, silu=True),
        # the prompt of two sequences of 2048 tokens; x is a slice of a wider projection
        dict(name="conv_prompt", op="conv", B=2, T=2048, C=2048, W=4, dtype=BF16, silu=True, seqs=0, wide=True),
        # ragged packed sequences in full precision, odd sizes, no activation, from states
        dict(name="conv_packed_fp32", op="conv", B=1, T=5003, C=1000, W=3, dtype=FP32, silu=False, seqs=7, wide=False),
        # the backward pass of a training step, a wide batch
        dict(name="conv_backward", op="conv_bwd", B=4, T=8192, C=2048, W=4, dtype=BF16, silu=True, seqs=0),
        # one token for each of 64 decoding sequences
        dict(name="scan_step", op="scan_step", B=64, T=1, D=2048, N=16, G=1, dtype=BF16),
        # the prompt of two sequences of 2048 tokens; x and z are halves of one projection
        dict(name="scan_prompt", op="scan", B=2, T=2048, D=2048, N=16, G=1, dtype=BF16, gated=True, seqs=0, wide=True),
        # twelve packed prompts of 32768 tokens in all: the longest call
        dict(name="scan_packed_long", op="scan", B=1, T=32768, D=2048, N=16, G=1, dtype=BF16, gated=True, seqs=12, wide=False),
        # full precision, odd sizes, two groups of B and C, no gate
        dict(name="scan_fp32_odd", op="scan", B=3, T=777, D=1002, N=13, G=2, dtype=FP32, gated=False, seqs=0, wide=False),
        # the backward pass of a training step
        dict(name="scan_backward", op="scan_bwd", B=2, T=2048, D=2048, N=16, G=1, dtype=BF16, gated=True, seqs=0),
        # what a training step keeps of the queries, keys or values of 16 heads of 128:
        # packed in the forward pass, restored in the backward pass
        dict(name="checkpoint_bf16", op="ckpt", rows=32768, C=2048, dtype=BF16),
        # restoring a checkpoint in full precision, an odd number of channels
        dict(name="restore_fp32_odd", op="restore", rows=5003, C=1000, dtype=FP32),
        # forward and backward pass of the scan, x and z kept in 8 bits in between
        dict(name="scan_train_8bit", op="scan_train", B=2, T=1024, D=1024, N=16, G=1, dtype=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "conv_bwd", "scan_step", "scan", "scan_bwd", "ckpt", "restore", "scan_train"])
    dtype = rng.choice([BF16, BF16, FP32])
    if op == "conv_step":
        return dict(op=op, B=_log(rng, 1, 256), T=rng.choice([1, 1, 2, 4]), C=_log(rng, 64, 8192), W=rng.choice([2, 3, 4]), dtype=dtype, silu=rng.random() < 0.7)
    if op == "scan_step":
        G = rng.choice([1, 1, 2])
        return dict(op=op, B=_log(rng, 1, 256), T=rng.choice([1, 1, 2, 4]), D=G * _log(rng, 32, 2048), N=rng.choice([8, 16, 16, 13, 32]), G=G, dtype=dtype)
    if op in ("ckpt", "restore"):
        C = _log(rng, 64, 8192)
        return dict(op=op, rows=min(_log(rng, 16, 32768), (1 << 25) // C), C=C, dtype=dtype)
    if op in ("conv", "conv_bwd"):
        C, seqs = _log(rng, 64, 8192), rng.choice([0, 0, 3, 9])
        B = 1 if seqs else rng.choice([1, 2, 3, 4])
        T = max(1, min(_log(rng, 16, 32768 if seqs else 8192), (1 << 25) // (B * C)))
        c = dict(op=op, B=B, T=T, C=C, W=rng.choice([2, 3, 4]), dtype=dtype, silu=rng.random() < 0.7, seqs=seqs)
        return dict(c, wide=rng.random() < 0.5) if op == "conv" else c
    G, N, seqs = rng.choice([1, 1, 2]), rng.choice([8, 16, 16, 13, 32]), rng.choice([0, 0, 3, 9])
    D = G * _log(rng, 64, 2048)
    if op == "scan_train":
        seqs = 0
    B = 1 if seqs else rng.choice([1, 2, 3])
    T = max(1, min(_log(rng, 16, 16384 if op == "scan" else 4096), (1 << (28 if op == "scan" else 26)) // (B * D * N)))
    c = dict(op=op, B=B, T=T, D=D, N=N, G=G, dtype=dtype)
    if op != "scan_train":
        c = dict(c, gated=rng.random() < 0.7, seqs=seqs)
    return dict(c, wide=rng.random() < 0.5) if op == "scan" else c


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

    def normal(*shape, scale=1.0, shift=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)

    def uniform(*shape, lo, hi):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=case, dtype=dt)
    if op in ("ckpt", "restore"):
        rows, C = case["rows"], case["C"]
        if op == "ckpt":
            # activations: normal, with channels of very different size among them
            s["x"] = (normal(rows, C) * torch.exp2(uniform(C, lo=-4.0, hi=4.0))).to(dt)
        else:
            s["codes"] = torch.randint(-127, 128, (rows, C), generator=g, device="cuda").to(torch.int8)
            s["scales"] = torch.randint(110, 128, (rows, -(-C // BLOCK)), generator=g, device="cuda").to(torch.uint8)
        return s
    off = _offsets(case)
    s["cu"] = None if off is None else torch.tensor(off, dtype=torch.int64, device="cuda")
    B, T = case["B"], case["T"]
    S = B if off is None else len(off) - 1  # sequences
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        s["x"] = normal(B, T, 2 * C, dtype=dt)[..., C:] if case.get("wide") else normal(B, T, C, dtype=dt)
        s["weight"] = uniform(C, W, lo=-W ** -0.5, hi=W ** -0.5)
        s["bias"] = normal(C, scale=0.1)
        s["h0"] = normal(S, W - 1, C, dtype=dt)
        s["act"] = "silu" if case["silu"] else None
        if op == "conv_step":
            s["new"] = torch.empty_like(s["h0"])
        if op == "conv_bwd":
            s["d_y"] = normal(B, T, C, dtype=dt)
            s["d_fin"] = normal(S, W - 1, C, scale=0.1, dtype=dt)
        return s
    D, N, G = case["D"], case["N"], case["G"]
    if case.get("wide"):
        xz = normal(B, T, 2 * D, dtype=dt)
        s["x"], s["z"] = xz[..., :D], xz[..., D:]
    else:
        s["x"], s["z"] = normal(B, T, D, dtype=dt), normal(B, T, D, dtype=dt)
    if not case.get("gated", True):
        s["z"] = None
    s["dt"] = normal(B, T, D, scale=0.5, dtype=dt)
    # time steps between 1e-3 and 1e-1, decay rates from 1 to N as such layers start
    step = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A_log"] = torch.log(torch.arange(1, N + 1, device="cuda", dtype=torch.float32)).expand(D, N) + normal(D, N, scale=0.1)
    s["Bm"], s["Cm"] = normal(B, T, G, N, dtype=dt), normal(B, T, G, N, dtype=dt)
    s["skip"] = normal(D, scale=0.1, shift=1.0)
    s["h0"] = normal(S, D, N, scale=0.5)
    if op == "scan_step":
        s["new"] = torch.empty_like(s["h0"])
    if op in ("scan_bwd", "scan_train"):
        s["d_y"] = normal(B, T, D, dtype=dt)
        s["d_fin"] = normal(S, D, N, scale=0.1)
    return s


# ---- plain forms -------------------------------------------------------------


def _places(s):
    """Of every token (flattened): its sequence, its place in it, and the tokens of
    the sequence after it."""
    B, T = s["case"]["B"], s["case"]["T"]
    tok = torch.arange(B * T, device="cuda")
    if s["cu"] is None:
        seq = tok // T
        return seq, tok - seq * T, T - 1 - (tok - seq * T)
    seq = torch.searchsorted(s["cu"], tok, right=True) - 1
    return seq, tok - s["cu"][seq], s["cu"][seq + 1] - 1 - tok


def _ends(s):
    """Each sequence's end in the flattened tokens, and its length."""
    B, T = s["case"]["B"], s["case"]["T"]
    if s["cu"] is None:
        n = torch.arange(B, device="cuda")
        return (n + 1) * T, torch.full_like(n, T)
    return s["cu"][1:], s["cu"][1:] - s["cu"][:-1]


def _conv_windows(s):
    """[tokens, W, C]: the W inputs that each output reads, oldest first."""
    W, C = s["case"]["W"], s["case"]["C"]
    x, h0 = s["x"].float().reshape(-1, C), s["h0"].float()
    seq, pos, _ = _places(s)
    back = torch.arange(W - 1, -1, -1, device="cuda")
    at = pos[:, None] - back                                       # place in the sequence
    tok = torch.arange(pos.numel(), device="cuda")[:, None] - back
    inside = x[tok.clamp(min=0)]
    before = h0[seq[:, None], (W - 1 + at).clamp(0, W - 2)]
    return torch.where((at >= 0)[..., None], inside, before)


def _conv_final(s):
    W, C = s["case"]["W"], s["case"]["C"]
    x, h0 = s["x"].reshape(-1, C), s["h0"]
    end, length = _ends(s)
    r = torch.arange(W - 1, device="cuda")
    at = length[:, None] - (W - 1) + r
    tok = (end[:, None] - (W - 1) + r).clamp(min=0, max=x.shape[0] - 1)
    n = torch.arange(end.numel(), device="cuda")[:, None]
    return torch.where((at >= 0)[..., None], x[tok], h0[n, (W - 1 + at).clamp(0, W - 2)])


def _conv(s):
    pre = s["bias"] + (_conv_windows(s) * s["weight"].t()).sum(1)
    y = pre * torch.sigmoid(pre) if s["act"] else pre
    return y.view(s["x"].shape).to(s["dtype"]), _conv_final(s)


def _conv_bwd(s):
    W, C = s["case"]["W"], s["case"]["C"]
    win = _conv_windows(s)
    dpre = s["d_y"].float().reshape(-1, C)
    if s["act"]:
        pre = s["bias"] + (win * s["weight"].t()).sum(1)
        g = torch.sigmoid(pre)
        dpre = dpre * (g + pre * g * (1 - g))
    seq, pos, left = _places(s)
    ahead = torch.arange(W, device="cuda")
    tok = torch.arange(pos.numel(), device="cuda")
    later = dpre[(tok[:, None] + ahead).clamp(max=pos.numel() - 1)]
    later = torch.where((ahead <= left[:, None])[..., None], later, 0.0)
    dx = (later * s["weight"].t().flip(0)).sum(1)
    # the final state holds each sequence's last W-1 inputs, or rows of its initial state
    d_fin = s["d_fin"].float()
    row = W - 2 - left
    dx = dx + torch.where((row >= 0)[:, None], d_fin[seq, row.clamp(min=0)], 0.0)
    # initial-state row r stands at place r - (W-1); the output at place p reads it with
    # weight r - p, for p <= r
    end, length = _ends(s)
    r, p = torch.arange(W - 1, device="cuda")[:, None], torch.arange(W - 1, device="cuda")[None, :]
    use = (p <= r) & (p < length[:, None, None])                   # [S, r, p]
    first = dpre[((end - length)[:, None] + p).clamp(max=pos.numel() - 1)]  # [S, p, C]
    wt = s["weight"].t()[(r - p).clamp(min=0)]                     # [r, p, C]
    dh0 = (torch.where(use[..., None], first[:, None] * wt, 0.0)).sum(2)
    kept = r[:, 0] - length[:, None]                               # final row that holds row r
    n = torch.arange(end.numel(), device="cuda")[:, None]
    dh0 = dh0 + torch.where((kept >= 0)[..., None], d_fin[n, kept.clamp(min=0)], 0.0)
    return dict(dx=dx.view(s["x"].shape).to(s["dtype"]), dweight=(dpre[:, None] * win).sum(0).t().contiguous(),
                dbias=dpre.sum(0), dh0=dh0.to(s["dtype"]))


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _prefix(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 0, h_{-1} = 0, by doubling."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _scan_terms(s, x=None, z=None):
    """The flattened inputs in 32 bits, the decays [tokens, D, N] and the states."""
    c = s["case"]
    D, N, G = c["D"], c["N"], c["G"]
    x = (s["x"] if x is None else x).float().reshape(-1, D)
    z = s["z"] if z is None else z
    z = None if z is None else z.float().reshape(-1, D)
    raw = s["dt"].float().reshape(-1, D) + s["dt_bias"]
    delta = _softplus(raw)
    A = -torch.exp(s["A_log"])
    a = torch.exp(delta[..., None] * A)
    Bf = s["Bm"].float().reshape(-1, G, 1, N).expand(-1, G, D // G, N).reshape(-1, D, N)
    Cf = s["Cm"].float().reshape(-1, G, 1, N).expand(-1, G, D // G, N).reshape(-1, D, N)
    seq, pos, left = _places(s)
    head = pos == 0
    start = s["h0"][seq[head]] * a[head]
    b = (delta * x)[..., None] * Bf
    b[head] += start
    keep = torch.where(head[:, None, None], 0.0, a)  # nothing passes from sequence to sequence
    return x, z, raw, delta, A, a, Bf, Cf, seq, head, left, _prefix(keep, b)


def _last(s, h):
    end, length = _ends(s)
    return torch.where((length > 0)[:, None, None], h[(end - 1).clamp(min=0)], s["h0"])


def _scan(s):
    x, z, _, _, _, _, _, Cf, _, _, _, h = _scan_terms(s)
    y = (h * Cf).sum(-1) + s["skip"] * x
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return y.view(s["x"].shape).to(s["dtype"]), _last(s, h)


def _scan_bwd(s, x=None, z=None):
    D, N, G = s["case"]["D"], s["case"]["N"], s["case"]["G"]
    x, z, raw, delta, A, a, Bf, Cf, seq, head, left, h = _scan_terms(s, x, z)
    dy = s["d_y"].float().reshape(-1, D)
    dz = None
    if z is not None:
        g = torch.sigmoid(z)
        dz = dy * ((h * Cf).sum(-1) + s["skip"] * x) * (g + z * g * (1 - g))
        dy = dy * z * g
    # the states' gradient, backwards: l_t = a_{t+1} l_{t+1} + C_t dy_t, from d_final
    tail = left == 0
    src = dy[..., None] * Cf
    src[tail] += s["d_fin"][seq[tail]]
    nxt = torch.cat([a[1:], torch.zeros_like(a[:1])])
    nxt = torch.where(tail[:, None, None], 0.0, nxt)
    lam = _prefix(nxt.flip(0), src.flip(0)).flip(0)
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    prev[head] = s["h0"][seq[head]]
    da = lam * a * prev                                            # towards delta A
    u = (lam * Bf).sum(-1)
    ddelta = (da * A).sum(-1) + u * x
    draw_ = ddelta * torch.where(raw > 20, 1.0, torch.sigmoid(raw))
    dh0 = s["d_fin"].clone()
    dh0[seq[head]] = (lam * a)[head]
    shape, gn = s["x"].shape, s["Bm"].shape
    out = dict(dx=(u * delta + s["skip"] * dy).view(shape), ddt=draw_.view(shape),
               dBm=(lam * (delta * x)[..., None]).view(-1, G, D // G, N).sum(2).view(gn),
               dCm=(h * dy[..., None]).view(-1, G, D // G, N).sum(2).view(gn))
    if dz is not None:
        out["dz"] = dz.view(shape)
    out = {k: v.to(s["dtype"]) for k, v in out.items()}
    return dict(out, dA_log=(da * delta[..., None]).sum(0) * A, dskip=(dy * x).sum(0), ddt_bias=draw_.sum(0), dh0=dh0)


def _pack(x):
    """Codes and the biased exponents of the blocks' scales."""
    C = x.shape[-1]
    v = x.float().reshape(-1, C)
    v = torch.nn.functional.pad(v, (0, -C % BLOCK)).view(v.shape[0], -1, BLOCK)
    m, e = torch.frexp(v.abs().amax(-1))                           # max = m 2^e, m in [1/2, 1)
    e = torch.where(m == 0, -126, torch.where(m > 127 / 128, e - 6, e - 7)).clamp(min=-126)
    codes = torch.round(torch.ldexp(torch.ldexp(v, (-e // 2)[..., None]), (-e - (-e // 2))[..., None]))
    return codes.view(v.shape[0], -1)[:, :C].to(torch.int8), (e + 127).to(torch.uint8)


def _unpack(codes, scales, dtype):
    C = codes.shape[-1]
    return (codes.float() * torch.exp2(scales.float() - 127).repeat_interleave(BLOCK, -1)[:, :C]).to(dtype)


def _through(x):
    """x as a checkpoint gives it back."""
    return _unpack(*_pack(x), x.dtype).view(x.shape)


def run(s):
    op = s["case"]["op"]
    if op == "ckpt":
        if own:
            return gdn.unpack8(gdn.pack8(s["x"]))
        return _through(s["x"])
    if op == "restore":
        if own:
            return gdn.unpack8(gdn.Packed8(s["codes"], s["scales"], s["dtype"]))
        return _unpack(s["codes"], s["scales"], s["dtype"])
    if op == "conv":
        if own:
            y, fin = gdn.conv_fwd(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu"], initial_state=s["h0"], activation=s["act"])
        else:
            y, fin = _conv(s)
        return dict(y=y, final_state=fin)
    if op == "conv_step":
        if own:
            y = gdn.conv_decode(s["x"], s["weight"], s["h0"], s["bias"], activation=s["act"], new_state=s["new"])
            return dict(y=y, state=s["new"])
        y, fin = _conv(s)
        return dict(y=y, state=fin)
    if op == "conv_bwd":
        if own:
            return gdn.conv_bwd(s["x"], s["weight"], s["bias"], s["d_y"], s["d_fin"], cu_seqlens=s["cu"], initial_state=s["h0"], activation=s["act"])
        return _conv_bwd(s)
    if op == "scan":
        if own:
            y, fin = gdn.scan_fwd(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"], cu_seqlens=s["cu"], initial_state=s["h0"])
        else:
            y, fin = _scan(s)
        return dict(y=y, final_state=fin)
    if op == "scan_step":
        if own:
            y = gdn.scan_decode(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["h0"], skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"], new_state=s["new"])
            return dict(y=y, state=s["new"])
        y, fin = _scan(s)
        return dict(y=y, state=fin)
    if op == "scan_bwd":
        if own:
            return gdn.scan_bwd(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["d_y"], s["d_fin"], skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"], cu_seqlens=s["cu"], initial_state=s["h0"])
        return _scan_bwd(s)
    # scan_train: one training step of the scan, x and z held in 8 bits for its backward pass
    if own:
        names = ("x", "dt", "A_log", "Bm", "Cm", "skip", "z", "dt_bias", "h0")
        leaf = {k: s[k].detach().requires_grad_() for k in names}
        y, fin = gdn.selective_scan(leaf["x"], leaf["dt"], leaf["A_log"], leaf["Bm"], leaf["Cm"], skip=leaf["skip"], z=leaf["z"], dt_bias=leaf["dt_bias"],
                                    initial_state=leaf["h0"], checkpoint_bits=8)
        grads = torch.autograd.grad((y, fin), [leaf[k] for k in names], (s["d_y"], s["d_fin"]))
        return dict({"d" + k: v for k, v in zip(names, grads)}, y=y.detach(), final_state=fin.detach())
    y, fin = _scan(s)
    return dict(_scan_bwd(s, _through(s["x"]), _through(s["z"])), y=y, final_state=fin)


def work(case):
    op, e = case["op"], 2 if case["dtype"] == BF16 else 4
    if op in ("ckpt", "restore"):
        n = case["rows"] * case["C"]
        packed = n + case["rows"] * -(-case["C"] // BLOCK)
        # a checkpoint is held between the passes: it is written and read as well
        return dict(bytes=packed + n * e if op == "restore" else 2 * packed + 2 * n * e, flops=2 * n)
    tok = case["B"] * case["T"]
    S = case.get("seqs", 0) or case["B"]
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        state, par = 2 * S * (W - 1) * C * e, C * (W + 1) * 4
        if op == "conv_bwd":
            return dict(bytes=3 * tok * C * e + 2 * par + state + state // 2, flops=tok * C * (6 * W + 10))
        return dict(bytes=2 * tok * C * e + par + state, flops=tok * C * (2 * W + 5))
    D, N, G = case["D"], case["N"], case["G"]
    wide = 4 if case.get("gated", True) else 3                     # x, dt, y and z
    par, state, bc = D * (N + 2) * 4, S * D * N * 4, 2 * tok * G * N * e
    fwd = dict(bytes=wide * tok * D * e + bc + par + 2 * state, flops=tok * D * (7 * N + 12))
    # x, dt, dy and z in, dx, ddt and dz out; the states once more and their gradients back
    bwd = dict(bytes=(2 * wide - 1) * tok * D * e + 2 * bc + 2 * par + 3 * state, flops=tok * D * (22 * N + 40))
    if op == "scan_bwd":
        return bwd
    if op == "scan_train":
        packed = 2 * tok * (D + -(-D // BLOCK))
        return dict(bytes=fwd["bytes"] + bwd["bytes"] + 2 * packed - 2 * tok * D * e, flops=fwd["flops"] + bwd["flops"])
    return fwd


# ---- the definitions, token by token, in 64 bits --------------------------------


def _spans(s):
    """(sequence, rows of the flattened tokens) of every sequence."""
    off = _offsets(s["case"])
    if off is None:
        off = [b * s["case"]["T"] for b in range(s["case"]["B"] + 1)]
    return [(n, slice(off[n], off[n + 1])) for n in range(len(off) - 1)]


def _exact_conv(s, back):
    W, C = s["case"]["W"], s["case"]["C"]
    x, w, bias = s["x"].double().reshape(-1, C), s["weight"].double(), s["bias"].double()
    y, dx, dh0, fin = torch.empty_like(x), torch.empty_like(x), [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for n, rows in _spans(s):
        line = torch.cat([s["h0"][n].double(), x[rows]])
        L = line.shape[0] - (W - 1)
        pre = bias + sum(line[j:j + L] * w[:, j] for j in range(W))
        y[rows] = pre / (1 + torch.exp(-pre)) if s["act"] else pre
        fin.append(line[L:])
        if back:
            d = s["d_y"].reshape(-1, C)[rows].double()
            if s["act"]:
                e = torch.exp(-pre)
                d = d * (1 + e + pre * e) / (1 + e) ** 2
            dline = torch.zeros_like(line)
            dline[L:] += s["d_fin"][n].double()
            for j in range(W):
                dline[j:j + L] += d * w[:, j]
                dw[:, j] += (d * line[j:j + L]).sum(0)
            db += d.sum(0)
            dx[rows] = dline[W - 1:]
            dh0.append(dline[:W - 1])
    shape = s["x"].shape
    if back:
        return dict(dx=dx.view(shape), dweight=dw, dbias=db, dh0=torch.stack(dh0))
    return y.view(shape), torch.stack(fin)


def _exact_scan(s, back, x8=None, z8=None):
    """Token by token, all sequences side by side, shorter ones padded with steps of
    length 0 (which leave a state as it was)."""
    c = s["case"]
    D, N, G = c["D"], c["N"], c["G"]
    spans = _spans(s)
    L = max(r.stop - r.start for _, r in spans)

    def side(t):
        t = t.double().reshape(c["B"] * c["T"], -1)
        out = torch.zeros(L, len(spans), t.shape[1], dtype=torch.float64, device="cuda")
        for n, r in spans:
            out[:r.stop - r.start, n] = t[r]
        return out

    def flat(t, shape):
        out = torch.empty(c["B"] * c["T"], t.shape[-1], dtype=torch.float64, device="cuda")
        for n, r in spans:
            out[r] = t[:r.stop - r.start, n]
        return out.view(shape)

    live = side(torch.ones(c["B"] * c["T"], 1, device="cuda"))
    raw = side(s["dt"]) + s["dt_bias"].double()
    delta = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20)))) * live
    A = -torch.exp(s["A_log"].double())
    x, Bm, Cm = side(s["x"] if x8 is None else x8), side(s["Bm"]).view(L, -1, G, N), side(s["Cm"]).view(L, -1, G, N)
    z = None if s["z"] is None else side(s["z"] if z8 is None else z8)
    skip = s["skip"].double()
    h, hs, ys = s["h0"].double(), [], []
    for t in range(L):
        if back:
            hs.append(h)
        wide = Bm[t].repeat_interleave(D // G, 1)
        h = torch.exp(delta[t][..., None] * A) * h + (delta[t] * x[t])[..., None] * wide
        ys.append((h * Cm[t].repeat_interleave(D // G, 1)).sum(-1) + skip * x[t])
    inner = torch.stack(ys)
    if not back:
        y = inner if z is None else inner * z / (1 + torch.exp(-z))
        return flat(y, s["x"].shape), h
    dy, dz = side(s["d_y"]), None
    if z is not None:
        e = torch.exp(-z)
        dz = dy * inner * (1 + e + z * e) / (1 + e) ** 2
        dy = dy * z / (1 + e)
    lam = s["d_fin"].double()
    dA, dx, dd = torch.zeros_like(A), torch.empty_like(x), torch.empty_like(x)
    dB, dC = torch.empty_like(Bm), torch.empty_like(Cm)
    for t in range(L - 1, -1, -1):
        a = torch.exp(delta[t][..., None] * A)
        wide = Bm[t].repeat_interleave(D // G, 1)
        ht = a * hs[t] + (delta[t] * x[t])[..., None] * wide
        lam = lam + (dy[t] * live[t])[..., None] * Cm[t].repeat_interleave(D // G, 1)
        dC[t] = (ht * dy[t][..., None]).view(-1, G, D // G, N).sum(2)
        dB[t] = (lam * (delta[t] * x[t])[..., None]).view(-1, G, D // G, N).sum(2)
        through = lam * a * hs[t]
        u = (lam * wide).sum(-1)
        dd[t] = (through * A).sum(-1) + u * x[t]
        dx[t] = u * delta[t] + skip * dy[t]
        dA += (through * delta[t][..., None]).sum(0)
        lam = lam * a
    dd = dd * torch.where(raw > 20, 1.0, 1 / (1 + torch.exp(-raw))) * live
    shape, gn = s["x"].shape, s["Bm"].shape
    out = dict(dx=flat(dx, shape), ddt=flat(dd, shape), dBm=flat(dB.view(L, -1, G * N), gn), dCm=flat(dC.view(L, -1, G * N), gn),
               dA_log=dA * A, dskip=(dy * x * live).sum((0, 1)), ddt_bias=dd.sum((0, 1)), dh0=lam)
    if dz is not None:
        out["dz"] = flat(dz, shape)
    return out


def _exact_through(x):
    """Every block on its own: the scale by trying exponents, the codes from the quotient."""
    C = x.shape[-1]
    out = x.double().reshape(-1, C).clone()
    for c0 in range(0, C, BLOCK):
        v = out[:, c0:c0 + BLOCK]
        e = torch.full((v.shape[0], 1), -126.0, dtype=torch.float64, device="cuda")
        for k in range(-60, 60):
            e = torch.where(v.abs().amax(1, keepdim=True) > 127 * 2.0 ** (k - 1), torch.full_like(e, float(k)), e)
        out[:, c0:c0 + BLOCK] = torch.round(v / torch.exp2(e)) * torch.exp2(e)
    return out.view(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ckpt":
        return _exact_through(s["x"])
    if op == "restore":
        return s["codes"].double() * torch.exp2(s["scales"].double() - 127).repeat_interleave(BLOCK, -1)[:, :case["C"]]
    if op in ("conv", "conv_step"):
        y, fin = _exact_conv(s, False)
        return dict(y=y, final_state=fin) if op == "conv" else dict(y=y, state=fin)
    if op == "conv_bwd":
        return _exact_conv(s, True)
    if op in ("scan", "scan_step"):
        y, fin = _exact_scan(s, False)
        return dict(y=y, final_state=fin) if op == "scan" else dict(y=y, state=fin)
    if op == "scan_bwd":
        return _exact_scan(s, True)
    y, fin = _exact_scan(s, False)
    return dict(_exact_scan(s, True, _exact_through(s["x"]), _exact_through(s["z"])), y=y, final_state=fin)
