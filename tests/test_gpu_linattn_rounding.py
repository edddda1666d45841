"""What bf16 linear attention gives is what its 64-bit form gives, rounded to bf16 once: whatever
is rounded on the way (weighted products, states where they meet rows) is rounded far below that."""
import pytest
import torch

import block_oracle as bo
import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# B, T, H, HV, K, V, lengths
CASES = [
    (2, 1, 1, 2, 64, 128, None),
    (1, 64, 1, 1, 64, 64, None),
    (2, 150, 2, 2, 128, 128, None),
    (1, 200, 1, 2, 128, 64, None),
    (1, 190, 2, 4, 64, 128, [70, 0, 120]),
    (1, 700, 1, 1, 128, 128, None),
    (1, 640, 1, 2, 64, 64, [450, 1, 189]),
]
IDS = ["%dx%d-h%d-%d-k%d-v%d%s" % (*c[:6], "" if c[6] is None else "-packed") for c in CASES]


def once_rounded(got, ref, terms, case, what):
    """`terms`: the sums of the terms' absolute values.  Operands in two bf16 parts are off by
    2^-8 2^-8 of themselves, and a term meets two of those at most (carried in a state, and the
    state's own where it meets a row); sums of K, of V, of a chunk and of T terms in fp32 by 2^-24
    an addition, the powers of the decay by as much as a handful more.  Rounding to bf16 keeps
    the order, so the result lies between the two ends, rounded."""
    _, T, _, _, K, V, _ = case
    off = (2 * 2.0 ** -16 + (K + V + 64 + T) * 2.0 ** -24) * terms
    low, high = (ref - off).to(BF16), (ref + off).to(BF16)
    got = got.cpu()
    outside = ((got < low) | (got > high)).sum()
    rounded = float((ref.to(BF16).double() - ref).norm() / ref.norm())
    print("  %-4s rel_l2=%.3e (rounding alone %.3e), outside %d of %d" %
          (what, float((got.double() - ref).norm() / ref.norm()), rounded, outside, ref.numel()), flush=True)
    assert got.isfinite().all() and outside == 0, (what, int(outside))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_results_are_rounded_once(case):
    B, T, H, HV, K, V, lengths = case
    cu = None if lengths is None else lo.offsets(lengths)
    d, seeds, ld = bo.linattn_inputs(B, T, H, HV, K, V, BF16, 31, B if cu is None else len(lengths))
    scale = K ** -0.5

    def form(**x):
        return bo.linattn(log_decay=ld.double(), cu=cu, scale=scale, **x)

    def sizes(x):
        return {k: t.abs() for k, t in x.items()}
    x, s = lo.double(d), lo.double(seeds)
    g, c, cuc = lo.cuda(d), lo.cuda(seeds), None if cu is None else cu.cuda()
    o, _ = gdn.linear_attn_fwd(g["q"], g["k"], g["v"], ld.cuda(), cuc, g["h0"], scale)
    once_rounded(o, form(**x)[0], form(**sizes(x))[0], case, "o")
    ref = lo.gradients(form, x, tuple(s.values()))
    terms = lo.gradients(form, sizes(x), tuple(sizes(s).values()))
    got = gdn.linear_attn_bwd(g["q"], g["k"], g["v"], ld.cuda(), c["d_o"], c["d_fin"], cuc, g["h0"], scale)
    for n, of in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        once_rounded(got[n], ref[of], terms[of], case, n)
