"""Linear attention of millions of sequences: calls are taken up to the launches' own limit (2^32
threads), at the threads that they have."""
import ctypes

import pytest
import torch

import gated_deltanet_chunkwise_amd as gdn
from gated_deltanet_chunkwise_amd._linattn import LinattnParams

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_three_million_sequences_of_one_token():
    """o = scale (q.k) v and its gradients: results are rounded to bf16 once."""
    n = 3_000_000
    gen = torch.Generator(device="cuda").manual_seed(51)
    q, k, v, d_o = (torch.randn(n, 1, 1, 64, generator=gen, device="cuda", dtype=BF16) for _ in range(4))
    ld = torch.tensor([-0.5], device="cuda")

    def holds(got, a, b, c):
        """scale (a.b) c, the last rows of it and some of the rest (products of 64 terms in fp32
        apart from the rounding, relative to the terms)"""
        for rows in (slice(n - 4099, n), slice(0, 4099), slice(n // 2, n // 2 + 999)):
            x, y, z = (t[rows].double() for t in (a, b, c))
            ref = 0.25 * (x * y).sum(-1, keepdim=True) * z
            terms = 0.25 * (x * y).abs().sum(-1, keepdim=True) * z.abs()
            err = (got[rows].double() - ref).abs()
            assert (err <= 2.0 ** -8 * ref.abs() + (2.0 ** -15 + 64 * 2.0 ** -24) * terms).all()
    o, fin = gdn.linear_attn_fwd(q, k, v, ld, scale=0.25, output_final_state=False)
    assert fin is None
    holds(o, q, k, v)
    del o
    lib, s = gdn.load_library(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, k, v))
    p = LinattnParams(n, 1, 1, 1, 64, 64, 0, gdn.GDN_BF16, 0.25, 0, 0, 0)
    assert lib.gdn_linattn_bwd_workspace_size(ctypes.byref(p), 0) == 0
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert lib.gdn_linattn_bwd(ctypes.byref(p), P(q), P(k), P(v), P(ld), None, None, P(d_o), None, P(dq), P(dk), P(dv), None,
                               None, 0, s) == 0
    holds(dq, d_o, v, k)
    holds(dk, v, d_o, q)
    holds(dv, k, q, d_o)
    torch.cuda.empty_cache()


def test_as_many_sequences_without_a_token():
    """Their states pass through, whatever their number."""
    n = 1 << 23
    state = torch.randn(8, 64, 64, device="cuda")
    empty = torch.empty(n, 0, 1, 64, device="cuda", dtype=BF16)
    p = LinattnParams(n, 0, 1, 1, 64, 128, 0, gdn.GDN_BF16, 1.0, 0, 0, 0)
    s, ld = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), torch.zeros(1, device="cuda")
    # without states there is nothing to pass on and nothing to do
    assert gdn.load_library().gdn_linattn_fwd(ctypes.byref(p), None, None, None, ctypes.c_void_p(ld.data_ptr()), None, None, None,
                                              None, None, 0, s) == 0
    o, fin = gdn.linear_attn_fwd(empty[:8], empty[:8], empty[:8], ld, initial_state=state.unsqueeze(1))
    assert o.shape == (8, 0, 1, 64) and torch.equal(fin[:, 0], state)
