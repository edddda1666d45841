"""Linear attention's workspaces for packed sequences, on the CPU: states of segments are kept
for sequences of several segments only, so that short and empty sequences take none."""
import pytest

import gated_deltanet_chunkwise_amd as gdn
from test_abi_blocks import LP, size

PASSES = {"gdn_linattn_fwd_workspace_size": 1, "gdn_linattn_bwd_workspace_size": 2}  # kinds of states


@pytest.mark.parametrize("dtype", [gdn.GDN_BF16, gdn.GDN_F32])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("name", list(PASSES))
def test_short_and_empty_sequences_take_no_workspace(name, K, V, dtype):
    heads = 16

    def need(T, n):
        return size(name, LP(B=1, T=T, H=heads, HV=heads, K=K, V=V, num_seqs=n, dtype=dtype), 1)
    for T in (700, 5003, 64000):
        # a sequence of several segments takes at most twice the states that its tokens would as
        # part of one sequence, and no more than T / 64 segments are whole
        assert need(T, 1000) == need(T, 64000) == need(T, 1 << 20)
        assert need(T, 1 << 20) <= PASSES[name] * 2 * (T // 64) * heads * K * V * 4
    # 1000 sequences of 64 tokens on average: below the initial states' own size by far
    assert need(64000, 1000) <= PASSES[name] * 1000 * heads * K * V * 4 // 4
