"""fp32 rows as far apart as they may be (64 MB): a chunk's rows beyond 2^31 bytes from its first,
read by 32-bit offsets; whole chunks, and one that ends early."""
import pytest
import torch

import block_oracle as bo
import gated_deltanet_chunkwise_amd as gdn
import layer_oracle as lo

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.mark.parametrize("K,V", [(64, 64), (128, 64), (64, 128)])
def test_fp32_rows_64_mb_apart(K, V):
    far, T = (1 << 24) - 4, 191
    big = torch.empty(T * far, dtype=F32, device="cuda")
    d, s, ld = bo.linattn_inputs(1, T, 1, 2, K, V, F32, 81)
    g, s, ld = lo.cuda(d), lo.cuda(s), ld.cuda()

    def view(off, t):
        return big.as_strided(t.shape, (T * far, far, t.shape[3], 1), off).copy_(t)
    w = dict(g, q=view(0, g["q"]), k=view(1024, g["k"]), v=view(4096, g["v"]))
    assert w["q"].stride(1) == far and T * far * 4 > 1 << 33
    a, b = (gdn.linear_attn_fwd(x["q"], x["k"], x["v"], ld, initial_state=x["h0"]) for x in (w, g))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = (gdn.linear_attn_bwd(x["q"], x["k"], x["v"], ld, s["d_o"], s["d_fin"], initial_state=x["h0"]) for x in (w, g))
    assert all(torch.equal(a[n], b[n]) for n in a)
    wide = torch.empty(1, T, far + 4, dtype=F32, device="cuda")[..., :K].unflatten(-1, (1, K))
    with pytest.raises(gdn.GdnError) as e:  # one step further
        gdn.linear_attn_fwd(wide, g["k"], g["v"], ld)
    assert e.value.status == 4
    del big, w, view, wide
    torch.cuda.empty_cache()
