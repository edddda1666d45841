"""A decay that is a parameter of the model: refused where a gradient would be recorded, taken
where none is (as serving runs a model)."""
import pytest
import torch

import gated_deltanet_chunkwise_amd as gdn
from gated_deltanet_chunkwise_amd import _binding
from test_blocks_host import _NoCalls, attn_case


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_without_gradients_a_parameter_is_taken(mode, monkeypatch):
    monkeypatch.setattr(_binding, "_LIB", _NoCalls())
    d = attn_case()
    a = (d["q"], d["k"], d["v"], torch.nn.Parameter(d["ld"]))
    with mode(), pytest.raises(ValueError, match="GPU tensor"):  # the next check: tensors of the CPU
        gdn.linear_attention(*a)
    with pytest.raises(ValueError, match="log_decay"):
        gdn.linear_attention(*a)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_results_with_a_parameter(mode):
    gen = torch.Generator().manual_seed(61)
    q, k, v = (torch.randn(2, 70, 2, 64, generator=gen).to("cuda", torch.bfloat16) for _ in range(3))
    decay = torch.nn.Parameter(torch.tensor([-0.1, -1.0], device="cuda"))
    with mode():
        o, fin = gdn.linear_attention(q, k, v, decay)
    want, want_fin = gdn.linear_attention(q, k, v, decay.detach())
    assert torch.equal(o, want) and torch.equal(fin, want_fin) and not o.requires_grad
