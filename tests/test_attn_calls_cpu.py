"""The attention-layer binding without a GPU: what a caller gives beside the tensors that the kernels read."""
import pytest
import torch

from gated_deltanet_cpr_gb300 import attn


def test_a_workspace_is_memory_of_the_calls_device():
    host = torch.empty(512, dtype=torch.uint8)
    assert attn._given(host, host.device) == (host.data_ptr(), 512)
    for ws, device in ((host, torch.device("cuda", 0)), (host[:1].expand(512), host.device), (host.view(2, 256).t(), host.device)):
        with pytest.raises(ValueError, match="ws is on"):
            attn._given(ws, device)


def test_a_quant_caches_tensors_cannot_be_replaced():
    """Calls go to the memory that it was made with; another tensor in a name's place would leave that to be freed."""
    c = attn.QuantCache.__new__(attn.QuantCache)
    c._tensors = tuple(torch.full((1,), i) for i in range(6))
    for i, name in enumerate(("k", "v", "k_scale", "v_scale", "k_tail", "v_tail")):
        assert getattr(c, name) is c._tensors[i]
        with pytest.raises(AttributeError):
            setattr(c, name, torch.zeros(1))
