"""Streams given as handles: what a call makes for itself comes from the memory of
the stream that it runs on, since memory of another one may be handed out while the call's
kernels still use it."""
import pytest
import torch

import static_token_routed_b200 as l3

pytestmark = pytest.mark.gpu


def owner(t):
    """The stream whose memory a tensor is."""
    at = [s["stream"] for s in torch.cuda.memory_snapshot()
          if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
    assert len(at) == 1
    return at[0]


@pytest.mark.parametrize("which", ["0", "1", "default", "other", "other's handle", "none"])
def test_memory_is_the_streams_own(which):
    current, other = torch.cuda.Stream(), torch.cuda.Stream()
    stream = {"0": 0, "1": 1, "default": torch.cuda.default_stream(), "other": other,
              "other's handle": other.cuda_stream, "none": None}[which]
    want = {"other": other.cuda_stream, "other's handle": other.cuda_stream, "none": current.cuda_stream}.get(which, 0)
    x, W = torch.randn(300, 64, device="cuda"), torch.randn(500, 64, device="cuda")
    t, G = torch.zeros(300, dtype=torch.int32, device="cuda"), torch.randn(200, 300, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(current):
        loss, lse = l3.l3_xent_forward(x, W, t, stream=stream)
        dx, dW = l3.l3_xent_backward(x, W, t, lse, loss, stream=stream)
        O = l3.l3_orthogonalize(G, stream=stream)
        l3.l3_muon_step(G.clone(), torch.zeros_like(G), G, 0.1, stream=current)
    torch.cuda.synchronize()
    for v in (loss, lse, dx, dW, O):
        assert owner(v) == want and torch.isfinite(v).all()
