"""What the Python functions of the loss and the update hand to the library, with the
library's entry points replaced (no GPU needed)."""
import weakref

import pytest
import torch

import static_token_routed_b200 as l3
from static_token_routed_b200 import _binding as b
from static_token_routed_b200 import build as l3build


@pytest.fixture
def calls(monkeypatch):
    """The functions run on CPU tensors; each call into the library appends
    (arguments, whether the workspace made for it is alive)."""
    l3build.build()
    made, seen = [], []

    def empty(like, shape, dtype, stream):
        t = torch.empty(shape, dtype=dtype)
        if dtype == torch.uint8:
            made.append((weakref.ref(t), t.data_ptr()))
        return t

    def call(fn, device, *args):
        ref, at = made[-1]
        seen.append((args, at in args and ref() is not None))

    monkeypatch.setattr(b, "_cuda_device", lambda t, name: t.device)
    monkeypatch.setattr(b, "_empty", empty)
    monkeypatch.setattr(b, "_stream_of", lambda stream, device: 0)
    monkeypatch.setattr(b, "_call", call)
    return seen


X, W, T, F = torch.ones(4, 16), torch.ones(8, 16), torch.zeros(4, dtype=torch.int32), torch.ones(4)


@pytest.mark.parametrize("run", [
    lambda: l3.l3_xent_forward(X, W, T),
    lambda: l3.l3_xent_backward(X, W, T, F, F),
    lambda: l3.l3_orthogonalize(X),
    lambda: l3.l3_muon_step(X.clone(), X.clone(), X, 0.1),
])
def test_the_workspace_lives_until_its_kernels_are_enqueued(calls, run):
    run()
    assert len(calls) == 1 and calls[0][1]


def test_status_needs_room_for_the_word(monkeypatch):
    with pytest.raises(ValueError):
        l3.l3_workspace_status(torch.zeros(16, dtype=torch.uint8))
    monkeypatch.setattr(b, "_cuda_device", lambda t, name: t.device)
    with pytest.raises(ValueError):
        l3.l3_workspace_status(torch.zeros(3, dtype=torch.uint8))
