"""What a caller learns when a wait inside the loss's or the update's kernels gives up:
the error word of its workspace, written here from the host, and results of NaN (the
launch that writes them is part of l3_check_bounded_wait)."""
import pytest
import torch

import static_token_routed_b200 as l3

pytestmark = pytest.mark.gpu


def test_status_reads_the_word_of_the_last_call():
    x = torch.randn(200, 64, device="cuda")
    ws = torch.empty(l3.l3_muon_workspace(1, 200, 64), dtype=torch.uint8, device="cuda")
    l3.l3_orthogonalize(x, workspace=ws)
    l3.l3_workspace_status(ws)
    ws[:4].view(torch.int32).fill_(4)   # as a give-up leaves it
    with pytest.raises(l3.L3Error) as e:
        l3.l3_workspace_status(ws)
    assert e.value.status == 6
    l3.l3_orthogonalize(x, workspace=ws)   # a call begins with a clear word
    l3.l3_workspace_status(ws)


def test_results_of_kernels_that_gave_up_are_nan_and_others_are_not_touched():
    assert l3.l3_check_bounded_wait() == 6, l3.l3_last_error()
    assert "results" not in l3.l3_last_error()


@pytest.mark.parametrize("empty", [
    lambda ws: l3.l3_orthogonalize(torch.empty(0, 5, device="cuda"), workspace=ws),
    lambda ws: l3.l3_muon_step(*[torch.empty(2, 0, 5, device="cuda") for _ in range(3)], 0.1, workspace=ws),
    lambda ws: l3.l3_xent_forward(torch.empty(0, 16, device="cuda"), torch.ones(9, 16, device="cuda"),
                                  torch.empty(0, dtype=torch.int32, device="cuda"), workspace=ws),
    lambda ws: l3.l3_xent_backward(torch.empty(0, 16, device="cuda"), torch.ones(9, 16, device="cuda"),
                                   torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda"),
                                   torch.empty(0, device="cuda"), workspace=ws),
])
def test_a_call_with_nothing_to_do_clears_the_word_too(empty):
    ws = torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    empty(ws)
    l3.l3_workspace_status(ws)
    empty(ws[:0])   # and writes nothing where there is no room
