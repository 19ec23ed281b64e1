"""The workspace functions of the loss and the update (no GPU needed): a size for what
the calls take, -1 for what they reject."""
import ctypes

import pytest
import torch

import static_token_routed_b200 as l3
from static_token_routed_b200 import build as l3build

P, BIG = ctypes.c_void_p(1 << 20), 1 << 60


@pytest.fixture(scope="module")
def lib():
    l3build.build()
    return l3.library()


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("n,vocab,d,dtype", [
    (-1, 100, 64, 0), (8, 0, 64, 0), (8, 100, 0, 0), (8, 100, 24, 0), (8, 100, 62, 1), (8, 100, 64, 2),
    (8, 100, 16400, 0), ((1 << 20) + 1, 100, 64, 0), (8, (1 << 24) + 1, 64, 0), (1 << 62, 100, 64, 0),
    (8, (1 << 63) - 1, 64, 1), (8, 100, (1 << 63) - 16, 0),
])
def test_xent_workspace_of_rejected_sizes(lib, n, vocab, d, dtype, backward):
    assert lib.l3_xent_workspace(n, vocab, d, dtype, backward) == -1 and l3.l3_last_error()
    call = (lambda: lib.l3_xent_backward(P, P, P, P, P, n, vocab, d, dtype, P, P, P, BIG, None)) if backward \
        else (lambda: lib.l3_xent_forward(P, P, P, n, vocab, d, dtype, P, P, P, BIG, None))
    assert call() in (1, 4)


@pytest.mark.parametrize("batch,rows,cols", [
    (-1, 8, 8), (1, -1, 8), (1, 8, -1), (1, 65537, 8), (1, 8, 65537), (4097, 8, 8), (4096, 32769, 65536),
    (1, 1 << 40, 1 << 40), (1 << 62, 8, 8), (1, 8, (1 << 63) - 1),
])
def test_muon_workspace_of_rejected_sizes(lib, batch, rows, cols):
    assert lib.l3_muon_workspace(batch, rows, cols) == -1 and l3.l3_last_error()
    assert lib.l3_orthogonalize(P, batch, rows, cols, 1, 5, 1e-7, P, P, BIG, None) in (1, 4)
    assert lib.l3_muon_step(P, P, P, batch, rows, cols, 1, 0.1, 0.9, 1, 0.0, 1.0, 5, 1e-7, P, BIG, None) in (1, 4)


@pytest.mark.parametrize("n,vocab,d,dtype", [(1 << 20, 1, 16, 0), (1, 1 << 24, 4, 1), (1, 1, 16384, 0),
                                             (1 << 20, 1 << 24, 16384, 1), (0, 5, 16, 0)])
def test_xent_workspace_at_the_limits(lib, n, vocab, d, dtype):
    for backward in (0, 1):
        assert lib.l3_xent_workspace(n, vocab, d, dtype, backward) > 0


@pytest.mark.parametrize("batch,rows,cols", [(4096, 1, 1), (1, 65536, 65536), (4096, 32768, 32768), (2048, 65536, 65536)])
def test_muon_workspace_at_the_limits(lib, batch, rows, cols):
    assert lib.l3_muon_workspace(batch, rows, cols) > 0


def test_python_names_the_refusal():
    with pytest.raises(l3.L3Error):
        l3.l3_xent_workspace(8, 100, 24)
    with pytest.raises(l3.L3Error):
        l3.l3_muon_workspace(1, 65537, 8)
    with pytest.raises(TypeError):
        l3.l3_xent_workspace(8, 100, 64, torch.float16)


@pytest.mark.parametrize("batch,rows,cols,most", [
    (1024, 32, 512, 4096), (4096, 128, 2048, 4096), (4096, 2048, 1, 4096),   # one launch: the error word alone
    (4096, 1, 65536, 3 << 29), (600, 33, 4200, 3 << 29), (4096, 512, 2048, 3 << 29),
    (1, 2048, 4096, 120 << 20),
])
def test_muon_workspace_is_bounded_in_the_batch(lib, batch, rows, cols, most):
    assert 0 < lib.l3_muon_workspace(batch, rows, cols) <= most
    assert 0 < lib.l3_muon_workspace(batch, cols, rows) <= most
