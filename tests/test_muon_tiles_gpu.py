"""Every tile of the orthogonalised update's products: A = X X^T in 256- and 128-column
tiles with and without shares of its depth, B in both, X' in both, ragged in each direction,
tall and wide, in every result's form. Tolerances: test_muon_gpu.py's for X, and
test_muon_update_gpu.py's for an update of nothing."""
import pytest
import torch

import static_token_routed_b200 as l3
from test_muon_gpu import BF, FP, TOL, close, exact, make
from test_muon_update_gpu import X_OFF

pytestmark = pytest.mark.gpu

# columns of A's tiles and shares, of B's, of X''s:
SHAPES = [(2, 2048, 2048),   # 256 1, 256, 256
          (3, 747, 3003),    # 256 4, 128, 256
          (2260, 2612),      # 256 1, 256, 128
          (2612, 2260),
          (3, 2076, 1331),   # 256 1, 256, 256
          (1000, 3000),      # 128 3, 128, 256
          (8000, 300),       # 256 24, 128, 256
          (40, 200, 4224),   # 256 3, 256, 256
          (304, 704)]        # 128 6, 128, 128


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [FP, BF])
def test_orthogonalize(shape, dtype):
    G = make(*shape, dtype=dtype, strong=20.0)
    X = exact(G)
    O = l3.l3_orthogonalize(G)
    close(O, X, TOL[dtype])
    assert torch.equal(O, l3.l3_orthogonalize(G, O=G))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [FP, BF])
def test_update(shape, dtype):
    W, M, G = torch.zeros(shape, dtype=dtype, device="cuda"), make(*shape, seed=1), make(*shape, seed=2, strong=20.0)
    U = G.double() + 0.9 * (0.9 * M.double() + G.double())
    l3.l3_muon_step(W, M, G, lr=1.0, momentum=0.9, scale=1.0)
    X = exact(U)
    own = (X.to(BF).double() - X).norm() if dtype == BF else 0.0
    assert (W.double() + X).norm() <= own + 2 * X_OFF * X.norm()
