"""What l3_muon_step adds to a weight, by itself: with W = 0, no decay, no momentum and
lr = scale = 1, W becomes -X, and no larger W hides how far X is off.

Tolerance, as |error|_F: X as in test_muon_gpu.py, 1.2e-4 |X|. A bf16 W is the
nearest value to what the kernel has, a, and that is no farther from a than the one
nearest to the exact x, so that |bf16(a) - x| <= |bf16(x) - x| + 2 |a - x|."""
import pytest
import torch

import static_token_routed_b200 as l3
from test_muon_gpu import BF, FP, exact, make

pytestmark = pytest.mark.gpu
X_OFF = 1.2e-4

# up to 32 rows, up to 128 x 4096, and tiles: aligned rows or not, A X X^T in shares
# (300 x 704, 512 x 2048) or not, stacks
SHAPES = [(16, 700), (900, 9), (64, 64), (128, 256), (131, 77), (100, 4000), (2, 90, 600),
          (200, 304), (150, 301), (300, 704), (704, 300), (512, 2048), (2, 260, 520), (1100, 1100)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("kind", ["noise", "strong", "equal"])
def test_update_of_a_zero_weight(shape, dtype, kind):
    if kind == "equal":  # orthonormal rows or columns: the roundings of A add up
        G = make(*shape).double()
        Q = torch.linalg.qr(G if shape[-2] >= shape[-1] else G.mT)[0]
        G = (Q if shape[-2] >= shape[-1] else Q.mT).float().contiguous()
    else:
        G = make(*shape, strong=20.0 if kind == "strong" else 0.0)
    W = torch.zeros(shape, dtype=dtype, device="cuda")
    M = torch.zeros(shape, device="cuda")
    l3.l3_muon_step(W, M, G, lr=1.0, momentum=0.0, nesterov=False, scale=1.0)
    X = exact(G)
    assert torch.equal(M, G) and torch.isfinite(W).all()
    if dtype == FP:
        assert (W.double() + X).norm() <= X_OFF * X.norm()
    else:
        own = (X.to(BF).double() - X).norm()
        assert (W.double() + X).norm() <= own + 2 * X_OFF * X.norm()


@pytest.mark.parametrize("shape", [(520, 33, 4200), (530, 4100, 5)])
@pytest.mark.parametrize("dtype", [FP, BF])
def test_stacks_larger_than_their_workspace(shape, dtype):
    """Stacks that go through the workspace in slices (5 rows and 9 steps take that way
    too): every matrix, the last slice's among them, its own results, and nothing
    outside of the workspace."""
    steps = 9 if min(shape) == 5 else 5
    size = l3.l3_muon_workspace(*shape)
    per_matrix = 8 * 64 * 4160   # X twice, in two fp16 parts, at the least
    assert size < shape[0] * per_matrix
    ws = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    G = torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    O = l3.l3_orthogonalize(G.to(dtype), steps=steps, workspace=ws[:size])
    l3.l3_workspace_status(ws)
    assert (ws[size:] == 0xFF).all()
    W, M = torch.zeros(shape, dtype=dtype, device="cuda"), torch.zeros(shape, device="cuda")
    l3.l3_muon_step(W, M, G, lr=1.0, momentum=0.0, nesterov=False, scale=1.0, steps=steps, workspace=ws[:size])
    assert (ws[size:] == 0xFF).all() and torch.equal(M, G)
    for i in list(range(0, shape[0], 37)) + [shape[0] - 1]:
        for got, of in ((O[i], G[i].to(dtype)), (-W[i], G[i])):
            X = exact(of, steps)
            own = (X.to(BF).double() - X).norm() if dtype == BF else 0.0
            assert (got.double() - X).norm() <= own + 2 * X_OFF * X.norm()
