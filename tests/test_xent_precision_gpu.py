"""Inputs on which the cross entropy's arithmetic shows: what a chain, a part or a
rounding loses is not hidden under bounds for any input."""
import pytest
import torch

import static_token_routed_b200 as l3

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("n", [3, 20, 100, 200, 500])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_sure_tokens_gradient_is_nothing(n, dtype):
    """Targets 50 to 100 above every other logit, all terms of one sign, so that a chain
    drops bits in each of its 16-deep steps. lse is then s_t to the last bit (the others'
    sum is below 300 e^-50), and p_t - 1 what the two passes' s_t differ by: nothing where
    they add the same operands up in the same order. Up to 128 tokens one of them has W's
    rows as M and the other the tokens. If that changes what a chain drops: a chain of
    128 (n <= 32) or 256 terms holds s / 32 or s / 16 with s < 128, a step drops up to 2^-23 of
    it, in 8 or 16 steps of 32 or 16 chains, 2.4e-4 at worst; adding up to 32 chains rounds
    by 2^-24 of s each, 2.4e-4; together 5e-4. One chain of all 4096 terms may drop 256
    times 2^-23 of s, 4e-3, and 1.5e-3 was seen."""
    d, vocab = 4096, 300
    g = torch.Generator().manual_seed(n)
    t = torch.randint(0, vocab, (n,), generator=g)
    W = (torch.randn(vocab, d, generator=g) / 64).to(dtype)
    x = (W.float()[t] * (60 + 40 * torch.rand(n, 1, generator=g)) / W.float()[t].square().sum(1, keepdim=True)).to(dtype)
    x, W, t = x.cuda(), W.cuda(), t.to(torch.int32).cuda()
    s = x.double() @ W.double().T
    at = t.long()[:, None]
    rest = s.scatter(1, at, float("-inf")).amax(1)
    assert (s.gather(1, at)[:, 0] - rest).min() > 50 and s.max() < 128
    loss, lse = l3.l3_xent_forward(x, W, t)
    dx, dW = l3.l3_xent_backward(x, W, t, lse, torch.ones(n, device="cuda"))
    # dx = G_t W_t, and less than 300 e^-50 of other rows of W
    G = (dx.double() * W.double()[t.long()]).sum(1) / W.double()[t.long()].square().sum(1)
    assert G.abs().max() <= (5e-4 if n <= 128 else 2.0 ** -24)
