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


@pytest.mark.parametrize("n,vocab,d,out", [(129, 20000, 512, 0.0), (300, 20000, 512, 0.2), (700, 30011, 272, 0.0),
                                           (2000, 70000, 272, 0.3)])
def test_the_targets_element_of_g_is_not_rounded_away_in_dw(n, vocab, d, out):
    """Most rows of dW have one token whose target they are, and every other element of
    their G is small: dW is off by its own rounding, not by that of the target's element.
    By norms: half a step of the other elements times |x|_2; 2^-16 of the targets' (two
    parts); the logits' errors (chains of 512: 32 steps, each 2^-23 of a sum of magnitudes)
    and 2^-17 for exponentials; the sums of n terms."""
    g = torch.Generator().manual_seed(n)
    W = (0.1 * torch.randn(vocab, d, generator=g) / d ** 0.5).to(BF).cuda()
    x = torch.randn(n, d, generator=g).to(BF).cuda()
    t = torch.randint(0, vocab, (n,), generator=g).to(torch.int32)
    t[torch.rand(n, generator=g) < out] = -1
    t, w = t.cuda(), ((0.5 + torch.rand(n, generator=g)) / n).cuda()
    _, lse = l3.l3_xent_forward(x, W, t)
    _, dW = l3.l3_xent_backward(x, W, t, lse, w)
    i = (t >= 0).nonzero()[:, 0]
    X, wd, at = x[i].double(), w[i].double()[:, None], t[i].long()[:, None]
    s = X @ W.double().T
    P = (s - torch.logsumexp(s, 1, keepdim=True)).exp() * wd
    ds = 36 * 2.0 ** -23 * (X.abs() @ W.double().abs().T).amax(1) * 2 + 2.0 ** -17 * (1 + s.abs().amax(1))
    spectral = torch.linalg.matrix_norm(X, 2)
    others = (P * (2.0 ** -8 + ds[:, None])).norm() * spectral
    target = (2.0 ** -16 + ds.max()) * wd.norm() * spectral
    del s
    G = P.scatter_add(1, at, -wd)
    ref = G.T @ X
    sums = (n + 64) * 2.0 ** -23 * (G.abs().T @ X.abs()).norm()
    own = (ref.to(BF).double() - ref).norm()
    assert others + target + sums < 0.3 * own   # what a rounded target's element, 1.3 own, would hide under
    assert (dW.double() - ref).norm() <= own + others + target + sums


@pytest.mark.parametrize("n", [2, 32, 60, 128, 200, 600])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("target", [0, 31, 32, 700])
def test_one_target_for_all_tokens(n, dtype, target):
    """d = 16 terms, exact for bf16 values and added in one step (2^-23 of a sum of
    magnitudes below 48); exponentials, their sums and the logarithm 2^-18."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, 16, generator=g, device="cuda").to(BF).to(dtype)
    W = (torch.randn(701, 16, generator=g, device="cuda") / 4).to(BF).to(dtype)
    t = torch.full((n,), target, dtype=torch.int32, device="cuda")
    s = x.double() @ W.double().T
    assert (x.double().abs() @ W.double().abs().T).max() < 48
    loss, lse = l3.l3_xent_forward(x, W, t)
    want = torch.logsumexp(s, 1)
    tol = 48 * 2.0 ** -23 + 2.0 ** -18
    assert (lse.double() - want).abs().max() <= tol
    assert (loss.double() - (want - s[:, target])).abs().max() <= 2 * tol


def mantissas(g, shape, bits):
    """Values in +-[1, 2) with that many random bits in all."""
    m = torch.randint(1 << (bits - 1), 1 << bits, shape, generator=g, device="cuda")
    return (m.double() / (1 << (bits - 1))).float() * (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1)


@pytest.mark.parametrize("n", [3, 200, 600])
@pytest.mark.parametrize("x_bits,w_bits", [(24, 1), (1, 24), (12, 12), (16, 8), (8, 16)])
def test_fp32_logits_keep_all_bits(n, x_bits, w_bits):
    """One column of W per row, so that each logit is a single product of 24 bits, which
    the parts of both factors hold exactly: off by 2^-23 of 16 twice at most, as the
    parts' products have either sign. The exponentials, their sum, the logarithm and the
    last rounding add 2^-18. Two parts of a factor would leave up to 2^-17 of a logit of 4 to
    16, 3e-5 to 1.2e-4."""
    d, vocab = 64, 300
    g = torch.Generator(device="cuda").manual_seed(n)
    x = mantissas(g, (n, d), x_bits) * 2
    W = torch.zeros(vocab, d, device="cuda")
    j = torch.arange(vocab, device="cuda")
    W[j, j % d] = mantissas(g, (vocab,), w_bits) * 2
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda").to(torch.int32)
    s = x.double() @ W.double().T
    assert (s.abs() > 0).all() and s.abs().max() < 16
    loss, lse = l3.l3_xent_forward(x, W, t)
    want = torch.logsumexp(s, 1)
    tol = 2 * 2.0 ** -23 * 16 + 2.0 ** -18
    assert (lse.double() - want).abs().max() <= tol
    assert (loss.double() - (want - s.gather(1, t.long()[:, None])[:, 0])).abs().max() <= tol


@pytest.mark.parametrize("which", ["dx", "dW"])
def test_fp32_gradients_keep_all_bits_of_g(which):
    """dW's x, or dx's W, has a single power of two in each column, so that the gradient's
    elements are G's times it. The probability: s is 2^-23 of 4 off, s - lse, below 14, half
    a step of 2^-20, its multiple by log2 e, below 21, half a step of 2^-19 (times log 2), the
    exponential 2^-22 (the reference takes the call's own lse): 2.1e-6 of it in all. The
    element: p - 1, the weight's ratio, two products by weights and three parts round by 2^-24
    each, their sum drops 2^-23 twice: 2^-21. Two parts would leave up to 2^-17, 7.6e-6."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n, vocab, d = (64, 300, 64) if which == "dW" else (300, 64, 64)
    eye = torch.eye(64, device="cuda") * 2.0 ** torch.randint(-1, 2, (64, 1), generator=g, device="cuda")
    full = torch.randn(max(n, vocab), d, generator=g, device="cuda").clamp(-2, 2)
    x, W = (eye, full) if which == "dW" else (full, eye)
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda").to(torch.int32)
    w = 0.5 + torch.rand(n, generator=g, device="cuda")
    _, lse = l3.l3_xent_forward(x, W, t)
    dx, dW = l3.l3_xent_backward(x, W, t, lse, w)
    s = x.double() @ W.double().T
    assert (s - lse.double()[:, None]).abs().max() < 14
    p = (s - lse.double()[:, None]).exp()
    hot = torch.zeros_like(p).scatter_(1, t.long()[:, None], 1.0)
    G, size = (p - hot) * w.double()[:, None], (p * 2.1e-6 + (p + hot) * 2.0 ** -21) * w.double()[:, None]
    got, want, tol = (dW, G.T @ x.double(), size.T @ x.double()) if which == "dW" else \
        (dx, G @ W.double(), size @ W.double())
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("n", [1, 20, 100, 200, 500])
def test_bf16_losses_keep_their_chains_short(n):
    """All terms of one sign, s near 100 from 4096 of them: a chain of 128 (n <= 32), 256
    (n <= 128) or 512 terms holds 1 / 32, 1 / 16 or 1 / 8 of s < 128, and each of its 8, 16
    or 32 steps drops up to 2^-23 of the power of two above that: 1.3e-4, 2.5e-4 and 4.9e-4 in
    all; adding the chains up rounds by 2^-24 of 128 each, 2.5e-4, 1.3e-4 and 6e-5. One
    chain of 4096 terms was 1.5e-3 off."""
    d, vocab = 4096, 40
    g = torch.Generator().manual_seed(n)
    W = (0.5 + torch.rand(vocab, d, generator=g)).to(BF).cuda()
    x = ((0.5 + torch.rand(n, d, generator=g)) / 40).to(BF).cuda()
    t = torch.randint(0, vocab, (n,), generator=g).to(torch.int32).cuda()
    s = x.double() @ W.double().T
    assert 90 < s.min() and s.max() < 128
    _, lse = l3.l3_xent_forward(x, W, t)
    assert (lse.double() - torch.logsumexp(s, 1)).abs().max() <= 5.5e-4
