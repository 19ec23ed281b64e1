"""Numbers of partials around which the loss's join takes one block or eight a row
group, against 64 bits. Tolerance of a loss or lse of order ten, from logits of which d = 16
products are exact and added in one step (2^-23 of a sum of magnitudes below 48: 6e-6)
and exponentials, sums and logarithms (2^-18 relative to the sum, as in test_xent_gpu.py:
4e-6)."""
import pytest
import torch

import static_token_routed_b200 as l3

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 33, 128, 129, 512, 513])
@pytest.mark.parametrize("parts", [159, 160, 161, 999, 1000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_join_of_any_number_of_partials(n, parts, dtype):
    for columns in (32, 64, 128):   # behind a partial, in one form or another
        vocab = columns * parts - 5
        g = torch.Generator(device="cuda").manual_seed(vocab + n)
        x = torch.randn(n, 16, generator=g, device="cuda").to(dtype)
        W = torch.randn(vocab, 16, generator=g, device="cuda").to(dtype) / 4
        t = torch.randint(0, vocab, (n,), generator=g, device="cuda").to(torch.int32)
        if dtype == torch.float32:   # a single part each: exact products
            x, W = x.to(torch.bfloat16).float(), W.to(torch.bfloat16).float()
        s = x.double() @ W.double().T
        assert (x.double().abs() @ W.double().abs().T).max() < 48
        lse = torch.logsumexp(s, 1)
        got_loss, got = l3.l3_xent_forward(x, W, t)
        tol = 48 * 2.0 ** -23 + 2.0 ** -18
        assert (got.double() - lse).abs().max() <= tol
        assert (got_loss.double() - (lse - s.gather(1, t.long()[:, None])[:, 0])).abs().max() <= 2 * tol
