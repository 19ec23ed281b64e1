"""The gradients' products in 256-column tiles, with shares of the depth and without,
in one piece of the vocabulary and several, in both types; bounds of test_xent_gpu.py."""
import pytest

from test_xent_gpu import BF, FP, make, run_and_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,vocab,d,dtype,out", [
    (1500, 6000, 1024, FP, 0.0),    # 256 columns, 3 shares of dx
    (777, 20011, 516, FP, 0.3),     # 256, 16 shares
    (2048, 60000, 132, FP, 0.0),    # two pieces
    (1500, 20003, 1024, BF, 0.4),   # 256
    (100, 9000, 592, BF, 0.0),      # 6 shares, G's second part everywhere
    (4, 30000, 1040, BF, 0.0),      # and in dx
])
def test_gradients(n, vocab, d, dtype, out):
    run_and_check(*make(n, vocab, d, dtype, out))
