"""The training operators at the ends of their ranges: what their formulas give where the
arithmetic could lose it, and every kernel that the sizes choose, against the 64-bit forms of
tests/training_ref.py (which derives the bounds)."""
import pytest
import torch

from tests.gpu_util import require_gpu
from tests.test_training_gpu import DTYPES, _check_balance, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ga():
    return require_gpu()


# -------------------------------------------------------------- balance loss

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e", [(1, 1), (13, 8), (700, 60), (14383, 8), (3000, 128)])
def test_balance_equal_counts_have_no_gradient(ga, t, e, dtype):
    # every token chooses every expert: the loss is the coefficient, whatever the logits, and the
    # gradient exactly 0
    logits = (1.5 * _randn(t, e, seed=t)).to(dtype)
    ids = torch.stack([torch.randperm(e, generator=torch.Generator().manual_seed(i % 7))
                       for i in range(t)])
    kept, grad = _check_balance(ga, logits, ids, _randn(t, seed=2) > -0.5)
    assert (grad == 0).all()
    kept, grad = _check_balance(ga, logits, ids, None, coef=0.25)
    assert (grad == 0).all() and abs(kept.loss.item() - 0.25) < 1e-5
