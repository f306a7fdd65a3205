"""What the head's gradient keeps of its accuracy where a result in fewer bits loses it: certain
targets, sums over very many rows, and the rounding of the logits' gradient D to bf16.

Expected values are the definitions in 64 bits; each tolerance is derived where it stands."""
import pytest
import torch

import masked_discrete_diffusion_sparse_b200 as smdm
from test_training_ends import BF16, Head, _gpu, f64  # noqa: F401

pytestmark = pytest.mark.gpu


def test_head_gradient_sums_over_very_many_rows():
    """grad_lm_head over 2^18 rows, its terms all of one sign: every row's target is id 0, whose
    gradient is left out, so D is positive elsewhere, and so are the hidden rows.

    A tensor-core step (16 rows) may cut 2^-23 of the final value off, always towards zero: 2^14
    steps in one accumulator up to 2^-9 (2e-3) of every output, as much as bf16's rounding, and the
    mean over the outputs shows it.  Summed 512 steps at a time it is 2^-14 at most; the outputs'
    rounding (uniform, 2^-8 / 3^0.5 of a value or less) leaves 2^-8 / (3 * 255 * 64)^0.5 = 1.8e-5
    in the mean, D's far less (2^18 independent ones); five times those."""
    rows, d, vocab = 1 << 18, 64, 256
    x = Head(rows, d, vocab, BF16, seed=1)
    x.h.abs_().add_(0.5)
    x.target.zero_()
    _, lse = x.check_loss()
    _, gw = x.check_grad(lse)
    z = x.h.to(f64) @ x.w.to(f64).T
    D = torch.exp(z - lse.to(f64)[:, None]) * x.weight.to(f64)[:, None]
    ref = D.T @ x.h.to(f64)
    rel = ((gw.to(f64) - ref) / ref)[1:]
    assert rel.mean().abs() <= 2.0 ** -14 + 5 * 1.8e-5, rel.mean().item()
