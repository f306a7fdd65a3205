"""The head's loss and gradient of more rows than one CTA can look through: the list of the rows that
take part is counted in a launch of its own."""
import pytest
import torch

from test_training_ends import BF16, F32, Head, _gpu, gen  # noqa: F401
from test_training_ends_precision import norm_error_bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,d,vocab,dt,ignored,pad", [
    (8192, 64, 130, BF16, 0.3, 0), (8193, 64, 130, BF16, 0.3, 0), (16385, 64, 130, BF16, 0.3, 0),
    (70001, 72, 100, BF16, 0.0, 0),
    (70001, 72, 100, BF16, 0.9, 3), (20000, 30, 70, F32, 0.5, 0), (40000, 64, 9, BF16, 0.9999, 8)])
def test_head_of_many_rows(rows, d, vocab, dt, ignored, pad):
    x = Head(rows, d, vocab, dt, ignored, pad, seed=rows + vocab)
    _, lse = x.check_loss()
    a = x.check_grad(lse)
    b = x.grad(lse)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_head_of_many_rows_with_few_or_none_that_take_part():
    x = Head(50000, 64, 100, BF16, seed=3)
    x.target.fill_(-1)
    nll, lse = x.loss()
    gh, gw = x.grad(lse)
    for t in (nll, lse, gh, gw):
        assert (t == 0).all()
    x.target[49999] = 7
    x.target[16400] = 100                  # beyond the vocabulary: takes no part
    nll, lse = x.loss()
    assert x.status.item() == 2
    assert (nll[:49999] == 0).all() and nll[49999] > 0
    gh, gw = x.grad(lse)
    assert (gh[:49999] == 0).all() and (gh[49999] != 0).any() and (gw[7] != 0).any()


@pytest.mark.parametrize("rows,vocab,hot", [(8000, 64, 0.0), (8000, 5000, 0.6), (30000, 64, 0.0),
                                            (30000, 5000, 0.6), (9000, 3, 0.0), (40000, 70000, 0.3)])
def test_head_gradient_of_many_rows_with_one_target(rows, vocab, hot):
    """Hundreds or thousands of rows share a target: their remainders are summed over the row's id."""
    x = Head(rows, 72, vocab, BF16, 0.2, seed=vocab)
    if hot:
        x.target[torch.rand(rows, generator=gen(2), device="cuda") < hot] = vocab - 2
    x.weight.fill_(1 / rows)
    _, lse = x.check_loss()
    a = x.check_grad(lse)
    ref, bound = norm_error_bounds(x, lse)[1]
    err = (a[1].to(torch.float64) - ref).norm().item()
    assert err <= 1.05 * bound, err / bound
    b = x.grad(lse)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("rows,d,vocab,pad", [
    (6000, 63, 32768, 0), (6000, 64, 32768, 3),     # weights copied, D in pieces
    (40, 16384, 20000, 0), (100, 16384, 16385, 8)])  # one row tile, a slot's ids in pieces
def test_head_gradient_in_several_pieces_of_other_kinds(rows, d, vocab, pad):
    x = Head(rows, d, vocab, BF16, 0.1, pad, seed=rows + d, wpad=pad if d == 64 else 0)
    _, lse = x.check_loss()
    a = x.check_grad(lse)
    b = x.grad(lse)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
