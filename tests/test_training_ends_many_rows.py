"""The head's loss and gradient of more rows than one CTA can look through: the list of the rows that
take part is counted in a launch of its own."""
import pytest
import torch

from test_training_ends import BF16, F32, Head, _gpu, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,d,vocab,dt,ignored,pad", [
    (16384, 64, 130, BF16, 0.3, 0), (16385, 64, 130, BF16, 0.3, 0), (70001, 72, 100, BF16, 0.0, 0),
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
