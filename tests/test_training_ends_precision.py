"""What the head's gradient keeps of its accuracy where a result in fewer bits loses it: certain
targets, sums over very many rows, and the rounding of the logits' gradient D to bf16.

Expected values are the definitions in 64 bits; each tolerance is derived where it stands."""
import pytest
import torch

import masked_discrete_diffusion_sparse_b200 as smdm
from test_training_ends import BF16, F32, Head, _gpu, f64, gen, rand, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [40, 200])
@pytest.mark.parametrize("rest", [1e-2, 1e-3])
def test_head_gradient_of_certain_targets(rows, rest):
    """p_target = 1 - rest at a logit of 30: D at the target is -rest, the difference of exp(z - lse)
    and 1, and every other entry is about rest / vocab.

    z_target and lse come from the same kind of sum, off by at most dz: the tensor core cuts up to
    2^-23 of a segment's value off in each of its 32 steps, the 8 segments are added with 2^-24 of a
    growing sum each, and z, lse and z - lse are rounded to 2^-24: 30 (2^-18 + 2^-22 + 3 2^-24), and
    2^-22 of exp.  grad_hidden is rest times a difference of weight rows, so dz / rest is its
    relative error, plus the output's rounding and D's (2^-9 in the norm each, 2^-8 together).
    With K summed whole (256 steps) dz alone would be 30 2^-15."""
    d, vocab, top = 4096, 500, 30.0
    g = gen(rows)
    u = rand(g, d, std=0.02)
    w = (u + rand(g, vocab, d, std=0.002)).to(BF16)
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    # z_v = other for all v, top at the target: rest = vocab exp(other - top)
    other = top + float(torch.log(torch.tensor(rest / vocab)))
    lift = w[target].float() - u
    lift -= (lift @ u)[:, None] / u.square().sum() * u
    h = other * u / u.square().sum() + (top - other) * lift / lift.square().sum(dim=1, keepdim=True)
    h = h.to(BF16)
    weight = torch.rand(rows, generator=g, device="cuda") + 0.5
    ws = workspace(max(smdm.smdm_head_loss_workspace_bytes(rows, d, vocab, BF16, grad=b)
                       for b in (False, True)))
    nll, lse = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    smdm.smdm_head_loss(h, w, target.int(), nll, lse, ws)
    gh, gw = torch.empty_like(h), torch.empty_like(w)
    smdm.smdm_head_loss_grad(h, w, target.int(), lse, weight, gh, gw, ws)
    z = h.to(f64) @ w.to(f64).T
    log_p = z - torch.logsumexp(z, dim=1, keepdim=True)
    at = torch.arange(rows, device="cuda")
    assert (log_p[at, target].neg().log() - torch.log(torch.tensor(rest))).abs().max() < 1
    D = log_p.exp()
    D[at, target] = torch.expm1(log_p[at, target])
    ref = (D * weight.to(f64)[:, None]) @ w.to(f64)
    dz = top * (2.0 ** -18 + 2.0 ** -22 + 3 * 2.0 ** -24) + 2.0 ** -22
    err = (gh.to(f64) - ref).norm(dim=1) / ref.norm(dim=1)
    tol = dz / -D[at, target] + 2.0 ** -8
    assert (err <= tol).all(), (err / tol).max().item()


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


def norm_error_bounds(x, lse):
    """The gradients of a Head case and, for each output, its value in 64 bits and the error that
    rounding the output once and D off the targets may leave, in the Frobenius norm: D's rounding
    is off by at most half a step u = 2^-8 of its value, independently from entry to entry, so the
    squares add up to at most u^2 / 3 D_rv^2 |w_v|^2 (or |h_r|^2) over r and v != t(r)."""
    on, h, w, z, t, _, _, _ = x.reference()
    p = torch.exp(z - lse.to(f64)[:, None])
    g = torch.where(on, x.weight, torch.zeros_like(x.weight)).to(f64)[:, None]
    D = p * g
    off = D.scatter(1, t, 0.0).square()
    D.scatter_add_(1, t, -g)
    out = []
    for ref, var in ((D @ w, (off @ w.square()).sum()), (D.T @ h, (off.T @ h.square()).sum())):
        own = (ref.to(BF16).to(f64) - ref).norm()
        out.append((ref, (own.square() + 2.0 ** -16 / 3 * var).sqrt().item()))
    return out


@pytest.mark.parametrize("kind", ["row", "equal", "sequence"])
@pytest.mark.parametrize("case", [(1024, 512, 2048, 0.0), (300, 128, 700, 0.1),
                                  (2000, 256, 5000, 0.25), (333, 251, 1001, 0.5)],
                         ids=lambda c: "-".join(map(str, c)))
def test_head_gradients_keep_their_own_rounding(case, kind):
    """Weights per row, the same for all rows (the mean), and per sequence of rows (1 / t): both
    gradients' errors are their own rounding's (at least 2^18 outputs: the norms' spread is below
    1 %; 3 % of room).  With D's rounding at the targets in them they are up to 1.45 times as large."""
    rows, d, vocab, ignored = case
    x = Head(rows, d, vocab, BF16, ignored, seed=rows)
    if kind == "equal":
        x.weight.fill_(1 / rows)
    elif kind == "sequence":
        x.weight = (1 / torch.tensor([0.05, 0.2, 0.5, 0.9], device="cuda") / rows) \
            .repeat_interleave((rows + 3) // 4)[:rows].contiguous()
    _, lse = x.check_loss()
    got = x.check_grad(lse)
    for what, o, (ref, bound) in zip(("grad_hidden", "grad_lm_head"), got,
                                     norm_error_bounds(x, lse)):
        err = (o.to(f64) - ref).norm().item()
        assert err <= 1.03 * bound, f"{what}: {err / bound:.3f} times its rounding"


@pytest.mark.parametrize("rows,d,vocab", [(700, 96, 40), (5000, 264, 3), (400, 1000, 1),
                                          (1500, 320, 900)])
def test_head_gradient_of_targets_with_many_rows(rows, d, vocab):
    """Few ids take all targets, or one id most of them: hundreds of remainders add to one row."""
    x = Head(rows, d, vocab, BF16, 0.2, pad=3 if d == 264 else 0, seed=d)
    if vocab == 900:
        x.target[torch.rand(rows, generator=gen(1), device="cuda") < 0.7] = 571
    x.weight.fill_(1 / rows)
    _, lse = x.check_loss()
    got = x.check_grad(lse)
    if vocab > 1:                      # (one id: D is nothing but the error of exp)
        ref, bound = norm_error_bounds(x, lse)[1]
        err = (got[1].to(f64) - ref).norm().item()
        assert err <= 1.05 * bound, err / bound
    again = x.grad(lse)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("rows,d,vocab", [(96, 64, 200), (12, 64, 200), (300, 96, 700)])
def test_head_gradients_against_differences(rows, d, vocab):
    """Each gradient alone against the central difference of the kernel's loss along it (fp32).

    The loss f is the weighted sum of nll, its weights add up to 1.  The difference over 2 e is off
    by what the same difference of the definition in 64 bits is off from its derivative, and by
    1 / e times the error of nll: at most 2^-20 of exp and log, 2^-23 of values up to 32, and a
    logit's, six products of d / 16 steps of 2^-23 of about (d / 2)^0.5 (the terms' signs are random),
    twice."""
    x = Head(rows, d, vocab, F32, 0.2, seed=11, std=0.3)
    x.weight /= x.weight[x.target >= 0].sum()
    _, lse = x.loss()
    gh, gw = x.grad(lse)
    on = x.target >= 0
    wt = torch.where(on, x.weight, torch.zeros_like(x.weight)).to(f64)
    t = x.target.long().clamp(min=0)[:, None]
    h0, w0 = x.h.clone(), x.w.clone()

    def exact(h, w):
        z = h.to(f64) @ w.to(f64).T
        return ((torch.logsumexp(z, 1) - z.gather(1, t)[:, 0]) * wt).sum().item()

    def kernel(h, w):
        x.h.copy_(h)
        x.w.copy_(w)
        return (x.loss()[0].to(f64) * wt).sum().item()

    err = 2 * (2.0 ** -20 + 2.0 ** -18 + 2 * 6 * d / 16 * 2.0 ** -23 * (d / 2) ** 0.5)
    e = 0.05
    for which, got in ((0, gh), (1, gw)):
        z = h0.to(f64).requires_grad_(which == 0), w0.to(f64).requires_grad_(which == 1)
        logits = z[0] @ z[1].T
        f = ((torch.logsumexp(logits, 1) - logits.gather(1, t)[:, 0]) * wt).sum()
        ref, = torch.autograd.grad(f, z[which])
        dirn = (ref / ref.norm()).float()
        at = lambda s: (h0 + s * dirn, w0) if which == 0 else (h0, w0 + s * dirn)  # noqa: E731
        true = (ref * dirn.to(f64)).sum().item()
        trunc = abs((exact(*at(e)) - exact(*at(-e))) / (2 * e) - true)
        diff = (kernel(*at(e)) - kernel(*at(-e))) / (2 * e)
        tol = trunc + err / e
        mine = (got.to(f64) * dirn.to(f64)).sum().item()
        assert tol < 0.1 * abs(diff), (which, tol, diff)
        assert abs(mine - diff) <= tol, (which, mine, diff, tol)
