"""The training form's ends on the GPU: the LM head's loss, RMSNorm and the embedding, each with
its gradient, against their definitions in 64 bits on the same inputs.

Tolerances are bounds computed from the inputs before the comparison.  With u = finfo.eps / 2, the
half step of a type:
  - a product summed on the tensor cores in fp32 over K terms is off by at most
    (K / 16 + 17) 2^-23 times the sum of the terms' magnitudes (one addition, rounded or cut, per
    16 terms, and the terms of one step among themselves);
  - values rounded to type T before a sum (the logits' gradient, bf16) are off by at most u(T)
    each, independently: their sum by at most 6 sigma, sigma^2 = sum (u value weight)^2 / 3;
  - the fp32 path drops products below 2^-23 of the factors' magnitudes;
  - every output is rounded once: u(out) times its value;
  - exp2 and log are good to a few 2^-23 relative; 2^-20 covers them with the scaling by log2 e.
"""
import math

import numpy as np
import pytest
import torch

import masked_discrete_diffusion_sparse_b200 as smdm
import oracle
import synth
from smdm_testlib import config_for, i32, upload_weights

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
f64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from masked_discrete_diffusion_sparse_b200 import build
    build.build()


def u_of(dt):
    return torch.finfo(dt).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape, std=1.0):
    return torch.empty(shape, device="cuda").normal_(0, std, generator=g)


def rows_apart(t, pad, dt, offset=0):
    """The same rows in a wider buffer (filled with NaN), `pad` elements apart, starting
    `offset` elements into the buffer."""
    n, d = t.shape
    buf = torch.full((n * (d + pad) + offset,), float("nan"), device="cuda", dtype=dt)
    v = buf[offset:].view(n, d + pad)[:, :d]
    v.copy_(t)
    return v


def within(got, ref, bound, what):
    got = got.to(f64)
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    excess = (got - ref).abs() - bound
    assert (excess <= 0).all(), \
        f"{what}: {(excess > 0).sum().item()} beyond the bound, worst {excess.max().item():.3g}, " \
        f"bound there {bound.flatten()[excess.argmax()].item():.3g}"


def workspace(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN patterns


# ------------------------------------------------------------------------------------------------
# LM-head loss
# ------------------------------------------------------------------------------------------------
class Head:
    def __init__(self, rows, d, vocab, dt, ignored=0.0, pad=0, offset=0, seed=0, std=0.02, wpad=0):
        g = gen(seed)
        self.dt, self.rows, self.d, self.vocab = dt, rows, d, vocab
        self.w = rows_apart(rand(g, vocab, d, std=std).to(dt), wpad, dt)
        self.target = torch.randint(0, vocab, (rows,), generator=g, device="cuda").int()
        h = rand(g, rows, d) + 0.4 * torch.rand((rows, 1), generator=g, device="cuda") / std * \
            self.w[self.target.long()].float()
        self.h = rows_apart(h.to(dt), pad, dt, offset)
        drop = torch.rand(rows, generator=g, device="cuda") < ignored
        self.target[drop] = -1
        self.weight = 1.0 / (0.02 + torch.rand(rows, generator=g, device="cuda")) / rows
        self.ws = workspace(max(smdm.smdm_head_loss_workspace_bytes(rows, d, vocab, dt, grad=b)
                                for b in (False, True)))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def loss(self, **kw):
        nll = torch.full((self.rows,), float("nan"), device="cuda")
        lse = torch.full_like(nll, float("nan"))
        smdm.smdm_head_loss(self.h, self.w, self.target, nll, lse, self.ws, status=self.status, **kw)
        return nll, lse

    def grad(self, lse, weight=None, want=(True, True), **kw):
        gh = torch.full((self.rows, self.d), float("nan"), dtype=self.dt, device="cuda")
        gw = torch.full((self.vocab, self.d), float("nan"), dtype=self.dt, device="cuda")
        smdm.smdm_head_loss_grad(self.h, self.w, self.target, lse,
                                 self.weight if weight is None else weight,
                                 gh if want[0] else None, gw if want[1] else None, self.ws,
                                 status=self.status, **kw)
        return gh, gw

    def reference(self):
        on = (self.target >= 0) & (self.target < self.vocab)
        h = torch.where(on[:, None], self.h, torch.zeros_like(self.h)).to(f64)
        w = self.w.to(f64)
        z = h @ w.T
        t = self.target.long().clamp(0, self.vocab - 1)[:, None]
        lse = torch.logsumexp(z, dim=1)
        zero = torch.zeros_like(lse)
        nll = torch.where(on, lse - z.gather(1, t)[:, 0], zero)
        # largest error of a logit of the row
        terms = 6 if self.dt == F32 else 1
        per = (terms * self.d / 16 + 17) * 2.0 ** -23 + (2.0 ** -23 if self.dt == F32 else 0)
        dz = per * (h.abs() @ w.abs().T).max(dim=1).values
        return on, h, w, z, t, torch.where(on, lse, zero), nll, dz

    def check_loss(self):
        nll, lse = self.loss()
        on, h, w, z, t, rlse, rnll, dz = self.reference()
        small = dz + 2.0 ** -20
        within(lse, rlse, torch.where(on, small + 2.0 ** -23 * rlse.abs(), torch.zeros_like(dz)),
               "lse")
        zt = z.gather(1, t)[:, 0].abs()
        within(nll, rnll, torch.where(on, 2 * small + 2.0 ** -23 * (rlse.abs() + zt),
                                      torch.zeros_like(dz)), "nll")
        assert self.status.item() == 0
        return nll, lse

    def check_grad(self, lse):
        gh, gw = self.grad(lse)
        on, h, w, z, t, _, _, dz = self.reference()
        p = torch.exp(z - lse.to(f64)[:, None])
        g = torch.where(on, self.weight, torch.zeros_like(self.weight)).to(f64)[:, None]
        D = p.clone()
        D.scatter_add_(1, t, torch.full_like(g, -1.0))
        D *= g
        # errors of D: the logit's and exp's (systematic), its rounding (independent; with 128 rows
        # or fewer D keeps two bf16 parts: 2^-16)
        sys_d = g.abs() * p * (dz[:, None] + 2.0 ** -20)
        u = (2.0 ** -8 if self.rows > 128 else 2.0 ** -16) if self.dt == BF16 else 2.0 ** -23
        out = u_of(self.dt)
        for what, got, ref, s, q, mag, k in (
                ("grad_hidden", gh, D @ w, sys_d @ w.abs(), (D * D) @ (w * w), D.abs() @ w.abs(),
                 self.vocab),
                ("grad_lm_head", gw, D.T @ h, sys_d.T @ h.abs(), (D * D).T @ (h * h),
                 D.abs().T @ h.abs(), self.rows)):
            terms = 6 if self.dt == F32 else 2
            acc = (terms * k / 16 + 17) * 2.0 ** -23 + (2.0 ** -23 if self.dt == F32 else 0)
            bound = s + 6 * u * (q / 3).sqrt() + acc * mag
            within(got, ref, bound + out * (ref.abs() + bound) + 1e-37, what)
        off = ~on
        assert (gh[off] == 0).all()
        return gh, gw


HEAD_CASES = [
    # rows, d, vocab, dtype, ignored, pad, offset
    (1, 64, 1, BF16, 0, 0, 0),             # one id: nll = 0
    (1, 128, 257, BF16, 0, 0, 0),
    (8, 1024, 32000, BF16, 0, 0, 0),
    (5, 8, 40, BF16, 0, 0, 0),
    (129, 72, 1000, BF16, 0.3, 0, 0),
    (130, 200, 513, BF16, 0.5, 1, 3),      # rows neither aligned nor together
    (300, 251, 1001, BF16, 0.2, 0, 0),     # no row of either operand on 16 bytes
    (257, 64, 130, BF16, 0.9, 8, 0),
    (700, 512, 4100, BF16, 0.15, 0, 0),
    (2000, 256, 5000, BF16, 0, 0, 0),      # CTA pairs, every row taken in place
    (2000, 256, 5000, BF16, 0.25, 0, 0),
    (1, 64, 33, F32, 0, 0, 0),
    (66, 1, 3, F32, 0, 0, 0),
    (331, 256, 1001, F32, 0.3, 5, 1),
    (1024, 256, 1024, F32, 0.5, 0, 0),
    (640, 130, 2111, F32, 0, 0, 0),
    # a handful of rows
    (16, 589, 3001, F32, 0, 0, 0), (16, 120, 1030, BF16, 0.4, 1, 3), (3, 589, 1999, BF16, 0, 0, 0),
    (7, 4096, 700, F32, 0.2, 4, 0), (13, 4096, 515, F32, 0, 0, 0), (9, 8, 2, BF16, 0, 0, 0),
    (4, 1000, 5003, F32, 0, 0, 0), (12, 2048, 4099, BF16, 0.3, 0, 0), (2, 1, 70, F32, 0, 0, 0),
    (17, 256, 900, F32, 0, 0, 0), (10, 3219, 1122, F32, 0.5, 0, 0), (16, 6401, 140, BF16, 0, 0, 0),
    (13, 2834, 333, BF16, 0, 2, 0), (3, 2834, 333, BF16, 0, 0, 0),
    # one row of tiles
    (128, 320, 1500, BF16, 0.3, 0, 0), (100, 1024, 8200, BF16, 0, 8, 0),
]


@pytest.mark.parametrize("case", HEAD_CASES, ids=lambda c: "-".join(map(str, c[:3])) + str(c[3])[6:])
def test_head_loss_and_gradient(case):
    rows, d, vocab, dt, ignored, pad, offset = case
    x = Head(rows, d, vocab, dt, ignored, pad, offset, seed=rows + d)
    _, lse = x.check_loss()
    x.check_grad(lse)


@pytest.mark.parametrize("dt,rows,wpad", [(BF16, 150, 8), (BF16, 150, 3), (BF16, 20, 24), (F32, 150, 1),
                                          (F32, 9, 5), (BF16, 9, 1), (F32, 9, 4)])
def test_head_weight_rows_apart(dt, rows, wpad):
    x = Head(rows, 96, 800, dt, 0.2, seed=13, wpad=wpad)
    _, lse = x.check_loss()
    x.check_grad(lse)


@pytest.mark.parametrize("dt,rows,vocab", [(BF16, 6000, 32768), (F32, 3500, 16000)])
def test_head_gradient_in_several_pieces(dt, rows, vocab):
    """The logits' gradient exceeds one piece: grad_hidden is summed over the pieces."""
    x = Head(rows, 64, vocab, dt, 0.1, seed=3)
    _, lse = x.check_loss()
    x.check_grad(lse)


@pytest.mark.parametrize("many", [300, 40])
def test_head_rows_of_equal_weight(many):
    """More rows share the largest weight than keep their remainders, or fewer."""
    x = Head(300, 128, 700, BF16, 0.1, seed=31)
    x.weight.fill_(1 / 300)
    x.weight[many:] /= 64
    _, lse = x.check_loss()
    x.check_grad(lse)


@pytest.mark.parametrize("rows", [40, 200])
def test_head_weights_past_32_bit_offsets(rows):
    """More than 2^31 weights, their gradient too; against the definition, 20000 ids at a time."""
    d, v, step = 4096, 540000, 20000
    g = gen(rows)
    w = torch.empty((v, d), dtype=BF16, device="cuda").normal_(0, 0.02, generator=g)
    h = rand(g, rows, d).to(BF16)
    target = torch.randint(0, v, (rows,), generator=g, device="cuda").int()
    target[:2] = torch.tensor([v - 1, 0])
    weight = (torch.rand(rows, generator=g, device="cuda") + 0.1) / rows
    ws = workspace(max(smdm.smdm_head_loss_workspace_bytes(rows, d, v, BF16, grad=b)
                       for b in (False, True)))
    nll, lse = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    smdm.smdm_head_loss(h, w, target, nll, lse, ws)
    gh, gw = torch.full_like(h, float("nan")), torch.empty_like(w)
    smdm.smdm_head_loss_grad(h, w, target, lse, weight, gh, gw, ws)
    hd, wt, l64 = h.to(f64), weight.to(f64)[:, None], lse.to(f64)[:, None]
    per = (d / 16 + 17) * 2.0 ** -23
    parts, dz = [], torch.zeros((rows, 1), dtype=f64, device="cuda")
    sums = [torch.zeros((rows, d), dtype=f64, device="cuda") for _ in range(4)]
    for a in range(0, v, step):
        c = w[a:a + step].to(f64)
        z = hd @ c.T
        dz = torch.maximum(dz, per * (hd.abs() @ c.abs().T).max(dim=1, keepdim=True).values)
        parts.append(torch.logsumexp(z, dim=1))
        p = torch.exp(z - l64)
        D = p * wt
        t = target.long() - a
        on = (t >= 0) & (t < len(c))
        D[on.nonzero()[:, 0], t[on]] -= wt[on, 0]
        for s, m in zip(sums, (D @ c, (D * D) @ (c * c), D.abs() @ c.abs(), (p * wt) @ c.abs())):
            s += m
    rlse = torch.logsumexp(torch.stack(parts), dim=0)
    dz = dz + 2.0 ** -20
    within(lse, rlse, dz[:, 0] + 2.0 ** -23 * rlse.abs(), "lse")
    # (as Head.check_grad)
    u = 2.0 ** -8 if rows > 128 else 2.0 ** -16
    ref, q, mag, sp = sums
    bound = dz * sp + 6 * u * (q / 3).sqrt() + (2 * v / 16 + 17) * 2.0 ** -23 * mag
    within(gh, ref, bound + u_of(BF16) * (ref.abs() + bound) + 1e-37, "grad_hidden")
    D, p = D[:, -64:], p[:, -64:]              # the last ids
    ref = D.T @ hd
    bound = (p * wt * dz).T @ hd.abs() + 6 * u * ((D * D).T @ (hd * hd) / 3).sqrt() + \
        (2 * rows / 16 + 17) * 2.0 ** -23 * (D.abs().T @ hd.abs())
    within(gw[-64:], ref, bound + u_of(BF16) * (ref.abs() + bound) + 1e-37, "grad_lm_head")
    assert torch.isfinite(gw[::997]).all()


@pytest.mark.parametrize("rows,d,dt", [(200, 128, BF16), (100, 64, BF16), (14, 128, BF16),
                                       (14, 30, F32), (150, 30, F32)])
def test_head_rows_without_a_target_reach_nothing(rows, d, dt):
    x = Head(rows, d, 700, dt, 0.4, seed=5)
    nll, lse = x.loss()
    a = x.grad(lse)
    off = x.target < 0
    for bad in (float("nan"), float("inf"), torch.finfo(dt).min):
        x.h[off] = bad
        lse2 = lse.clone()
        lse2[off] = float("nan")
        wt = x.weight.clone()
        wt[off] = float("nan")
        nll3, lse3 = x.loss()
        assert torch.equal(nll, nll3) and torch.equal(lse, lse3)
        b = x.grad(lse2, weight=wt)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("rows", [70, 5, 300])
def test_head_no_row_takes_part(dt, rows):
    x = Head(rows, 96, 300, dt, seed=6)
    x.target.fill_(-7)
    nll, lse = x.loss()
    gh, gw = x.grad(lse)
    for t in (nll, lse, gh, gw):
        assert (t == 0).all()
    e = Head(0, 96, 300, dt, seed=6)
    nll, lse = e.loss()
    _, gw = e.grad(lse)
    assert (gw == 0).all()


@pytest.mark.parametrize("rows,dt", [(50, BF16), (10, BF16), (10, F32), (150, F32)])
def test_head_target_beyond_the_vocabulary_sets_the_status(rows, dt):
    x = Head(rows, 64, 100, dt, seed=7)
    x.target[3] = 100
    x.target[9] = 2 ** 31 - 1
    nll, lse = x.loss()
    assert x.status.item() == 2
    assert nll[3] == 0 and lse[9] == 0
    x.status.zero_()
    gh, _ = x.grad(lse)
    assert x.status.item() == 2
    assert (gh[3] == 0).all() and (gh[9] == 0).all() and (gh[4] != 0).any()


@pytest.mark.parametrize("rows", [300, 11])
def test_head_one_gradient_alone(rows):
    x = Head(rows, 136, 900, BF16, 0.3, seed=8)
    _, lse = x.loss()
    gh, gw = x.grad(lse)
    assert torch.equal(x.grad(lse, want=(True, False))[0], gh)
    assert torch.equal(x.grad(lse, want=(False, True))[1], gw)


def test_head_large_logits_and_a_certain_target():
    """Logits of several hundred: the maximum is taken out before any exponential."""
    x = Head(64, 64, 512, F32, seed=9, std=4.0)
    nll, _ = x.check_loss()
    assert (nll >= 0).all()
    assert nll.max() > 20


@pytest.mark.parametrize("rows", [900, 12])
def test_head_same_bits_every_time(rows):
    x = Head(rows, 320, 3001, BF16, 0.2, seed=10)
    nll, lse = x.loss()
    a = x.grad(lse)
    for _ in range(3):
        assert torch.equal(x.loss()[0], nll)
        b = x.grad(lse)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_head_directional_difference():
    """The gradient against a central difference of the loss itself (fp32).  With step e along
    directions of unit size the difference is off by e^2 / 6 times the third derivative, here at
    most sum(weight) (2 |direction . row|)^3 < 1e-4 at e = 1e-2, plus 2 * 1e-5 / e of rounding."""
    x = Head(96, 64, 200, F32, 0.2, seed=11, std=0.3)
    x.weight /= x.weight.sum()
    _, lse = x.loss()
    gh, gw = x.grad(lse)
    g = gen(12)
    dh = rand(g, 96, 64) / 8
    dw = rand(g, 200, 64) / 8
    e = 1e-2

    def at(s):
        y = Head(96, 64, 200, F32, 0.2, seed=11, std=0.3)
        y.h.add_(s * dh)
        y.w.add_(s * dw)
        return (y.loss()[0].to(f64) * x.weight.to(f64)).sum().item()

    got = (gh.to(f64) * dh).sum().item() + (gw.to(f64) * dw).sum().item()
    diff = (at(e) - at(-e)) / (2 * e)
    third = 8 * max((dh.abs() * x.w.abs().max() + x.h.abs().max() * dw.abs().max()).max().item(), 1)
    assert abs(got - diff) <= e * e / 6 * third ** 3 + 2e-5 / e, (got, diff)


# ------------------------------------------------------------------------------------------------
# RMSNorm
# ------------------------------------------------------------------------------------------------
NORM_CASES = [
    # rows, d, x type, type, pad, add
    (1, 1, F32, F32, 0, False), (3, 7, F32, BF16, 1, True), (1, 4096, F32, BF16, 0, True),
    (66, 4096, F32, BF16, 0, False), (700, 251, F32, F32, 3, True), (129, 512, BF16, BF16, 0, True),
    (1000, 1024, BF16, F32, 4, False), (37, 1028, F32, BF16, 0, True),
    (500, 8192, F32, F32, 0, False), (9, 8191, BF16, BF16, 0, True), (2500, 64, F32, BF16, 8, True),
]


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: f"{c[0]}-{c[1]}")
def test_rmsnorm_and_gradient(case):
    rows, d, xt, dt, pad, add = case
    g = gen(rows * 7 + d)
    x = rows_apart(rand(g, rows, d, std=1.5).to(xt), pad, xt)
    gain = (1 + 0.1 * rand(g, d)).to(dt)
    gy = rows_apart(rand(g, rows, d).to(dt), pad, dt)
    ga = rand(g, rows, d).to(xt) if add else None
    ybuf = torch.full((rows, d + pad), 7.0, dtype=dt, device="cuda")
    y, rstd = ybuf[:, :d], torch.full((rows,), float("nan"), device="cuda")
    smdm.smdm_rmsnorm(x, gain, y, rstd, eps=1e-6)
    X, G = x.to(f64), gain.to(f64)
    r = 1 / (X.square().mean(dim=1) + 1e-6).sqrt()
    # the sum of squares: at most 32 additions in a thread, 8 shuffles and warps, then sqrt,
    # the quotient and the products: 48 half steps
    e = 48 * 2.0 ** -24
    within(rstd, r, e * r, "rstd")
    ref = X * r[:, None] * G
    within(y, ref, (2 * e + u_of(dt)) * ref.abs() + 1e-37, "y")
    assert (ybuf[:, d:] == 7.0).all(), "the columns between the rows were written"
    gx = torch.full((rows, d), float("nan"), dtype=xt, device="cuda")
    gg = torch.full((d,), float("nan"), dtype=dt, device="cuda")
    ws = workspace(smdm.smdm_rmsnorm_grad_workspace_bytes(rows, d))
    smdm.smdm_rmsnorm_grad(x, gain, rstd, gy, gx, gg, ws, grad_add=ga)
    R, GY = rstd.to(f64)[:, None], gy.to(f64)
    u = GY * G
    m = (u * X).mean(dim=1, keepdim=True)
    ref = R * (u - X * (R * R * m))
    A = ga.to(f64) if add else torch.zeros_like(ref)
    mag = R * (u.abs() + X.abs() * R * R * (u * X).abs().mean(dim=1, keepdim=True)) + A.abs()
    within(gx, ref + A, e * mag + u_of(xt) * (ref + A).abs() + 1e-37, "grad_x")
    terms = GY * X * R
    # rows of one thread in order, then the CTAs' shares: rows / (2 * 148) + 8 + 20 additions
    n_add = rows / 296 + 8 + rows / 32 + 40
    within(gg, terms.sum(0), n_add * 2.0 ** -24 * terms.abs().sum(0) +
           u_of(dt) * terms.sum(0).abs() + 1e-37, "grad_gain")
    if add:   # in place of grad_add
        smdm.smdm_rmsnorm_grad(x, gain, rstd, gy, ga, gg, ws, grad_add=ga)
        assert torch.equal(ga, gx)


def test_rmsnorm_no_rows_and_zero_rows():
    gain = torch.ones(64, device="cuda")
    gg = torch.full((64,), float("nan"), device="cuda")
    e = torch.empty((0, 64), device="cuda")
    smdm.smdm_rmsnorm(e, gain, e)
    smdm.smdm_rmsnorm_grad(e, gain, torch.empty(0, device="cuda"), e, e, gg,
                           workspace(smdm.smdm_rmsnorm_grad_workspace_bytes(0, 64)))
    assert (gg == 0).all()
    z = torch.zeros((5, 64), device="cuda")     # a zero row: rstd = eps^-1/2, y = 0
    y, r = torch.empty_like(z), torch.empty(5, device="cuda")
    smdm.smdm_rmsnorm(z, gain, y, r, eps=1e-4)
    assert (y == 0).all() and torch.allclose(r, torch.full_like(r, 100.0))


# ------------------------------------------------------------------------------------------------
# Embedding
# ------------------------------------------------------------------------------------------------
EMBED_CASES = [
    # rows, d, table rows, table type, row type, ids, pad, scale
    (1, 1, 1, F32, F32, "uniform", 0, 1.0), (5, 72, 3, BF16, F32, "uniform", 0, 1.0),
    (300, 64, 1000, BF16, BF16, "pad", 8, 8.0), (2048, 40, 50, F32, BF16, "uniform", 0, 0.5),
    (2049, 251, 700, BF16, BF16, "zipf", 3, 1.0), (5000, 256, 130, F32, F32, "mask", 0, 16.0),
    (17000, 264, 9000, BF16, F32, "mask", 0, 1.0), (40000, 16, 300, BF16, BF16, "one", 0, 1.0),
    (140000, 8, 70000, F32, F32, "pad", 0, 1.0), (64, 4096, 40, BF16, BF16, "one", 0, 1.0),
]


@pytest.mark.parametrize("case", EMBED_CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[5]}")
def test_embedding_and_gradient(case):
    rows, d, n_emb, dt, ot, kind, pad, scale = case
    g = gen(rows + d)
    ids = torch.randint(0, n_emb, (rows,), generator=g, device="cuda")
    if kind == "pad":
        ids[torch.rand(rows, generator=g, device="cuda") < 0.3] = -1
    elif kind == "mask":        # half of the rows carry one id, as [MASK] does
        ids[torch.rand(rows, generator=g, device="cuda") < 0.5] = n_emb - 2
    elif kind == "one":
        ids.fill_(n_emb // 2)
    elif kind == "zipf":
        ids = (n_emb * torch.rand(rows, generator=g, device="cuda") ** 6).long()
    ids = ids.int()
    table = rows_apart(rand(g, n_emb, d).to(dt), pad, dt)
    out = torch.full((rows, d), float("nan"), dtype=ot, device="cuda")
    smdm.smdm_embed(ids, table, out, scale=scale)
    on = (ids >= 0)[:, None]
    ref = torch.where(on, table[ids.clamp(min=0).long()].to(f64) * scale, torch.zeros((), dtype=f64,
                                                                                      device="cuda"))
    within(out, ref, (2.0 ** -24 + u_of(ot)) * ref.abs(), "rows")
    go = rows_apart(rand(g, rows, d).to(ot), pad, ot)
    gt = torch.full((n_emb, d), float("nan"), dtype=dt, device="cuda")
    ws = workspace(smdm.smdm_embed_grad_workspace_bytes(rows, d, n_emb))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    smdm.smdm_embed_grad(ids, go, gt, ws, scale=scale, status=status)
    G = torch.where(on, go.to(f64), torch.zeros((), dtype=f64, device="cuda"))
    i = ids.clamp(min=0).long()
    ref = torch.zeros((n_emb, d), dtype=f64, device="cuda").index_add_(0, i, G) * scale
    mag = torch.zeros_like(ref).index_add_(0, i, G.abs()) * scale
    cnt = torch.bincount(i[on[:, 0]], minlength=n_emb).to(f64)[:, None]
    # a piece's rows in order (at most 128), then an eighth of the pieces, the groups, the scale
    adds = torch.minimum(cnt, torch.full_like(cnt, 128)) + cnt / 64 + 12
    within(gt, ref, adds * 2.0 ** -24 * mag + u_of(dt) * ref.abs() + 1e-37, "grad_table")
    assert (gt[(cnt == 0)[:, 0]] == 0).all()
    assert status.item() == 0
    again = torch.empty_like(gt)
    smdm.smdm_embed_grad(ids, go, again, ws, scale=scale)
    assert torch.equal(gt, again)


def test_embedding_ids_beyond_the_table_and_no_rows():
    table = torch.ones((10, 16), device="cuda")
    ids = torch.tensor([0, 10, 3, -5], dtype=torch.int32, device="cuda")
    out = torch.full((4, 16), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    smdm.smdm_embed(ids, table, out, status=status)
    assert status.item() == 2 and out[:, 0].tolist() == [1, 0, 1, 0]
    status.zero_()
    gt = torch.empty_like(table)
    ws = workspace(smdm.smdm_embed_grad_workspace_bytes(4, 16, 10))
    go = torch.ones((4, 16), device="cuda")
    go[1] = float("nan")
    go[3] = float("inf")
    smdm.smdm_embed_grad(ids, go, gt, ws, status=status)
    assert status.item() == 2
    assert gt[:, 0].tolist() == [1, 0, 0, 1, 0, 0, 0, 0, 0, 0]
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 16), device="cuda")
    smdm.smdm_embed(none, table, e)
    smdm.smdm_embed_grad(none, e, gt, ws)
    assert (gt == 0).all()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_row_strides_past_32_bit_offsets(dt):
    """Rows 2^26 elements apart: the last ones lie past 2^31.  The same bits as rows together."""
    n, d, ld = 36, 128, 1 << 26
    g = gen(40)
    buf = torch.empty((n - 1) * ld + 4 * d, dtype=dt, device="cuda")
    near = [rand(g, n, d).to(dt) for _ in range(3)]
    near[1] *= 0.1
    far = [buf[i * d:].as_strided((n, d), (ld, 1)) for i in range(4)]
    for f, t in zip(far, near):
        f.copy_(t)
    x, w, y = near
    fx, fw, fy, fo = far
    target = torch.arange(n, device="cuda").int()
    target[5] = -1
    weight = torch.rand(n, generator=g, device="cuda")
    gain = rand(g, d).to(dt)
    ws = workspace(max(smdm.smdm_head_loss_workspace_bytes(n, d, n, dt),
                       smdm.smdm_head_loss_workspace_bytes(n, d, n, dt, grad=True),
                       smdm.smdm_head_loss_workspace_bytes(9, d, n, dt),
                       smdm.smdm_head_loss_workspace_bytes(9, d, n, dt, grad=True),
                       smdm.smdm_rmsnorm_grad_workspace_bytes(n, d),
                       smdm.smdm_embed_grad_workspace_bytes(n, d, n)))

    def run(x, w, y, out, rows):
        r = [torch.full((n,), float("nan"), device="cuda") for _ in range(3)]
        m = [torch.full((n, d), float("nan"), dtype=dt, device="cuda") for _ in range(5)]
        gg = torch.empty_like(gain)
        smdm.smdm_head_loss(x[:rows], w, target[:rows], r[0][:rows], r[1][:rows], ws)
        smdm.smdm_head_loss_grad(x[:rows], w, target[:rows], r[1][:rows], weight[:rows], m[0][:rows],
                                 m[1], ws)
        smdm.smdm_rmsnorm(x, gain, out, r[2])
        smdm.smdm_rmsnorm_grad(x, gain, r[2], y, m[2], gg, ws)
        smdm.smdm_embed(target, w, m[3])
        smdm.smdm_embed_grad(target, y, m[4], ws)
        return [t[:rows] for t in r[:2]] + [m[0][:rows], r[2], *m[1:], gg, out]

    for rows in (n, 9):
        a = run(x, w, y, torch.empty_like(x), rows)
        b = run(fx, fw, fy, fo, rows)
        for i, (s, t) in enumerate(zip(a, b)):
            assert torch.equal(s, t), i
            assert torch.isfinite(s.float()).all(), i


def test_embedding_past_32_bit_offsets():
    n, d = 40000, 65536
    g = gen(41)
    table = rand(g, 50, d).to(BF16)
    ids = torch.randint(0, 50, (n,), generator=g, device="cuda").int()
    out = torch.empty((n, d), dtype=BF16, device="cuda")
    smdm.smdm_embed(ids, table, out)
    for a in range(0, n, 5000):
        assert torch.equal(out[a:a + 5000], table[ids[a:a + 5000].long()])
    rows = torch.tensor([0, n - 1, 17, n - 1, 32769, n - 2], dtype=torch.int32, device="cuda")
    go = rand(g, 6, d).to(BF16)
    out.fill_(float("nan"))
    smdm.smdm_embed_grad(rows, go, out, workspace(smdm.smdm_embed_grad_workspace_bytes(6, d, n)))
    twice = (go[1].float() + go[3].float()).to(BF16)      # one fp32 addition, rounded once
    for row, want in ((0, go[0]), (17, go[2]), (32769, go[4]), (n - 2, go[5]), (n - 1, twice)):
        assert torch.equal(out[row], want), row
    assert sum(int(out[a:a + 5000].any(dim=1).sum()) for a in range(0, n, 5000)) == 5


# ------------------------------------------------------------------------------------------------
# Together, on streams and in graphs
# ------------------------------------------------------------------------------------------------
class Chain:
    """Embedding -> RMSNorm -> head loss and back: a model without layers."""

    def __init__(self, dt, rows=700, d=192, vocab=900, seed=20):
        g = gen(seed)
        self.dt, self.rows, self.d, self.vocab = dt, rows, d, vocab
        self.table = rand(g, vocab + 2, d).to(dt)
        self.gain = (1 + 0.1 * rand(g, d)).to(dt)
        self.w = rand(g, vocab, d, std=0.1).to(dt)
        self.ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda").int()
        masked = torch.rand(rows, generator=g, device="cuda") < 0.5
        self.target = torch.where(masked, self.ids, -1)
        self.ids[masked] = vocab                       # [MASK]
        self.weight = torch.rand(rows, generator=g, device="cuda") / rows

        def new(*s, dtype=dt):
            return torch.full(s, float("nan"), dtype=dtype, device="cuda")

        self.x, self.gx = new(rows, d, dtype=F32), new(rows, d, dtype=F32)
        self.y, self.gy = new(rows, d), new(rows, d)
        self.rstd, self.nll, self.lse = (new(rows, dtype=F32) for _ in range(3))
        self.gt, self.gg, self.gw = new(vocab + 2, d), new(d), new(vocab, d)
        self.ws = workspace(max(
            smdm.smdm_head_loss_workspace_bytes(rows, d, vocab, dt, grad=False),
            smdm.smdm_head_loss_workspace_bytes(rows, d, vocab, dt, grad=True),
            smdm.smdm_rmsnorm_grad_workspace_bytes(rows, d),
            smdm.smdm_embed_grad_workspace_bytes(rows, d, vocab + 2)))

    def outputs(self):
        return [self.nll, self.gt, self.gg, self.gw, self.gx]

    def step(self, stream=None):
        k = dict(stream=stream)
        smdm.smdm_embed(self.ids, self.table, self.x, **k)
        smdm.smdm_rmsnorm(self.x, self.gain, self.y, self.rstd, **k)
        smdm.smdm_head_loss(self.y, self.w, self.target, self.nll, self.lse, self.ws, **k)
        smdm.smdm_head_loss_grad(self.y, self.w, self.target, self.lse, self.weight, self.gy,
                                 self.gw, self.ws, **k)
        smdm.smdm_rmsnorm_grad(self.x, self.gain, self.rstd, self.gy, self.gx, self.gg, self.ws, **k)
        smdm.smdm_embed_grad(self.ids, self.gx, self.gt, self.ws, **k)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_chain_against_automatic_differentiation(dt):
    c = Chain(dt)
    c.step()
    t, gain, w = (v.to(f64).requires_grad_() for v in (c.table, c.gain, c.w))
    x = t[c.ids.long()]
    y = x / (x.square().mean(dim=1, keepdim=True) + 1e-6).sqrt() * gain
    on = c.target >= 0
    nll = torch.nn.functional.cross_entropy((y @ w.T)[on], c.target[on].long(), reduction="none")
    (nll * c.weight[on].to(f64)).sum().backward()
    # Intermediate roundings are independent, so relative errors in the Frobenius norm add up in
    # quadrature: at most four tensors rounded to the type (y, D, grad_y, the output), each by
    # u / sqrt(3) or less; times 3 for the propagation through the products.  fp32: 2^-23 sums.
    tol = 3 * 2 * u_of(dt) if dt == BF16 else 2.0 ** -16
    # y's rounding moves a logit by u |y| |w| / sqrt(3): sqrt(192) * 0.1 * 2^-8 / 1.7 = 3.2e-3
    # (one sigma); 6 sigma for bf16
    assert (c.nll[on].to(f64) - nll).abs().max() < (6 * 2 * 3.2e-3 if dt == BF16 else 2e-5)
    for name, got, ref in (("table", c.gt, t.grad), ("gain", c.gg, gain.grad), ("lm_head", c.gw, w.grad)):
        err = ((got.to(f64) - ref).norm() / ref.norm()).item()
        assert err < tol, f"{name}: {err:.3g} of {tol:.3g}"


def test_chain_on_another_stream_and_twice_at_once():
    a, b = Chain(BF16, seed=21), Chain(BF16, seed=22)
    a.step()
    b.step()
    torch.cuda.synchronize()
    want = [[t.clone() for t in c.outputs()] for c in (a, b)]
    for c in (a, b):
        for t in c.outputs():
            t.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        a.step(streams[0])
        b.step(streams[1])
    torch.cuda.synchronize()
    for c, ws in zip((a, b), want):
        for t, r in zip(c.outputs(), ws):
            assert torch.equal(t, r)


def test_chain_captured_and_replayed_with_a_shared_workspace():
    a, b = Chain(BF16, seed=23), Chain(BF16, seed=24)
    b.ws = a.ws
    a.step()
    b.step()
    torch.cuda.synchronize()
    want = [[t.clone() for t in c.outputs()] for c in (a, b)]
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.step()
        graphs.append(g)
    for c in (a, b):
        for t in c.outputs():
            t.fill_(float("nan"))
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, ws in zip((a, b), want):
        for t, r in zip(c.outputs(), ws):
            assert torch.equal(t, r)
    # the captured call reads the data, not what it was at capture
    a.target.fill_(-1)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert (a.nll == 0).all() and (a.gw == 0).all()


FIRST_CALL_CAPTURED = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from test_training_ends import BF16, Chain
a = Chain(BF16, seed=25)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a.step()
for t in a.outputs():
    t.fill_(float("nan"))
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in a.outputs()]
a.step()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, a.outputs()))
print("captured")
"""


def test_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL_CAPTURED.format(root=os.path.dirname(here), tests=here)
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "captured" in out.stdout, out.stderr[-2000:]


# ------------------------------------------------------------------------------------------------
# The model's path
# ------------------------------------------------------------------------------------------------
def residual_rows(m, ids, pos, types, labels, rows):
    """Rows of the residual stream behind the last layer (oracle.forward_stepcausal without its
    head)."""
    vis = oracle.cross_mask(types, labels, types, labels)
    x = m.emb[np.asarray(ids, dtype=np.int64)]
    for l in range(m.shape.n_layers):
        q, k, v = m.qkv(l, x, np.asarray(pos, dtype=np.int64))
        x = m.attn_out(l, x, oracle.attention(q, k, v, vis))
        x = m.mlp(l, x)
    return x[np.asarray(rows, dtype=np.int64)]


@pytest.mark.parametrize("name", ["tiny-f32-cos", "tiny-bf16-cos"])
def test_loss_stepcausal_against_the_oracle(name):
    wl = synth.WORKLOADS[name]
    w = synth.make_weights(wl.model, wl.seed, gain_std=0.02)
    om = oracle.Model(w)
    prompt = synth.make_prompt(wl)
    _, recs = oracle.generate(om, prompt, wl.gen_len, synth.make_plan(wl), max_steps=3)
    ids, pos, types, labels, qrows = oracle.trajectory(prompt, wl.model, wl.gen_len, recs)
    rows = np.concatenate([qrows[k] for k in sorted(qrows)])
    rows = np.concatenate([rows, rows[:3]])            # listed twice
    rng = np.random.default_rng(5)
    target = rng.integers(0, wl.model.vocab, len(rows)).astype(np.int32)
    target[::4] = -1
    on = target >= 0
    weight = (rng.random(len(rows)) / len(rows)).astype(np.float32)
    f32 = wl.model.dtype == synth.F32
    dt = F32 if f32 else BF16
    model = smdm.Model(config_for(wl, train_rows=len(ids)), upload_weights(w))
    try:
        m, d, v = len(rows), wl.model.d_model, wl.model.vocab
        nll, lse = (torch.full((m,), float("nan"), device="cuda") for _ in range(2))
        gx = torch.full((m, d), float("nan"), device="cuda")
        gn = torch.full((d,), float("nan"), dtype=dt, device="cuda")
        gw = torch.full((v, d), float("nan"), dtype=dt, device="cuda")
        args = [i32(a) for a in (ids, pos, types, labels, rows, target)]
        ws = workspace(model.smdm_loss_stepcausal_workspace_bytes(m, grad=True))
        model.smdm_loss_stepcausal(*args, nll, lse, ws)
        only = nll.clone()
        model.smdm_loss_stepcausal(*args, nll, lse, ws, grad_nll=torch.from_numpy(weight).cuda(),
                                   grad_x=gx, grad_final_norm=gn, grad_lm_head=gw)
        assert model.smdm_device_status() == 0
        logits = torch.empty((m, v), device="cuda")
        model.smdm_forward_stepcausal(*args[:5], logits)
        torch.cuda.synchronize()
    finally:
        model.close()
    x = torch.from_numpy(residual_rows(om, ids, pos, types, labels, rows)).requires_grad_()
    gain = torch.from_numpy(np.asarray(om.final_norm, dtype=np.float64)).requires_grad_()
    lm = torch.from_numpy(np.asarray(om.lm_head, dtype=np.float64)).requires_grad_()
    y = x / (x.square().mean(dim=1, keepdim=True) + wl.model.rms_eps).sqrt() * gain
    z = y @ lm.T
    ref = torch.logsumexp(z, 1) - z.gather(1, torch.from_numpy(target).long().clamp(min=0)[:, None])[:, 0]
    ref = torch.where(torch.from_numpy(on), ref, torch.zeros_like(ref))
    (ref * torch.from_numpy(weight).to(f64)).sum().backward()
    # the logits of this path meet the library's own bar (2e-2 / 1e-4 of the logit scale); a loss
    # is the difference of two functions of them, each moved by no more than the largest error
    bar = (1e-4 if f32 else 2e-2) * max(1.0, z.detach().abs().max().item())
    assert (nll.cpu().to(f64) - ref).abs().max().item() <= 2 * bar
    assert (only.cpu().to(f64) - ref).abs().max().item() <= 2 * bar
    assert (nll.cpu()[~torch.from_numpy(on)] == 0).all()
    own = torch.logsumexp(logits.cpu().to(f64), 1)
    assert (lse.cpu().to(f64) - own)[torch.from_numpy(on)].abs().max().item() <= 2 * bar
    # gradients: relative in the norm; the softmax moves by at most 2 bar, and bf16 rounds the
    # normalised rows, D, the gradient of the rows and the outputs
    tol = 2 * bar + (6 * 2.0 ** -8 if not f32 else 2.0 ** -16)
    for name, got, r in (("grad_x", gx, x.grad), ("grad_final_norm", gn, gain.grad),
                         ("grad_lm_head", gw, lm.grad)):
        err = ((got.cpu().to(f64) - r).norm() / r.norm()).item()
        assert err <= tol, f"{name}: {err:.3g} of {tol:.3g}"
    assert (gx.cpu()[~torch.from_numpy(on)] == 0).all()
