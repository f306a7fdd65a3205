"""smdm_loss_stepcausal against the library's own logits, on other streams, captured and replayed.

The forward adds into its residual rows in an order that depends on timing, so two calls agree to its
rounding and not to the bit.  Where outputs of two calls are compared, the largest difference
between any two of five plain calls, four times it, is what their noise may make."""
import numpy as np
import pytest
import torch

import masked_discrete_diffusion_sparse_b200 as smdm
import oracle
import synth
from smdm_testlib import config_for, i32, upload_weights
from test_training_ends import _gpu, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


class Trajectory:
    def __init__(self, name, seed=5):
        self.wl = wl = synth.WORKLOADS[name]
        w = synth.make_weights(wl.model, wl.seed, gain_std=0.02)
        prompt = synth.make_prompt(wl)
        _, recs = oracle.generate(oracle.Model(w), prompt, wl.gen_len, synth.make_plan(wl),
                                  max_steps=3)
        ids, pos, types, labels, qrows = oracle.trajectory(prompt, wl.model, wl.gen_len, recs)
        rows = np.concatenate([qrows[k] for k in sorted(qrows)])
        rng = np.random.default_rng(seed)
        target = rng.integers(0, wl.model.vocab, len(rows)).astype(np.int32)
        target[::5] = -1
        self.m, self.d, self.v = len(rows), wl.model.d_model, wl.model.vocab
        dt = torch.float32 if wl.model.dtype == synth.F32 else torch.bfloat16
        self.weights = upload_weights(w)
        self.model = smdm.Model(config_for(wl, train_rows=max(len(ids), 200)), self.weights)
        self.seq = [i32(a) for a in (ids, pos, types, labels, rows)]
        self.target = i32(target)
        self.weight = torch.rand(self.m, device="cuda") / self.m
        nan = float("nan")
        self.nll, self.lse = (torch.full((self.m,), nan, device="cuda") for _ in range(2))
        self.gx = torch.full((self.m, self.d), nan, device="cuda")
        self.gn = torch.full((self.d,), nan, dtype=dt, device="cuda")
        self.gw = torch.full((self.v, self.d), nan, dtype=dt, device="cuda")
        self.ws = workspace(self.model.smdm_loss_stepcausal_workspace_bytes(self.m, grad=True))

    def outputs(self):
        return [self.nll, self.lse, self.gx, self.gn, self.gw]

    def clear(self):
        for t in self.outputs():
            t.fill_(float("nan"))

    def run(self, grad=True, stream=None):
        kw = dict(grad_nll=self.weight, grad_x=self.gx, grad_final_norm=self.gn,
                  grad_lm_head=self.gw) if grad else {}
        self.model.smdm_loss_stepcausal(*self.seq, self.target, self.nll, self.lse, self.ws,
                                        stream=stream, **kw)


@pytest.fixture(params=["tiny-bf16-cos", "tiny-f32-cos"])
def traj(request):
    t = Trajectory(request.param)
    yield t
    torch.cuda.synchronize()
    t.model.close()


def spread(runs):
    """Four times the largest difference between any two of the runs, output by output."""
    return [4 * max((a.double() - b.double()).abs().max().item() for a in r for b in r)
            for r in zip(*runs)]


def eager(traj, times=5):
    runs = []
    for _ in range(times):
        traj.run()
        torch.cuda.synchronize()
        runs.append([t.clone() for t in traj.outputs()])
    return runs


def assert_close(got, want, noise):
    for name, t, w, n in zip(("nll", "lse", "grad_x", "grad_final_norm", "grad_lm_head"), got, want,
                             noise):
        assert (t.double() - w.double()).abs().max().item() <= n, name


def test_loss_is_that_of_the_forward_s_logits(traj):
    """lse and nll are those of smdm_forward_stepcausal's logits: the same rows times the same
    weights, summed in fp32 on both sides, each off by at most (d / 16 + 17) 2^-23 of the sum of
    the terms' magnitudes, which is at most |row| |w_v|, and |row| at most d^0.5 max |gain|; 2^-20
    for exp and log, 2^-23 of the values for their rounding.  (Six products on the fp32 path.)"""
    traj.run(grad=False)
    runs = []
    for _ in range(5):
        logits = torch.empty((traj.m, traj.v), device="cuda")
        traj.model.smdm_forward_stepcausal(*traj.seq, logits)
        runs.append([logits])
    torch.cuda.synchronize()
    noise = spread(runs)[0]
    z = logits.double()
    on = traj.target >= 0
    lse = torch.logsumexp(z, dim=1)
    nll = lse - z.gather(1, traj.target.clamp(min=0).long()[:, None])[:, 0]
    f32 = traj.wl.model.dtype == synth.F32
    steps = ((6 if f32 else 1) * traj.d / 16 + 17) * 2.0 ** -23
    mag = traj.d ** 0.5 * traj.weights["final_norm"].abs().max().item() * 1.01 * \
        traj.weights["lm_head"].double().norm(dim=1).max().item()
    tol = 2 * steps * mag + 2.0 ** -20 + 2.0 ** -22 * z.abs().max().item() + noise
    err = (traj.lse.double() - lse)[on].abs().max().item()
    assert err <= tol, (err, tol)
    err = (traj.nll.double() - nll)[on].abs().max().item()
    assert err <= 2 * tol, (err, tol)
    assert (traj.nll[~on] == 0).all() and (traj.lse[~on] == 0).all()


def test_loss_s_rows_are_as_exact_as_the_forward_s(traj):
    """The logits of 200 (row, target) pairs, z = lse - nll, differ from one forward's as two forwards'
    do from each other (s, the root of the mean square over the same 200; twice that is allowed).
    Rows rounded to bf16 instead of the forward's fp16 would add 2^-8 / 3^0.5 of |row * w_v|, which
    is what a logit is, to every one: four times s here."""
    m = 200
    g = torch.Generator(device="cuda").manual_seed(3)
    pick = torch.randint(0, traj.m, (m,), generator=g, device="cuda")
    target = torch.randint(0, traj.v, (m,), generator=g, device="cuda")
    rows = traj.seq[4][pick].contiguous()
    nll, lse = (torch.full((m,), float("nan"), device="cuda") for _ in range(2))
    ws = workspace(traj.model.smdm_loss_stepcausal_workspace_bytes(m))
    zs, own = [], []
    for _ in range(6):
        logits = torch.empty((m, traj.v), device="cuda")
        traj.model.smdm_forward_stepcausal(*traj.seq[:4], rows, logits)
        zs.append(logits.double().gather(1, target[:, None])[:, 0])
        traj.model.smdm_loss_stepcausal(*traj.seq[:4], rows, target.int(), nll, lse, ws)
        own.append(lse.double() - nll.double())
    torch.cuda.synchronize()

    def rms(pairs):
        return sum((a - b).square().mean().item() for a, b in pairs) ** 0.5 / len(pairs) ** 0.5

    s = rms([(a, b) for i, a in enumerate(zs) for b in zs[:i]])
    err = rms([(a, b) for a in zs for b in own])
    # (2^-23 of values up to 8 in lse and nll, and the products' sums)
    steps = ((6 if traj.wl.model.dtype == synth.F32 else 1) * traj.d / 16 + 17) * 2.0 ** -23
    assert err <= 2 * s + 2.0 ** -20 + steps * zs[0].abs().max().item() * 8, (err, s)


@pytest.mark.parametrize("ignored", [0.0, 0.3])
def test_gradients_of_many_rows_are_those_of_its_parts(traj, ignored):
    """200 listed rows at once against 100 and 100 (other kernels): grad_x row by row, the weights'
    gradients as their sum.  Every output rounded once, the parts' too, D's entries to bf16, and the
    forwards' noise in z (1e-4 of p): together below 4 half steps of bf16 in the norm."""
    m, v, d = 200, traj.v, traj.d
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = traj.seq[4][torch.randint(0, traj.m, (m,), generator=g, device="cuda")].contiguous()
    target = torch.randint(0, v, (m,), generator=g, device="cuda").int()
    target[:40] = target[100]                       # shared targets
    target[torch.rand(m, generator=g, device="cuda") < ignored] = -1
    weight = torch.rand(m, generator=g, device="cuda") / m
    ws = workspace(max(traj.model.smdm_loss_stepcausal_workspace_bytes(k, grad=True)
                       for k in (100, m)))

    def grads(a, b):
        k = b - a
        nll, lse = (torch.full((k,), float("nan"), device="cuda") for _ in range(2))
        gx = torch.full((k, d), float("nan"), device="cuda")
        gn, gw = torch.empty_like(traj.gn), torch.full_like(traj.gw, float("nan"))
        traj.model.smdm_loss_stepcausal(
            *traj.seq[:4], rows[a:b].contiguous(), target[a:b].contiguous(), nll, lse, ws,
            grad_nll=weight[a:b].contiguous(), grad_x=gx, grad_final_norm=gn, grad_lm_head=gw)
        torch.cuda.synchronize()
        return nll, gx, gn, gw

    whole, one, two = grads(0, m), grads(0, 100), grads(100, m)
    for name, w, p in (("nll", whole[0], torch.cat([one[0], two[0]])),
                       ("grad_x", whole[1], torch.cat([one[1], two[1]])),
                       ("grad_final_norm", whole[2], one[2].double() + two[2].double()),
                       ("grad_lm_head", whole[3], one[3].double() + two[3].double())):
        err = (w.double() - p.double()).norm() / p.double().norm()
        assert err <= 4 * 2.0 ** -8, (name, err.item())
    assert (whole[1][target < 0] == 0).all()


def test_loss_on_another_stream_and_after_other_targets(traj):
    runs = eager(traj)
    s = torch.cuda.Stream()
    kept = traj.target.clone()
    for target in (torch.full_like(kept, 1), torch.full_like(kept, -1), kept):
        traj.target.copy_(target)
        traj.clear()
        torch.cuda.synchronize()
        traj.run(stream=s)
        torch.cuda.synchronize()
        for t in traj.outputs():
            assert torch.isfinite(t.float()).all()
        if (target < 0).all():
            assert all((t == 0).all() for t in traj.outputs())
    assert_close(traj.outputs(), runs[0], spread(runs))
    assert traj.model.smdm_device_status() == 0


def test_loss_on_another_stream_keeps_its_tensors(traj):
    """Tensors that the caller lets go of right after the call still hold their values when its
    kernels run."""
    traj.run()
    torch.cuda.synchronize()
    on = traj.target >= 0
    s = torch.cuda.Stream()
    target = traj.target.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)               # (about 50 ms: the call waits behind it)
    kept, traj.target = traj.target, target
    traj.clear()
    s.wait_stream(torch.cuda.current_stream())
    traj.run(grad=False, stream=s)
    traj.target = kept
    where = target.data_ptr()
    del target
    others = [torch.full_like(kept, -1) for _ in range(64)]     # would land in its memory
    assert all(t.data_ptr() != where for t in others)
    torch.cuda.synchronize()
    assert (traj.nll[on] != 0).all()


def test_loss_captured_and_replayed(traj):
    runs = eager(traj)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        traj.run()
    for _ in range(2):
        traj.clear()
        g.replay()
        torch.cuda.synchronize()
        assert_close(traj.outputs(), runs[0], spread(runs))
    # the captured call reads the data, not what it was at capture
    traj.target.fill_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert (traj.nll == 0).all() and (traj.gw == 0).all() and (traj.gx == 0).all()
    traj.run(grad=False)
    torch.cuda.synchronize()
    assert (traj.nll == 0).all()


def test_loss_of_a_target_beyond_the_vocabulary(traj):
    """It takes no part and sets the handle's status."""
    traj.target[1] = traj.v
    traj.run()
    with pytest.raises(smdm.SmdmError, match="bounds"):
        traj.model.smdm_device_status()
    assert traj.nll[1] == 0 and (traj.gx[1] == 0).all()
    assert torch.isfinite(traj.gw.float()).all()
