"""Operators at the vocabulary-sized ends of a masked diffusion model's training form: the
embedding lookup, the RMSNorm in front of the LM head, and the LM head's cross entropy, each with
its gradient.  Every case is one pass of one operator.

    head_loss   hidden [R][d], lm_head [V][d], target [R] -> nll [R], lse [R]
    head_grad   the same inputs, lse and the per-row weights of the loss (the gradient with
                respect to nll) -> grad_hidden [R][d], grad_lm_head [V][d]
    norm        x [R][d], gain [d] -> y [R][d], rstd [R]
    norm_grad   x, gain, rstd, grad_y, the residual branch's gradient -> grad_x, grad_gain
    embed       ids [n], table [N][d], scale -> rows [n][d]
    embed_grad  ids [n], grad_rows [n][d], scale -> grad_table [N][d]

A negative target or id is a row that takes no part (an unmasked position, padding).
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
DT = {F32: torch.float32, BF16: torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # the 8 tokens committed by one step of a semi-autoregressive text run, scored
        {"name": "head_loss-text-step", "op": "head_loss", "dtype": BF16, "rows": 8, "d": 1024,
         "vocab": 32000, "ignored": 0.0, "pad": 0},
        # every mask row of a 4096-token image trajectory
        {"name": "head_loss-image", "op": "head_loss", "dtype": BF16, "rows": 4096, "d": 4096,
         "vocab": 8192, "ignored": 0.0, "pad": 0},
        # an fp32 model with a ragged vocabulary; the rows are a slice of wider ones
        {"name": "head_loss-f32-ragged", "op": "head_loss", "dtype": F32, "rows": 331, "d": 256,
         "vocab": 1001, "ignored": 0.3, "pad": 5},
        # one 128-token block of text over the large vocabulary
        {"name": "head_grad-text-block", "op": "head_grad", "dtype": BF16, "rows": 128, "d": 1024,
         "vocab": 32000, "ignored": 0.0, "pad": 0},
        # a 4096-token image of which a quarter was given (inpainting), so carries no loss
        {"name": "head_grad-image", "op": "head_grad", "dtype": BF16, "rows": 4096, "d": 4096,
         "vocab": 8192, "ignored": 0.25, "pad": 0},
        # the small fp32 model: 32 x 32 positions over its 1024 ids
        {"name": "head_grad-f32", "op": "head_grad", "dtype": F32, "rows": 1024, "d": 256,
         "vocab": 1024, "ignored": 0.5, "pad": 0},
        # one query and one new token with the 64 registers: a sampling step's smallest row set
        {"name": "norm-step", "op": "norm", "x": F32, "dtype": BF16, "rows": 66, "d": 4096,
         "pad": 0},
        # the whole step-labelled trajectory of the 4096-token image
        {"name": "norm_grad-image", "op": "norm_grad", "x": F32, "dtype": BF16, "rows": 12544,
         "d": 4096, "pad": 0, "add": True},
        # odd width, rows apart
        {"name": "norm_grad-odd", "op": "norm_grad", "x": F32, "dtype": F32, "rows": 777,
         "d": 251, "pad": 3, "add": False},
        # the trajectory's ids: prompt, clean tokens, 4096 [MASK] rows, 64 x 64 registers
        {"name": "embed-image", "op": "embed", "dtype": BF16, "out": F32, "ids": "trajectory",
         "rows": 12544, "d": 4096, "table": 8258, "scale": 1.0},
        {"name": "embed_grad-image", "op": "embed_grad", "dtype": BF16, "out": BF16,
         "ids": "trajectory", "rows": 12544, "d": 4096, "table": 8258, "scale": 1.0},
        # a text prompt: Zipf-distributed ids over the large table, scaled embeddings
        {"name": "embed_grad-text", "op": "embed_grad", "dtype": BF16, "out": F32, "ids": "zipf",
         "rows": 512, "d": 1024, "table": 32066, "scale": 32.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row width: a multiple of 64, of 8, or any number."""
    d = _log(rng, lo, hi)
    step = rng.choice([64, 64, 8, 1])
    return max(step, d // step * step)


def draw(rng):
    op = rng.choice(["head_loss", "head_grad", "head_loss", "head_grad", "norm", "norm_grad",
                     "embed", "embed_grad"])
    dtype = rng.choice([BF16, BF16, F32])
    if op in ("head_loss", "head_grad"):
        rows = _log(rng, 1, 4096)
        vocab = _log(rng, 257, 32768)
        d = _width(rng, 64, 4096)
        # fp32 models are the small ones; every case costs at most the largest listed one
        top = 4096 * 4096 * 8192 if dtype == BF16 else 2048 * 1024 * 4096
        while rows * vocab * d > top:
            if d > 1024:
                d = _width(rng, 64, 1024)
            else:
                vocab = max(257, vocab // 2)
                rows = max(1, rows * 3 // 4)
        return {"op": op, "dtype": dtype, "rows": rows, "d": d, "vocab": vocab,
                "ignored": rng.choice([0.0, 0.15, 0.5, 0.85]), "pad": rng.choice([0, 0, 1, 8])}
    if op in ("norm", "norm_grad"):
        d = _width(rng, 64, 8192)
        rows = min(_log(rng, 1, 12544), 12544 * 4096 // d)
        c = {"op": op, "x": rng.choice([F32, dtype]), "dtype": dtype, "rows": rows, "d": d,
             "pad": rng.choice([0, 0, 1, 8])}
        if op == "norm_grad":
            c["add"] = rng.choice([True, False])
        return c
    d = _width(rng, 64, 4096)
    table = _log(rng, 100, 32768)
    rows = min(_log(rng, 1, 32768), 12544 * 4096 // d)
    while table * d > 8258 * 4096:
        table //= 2
    return {"op": op, "dtype": dtype, "out": rng.choice([F32, dtype]),
            "ids": rng.choice(["trajectory", "zipf", "uniform"]), "rows": rows, "d": d,
            "table": table, "scale": rng.choice([1.0, math.sqrt(d)])}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def _rows(gen, n, d, dtype, pad, std=1.0):
    """[n][d] values N(0, std), every row `pad` elements apart from the next."""
    t = torch.empty((n, d + pad), dtype=torch.float32, device="cuda").normal_(0, std, generator=gen)
    return t.to(DT[dtype])[:, :d]


def _active(gen, n, ignored):
    """Which rows take part: a fixed number of them, placed at random."""
    order = torch.rand(n, generator=gen, device="cuda").argsort()
    return order >= int(n * ignored)


def _ids(gen, case):
    n, table = case["rows"], case["table"]
    if case["ids"] == "uniform":
        ids = torch.randint(0, table, (n,), generator=gen, device="cuda")
        ids[torch.rand(n, generator=gen, device="cuda") < 0.05] = -1      # padding
        return ids.int()
    if case["ids"] == "zipf":
        w = torch.arange(1, table + 1, device="cuda", dtype=torch.float64).pow(-1.1)
        cdf = (w.cumsum(0) / w.sum()).float()
        u = torch.rand(n, generator=gen, device="cuda")
        return torch.searchsorted(cdf, u).clamp_(max=table - 1).int()
    # a step-labelled trajectory: a third clean tokens, a third [MASK], a third registers
    regs = min(64, table // 4)
    vocab = table - 2 - regs
    clean = torch.randint(0, vocab, (n - 2 * (n // 3),), generator=gen, device="cuda")
    mask = torch.full((n // 3,), vocab, device="cuda")
    reg = vocab + 2 + torch.arange(n // 3, device="cuda") % regs
    return torch.cat([clean, mask, reg]).int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, n, d = case["op"], case["rows"], case["d"]
    s = {"case": case}
    if op in ("head_loss", "head_grad"):
        v = case["vocab"]
        s["lm_head"] = _rows(gen, v, d, case["dtype"], 0, 0.02)
        target = torch.randint(0, v, (n,), generator=gen, device="cuda")
        # normalised rows that lean towards their target's row, as a trained model's do: the
        # target's logit stands up to 8 above the others
        h = torch.empty((n, d + case["pad"]), device="cuda").normal_(generator=gen)
        lean = torch.rand((n, 1), generator=gen, device="cuda") * 8 / (0.02 * 0.02 * d)
        h[:, :d] += lean * s["lm_head"][target].float()
        s["hidden"] = h.to(DT[case["dtype"]])[:, :d]
        s["target"] = torch.where(_active(gen, n, case["ignored"]), target, -1).int()
        if op == "head_grad":
            # 1 / t weights of the masked diffusion objective, averaged over the rows
            t = torch.rand(n, generator=gen, device="cuda") * 0.98 + 0.02
            s["grad_nll"] = 1.0 / (t * n)
            lse = torch.empty(n, device="cuda")
            w = s["lm_head"].float()
            for i in range(0, n, 1024):
                lse[i:i + 1024] = torch.logsumexp(s["hidden"][i:i + 1024].float() @ w.T, dim=1)
            s["lse"] = torch.where(s["target"] >= 0, lse, torch.zeros_like(lse))
    elif op in ("norm", "norm_grad"):
        s["x"] = _rows(gen, n, d, case["x"], case["pad"], 1.5)
        s["gain"] = (1 + 0.1 * torch.empty(d, device="cuda").normal_(generator=gen)) \
            .to(DT[case["dtype"]])
        if op == "norm_grad":
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(dim=1) + EPS)
            s["grad_y"] = _rows(gen, n, d, case["dtype"], case["pad"], 0.01)
            s["grad_add"] = _rows(gen, n, d, case["x"], 0, 0.01) if case["add"] else None
    else:
        s["ids"] = _ids(gen, case)
        if op == "embed":
            s["table"] = _rows(gen, case["table"], d, case["dtype"], 0, 0.02)
        else:
            s["grad_rows"] = _rows(gen, n, d, case["out"], 0, 0.01)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The output tensors and the workspace that a user's program keeps from step to step."""
    import masked_discrete_diffusion_sparse_b200 as smdm
    case = s["case"]
    op, n, d = case["op"], case["rows"], case["d"]

    def new(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    size = 0
    if op in ("head_loss", "head_grad"):
        v, dt = case["vocab"], DT[case["dtype"]]
        size = smdm.smdm_head_loss_workspace_bytes(n, d, v, dt, grad=op == "head_grad")
        s["o"] = (new(n), new(n)) if op == "head_loss" else \
            (new(n, d, dtype=dt), new(v, d, dtype=dt))
    elif op == "norm":
        s["o"] = (new(n, d, dtype=DT[case["dtype"]]), new(n))
    elif op == "norm_grad":
        size = smdm.smdm_rmsnorm_grad_workspace_bytes(n, d)
        s["o"] = (new(n, d, dtype=DT[case["x"]]), new(d, dtype=DT[case["dtype"]]))
    elif op == "embed":
        s["o"] = new(n, d, dtype=DT[case["out"]])
    else:
        size = smdm.smdm_embed_grad_workspace_bytes(n, d, case["table"])
        s["o"] = new(case["table"], d, dtype=DT[case["dtype"]])
    s["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import masked_discrete_diffusion_sparse_b200 as smdm
    case, o = s["case"], s["o"]
    op = case["op"]
    if op == "head_loss":
        smdm.smdm_head_loss(s["hidden"], s["lm_head"], s["target"], o[0], o[1], s["ws"])
    elif op == "head_grad":
        smdm.smdm_head_loss_grad(s["hidden"], s["lm_head"], s["target"], s["lse"], s["grad_nll"],
                                 o[0], o[1], s["ws"])
    elif op == "norm":
        smdm.smdm_rmsnorm(s["x"], s["gain"], o[0], o[1], eps=EPS)
    elif op == "norm_grad":
        smdm.smdm_rmsnorm_grad(s["x"], s["gain"], s["rstd"], s["grad_y"], o[0], o[1], s["ws"],
                               grad_add=s["grad_add"])
    elif op == "embed":
        smdm.smdm_embed(s["ids"], s["table"], o, scale=case["scale"])
    else:
        smdm.smdm_embed_grad(s["ids"], s["grad_rows"], o, s["ws"], scale=case["scale"])
    return o


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("head_loss", "head_grad"):
        w, h = s["lm_head"].float(), s["hidden"].float()
        on = s["target"] >= 0
        t = s["target"].clamp(min=0).long()[:, None]
        logits = h @ w.T
        if op == "head_loss":
            top = logits.max(dim=1, keepdim=True).values
            lse = (logits - top).exp_().sum(dim=1).log_() + top[:, 0]
            zero = torch.zeros_like(lse)
            return torch.where(on, lse - logits.gather(1, t)[:, 0], zero), \
                torch.where(on, lse, zero)
        g = torch.where(on, s["grad_nll"], torch.zeros_like(s["grad_nll"]))[:, None]
        p = (logits - s["lse"][:, None]).exp_()
        p.scatter_add_(1, t, torch.full_like(g, -1.0))
        p *= g
        p = torch.where(on[:, None], p, torch.zeros_like(p))
        return (p @ w).to(s["hidden"].dtype), (p.T @ h).to(s["lm_head"].dtype)
    if op == "norm":
        x = s["x"].float()
        r = torch.rsqrt(x.square().mean(dim=1) + EPS)
        return (x * r[:, None] * s["gain"].float()).to(s["gain"].dtype), r
    if op == "norm_grad":
        x, gy, r = s["x"].float(), s["grad_y"].float(), s["rstd"][:, None]
        u = gy * s["gain"].float()
        gx = r * (u - x * (r * r * (u * x).mean(dim=1, keepdim=True)))
        if s["grad_add"] is not None:
            gx = gx + s["grad_add"].float()
        return gx.to(s["x"].dtype), (gy * x * r).sum(dim=0).to(s["gain"].dtype)
    on = (s["ids"] >= 0)[:, None]
    i = s["ids"].clamp(min=0).long()
    if op == "embed":
        rows = s["table"].float()[i] * case["scale"]
        return torch.where(on, rows, torch.zeros_like(rows)).to(DT[case["out"]])
    g = s["grad_rows"].float()
    out = torch.zeros((case["table"], case["d"]), device="cuda")
    out.index_add_(0, i, torch.where(on, g, torch.zeros_like(g)))
    return (out * case["scale"]).to(DT[case["dtype"]])


# ------------------------------------------------------------------------------------------------
# Work and exact values
# ------------------------------------------------------------------------------------------------
def work(case):
    op, n, d = case["op"], case["rows"], case["d"]
    size = {F32: 4, BF16: 2}
    e = size[case["dtype"]]
    if op in ("head_loss", "head_grad"):
        v = case["vocab"]
        on = n - int(n * case["ignored"])
        if op == "head_loss":
            return {"bytes": e * d * (on + v) + 12 * n, "flops": 2 * on * v * d}
        # the logits are not kept, so the gradient needs them once more: three products
        return {"bytes": e * d * (on + n + 2 * v) + 12 * n, "flops": 6 * on * v * d}
    if op == "norm":
        return {"bytes": n * d * (size[case["x"]] + e) + d * e + 4 * n, "flops": 4 * n * d}
    if op == "norm_grad":
        per = 2 * size[case["x"]] + e + (size[case["x"]] if case["add"] else 0)
        return {"bytes": n * d * per + 2 * d * e + 4 * n, "flops": 10 * n * d}
    t, o = case["table"], size[case["out"]]
    if op == "embed":
        distinct = min(n, t) if case["ids"] != "trajectory" else min(t, n - 2 * (n // 3) + 65)
        return {"bytes": n * d * o + distinct * d * e + 4 * n, "flops": n * d}
    return {"bytes": n * d * o + t * d * e + 4 * n, "flops": n * d}


def exact(case, seed):
    """The definitions in 64 bits: log-softmax row by row, gradients by the chain rule."""
    s = prepare(case, seed)
    op, n, d = case["op"], case["rows"], case["d"]
    f64 = torch.float64
    if op in ("head_loss", "head_grad"):
        w = s["lm_head"].to(f64)
        rows = (s["target"] >= 0).nonzero()[:, 0]
        tgt = s["target"][rows].long()
        nll = torch.zeros(n, dtype=f64, device="cuda")
        lse = torch.zeros_like(nll)
        gh = torch.zeros((n, d), dtype=f64, device="cuda")
        gw = torch.zeros_like(w)
        for a in range(0, len(rows), 1024):
            r, t = rows[a:a + 1024], tgt[a:a + 1024]
            h = s["hidden"][r].to(f64)
            z = torch.einsum("rd,vd->rv", h, w)
            if op == "head_loss":
                lse[r] = torch.logsumexp(z, dim=1)
                nll[r] = lse[r] - z[torch.arange(len(r), device="cuda"), t]
            else:
                p = torch.exp(z - s["lse"][r].to(f64)[:, None])
                p[torch.arange(len(r), device="cuda"), t] -= 1.0
                p = p * s["grad_nll"][r].to(f64)[:, None]
                gh[r] = torch.einsum("rv,vd->rd", p, w)
                gw += torch.einsum("rv,rd->vd", p, h)
        return (nll, lse) if op == "head_loss" else (gh, gw)
    if op in ("norm", "norm_grad"):
        x, gain = s["x"].to(f64), s["gain"].to(f64)
        if op == "norm":
            r = 1.0 / torch.sqrt((x * x).sum(dim=1) / d + EPS)
            return torch.einsum("rd,r,d->rd", x, r, gain), r
        r, gy = s["rstd"].to(f64), s["grad_y"].to(f64)
        xhat = x * r[:, None]
        u = gy * gain
        gx = r[:, None] * (u - xhat * (torch.einsum("rd,rd->r", u, xhat) / d)[:, None])
        if s["grad_add"] is not None:
            gx = gx + s["grad_add"].to(f64)
        return gx, torch.einsum("rd,rd->d", gy, xhat)
    ids = s["ids"].long()
    on = (ids >= 0).nonzero()[:, 0]
    if op == "embed":
        out = torch.zeros((n, d), dtype=f64, device="cuda")
        out[on] = s["table"].to(f64)[ids[on]] * case["scale"]
        return out
    # sums over each token's rows, taken from the rows in sorted order
    srt = ids[on].sort(stable=True)
    out = torch.zeros((case["table"], d), dtype=f64, device="cuda")
    if len(on):
        total = torch.cumsum(s["grad_rows"][on[srt.indices]].to(f64), dim=0)
        last = torch.ones(len(on), dtype=torch.bool, device="cuda")
        last[:-1] = srt.values[1:] != srt.values[:-1]
        ends = last.nonzero()[:, 0]
        seg = total[ends]
        seg[1:] -= total[ends[:-1]]
        out[srt.values[ends]] = seg * case["scale"]
    return out
