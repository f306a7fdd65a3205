"""Pointers off their element's boundary are refused by every entry point of the training form's
ends, on the host (a kernel that read or wrote them would fault)."""
import ctypes
import os

import pytest
import torch

import masked_discrete_diffusion_sparse_b200 as smdm

GOOD = 0x10000                        # never dereferenced: every call below is refused
WS = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(smdm.LIB_PATH):
        from masked_discrete_diffusion_sparse_b200 import build
        build.build()


def head(dtype):
    return ctypes.byref(smdm.smdm_head_shape(8, 64, 100, dtype, 64, 64))


def norm(xt, t):
    return ctypes.byref(smdm.smdm_rmsnorm_shape(8, 64, xt, t, 64, 64, 1e-6))


def embed(t, ot):
    return ctypes.byref(smdm.smdm_embed_shape(8, 64, 100, t, ot, 64, 1.0))


F, B = smdm.SMDM_F32, smdm.SMDM_BF16
# entry point, shape, pointers behind it as (name, element bytes) or a plain value
CALLS = [(e, s(*t), p(*t)) for e, s, ts, p in [
    ("smdm_head_loss", head, [(F,), (B,)], lambda t: [
        ("hidden", 4 if t == F else 2), ("lm_head", 4 if t == F else 16), ("target", 4), ("nll", 4),
        ("lse", 4), ("workspace", 256), WS, ("status", 4)]),
    ("smdm_head_loss_grad", head, [(F,), (B,)], lambda t: [
        ("hidden", 4 if t == F else 2), ("lm_head", 4 if t == F else 16), ("target", 4), ("lse", 4),
        ("grad_nll", 4), ("grad_hidden", 4 if t == F else 2), ("grad_lm_head", 4 if t == F else 2),
        ("workspace", 256), WS, ("status", 4)]),
    ("smdm_rmsnorm", norm, [(F, B), (B, F)], lambda x, t: [
        ("x", 4 if x == F else 2), ("gain", 4 if t == F else 2), ("y", 4 if t == F else 2),
        ("rstd", 4)]),
    ("smdm_rmsnorm_grad", norm, [(F, B), (B, F)], lambda x, t: [
        ("x", 4 if x == F else 2), ("gain", 4 if t == F else 2), ("rstd", 4),
        ("grad_y", 4 if t == F else 2), ("grad_add", 4 if x == F else 2),
        ("grad_x", 4 if x == F else 2), ("grad_gain", 4 if t == F else 2), ("workspace", 256), WS]),
    ("smdm_embed", embed, [(F, B), (B, F)], lambda t, o: [
        ("ids", 4), ("table", 4 if t == F else 2), ("out", 4 if o == F else 2), ("status", 4)]),
    ("smdm_embed_grad", embed, [(F, B), (B, F)], lambda t, o: [
        ("ids", 4), ("grad_out", 4 if o == F else 2), ("grad_table", 4 if t == F else 2),
        ("workspace", 256), WS, ("status", 4)]),
] for t in ts]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c[0])
def test_pointers_off_their_boundary_are_refused(call):
    entry, shape, params = call
    for i, p in enumerate(params):
        if not isinstance(p, tuple):
            continue
        name, size = p
        args = [GOOD if isinstance(q, tuple) else q for q in params]
        for shift in {1, size // 2}:
            args[i] = GOOD + shift
            r = getattr(smdm.lib(), entry)(shape, *args, None)
            assert r == smdm.SMDM_EINVAL, f"{entry}: {name} {shift} bytes off gives {r}"


def test_sizes_past_32_bits_are_refused_not_cut():
    for rows in (2 ** 32 + 8, 2 ** 31, -2 ** 32 + 8):
        with pytest.raises(smdm.SmdmError):
            smdm.smdm_head_loss_workspace_bytes(rows, 64, 100, torch.bfloat16)
        with pytest.raises(smdm.SmdmError):
            smdm.smdm_head_loss_workspace_bytes(8, 64, rows, torch.bfloat16)
        with pytest.raises(smdm.SmdmError):
            smdm.smdm_rmsnorm_grad_workspace_bytes(rows, 64)
        with pytest.raises(smdm.SmdmError):
            smdm.smdm_embed_grad_workspace_bytes(rows, 64, 100)
    assert smdm.smdm_head_loss_workspace_bytes(8, 64, 100, torch.bfloat16) > 0


def test_the_status_is_a_32_bit_integer():
    for bad in (torch.zeros(1), torch.zeros(1, dtype=torch.int64), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError, match="32-bit integer"):
            smdm._status(bad)
    with pytest.raises(ValueError, match="CUDA"):
        smdm._status(torch.zeros(1, dtype=torch.int32))


@pytest.mark.gpu
def test_loss_of_the_training_form_refuses_them_too():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import synth
    from smdm_testlib import config_for, upload_weights
    wl = synth.WORKLOADS["tiny-bf16-cos"]
    model = smdm.Model(config_for(wl, train_rows=64), upload_weights(synth.make_weights(wl.model, 1)))
    try:
        need = model.smdm_loss_stepcausal_workspace_bytes(8, grad=True)
        buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        good = buf.data_ptr()
        sizes = {"ids": 4, "pos": 4, "types": 4, "labels": 4, "rows": 4, "target": 4, "nll": 4,
                 "lse": 4, "grad_nll": 4, "grad_x": 4, "grad_final_norm": 2, "grad_lm_head": 2}
        for name, size in sizes.items():
            a = {k: good + (size // 2 if k == name else 0) for k in sizes}
            r = smdm.lib().smdm_loss_stepcausal(
                model.h, a["ids"], a["pos"], a["types"], a["labels"], 16, a["rows"], 8, a["target"],
                a["nll"], a["lse"], a["grad_nll"], a["grad_x"], a["grad_final_norm"],
                a["grad_lm_head"], ws.data_ptr(), need, None)
            assert r == smdm.SMDM_EINVAL, name
        torch.cuda.synchronize()
    finally:
        model.close()
