"""Argument checks of the training form's ends: refused on the host before any CUDA call (CPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import masked_discrete_diffusion_sparse_b200 as smdm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)       # never dereferenced: every call below is refused
OK_WS = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(smdm.LIB_PATH):
        from masked_discrete_diffusion_sparse_b200 import build
        build.build()


def at(offset):
    return ctypes.c_void_p(0x10000 + offset)


def head(rows=8, d=64, vocab=100, dtype=smdm.SMDM_BF16, ld_h=None, ld_w=None):
    return ctypes.byref(smdm.smdm_head_shape(rows, d, vocab, dtype, d if ld_h is None else ld_h,
                                             d if ld_w is None else ld_w))


def test_head_loss_refusals():
    L = smdm.lib()
    E, S, M = smdm.SMDM_EINVAL, smdm.SMDM_ESHAPE, smdm.SMDM_ENOMEM

    def loss(shape, h=FAKE, w=FAKE, t=FAKE, nll=FAKE, lse=FAKE, ws=FAKE, nb=OK_WS):
        return L.smdm_head_loss(shape, h, w, t, nll, lse, ws, nb, None, None)

    def grad(shape, h=FAKE, w=FAKE, t=FAKE, lse=FAKE, g=FAKE, gh=FAKE, gw=FAKE, ws=FAKE, nb=OK_WS):
        return L.smdm_head_loss_grad(shape, h, w, t, lse, g, gh, gw, ws, nb, None, None)

    for call in (loss, grad):
        assert call(None) == E
        assert call(head(dtype=7)) == E
        for bad in (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(d=0), dict(d=1 << 17),
                    dict(vocab=0), dict(vocab=(1 << 24) + 1)):
            assert call(head(**bad)) == S, bad
        assert call(head(ld_h=63)) == E and call(head(ld_w=63)) == E
        for missing in ("h", "w", "t", "ws", "lse"):
            assert call(head(), **{missing: None}) == E, missing
        assert call(head(), ws=at(16)) == E                  # 256-byte alignment
        assert call(head(), h=at(1)) == E                    # half an element
        assert call(head(), w=at(2)) == E                    # rows read in place need 16 bytes
        assert call(head(), nb=1000) == M
    assert loss(head(), nll=None) == E
    assert grad(head(), g=None) == E
    assert grad(head(), gh=None, gw=None) == E
    assert grad(head(), gw=at(1)) == E
    need = L.smdm_head_loss_workspace_bytes(head(), 1)
    assert need > 0 and grad(head(), nb=need - 1) == M
    assert L.smdm_head_loss_workspace_bytes(head(d=0), 0) == 0
    assert loss(head(rows=0), h=None, t=None, nll=None, lse=None) == smdm.SMDM_OK


def test_head_workspace_stays_bounded():
    """The gradient's workspace grows with rows x width, not with rows x vocabulary, once the
    logits' gradient of a piece reaches its limit of 256 MiB."""
    L = smdm.lib()
    small = L.smdm_head_loss_workspace_bytes(head(rows=16384, d=64, vocab=32768), 1)
    large = L.smdm_head_loss_workspace_bytes(head(rows=16384, d=64, vocab=1 << 20), 1)
    assert large < small + (300 << 20)
    assert large < 16384 * (1 << 20) * 2 // 8


def test_rmsnorm_refusals():
    L = smdm.lib()
    E, S, M = smdm.SMDM_EINVAL, smdm.SMDM_ESHAPE, smdm.SMDM_ENOMEM

    def shape(rows=4, d=64, xt=0, t=1, ld_x=None, ld_y=None, eps=1e-6):
        return ctypes.byref(smdm.smdm_rmsnorm_shape(rows, d, xt, t, ld_x or d, ld_y or d, eps))

    def fwd(s, x=FAKE, g=FAKE, y=FAKE):
        return L.smdm_rmsnorm(s, x, g, y, None, None)

    def bwd(s, x=FAKE, g=FAKE, r=FAKE, gy=FAKE, add=None, gx=FAKE, gg=FAKE, ws=FAKE, nb=OK_WS):
        return L.smdm_rmsnorm_grad(s, x, g, r, gy, add, gx, gg, ws, nb, None)

    for call in (fwd, bwd):
        assert call(None) == E
        assert call(shape(xt=2)) == E and call(shape(t=9)) == E
        assert call(shape(rows=-1)) == S and call(shape(d=0)) == S and call(shape(d=8193)) == S
        assert call(shape(ld_x=63)) == E and call(shape(ld_y=1)) == E
        assert call(shape(eps=-1.0)) == E and call(shape(eps=float("nan"))) == E
        assert call(shape(), x=None) == E and call(shape(), g=None) == E
        assert call(shape(), x=at(2)) == E
    assert fwd(shape(), y=None) == E
    for k in ("r", "gy", "gx", "gg", "ws"):
        assert bwd(shape(), **{k: None}) == E, k
    assert bwd(shape(), add=at(2)) == E
    assert bwd(shape(), nb=8) == M
    assert fwd(shape(rows=0), x=None, y=None) == smdm.SMDM_OK


def test_embed_refusals():
    L = smdm.lib()
    E, S, M = smdm.SMDM_EINVAL, smdm.SMDM_ESHAPE, smdm.SMDM_ENOMEM

    def shape(rows=4, d=64, n=10, t=1, ot=0, ld=None):
        return ctypes.byref(smdm.smdm_embed_shape(rows, d, n, t, ot, ld or d, 1.0))

    def fwd(s, i=FAKE, t=FAKE, o=FAKE):
        return L.smdm_embed(s, i, t, o, None, None)

    def bwd(s, i=FAKE, t=FAKE, o=FAKE, ws=FAKE, nb=OK_WS):
        return L.smdm_embed_grad(s, i, o, t, ws, nb, None, None)

    for call in (fwd, bwd):
        assert call(None) == E
        assert call(shape(t=3)) == E and call(shape(ot=-1)) == E and call(shape(ld=1)) == E
        assert call(shape(rows=-1)) == S and call(shape(d=0)) == S and call(shape(n=0)) == S
        assert call(shape(n=(1 << 24) + 1)) == S
        assert call(shape(), i=None) == E and call(shape(), t=None) == E
        assert call(shape(), o=None) == E
        assert call(shape(), t=at(1)) == E and call(shape(), o=at(2)) == E
    assert bwd(shape(), ws=None) == E and bwd(shape(), ws=at(128)) == E
    assert bwd(shape(), nb=16) == M
    assert fwd(shape(rows=0), i=None, o=None) == smdm.SMDM_OK


def test_loss_stepcausal_refusals():
    L = smdm.lib()
    assert L.smdm_loss_stepcausal(None, *[FAKE] * 4, 1, FAKE, 1, *[FAKE] * 8, OK_WS, None) == \
        smdm.SMDM_EINVAL
    cfg = smdm.make_config(2, 256, 2, 128, 704, 1000, dtype=smdm.SMDM_BF16, max_batch=1,
                           max_len=300, max_step_rows=200, max_rows=300)
    need = [L.smdm_loss_stepcausal_workspace_bytes(ctypes.byref(cfg), 100, g) for g in (0, 1)]
    assert 0 < need[0] < need[1]
    for n in (0, -1, 301):
        assert L.smdm_loss_stepcausal_workspace_bytes(ctypes.byref(cfg), n, 0) == 0


def test_binding_checks_tensors_before_the_call():
    """Shapes, types, strides and devices that the binding refuses (nothing is launched)."""
    h = torch.zeros((4, 8))
    t = torch.zeros(4, dtype=torch.int32)
    ws = torch.zeros(8, dtype=torch.uint8)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        smdm.smdm_head_loss(h, h, t, f, f, ws)
    with pytest.raises(ValueError, match="share"):
        smdm.smdm_head_loss(h, h.bfloat16(), t, f, f, ws)
    with pytest.raises(ValueError, match="contiguous"):
        smdm.smdm_rmsnorm(torch.zeros((8, 4)).T, torch.zeros(8), h)
    with pytest.raises(ValueError, match="overlap"):
        smdm.smdm_rmsnorm(torch.zeros(8).expand(4, 8), torch.zeros(8), h)
    with pytest.raises(ValueError, match="2-D"):
        smdm.smdm_embed(t, torch.zeros(8), h)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        smdm.smdm_head_loss_workspace_bytes(4, 8, 8, torch.float16)
    with pytest.raises(smdm.SmdmError):
        smdm.smdm_head_loss_workspace_bytes(-4, 8, 8, torch.float32)


def test_shape_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    structs = {c.__name__: c for c in (smdm.smdm_head_shape, smdm.smdm_rmsnorm_shape,
                                       smdm.smdm_embed_shape)}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "smdm.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'  printf("%zu\\n", sizeof({name}));')
        lines += [f'  printf("%zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), "-I", cuda_inc, str(src), "-o",
                    str(exe)], check=True)
    got = iter(subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    for cls in structs.values():
        assert int(next(got)) == ctypes.sizeof(cls)
        for f in cls._fields_:
            assert int(next(got)) == getattr(cls, f[0]).offset, f[0]
