"""Sparse masked-diffusion sampling on B200 (sm_100a).

Python binding of the C ABI in ``include/smdm.h`` (library ``libsmdm.so`` in this package).
The binding only marshals arguments: torch supplies device memory and streams, every step of
the computation runs in the library's CUDA kernels.  There is no CPU fallback: importing works
anywhere, but creating a model raises if the library is not built or no GPU is present.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsmdm.so")

# --- constants mirrored from smdm.h ----------------------------------------------------------
SMDM_OK, SMDM_EINVAL, SMDM_ESHAPE, SMDM_ENOMEM, SMDM_ECUDA, SMDM_ESTATE, SMDM_ETIMEOUT, \
    SMDM_EDEVICE = range(8)
SMDM_F32, SMDM_BF16 = 0, 1
SMDM_POLICY_ALL, SMDM_POLICY_TOPN = 0, 1
SMDM_MODE_SPARSE, SMDM_MODE_DENSE = 0, 1
SMDM_TYPE_PROMPT, SMDM_TYPE_CLEAN, SMDM_TYPE_MASK, SMDM_TYPE_REG = range(4)
SMDM_PLAN_ORDER, SMDM_PLAN_SEMIAR = 0, 1
SMDM_MAX_BATCH = 8
SMDM_REG_LEN = -1      # n_reg of the length-token variant (one [LEN] row, no registers)
SMDM_SW_CACHE_PROMPT, SMDM_SW_CACHE_RES, SMDM_SW_TRUNCATE, SMDM_SW_ALL = 1, 2, 4, 7

STATUS_NAMES = {0: "SMDM_OK", 1: "SMDM_EINVAL", 2: "SMDM_ESHAPE", 3: "SMDM_ENOMEM",
                4: "SMDM_ECUDA", 5: "SMDM_ESTATE", 6: "SMDM_ETIMEOUT", 7: "SMDM_EDEVICE"}

EXPORTED = ["smdm_workspace_bytes", "smdm_create", "smdm_destroy", "smdm_last_error",
            "smdm_prefill", "smdm_prefill_given", "smdm_step", "smdm_step_switched",
            "smdm_dense_step", "smdm_generate",
            "smdm_forward_stepcausal", "smdm_debug_mask", "smdm_debug_rows",
            "smdm_context_length", "smdm_device_status", "smdm_profile_begin",
            "smdm_profile_end", "smdm_forward_stepcausal_noalloc",
            "smdm_head_loss_workspace_bytes", "smdm_head_loss", "smdm_head_loss_grad",
            "smdm_rmsnorm", "smdm_rmsnorm_grad_workspace_bytes", "smdm_rmsnorm_grad",
            "smdm_embed", "smdm_embed_grad_workspace_bytes", "smdm_embed_grad",
            "smdm_loss_stepcausal_workspace_bytes", "smdm_loss_stepcausal"]

K_CLASSES = ["pack", "norm", "gemm_qkv", "attn", "gemm_o", "gemm_gateup", "gemm_down",
             "gemm_lmhead", "unmask", "other"]


class SmdmError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class smdm_config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("d_model", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("d_head", ctypes.c_int), ("d_ffn", ctypes.c_int), ("vocab", ctypes.c_int),
                ("n_reg", ctypes.c_int), ("dtype", ctypes.c_int), ("rope_theta", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("max_batch", ctypes.c_int),
                ("max_len", ctypes.c_int), ("max_step_rows", ctypes.c_int),
                ("max_rows", ctypes.c_int)]


_PP = ctypes.POINTER(ctypes.c_void_p)


class smdm_weights(ctypes.Structure):
    _fields_ = [("emb", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p), ("attn_norm", _PP), ("w_qkv", _PP), ("w_o", _PP),
                ("mlp_norm", _PP), ("w_gate", _PP), ("w_up", _PP), ("w_down", _PP)]


class smdm_step_desc(ctypes.Structure):
    _fields_ = [("seq", ctypes.c_int), ("d_query_pos", ctypes.c_void_p),
                ("n_query", ctypes.c_int), ("block_lo", ctypes.c_int), ("block_hi", ctypes.c_int),
                ("policy", ctypes.c_int), ("n_commit", ctypes.c_int)]


class smdm_plan(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("n_steps", ctypes.c_int),
                ("h_n_per_step", ctypes.POINTER(ctypes.c_int32)), ("d_order", ctypes.c_void_p),
                ("block", ctypes.c_int), ("steps_per_block", ctypes.c_int),
                ("commit", ctypes.c_int), ("h_block_order", ctypes.POINTER(ctypes.c_int32))]


class smdm_profile(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_ulonglong), ("class_launches", ctypes.c_ulonglong * 10),
                ("class_ms", ctypes.c_double * 10)]


class smdm_head_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("d_model", ctypes.c_int), ("vocab", ctypes.c_int),
                ("dtype", ctypes.c_int), ("ld_hidden", ctypes.c_longlong),
                ("ld_head", ctypes.c_longlong)]


class smdm_rmsnorm_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("d_model", ctypes.c_int), ("x_dtype", ctypes.c_int),
                ("dtype", ctypes.c_int), ("ld_x", ctypes.c_longlong),
                ("ld_y", ctypes.c_longlong), ("eps", ctypes.c_float)]


class smdm_embed_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("d_model", ctypes.c_int), ("n_emb", ctypes.c_int),
                ("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("ld", ctypes.c_longlong),
                ("scale", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libsmdm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m masked_discrete_diffusion_sparse_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int
    L.smdm_workspace_bytes.argtypes = [ctypes.POINTER(smdm_config)]
    L.smdm_workspace_bytes.restype = ctypes.c_size_t
    L.smdm_create.argtypes = [ctypes.POINTER(smdm_config), ctypes.POINTER(smdm_weights), vp,
                              ctypes.c_size_t, ctypes.POINTER(vp)]
    L.smdm_create.restype = st
    L.smdm_destroy.argtypes = [vp]
    L.smdm_destroy.restype = None
    L.smdm_last_error.argtypes = [vp]
    L.smdm_last_error.restype = ctypes.c_char_p
    L.smdm_prefill.argtypes = [vp, i32, vp, i32, i32, vp, vp]
    L.smdm_prefill.restype = st
    L.smdm_prefill_given.argtypes = [vp, i32, vp, i32, i32, vp, vp, i32, vp, vp]
    L.smdm_prefill_given.restype = st
    L.smdm_step.argtypes = [vp, i32, ctypes.POINTER(smdm_step_desc), vp, vp, vp, vp]
    L.smdm_step.restype = st
    L.smdm_step_switched.argtypes = [vp, ctypes.POINTER(smdm_step_desc), i32, vp, vp, vp, vp]
    L.smdm_step_switched.restype = st
    L.smdm_dense_step.argtypes = [vp, ctypes.POINTER(smdm_step_desc), vp, vp, vp, vp]
    L.smdm_dense_step.restype = st
    L.smdm_generate.argtypes = [vp, i32, vp, i32, i32, ctypes.POINTER(smdm_plan), i32, vp, vp]
    L.smdm_generate.restype = st
    L.smdm_forward_stepcausal.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, vp, vp]
    L.smdm_forward_stepcausal.restype = st
    L.smdm_debug_mask.argtypes = [vp, vp, vp, i32, vp, vp]
    L.smdm_debug_mask.restype = st
    L.smdm_debug_rows.argtypes = [vp, vp, vp, vp, vp, ctypes.POINTER(ctypes.c_int), vp]
    L.smdm_debug_rows.restype = st
    L.smdm_context_length.argtypes = [vp, i32]
    L.smdm_context_length.restype = ctypes.c_int
    L.smdm_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint), vp]
    L.smdm_device_status.restype = st
    L.smdm_profile_begin.argtypes = [vp, i32]
    L.smdm_profile_begin.restype = st
    L.smdm_profile_end.argtypes = [vp, ctypes.POINTER(smdm_profile), vp]
    L.smdm_profile_end.restype = st
    L.smdm_forward_stepcausal_noalloc.argtypes = [ctypes.POINTER(smdm_config),
                                                  ctypes.POINTER(smdm_weights), vp, vp, vp, vp,
                                                  i32, vp, i32, vp, vp]
    L.smdm_forward_stepcausal_noalloc.restype = st
    sz = ctypes.c_size_t
    hs, ns, es = (ctypes.POINTER(t) for t in (smdm_head_shape, smdm_rmsnorm_shape,
                                              smdm_embed_shape))
    for name, args, res in [
            ("smdm_head_loss_workspace_bytes", [hs, i32], sz),
            ("smdm_head_loss", [hs, vp, vp, vp, vp, vp, vp, sz, vp, vp], st),
            ("smdm_head_loss_grad", [hs, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp], st),
            ("smdm_rmsnorm", [ns, vp, vp, vp, vp, vp], st),
            ("smdm_rmsnorm_grad_workspace_bytes", [ns], sz),
            ("smdm_rmsnorm_grad", [ns, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], st),
            ("smdm_embed", [es, vp, vp, vp, vp, vp], st),
            ("smdm_embed_grad_workspace_bytes", [es], sz),
            ("smdm_embed_grad", [es, vp, vp, vp, vp, sz, vp, vp], st),
            ("smdm_loss_stepcausal_workspace_bytes", [ctypes.POINTER(smdm_config), i32, i32], sz),
            ("smdm_loss_stepcausal", [vp, vp, vp, vp, vp, i32, vp, i32] + [vp] * 8 + [sz, vp],
             st)]:
        getattr(L, name).argtypes = args
        getattr(L, name).restype = res
    _lib = L
    return L


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _i32(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.int32:
        raise ValueError("expected an int32 tensor")
    return t


class Model:
    """A handle plus the device memory it borrows.

    weights: dict with 'emb', 'final_norm', 'lm_head' and per-layer lists 'attn_norm', 'w_qkv',
    'w_o', 'mlp_norm', 'w_gate', 'w_up', 'w_down' (torch CUDA tensors in the model dtype, linear
    weights [out][in]).  Methods mirror the C entry points of the same name.
    """

    def __init__(self, cfg: smdm_config, weights: dict, device: str = "cuda"):
        L = lib()
        if not torch.cuda.is_available():
            raise RuntimeError("the sparse sampler needs a CUDA device (no CPU fallback)")
        self.cfg = cfg
        self.weights = weights
        self._layer_arrays = {}
        arr = {}
        for k in ("attn_norm", "w_qkv", "w_o", "mlp_norm", "w_gate", "w_up", "w_down"):
            ts = weights[k]
            a = (ctypes.c_void_p * cfg.n_layers)(*[t.data_ptr() for t in ts])
            self._layer_arrays[k] = a
            arr[k] = ctypes.cast(a, _PP)
        self._w = smdm_weights(weights["emb"].data_ptr(), weights["final_norm"].data_ptr(),
                               weights["lm_head"].data_ptr(), arr["attn_norm"], arr["w_qkv"],
                               arr["w_o"], arr["mlp_norm"], arr["w_gate"], arr["w_up"],
                               arr["w_down"])
        nbytes = L.smdm_workspace_bytes(ctypes.byref(cfg))
        if nbytes == 0:
            raise SmdmError(SMDM_ESHAPE, "invalid configuration")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        torch.cuda.synchronize()
        h = ctypes.c_void_p()
        s = L.smdm_create(ctypes.byref(cfg), ctypes.byref(self._w),
                          ctypes.c_void_p(self.workspace.data_ptr()), nbytes, ctypes.byref(h))
        if s != SMDM_OK:
            raise SmdmError(s, "smdm_create failed")
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            lib().smdm_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, s: int):
        if s != SMDM_OK:
            raise SmdmError(s, lib().smdm_last_error(self.h).decode())

    # -- entry points -------------------------------------------------------------------------
    def smdm_prefill(self, seq: int, prompt: torch.Tensor, gen_len: int, grid: torch.Tensor,
                     stream=None):
        self._check(lib().smdm_prefill(self.h, seq, _ptr(_i32(prompt)) if prompt.numel() else None,
                                       prompt.numel(), gen_len, _ptr(_i32(grid)), _stream(stream)))

    def smdm_prefill_given(self, seq: int, prompt: torch.Tensor, gen_len: int,
                           given_pos: torch.Tensor, given_tok: torch.Tensor, grid: torch.Tensor,
                           stream=None):
        """Prefill with given generation tokens (bidirectional tasks): 1-based absolute
        positions and their token ids, device int32 tensors of equal length."""
        if given_pos.numel() != given_tok.numel():
            raise ValueError("given_pos and given_tok differ in length")
        n = given_pos.numel()
        self._check(lib().smdm_prefill_given(
            self.h, seq, _ptr(_i32(prompt)) if prompt.numel() else None, prompt.numel(), gen_len,
            _ptr(_i32(given_pos)) if n else None, _ptr(_i32(given_tok)) if n else None, n,
            _ptr(_i32(grid)), _stream(stream)))

    def smdm_step(self, descs: Sequence[dict], logits: Optional[torch.Tensor] = None,
                  tok: Optional[torch.Tensor] = None, conf: Optional[torch.Tensor] = None,
                  stream=None):
        """descs: dicts with seq, query_pos (int32 CUDA tensor or None), n_query, block_lo,
        block_hi, policy, n_commit."""
        arr = (smdm_step_desc * len(descs))()
        for i, d in enumerate(descs):
            qp = d.get("query_pos")
            arr[i] = smdm_step_desc(d["seq"], _ptr(_i32(qp)) if qp is not None else None,
                                    d["n_query"], d.get("block_lo", 0), d.get("block_hi", 0),
                                    d.get("policy", SMDM_POLICY_ALL), d.get("n_commit", 0))
        self._check(lib().smdm_step(self.h, len(descs), arr, _ptr(logits), _ptr(tok), _ptr(conf),
                                    _stream(stream)))

    def smdm_step_switched(self, desc: dict, switches: int, logits=None, tok=None, conf=None,
                           stream=None):
        """One step of one sequence with the Table-6 speed switches (SMDM_SW_* bits); desc as
        in smdm_step, with query_pos required."""
        qp = desc["query_pos"]
        d = smdm_step_desc(desc["seq"], _ptr(_i32(qp)), desc["n_query"], 0, 0,
                           desc.get("policy", SMDM_POLICY_ALL), desc.get("n_commit", 0))
        self._check(lib().smdm_step_switched(self.h, ctypes.byref(d), switches, _ptr(logits),
                                             _ptr(tok), _ptr(conf), _stream(stream)))

    def smdm_dense_step(self, desc: dict, logits=None, tok=None, conf=None, stream=None):
        qp = desc.get("query_pos")
        d = smdm_step_desc(desc["seq"], _ptr(_i32(qp)) if qp is not None else None,
                           desc["n_query"], desc.get("block_lo", 0), desc.get("block_hi", 0),
                           desc.get("policy", SMDM_POLICY_ALL), desc.get("n_commit", 0))
        self._check(lib().smdm_dense_step(self.h, ctypes.byref(d), _ptr(logits), _ptr(tok),
                                          _ptr(conf), _stream(stream)))

    def smdm_generate(self, prompts: torch.Tensor, gen_len: int, plans: Sequence[dict],
                      grids: torch.Tensor, mode: int = SMDM_MODE_SPARSE, stream=None):
        """plans: dicts with kind, n_steps, n_per_step (host int list), order (int32 CUDA
        tensor), block, steps_per_block, commit, block_order (host int list, optional)."""
        B = len(plans)
        arr = (smdm_plan * B)()
        keep = []
        for i, p in enumerate(plans):
            nps = p.get("n_per_step")
            h_n = None
            if nps is not None:
                h_n = (ctypes.c_int32 * len(nps))(*[int(v) for v in nps])
                keep.append(h_n)
            bo = p.get("block_order")
            h_bo = None
            if bo is not None:
                h_bo = (ctypes.c_int32 * len(bo))(*[int(v) for v in bo])
                keep.append(h_bo)
            order = p.get("order")
            arr[i] = smdm_plan(p["kind"], p["n_steps"],
                               ctypes.cast(h_n, ctypes.POINTER(ctypes.c_int32)) if h_n else None,
                               _ptr(_i32(order)) if order is not None else None,
                               p.get("block", 0), p.get("steps_per_block", 0), p.get("commit", 0),
                               ctypes.cast(h_bo, ctypes.POINTER(ctypes.c_int32)) if h_bo else None)
        P = prompts.shape[-1] if prompts.numel() else 0
        self._check(lib().smdm_generate(self.h, B, _ptr(_i32(prompts)) if P else None, P, gen_len,
                                        arr, mode, _ptr(_i32(grids)), _stream(stream)))

    def smdm_forward_stepcausal(self, ids, pos, types, labels, logit_rows, logits, stream=None):
        self._check(lib().smdm_forward_stepcausal(
            self.h, _ptr(_i32(ids)), _ptr(_i32(pos)), _ptr(_i32(types)), _ptr(_i32(labels)),
            ids.numel(), _ptr(_i32(logit_rows)), logit_rows.numel(), _ptr(logits),
            _stream(stream)))

    def smdm_loss_stepcausal(self, ids, pos, types, labels, loss_rows, target, nll, lse, workspace,
                             grad_nll=None, grad_x=None, grad_final_norm=None, grad_lm_head=None,
                             stream=None):
        """Training-form forward over the step-labelled rows, then the cross entropy of the rows
        in loss_rows against target (int32, negative: takes no part) into nll and lse (fp32).
        With grad_nll (fp32, the loss weight of every row) also the gradients through the head:
        grad_x (fp32 [n_rows][d_model]), grad_final_norm and grad_lm_head (model dtype).
        workspace: uint8 tensor of smdm_loss_stepcausal_workspace_bytes."""
        m = _count(loss_rows.numel())
        d, v = self.cfg.d_model, self.cfg.vocab
        dt = torch.float32 if self.cfg.dtype == SMDM_F32 else torch.bfloat16
        for t in (pos, types, labels):
            _shape(t, (ids.numel(),), "pos / types / labels")
        for name, t, shape, want in (
                ("target", target, (m,), torch.int32), ("nll", nll, (m,), torch.float32),
                ("lse", lse, (m,), torch.float32), ("grad_nll", grad_nll, (m,), torch.float32),
                ("grad_x", grad_x, (m, d), torch.float32),
                ("grad_final_norm", grad_final_norm, (d,), dt),
                ("grad_lm_head", grad_lm_head, (v, d), dt)):
            if t is not None:
                _shape(t, shape, name)
                _typed(t, want, name)
        if stream is not None and stream != torch.cuda.current_stream(stream.device):
            # (the allocator must not hand their memory out while the kernels run)
            for t in (ids, pos, types, labels, loss_rows, target, nll, lse, grad_nll, grad_x,
                      grad_final_norm, grad_lm_head, workspace):
                if t is not None and t.is_cuda:
                    t.record_stream(stream)
        self._check(lib().smdm_loss_stepcausal(
            self.h, _ptr(_i32(ids)), _ptr(_i32(pos)), _ptr(_i32(types)), _ptr(_i32(labels)),
            _count(ids.numel()), _ptr(_i32(loss_rows)), m, _ptr(target), _ptr(nll), _ptr(lse),
            _ptr(grad_nll), _ptr(grad_x), _ptr(grad_final_norm), _ptr(grad_lm_head),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))

    def smdm_loss_stepcausal_workspace_bytes(self, n_rows: int, grad: bool = False) -> int:
        return _bytes(lib().smdm_loss_stepcausal_workspace_bytes(
            ctypes.byref(self.cfg), _count(n_rows), 1 if grad else 0))

    def smdm_debug_mask(self, types, labels, bitmap, stream=None):
        self._check(lib().smdm_debug_mask(self.h, _ptr(_i32(types)), _ptr(_i32(labels)),
                                          types.numel(), _ptr(bitmap), _stream(stream)))

    def smdm_debug_rows(self, ids=None, pos=None, types=None, labels=None, stream=None) -> int:
        n = ctypes.c_int(0)
        self._check(lib().smdm_debug_rows(self.h, _ptr(ids), _ptr(pos), _ptr(types), _ptr(labels),
                                          ctypes.byref(n), _stream(stream)))
        return n.value

    def smdm_context_length(self, seq: int) -> int:
        return lib().smdm_context_length(self.h, seq)

    def smdm_profile_begin(self, timed: bool = False):
        self._check(lib().smdm_profile_begin(self.h, 1 if timed else 0))

    def smdm_profile_end(self, stream=None) -> dict:
        p = smdm_profile()
        self._check(lib().smdm_profile_end(self.h, ctypes.byref(p), _stream(stream)))
        return {"launches": int(p.launches),
                "class_launches": {K_CLASSES[i]: int(p.class_launches[i]) for i in range(10)},
                "class_ms": {K_CLASSES[i]: float(p.class_ms[i]) for i in range(10)}}

    def smdm_device_status(self, stream=None) -> int:
        bits = ctypes.c_uint(0)
        self._check(lib().smdm_device_status(self.h, ctypes.byref(bits), _stream(stream)))
        return bits.value


def smdm_forward_stepcausal_noalloc(cfg: smdm_config, weights: dict, ids, pos, types, labels,
                                    logit_rows, logits, stream=None):
    """Training-form forward without a handle and without any device allocation.

    For callers that may not allocate device memory at the point of the call (a frozen
    allocator, a plug-in handed only pointers by its host program): all scratch lives in a
    16 MiB array built into the library.  Same arguments and result as
    Model.smdm_forward_stepcausal, plus the config and the weights dict.  Shapes whose scratch
    does not fit raise SmdmError(SMDM_ESHAPE).  Calls share that array: do not overlap them on
    the GPU.  Make the first call on a device outside CUDA-graph capture (it looks up the
    array's device address).
    """
    keep = []
    arr = {}
    for k in ("attn_norm", "w_qkv", "w_o", "mlp_norm", "w_gate", "w_up", "w_down"):
        a = (ctypes.c_void_p * cfg.n_layers)(*[t.data_ptr() for t in weights[k]])
        keep.append(a)
        arr[k] = ctypes.cast(a, _PP)
    w = smdm_weights(weights["emb"].data_ptr(), weights["final_norm"].data_ptr(),
                     weights["lm_head"].data_ptr(), arr["attn_norm"], arr["w_qkv"], arr["w_o"],
                     arr["mlp_norm"], arr["w_gate"], arr["w_up"], arr["w_down"])
    s = lib().smdm_forward_stepcausal_noalloc(
        ctypes.byref(cfg), ctypes.byref(w), _ptr(_i32(ids)), _ptr(_i32(pos)), _ptr(_i32(types)),
        _ptr(_i32(labels)), ids.numel(), _ptr(_i32(logit_rows)), logit_rows.numel(),
        _ptr(logits), _stream(stream))
    if s != SMDM_OK:
        raise SmdmError(s, "smdm_forward_stepcausal_noalloc failed")


# --- the training form's ends (no handle) -----------------------------------------------------
_DTYPES = {torch.float32: SMDM_F32, torch.bfloat16: SMDM_BF16}


def _dtype(dt) -> int:
    """SMDM_* constant of a torch dtype (or of itself)."""
    c = _DTYPES.get(dt)
    if c is None:
        if not isinstance(dt, int) or dt not in (SMDM_F32, SMDM_BF16):
            raise ValueError(f"expected float32 or bfloat16, got {dt}")
        c = dt
    return c


def _count(n: int) -> int:
    if not -2 ** 31 <= n < 2 ** 31:
        raise SmdmError(SMDM_ESHAPE, f"{n} elements")
    return n


def _struct(t, *a):
    """A shape struct; a size that its field cannot hold is refused, not cut."""
    for (_, kind), v in zip(t._fields_, a):
        if kind is ctypes.c_int:
            _count(v)
    return ctypes.byref(t(*a))


# Shape arguments of recent calls: building one takes as long as the call that it is passed to.
_head_struct, _norm_struct, _embed_struct = (
    functools.lru_cache(maxsize=256)(functools.partial(_struct, t))
    for t in (smdm_head_shape, smdm_rmsnorm_shape, smdm_embed_shape))


def _typed(t: torch.Tensor, dt: torch.dtype, name: str):
    if t.dtype != dt:
        raise ValueError(f"{name}: expected {dt}, got {t.dtype}")


def _shape(t: torch.Tensor, shape: tuple, name: str):
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _bytes(n: int) -> int:
    if n == 0:
        raise SmdmError(SMDM_ESHAPE, "invalid shape")
    return n


def _adr(t: Optional[torch.Tensor], name: str):
    """Address of a contiguous CUDA tensor (None stays None)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str):
    """Address and row stride of a 2-D CUDA tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    n, d = t.shape
    ld, step = t.stride()
    if d > 1 and step != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if n < 2:
        ld = d
    if ld < d:
        raise ValueError(f"{name}: rows overlap")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    return t.data_ptr(), ld


def _call(fn: str, stream, tensors, *args):
    """Run one entry point on the tensors' device and the given (or that device's current)
    stream; a tensor used on another stream than the current one is recorded there, so that the
    allocator does not hand its memory out while the kernels run."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")
    f = getattr(_lib or lib(), fn)
    if stream is None and dev == torch.cuda.current_device():
        r = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        if stream is not None and stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        with torch.cuda.device(dev):
            cur = torch.cuda.current_stream(dev)
            s = cur if stream is None else stream
            if s != cur:
                for t in tensors:
                    if t is not None:
                        t.record_stream(s)
            r = f(*args, s.cuda_stream)
    if r != SMDM_OK:
        raise SmdmError(r, f"{fn} failed")


def _status(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if t.numel() < 1 or t.dtype not in (torch.int32, torch.uint32):
        raise ValueError("status: expected a 32-bit integer tensor of one element")
    return _adr(t, "status")


def _ws(t: torch.Tensor):
    return _adr(t, "workspace"), t.nbytes


def _head_shape(hidden, lm_head, target):
    if lm_head.dtype != hidden.dtype:
        raise ValueError("hidden and lm_head must share their dtype")
    h, ld_h = _rows(hidden, "hidden")
    w, ld_w = _rows(lm_head, "lm_head")
    n, d = hidden.shape
    if lm_head.shape[1] != d:
        raise ValueError("hidden and lm_head must share their width")
    _shape(target, (n,), "target")
    v = lm_head.shape[0]
    return _head_struct(n, d, v, _dtype(hidden.dtype), ld_h, ld_w), h, w, n, d, v


def smdm_head_loss_workspace_bytes(rows: int, d_model: int, vocab: int, dtype,
                                   grad: bool = False) -> int:
    """dtype: torch.float32, torch.bfloat16 or the SMDM_* constant."""
    s = _head_struct(rows, d_model, vocab, _dtype(dtype), d_model, d_model)
    return _bytes(lib().smdm_head_loss_workspace_bytes(s, 1 if grad else 0))


def smdm_head_loss(hidden, lm_head, target, nll, lse, workspace, status=None, stream=None):
    """Cross entropy of the LM head without its logits: hidden [R][d] and lm_head [V][d] (float32
    or bfloat16, rows may lie apart), target int32 [R] (negative: the row takes no part) ->
    nll, lse (fp32 [R])."""
    s, h, w, n, _, _ = _head_shape(hidden, lm_head, target)
    for name, t in (("nll", nll), ("lse", lse)):
        _shape(t, (n,), name)
        _typed(t, torch.float32, name)
    ws, nb = _ws(workspace)
    _call("smdm_head_loss", stream, (hidden, lm_head, target, nll, lse, workspace, status), s, h,
          w, _adr(_i32(target), "target"), _adr(nll, "nll"), _adr(lse, "lse"), ws, nb,
          _status(status))


def smdm_head_loss_grad(hidden, lm_head, target, lse, grad_nll, grad_hidden, grad_lm_head,
                        workspace, status=None, stream=None):
    """Gradient of smdm_head_loss: lse from it and grad_nll (fp32 [R], the rows' weights) ->
    grad_hidden [R][d] and grad_lm_head [V][d] in hidden's dtype (either may be None)."""
    s, h, w, n, d, v = _head_shape(hidden, lm_head, target)
    for name, t in (("lse", lse), ("grad_nll", grad_nll)):
        _shape(t, (n,), name)
        _typed(t, torch.float32, name)
    for name, t, shape in (("grad_hidden", grad_hidden, (n, d)),
                           ("grad_lm_head", grad_lm_head, (v, d))):
        if t is not None:
            _shape(t, shape, name)
            _typed(t, hidden.dtype, name)
    ws, nb = _ws(workspace)
    _call("smdm_head_loss_grad", stream,
          (hidden, lm_head, target, lse, grad_nll, grad_hidden, grad_lm_head, workspace, status),
          s, h, w, _adr(_i32(target), "target"), _adr(lse, "lse"), _adr(grad_nll, "grad_nll"),
          _adr(grad_hidden, "grad_hidden"), _adr(grad_lm_head, "grad_lm_head"), ws, nb,
          _status(status))


def smdm_rmsnorm(x, gain, y, rstd=None, eps: float = 1e-6, stream=None):
    """y = x rstd gain, rstd = (mean x^2 + eps)^(-1/2): x [R][d] and y [R][d] (rows may lie
    apart), gain [d] in y's dtype, rstd fp32 [R] (optional, for the gradient)."""
    px, ld_x = _rows(x, "x")
    py, ld_y = _rows(y, "y")
    _shape(y, x.shape, "y")
    _shape(gain, (x.shape[1],), "gain")
    _typed(gain, y.dtype, "gain")
    if rstd is not None:
        _shape(rstd, (x.shape[0],), "rstd")
        _typed(rstd, torch.float32, "rstd")
    n, d = x.shape
    s = _norm_struct(n, d, _dtype(x.dtype), _dtype(y.dtype), ld_x, ld_y, eps)
    _call("smdm_rmsnorm", stream, (x, gain, y, rstd), s, px, _adr(gain, "gain"), py,
          _adr(rstd, "rstd"))


def smdm_rmsnorm_grad_workspace_bytes(rows: int, d_model: int) -> int:
    s = _norm_struct(rows, d_model, SMDM_F32, SMDM_F32, d_model, d_model, 0.0)
    return _bytes(lib().smdm_rmsnorm_grad_workspace_bytes(s))


def smdm_rmsnorm_grad(x, gain, rstd, grad_y, grad_x, grad_gain, workspace, grad_add=None,
                      stream=None):
    """Gradient of smdm_rmsnorm: grad_x [R][d] in x's dtype (plus grad_add, the gradient that
    reaches x past the norm; the two may be one tensor) and grad_gain [d]."""
    px, ld_x = _rows(x, "x")
    pg, ld_y = _rows(grad_y, "grad_y")
    n, d = x.shape
    _shape(grad_y, (n, d), "grad_y")
    for name, t, shape, want in (
            ("gain", gain, (d,), grad_y.dtype), ("grad_gain", grad_gain, (d,), grad_y.dtype),
            ("rstd", rstd, (n,), torch.float32), ("grad_x", grad_x, (n, d), x.dtype),
            ("grad_add", grad_add, (n, d), x.dtype)):
        if t is not None:
            _shape(t, shape, name)
            _typed(t, want, name)
    s = _norm_struct(n, d, _dtype(x.dtype), _dtype(grad_y.dtype), ld_x, ld_y, 0.0)
    ws, nb = _ws(workspace)
    _call("smdm_rmsnorm_grad", stream,
          (x, gain, rstd, grad_y, grad_x, grad_gain, workspace, grad_add), s, px,
          _adr(gain, "gain"), _adr(rstd, "rstd"), pg, _adr(grad_add, "grad_add"), _adr(grad_x, "grad_x"), _adr(grad_gain, "grad_gain"), ws, nb)


def smdm_embed(ids, table, out, scale: float = 1.0, status=None, stream=None):
    """out[i] = scale * table[ids[i]] (float32 or bfloat16 each); a negative id gives zeros."""
    pt, ld = _rows(table, "table")
    _shape(ids, (out.shape[0],), "ids")
    _shape(out, (out.shape[0], table.shape[1]), "out")
    n_emb, d = table.shape
    s = _embed_struct(ids.numel(), d, n_emb, _dtype(table.dtype), _dtype(out.dtype), ld, scale)
    _call("smdm_embed", stream, (ids, table, out, status), s, _adr(_i32(ids), "ids"), pt,
          _adr(out, "out"), _status(status))


def smdm_embed_grad_workspace_bytes(rows: int, d_model: int, n_emb: int) -> int:
    s = _embed_struct(rows, d_model, n_emb, SMDM_F32, SMDM_F32, d_model, 1.0)
    return _bytes(lib().smdm_embed_grad_workspace_bytes(s))


def smdm_embed_grad(ids, grad_out, grad_table, workspace, scale: float = 1.0, status=None,
                    stream=None):
    """grad_table[v] = scale * sum of grad_out[i] over ids[i] == v, every row written."""
    pg, ld = _rows(grad_out, "grad_out")
    _shape(ids, (grad_out.shape[0],), "ids")
    _shape(grad_table, (grad_table.shape[0], grad_out.shape[1]), "grad_table")
    s = _embed_struct(ids.numel(), grad_out.shape[1], grad_table.shape[0],
                      _dtype(grad_table.dtype), _dtype(grad_out.dtype), ld, scale)
    ws, nb = _ws(workspace)
    _call("smdm_embed_grad", stream, (ids, grad_out, grad_table, workspace, status), s,
          _adr(_i32(ids), "ids"), pg, _adr(grad_table, "grad_table"), ws, nb, _status(status))


def make_config(n_layers, d_model, n_heads, d_head, d_ffn, vocab, n_reg=64, dtype=SMDM_BF16,
                rope_theta=10000.0, rms_eps=1e-6, max_batch=1, max_len=1, max_step_rows=1,
                max_rows=1) -> smdm_config:
    return smdm_config(n_layers, d_model, n_heads, d_head, d_ffn, vocab, n_reg, dtype, rope_theta,
                       rms_eps, max_batch, max_len, max_step_rows, max_rows)
