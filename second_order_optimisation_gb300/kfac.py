"""Thin ctypes binding of libkfac_gb300.so (C ABI in include/kfac.h).

Argument marshalling only: every step of the K-FAC curvature path runs in the
library's CUDA kernels.  PyTorch supplies device memory (tensors, the
workspace) and the stream.  There is no CPU or PyTorch fallback: if the
library is missing, loading it raises.

The functions keep the C names:
  kfac_factor_update   (Osawa et al. section 3.2, Eq. 5 + running average)
  kfac_damp_invert     (Eq. 6, pi-split Tikhonov damping)
  kfac_precondition    (Eq. 7)
  kfac_bn_diag_fisher  (diagonal BatchNorm Fisher, section 1)
and, next to the step, the losses that make a policy's or language model's
output gradients and the bound on the step over all tensors:
  kfac_token_logprob, kfac_token_logprob_grad, kfac_policy_loss,
  kfac_preference_loss, kfac_clip_norm
and what a policy's tokens are drawn with and a layer's input is kept in until the
backward pass:
  kfac_verify_draft, kfac_checkpoint_store, kfac_checkpoint_load, kfac_weight_grad
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkfac_gb300.so")

KFAC_OK, KFAC_ERR_INVALID, KFAC_ERR_UNSUPPORTED, KFAC_ERR_NOT_PD, KFAC_ERR_CUDA, KFAC_ERR_WORKSPACE = range(6)
KFAC_BF16, KFAC_F32, KFAC_F16, KFAC_E4M3 = 0, 1, 2, 3
KFAC_LAYOUT_FULL, KFAC_LAYOUT_PACKED_UPPER = 0, 1
# bits of the device error word (the first int32 of a call's workspace)
ERRW_TIMEOUT_OPERAND, ERRW_TIMEOUT_STAGE, ERRW_TIMEOUT_ACCUM, ERRW_TIMEOUT_DRAIN, ERRW_NONFINITE = 1, 2, 4, 8, 16
ERRW_TARGET = 32
KFAC_PREF_SIGMOID, KFAC_PREF_HINGE, KFAC_PREF_IPO = 0, 1, 2

EXPORTS = ("kfac_status_string", "kfac_version", "kfac_launch_count", "kfac_timing_enable",
           "kfac_timing_read", "kfac_timing_kind_name", "kfac_factor_update_workspace_size",
           "kfac_factor_update", "kfac_damp_invert_workspace_size", "kfac_damp_invert",
           "kfac_precondition_workspace_size", "kfac_precondition", "kfac_bn_diag_fisher",
           "kfac_noalloc_scratch_bytes", "kfac_precondition_noalloc", "kfac_timing_read_launches",
           "kfac_token_logprob", "kfac_token_logprob_grad", "kfac_policy_loss_workspace_size", "kfac_policy_loss",
           "kfac_preference_loss_workspace_size", "kfac_preference_loss", "kfac_clip_norm_workspace_size",
           "kfac_clip_norm", "kfac_checkpoint_scale_bytes", "kfac_checkpoint_store", "kfac_checkpoint_load",
           "kfac_weight_grad_workspace_size", "kfac_weight_grad", "kfac_verify_draft_workspace_size",
           "kfac_verify_draft")


class KfacError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)}")
        self.status = status


class FactorDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("x", ctypes.c_void_p),
                ("n", ctypes.c_int32), ("h", ctypes.c_int32), ("w", ctypes.c_int32), ("c", ctypes.c_int32),
                ("kh", ctypes.c_int32), ("kw", ctypes.c_int32),
                ("stride_h", ctypes.c_int32), ("stride_w", ctypes.c_int32),
                ("pad_h", ctypes.c_int32), ("pad_w", ctypes.c_int32),
                ("append_one", ctypes.c_int32),
                ("F", ctypes.c_void_p), ("ldf", ctypes.c_int64),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("layout", ctypes.c_int32), ("scales", ctypes.c_void_p), ("ldx", ctypes.c_int64)]


class InvertDesc(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("dA", ctypes.c_int32), ("lda", ctypes.c_int64),
                ("G", ctypes.c_void_p), ("dG", ctypes.c_int32), ("ldg", ctypes.c_int64),
                ("A_inv", ctypes.c_void_p), ("ld_ainv", ctypes.c_int64),
                ("G_inv", ctypes.c_void_p), ("ld_ginv", ctypes.c_int64),
                ("A_inv_bf16", ctypes.c_void_p), ("ld_ainv_bf16", ctypes.c_int64),
                ("G_inv_bf16", ctypes.c_void_p), ("ld_ginv_bf16", ctypes.c_int64),
                ("layout_A", ctypes.c_int32), ("layout_G", ctypes.c_int32),
                ("copy_dtype", ctypes.c_int32)]


class PrecondDesc(ctypes.Structure):
    _fields_ = [("dG", ctypes.c_int32), ("dA", ctypes.c_int32),
                ("G_inv", ctypes.c_void_p), ("ld_ginv", ctypes.c_int64),
                ("A_inv", ctypes.c_void_p), ("ld_ainv", ctypes.c_int64),
                ("grad", ctypes.c_void_p), ("ld_grad", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64),
                ("w", ctypes.c_void_p), ("ld_w", ctypes.c_int64),
                ("eta", ctypes.c_float)]


class BnDesc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("C", ctypes.c_int32), ("F", ctypes.c_void_p),
                ("grad_mean", ctypes.c_void_p), ("precond", ctypes.c_void_p)]


class LogprobDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int32),
                ("target", ctypes.c_void_p), ("target_i32", ctypes.c_int32), ("temperature", ctypes.c_float),
                ("logp", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
                ("saved", ctypes.c_void_p)]


class LogprobGradDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int32),
                ("target", ctypes.c_void_p), ("target_i32", ctypes.c_int32), ("temperature", ctypes.c_float),
                ("saved", ctypes.c_void_p), ("entropy", ctypes.c_void_p), ("dlogp", ctypes.c_void_p),
                ("dentropy", ctypes.c_void_p), ("dlogits", ctypes.c_void_p), ("ld_d", ctypes.c_int64)]


class PolicyDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int32),
                ("target", ctypes.c_void_p), ("target_i32", ctypes.c_int32), ("temperature", ctypes.c_float),
                ("advantage", ctypes.c_void_p), ("old_logp", ctypes.c_void_p), ("ref_logp", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("seq_offsets", ctypes.c_void_p), ("seqs", ctypes.c_int32),
                ("seq_mean", ctypes.c_int32),
                ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float), ("kl_coef", ctypes.c_float),
                ("entropy_coef", ctypes.c_float), ("grad_scale", ctypes.c_float),
                ("stats", ctypes.c_void_p), ("logp", ctypes.c_void_p), ("kl", ctypes.c_void_p),
                ("entropy", ctypes.c_void_p), ("dlogits", ctypes.c_void_p), ("ld_d", ctypes.c_int64)]


class PreferenceDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int32),
                ("target", ctypes.c_void_p), ("target_i32", ctypes.c_int32), ("temperature", ctypes.c_float),
                ("seq_offsets", ctypes.c_void_p), ("pairs", ctypes.c_int32),
                ("ref_logp", ctypes.c_void_p), ("pair_weight", ctypes.c_void_p),
                ("kind", ctypes.c_int32), ("average", ctypes.c_int32),
                ("beta", ctypes.c_float), ("label_smoothing", ctypes.c_float), ("grad_scale", ctypes.c_float),
                ("loss", ctypes.c_void_p), ("pair_loss", ctypes.c_void_p), ("seq_logp", ctypes.c_void_p),
                ("token_logp", ctypes.c_void_p), ("dlogits", ctypes.c_void_p), ("ld_d", ctypes.c_int64)]


class ClipDesc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ld", ctypes.c_int64), ("y", ctypes.c_void_p), ("ld_y", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64), ("w", ctypes.c_void_p), ("ld_w", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class CheckpointDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("x", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("append_one", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("scales", ctypes.c_void_p)]


class WeightGradDesc(ctypes.Structure):
    _fields_ = [("q_a", ctypes.c_void_p), ("ldq_a", ctypes.c_int64), ("scales_a", ctypes.c_void_p),
                ("q_g", ctypes.c_void_p), ("ldq_g", ctypes.c_int64), ("scales_g", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("dA", ctypes.c_int32), ("dG", ctypes.c_int32),
                ("out", ctypes.c_void_p), ("ld", ctypes.c_int64), ("out_dtype", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float)]


class VerifyDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int32),
                ("tokens", ctypes.c_void_p), ("token_i32", ctypes.c_int32), ("temperature", ctypes.c_float),
                ("seq_offsets", ctypes.c_void_p), ("seqs", ctypes.c_int32),
                ("draft", ctypes.c_void_p), ("ld_draft", ctypes.c_int64), ("draft_saved", ctypes.c_void_p),
                ("draft_temperature", ctypes.c_float), ("uniform", ctypes.c_void_p),
                ("noise", ctypes.c_void_p), ("ld_noise", ctypes.c_int64), ("greedy", ctypes.c_int32),
                ("accepted", ctypes.c_void_p), ("out_tokens", ctypes.c_void_p), ("logp", ctypes.c_void_p)]


_lib = None


def library_path() -> str:
    return LIB_PATH


def load() -> ctypes.CDLL:
    """Load libkfac_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.kfac_status_string.argtypes = [i32]
        lib.kfac_status_string.restype = ctypes.c_char_p
        lib.kfac_version.restype = i32
        lib.kfac_launch_count.restype = ctypes.c_longlong
        lib.kfac_timing_enable.argtypes = [i32]
        lib.kfac_timing_enable.restype = i32
        lib.kfac_timing_read.argtypes = [vp, vp, i32]
        lib.kfac_timing_read.restype = i32
        lib.kfac_timing_read_launches.argtypes = [vp, vp, vp, vp, i32]
        lib.kfac_timing_read_launches.restype = i32
        lib.kfac_timing_kind_name.argtypes = [i32]
        lib.kfac_timing_kind_name.restype = ctypes.c_char_p
        lib.kfac_factor_update_workspace_size.argtypes = [vp, i32]
        lib.kfac_factor_update_workspace_size.restype = sz
        lib.kfac_factor_update.argtypes = [vp, i32, vp, sz, vp]
        lib.kfac_damp_invert_workspace_size.argtypes = [vp, i32]
        lib.kfac_damp_invert_workspace_size.restype = sz
        lib.kfac_damp_invert.argtypes = [vp, i32, f32, i32, vp, vp, vp, sz, vp]
        lib.kfac_precondition_workspace_size.argtypes = [vp, i32, i32]
        lib.kfac_precondition_workspace_size.restype = sz
        lib.kfac_precondition.argtypes = [vp, i32, i32, vp, sz, vp]
        lib.kfac_bn_diag_fisher.argtypes = [vp, i32, i32, f32, f32, vp]
        lib.kfac_noalloc_scratch_bytes.restype = sz
        lib.kfac_precondition_noalloc.argtypes = [vp, i32, i32, vp]
        lib.kfac_token_logprob.argtypes = [vp, vp]
        lib.kfac_token_logprob_grad.argtypes = [vp, vp]
        for f in ("kfac_policy_loss", "kfac_preference_loss"):
            getattr(lib, f).argtypes = [vp, vp, sz, vp]
            getattr(lib, f + "_workspace_size").argtypes = [vp]
            getattr(lib, f + "_workspace_size").restype = sz
        lib.kfac_clip_norm_workspace_size.argtypes = [vp, i32]
        lib.kfac_clip_norm_workspace_size.restype = sz
        lib.kfac_clip_norm.argtypes = [vp, i32, f32, f32, vp, vp, vp, sz, vp]
        lib.kfac_checkpoint_scale_bytes.argtypes = [ctypes.c_int64, ctypes.c_int32]
        lib.kfac_checkpoint_scale_bytes.restype = sz
        lib.kfac_checkpoint_store.argtypes = [vp, i32, vp]
        lib.kfac_checkpoint_load.argtypes = [vp, i32, vp]
        lib.kfac_weight_grad_workspace_size.argtypes = [vp, i32]
        lib.kfac_weight_grad_workspace_size.restype = sz
        lib.kfac_weight_grad.argtypes = [vp, i32, vp, sz, vp]
        lib.kfac_verify_draft_workspace_size.argtypes = [vp]
        lib.kfac_verify_draft_workspace_size.restype = sz
        lib.kfac_verify_draft.argtypes = [vp, vp, sz, vp]
        for f in ("kfac_factor_update", "kfac_damp_invert", "kfac_precondition", "kfac_bn_diag_fisher",
                  "kfac_precondition_noalloc", "kfac_token_logprob", "kfac_token_logprob_grad", "kfac_policy_loss",
                  "kfac_preference_loss", "kfac_clip_norm", "kfac_checkpoint_store", "kfac_checkpoint_load",
                  "kfac_weight_grad", "kfac_verify_draft"):
            getattr(lib, f).restype = i32
        _lib = lib
    return _lib


def launch_count() -> int:
    """Kernel launches the library has enqueued in this process."""
    return int(load().kfac_launch_count())


def timing_enable(on: bool = True) -> bool:
    """Turn the library's per-kernel event timing on or off (diagnostic)."""
    return bool(load().kfac_timing_enable(int(bool(on))))


def timing_read() -> dict:
    """{kernel kind: (total ms, launches)} since the last read (synchronises)."""
    lib = load()
    n = 32
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_longlong * n)()
    _check(lib.kfac_timing_read(ms, cnt, n), "kfac_timing_read")
    out = {}
    for k in range(n):
        name = lib.kfac_timing_kind_name(k).decode()
        if name and cnt[k]:
            out[name] = (ms[k], int(cnt[k]))
    return out


def timing_read_launches(n: int = 65536) -> list:
    """[(start ms, duration ms, kernel kind name, stream id)] of every recorded
    launch in enqueue order, since the last read (synchronises); stream ids
    number the launch streams 0, 1, ... in order of first appearance."""
    lib = load()
    st = (ctypes.c_double * n)()
    du = (ctypes.c_double * n)()
    kd = (ctypes.c_int * n)()
    sm = (ctypes.c_ulonglong * n)()
    cnt = lib.kfac_timing_read_launches(st, du, kd, sm, n)
    if cnt < 0:
        raise KfacError(KFAC_ERR_CUDA, "kfac_timing_read_launches")
    ids = {}
    return [(st[i], du[i], lib.kfac_timing_kind_name(kd[i]).decode(), ids.setdefault(sm[i], len(ids)))
            for i in range(min(cnt, n))]


def status_string(status: int) -> str:
    return load().kfac_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:  # (the raw handle: making a Stream object costs microseconds)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, what: str):
    if status != KFAC_OK:
        raise KfacError(status, what)


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise KfacError(KFAC_ERR_WORKSPACE, "workspace too small")
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _ld(t: torch.Tensor) -> int:
    assert t.dim() == 2 and t.stride(1) == 1, "matrices must be row-major with unit column stride"
    return t.stride(0)


# ------------------------------------------------------------ checkpoints

@dataclass
class Checkpoint:
    """A matrix [rows, width] kept in 8 bits (format in kfac.h): q uint8 with at least
    that shape, unit column stride and a row pitch of a multiple of 16 (better 32), scales the
    dense uint8 exponents.  Checkpoint.empty makes the buffers."""
    q: torch.Tensor
    scales: torch.Tensor
    rows: int
    width: int

    @property
    def device(self) -> torch.device:
        return self.q.device

    @staticmethod
    def empty(rows: int, cols: int, append_one: bool = False, device="cuda") -> "Checkpoint":
        width = cols + bool(append_one)
        # (a pitch of whole sectors of 32 bytes: the products' copies then touch a fifth fewer of them)
        return Checkpoint(torch.empty(rows, (width + 31) // 32 * 32, dtype=torch.uint8, device=device),
                          torch.empty(checkpoint_scale_bytes(rows, width), dtype=torch.uint8, device=device), rows, width)


def checkpoint_scale_bytes(rows: int, width: int) -> int:
    """Bytes of a checkpoint's exponents: 512 for each 128 x 128 values, begun ones whole."""
    return (rows + 127) // 128 * ((width + 127) // 128) * 512


def _checkpoint_args(c: Checkpoint):
    """A checkpoint's elements, pitch and exponents.  (Few questions to the tensors: each costs
    as much as the rest of a field.)"""
    q, sc, rows, width = c.q, c.scales, c.rows, c.width
    if q.dtype is not torch.uint8 or sc.dtype is not torch.uint8:
        raise TypeError("a checkpoint's q and scales must be uint8")
    shape = q.shape
    if len(shape) != 2 or shape[0] < rows or shape[1] < width:
        raise ValueError(f"q must be at least [{rows}, {width}], got {tuple(shape)}")
    ld, unit = q.stride()
    if unit != 1 and shape[1] > 1 and rows > 0:
        raise ValueError("q must have unit column stride")
    if not sc.is_contiguous() or sc.numel() < checkpoint_scale_bytes(rows, width):
        raise ValueError(f"scales must be {checkpoint_scale_bytes(rows, width)} dense bytes, got {tuple(sc.shape)}")
    # (one row has no pitch)
    return q.data_ptr(), ld if shape[0] > 1 else (width + 15) // 16 * 16, sc.data_ptr()


@dataclass
class CheckpointItem:
    """A matrix x [rows, cols] (bf16, fp16 or fp32, unit column stride, any pitch) and the
    checkpoint that keeps it; with append_one the checkpoint has a column of ones more."""
    x: torch.Tensor
    checkpoint: Checkpoint
    append_one: bool = False


def _checkpoint_desc(it: CheckpointItem) -> CheckpointDesc:
    x, c, one = it.x, it.checkpoint, bool(it.append_one)
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {x.dtype}")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must be [rows, cols], got {tuple(shape)}")
    rows, cols = shape
    ld, unit = x.stride()
    if unit != 1 and cols > 1 and rows > 0:
        raise ValueError("x must have unit column stride")
    if c.rows != rows or c.width != cols + one:
        raise ValueError(f"the checkpoint is [{c.rows}, {c.width}], x is {tuple(shape)}, append_one {one}")
    return CheckpointDesc(dtype, x.data_ptr(), ld if rows > 1 else cols, rows, cols, one, *_checkpoint_args(c))


def _checkpoint_descs(items: Sequence[CheckpointItem]):
    if len(items) == 1:
        return ctypes.byref(_checkpoint_desc(items[0]))
    return (CheckpointDesc * max(len(items), 1))(*[_checkpoint_desc(it) for it in items])


def kfac_checkpoint_store(items: Sequence[CheckpointItem], stream=None) -> None:
    """Keep every x in its checkpoint."""
    _check(load().kfac_checkpoint_store(_checkpoint_descs(items), len(items), _stream(stream)), "kfac_checkpoint_store")


def kfac_checkpoint_load(items: Sequence[CheckpointItem], stream=None) -> None:
    """Write every checkpoint's values to its x (a column of ones is left out)."""
    _check(load().kfac_checkpoint_load(_checkpoint_descs(items), len(items), _stream(stream)), "kfac_checkpoint_load")


@dataclass
class WeightGrad:
    """out [dG, dA] (fp32, bf16 or fp16) <- beta out + alpha g^T a, from the checkpoints of
    a layer's input a [rows, dA] and of its output gradients g [rows, dG].  The outs of one
    call must not overlap."""
    a: Checkpoint
    g: Checkpoint
    out: torch.Tensor
    alpha: float = 1.0
    beta: float = 0.0


def _weight_grad_desc(it: WeightGrad) -> WeightGradDesc:
    a, g, out = it.a, it.g, it.out
    dtype, dA, dG = _DTYPES.get(out.dtype), a.width, g.width
    if dtype is None:
        raise TypeError(f"unsupported dtype {out.dtype}")
    if a.rows != g.rows:
        raise ValueError(f"a has {a.rows} rows, g {g.rows}")
    if out.shape != (dG, dA):
        raise ValueError(f"out must be [{dG}, {dA}], got {tuple(out.shape)}")
    ld, unit = out.stride()
    if unit != 1 and dA > 1:
        raise ValueError("out must have unit column stride")
    return WeightGradDesc(*_checkpoint_args(a), *_checkpoint_args(g), a.rows, dA, dG, out.data_ptr(),
                          ld if dG > 1 else dA, dtype, it.alpha, it.beta)


def _weight_grad_descs(items: Sequence[WeightGrad]):
    if len(items) == 1:
        return ctypes.byref(_weight_grad_desc(items[0]))
    return (WeightGradDesc * max(len(items), 1))(*[_weight_grad_desc(it) for it in items])


def kfac_weight_grad_workspace_size(items: Sequence[WeightGrad]) -> int:
    return int(load().kfac_weight_grad_workspace_size(_weight_grad_descs(items), len(items)))


def kfac_weight_grad(items: Sequence[WeightGrad], workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Enqueue the weight gradients; returns the workspace used (its first int32 is the
    device error word: ERRW_NONFINITE, ERRW_TIMEOUT_*)."""
    lib = load()
    arr = _weight_grad_descs(items)
    n = len(items)
    ws = _scratch(lib.kfac_weight_grad_workspace_size(arr, n), items[0].out.device if n else "cuda", workspace, stream)
    _check(lib.kfac_weight_grad(arr, n, ws.data_ptr(), ws.nbytes, _stream(stream)), "kfac_weight_grad")
    return ws


# ------------------------------------------------------------ factor update

@dataclass
class FactorSource:
    """One factor update: F[:d, :d] (upper) <- beta F + alpha P^T P, P the patch
    matrix of x.  x: NHWC [n, h, w, c] (conv) or [rows, c] (FC / output grads),
    bf16, fp16 or fp32, or a Checkpoint of [rows, c].  With packed, F is the packed upper triangle (a 1-D
    tensor of d(d+1)/2 floats, see pack_upper)."""
    x: torch.Tensor
    F: torch.Tensor
    kh: int = 1
    kw: int = 1
    stride: tuple = (1, 1)
    pad: tuple = (0, 0)
    append_one: bool = False
    alpha: float = 1.0
    beta: float = 0.0
    packed: bool = False


_DTYPES = {torch.bfloat16: KFAC_BF16, torch.float16: KFAC_F16, torch.float32: KFAC_F32}


def packed_size(d: int) -> int:
    """Floats of a packed upper triangle of order d."""
    return d * (d + 1) // 2


def pack_upper(F: torch.Tensor) -> torch.Tensor:
    """The packed upper triangle (KFAC_LAYOUT_PACKED_UPPER) of a square
    matrix: row i's entries j >= i, row after row (a layout conversion)."""
    d = F.shape[0]
    iu = torch.triu_indices(d, d, device=F.device)
    return F[iu[0], iu[1]].contiguous()


def unpack_upper(Fp: torch.Tensor, d: int) -> torch.Tensor:
    """Square matrix holding a packed upper triangle (zeros below)."""
    out = torch.zeros(d, d, dtype=Fp.dtype, device=Fp.device)
    iu = torch.triu_indices(d, d, device=Fp.device)
    out[iu[0], iu[1]] = Fp
    return out


def _fld(F: torch.Tensor, packed: bool) -> int:
    if packed:
        assert F.dim() == 1 and F.is_contiguous() and F.dtype == torch.float32
        return 0
    return _ld(F)


def _factor_descs(sources: Sequence[FactorSource]):
    arr = (FactorDesc * max(len(sources), 1))()
    for i, s in enumerate(sources):
        x = s.x
        if isinstance(x, Checkpoint):
            assert s.F.dtype == torch.float32
            q, ldq, scales = _checkpoint_args(x)
            if s.F.numel() < packed_size(x.width) if s.packed else min(s.F.shape) < x.width:
                raise KfacError(KFAC_ERR_INVALID, f"F is {tuple(s.F.shape)}, the checkpoint has {x.width} columns")
            arr[i] = FactorDesc(KFAC_E4M3, q, x.rows, 1, 1, x.width, s.kh, s.kw, s.stride[0], s.stride[1],
                                s.pad[0], s.pad[1], int(bool(s.append_one)), s.F.data_ptr(), _fld(s.F, s.packed),
                                float(s.alpha), float(s.beta),
                                KFAC_LAYOUT_PACKED_UPPER if s.packed else KFAC_LAYOUT_FULL, scales, ldq)
            continue
        assert x.is_contiguous(), "x must be dense"
        if x.dim() == 2:
            n, h, w, c = x.shape[0], 1, 1, x.shape[1]
        else:
            n, h, w, c = x.shape
        if x.dtype not in _DTYPES:
            raise TypeError(f"unsupported source dtype {x.dtype}")
        assert s.F.dtype == torch.float32
        arr[i] = FactorDesc(_DTYPES[x.dtype], x.data_ptr(), n, h, w, c, s.kh, s.kw, s.stride[0], s.stride[1],
                            s.pad[0], s.pad[1], int(bool(s.append_one)), s.F.data_ptr(), _fld(s.F, s.packed),
                            float(s.alpha), float(s.beta),
                            KFAC_LAYOUT_PACKED_UPPER if s.packed else KFAC_LAYOUT_FULL)
    return arr


def kfac_factor_update_workspace_size(sources: Sequence[FactorSource]) -> int:
    arr = _factor_descs(sources)
    return int(load().kfac_factor_update_workspace_size(arr, len(sources)))


def kfac_factor_update(sources: Sequence[FactorSource], workspace: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Enqueue the factor updates; returns the workspace used (its first int32
    is the library's device error word: 0 = no timeout and no NaN or infinite
    output; ERRW_* bits otherwise)."""
    lib = load()
    arr = _factor_descs(sources)
    need = int(lib.kfac_factor_update_workspace_size(arr, len(sources)))
    if need == 0 and len(sources):
        _check(lib.kfac_factor_update(arr, len(sources), None, 0, _stream(stream)), "kfac_factor_update")
    ws = _workspace(need, sources[0].x.device if sources else "cuda", workspace)
    _check(lib.kfac_factor_update(arr, len(sources), ws.data_ptr(), ws.numel() * ws.element_size(),
                                  _stream(stream)), "kfac_factor_update")
    return ws


# ------------------------------------------------------------ damp + invert

@dataclass
class InvertPair:
    """Both factors of one layer and where their damped inverses go.  The
    optional 16-bit copies are bf16 or fp16 (both the same dtype); a packed
    factor is a 1-D tensor of d(d+1)/2 floats (then dA / dG are required)."""
    A: torch.Tensor
    G: torch.Tensor
    A_inv: torch.Tensor
    G_inv: torch.Tensor
    A_inv_bf16: Optional[torch.Tensor] = None
    G_inv_bf16: Optional[torch.Tensor] = None
    dA: Optional[int] = None
    dG: Optional[int] = None
    packed_A: bool = False
    packed_G: bool = False


def _invert_descs(pairs: Sequence[InvertPair]):
    arr = (InvertDesc * max(len(pairs), 1))()
    for i, p in enumerate(pairs):
        dA = p.dA or p.A_inv.shape[0]
        dG = p.dG or p.G_inv.shape[0]
        copies = {t.dtype for t in (p.A_inv_bf16, p.G_inv_bf16) if t is not None}
        if not copies <= {torch.bfloat16, torch.float16} or len(copies) > 1:
            raise TypeError(f"16-bit inverse copies must be both bf16 or both fp16, got {copies}")
        cdt = KFAC_F16 if copies == {torch.float16} else KFAC_BF16
        arr[i] = InvertDesc(p.A.data_ptr(), dA, _fld(p.A, p.packed_A), p.G.data_ptr(), dG, _fld(p.G, p.packed_G),
                            p.A_inv.data_ptr(), _ld(p.A_inv), p.G_inv.data_ptr(), _ld(p.G_inv),
                            _ptr(p.A_inv_bf16), _ld(p.A_inv_bf16) if p.A_inv_bf16 is not None else 0,
                            _ptr(p.G_inv_bf16), _ld(p.G_inv_bf16) if p.G_inv_bf16 is not None else 0,
                            KFAC_LAYOUT_PACKED_UPPER if p.packed_A else KFAC_LAYOUT_FULL,
                            KFAC_LAYOUT_PACKED_UPPER if p.packed_G else KFAC_LAYOUT_FULL, cdt)
    return arr


def kfac_damp_invert_workspace_size(pairs: Sequence[InvertPair]) -> int:
    return int(load().kfac_damp_invert_workspace_size(_invert_descs(pairs), len(pairs)))


def kfac_damp_invert(pairs: Sequence[InvertPair], gamma: float, pi_split: bool = True,
                     info: Optional[torch.Tensor] = None, damp: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Enqueue the damped inversions; returns the workspace used (its first
    int32 is the library's device error word: 0 = no timeout and no NaN or
    infinite output; ERRW_* bits otherwise)."""
    lib = load()
    arr = _invert_descs(pairs)
    need = int(lib.kfac_damp_invert_workspace_size(arr, len(pairs)))
    ws = _workspace(need, pairs[0].A.device if pairs else "cuda", workspace)
    if info is not None:
        assert info.dtype == torch.int32 and info.numel() >= 2 * len(pairs)
    if damp is not None:
        assert damp.dtype == torch.float32 and damp.numel() >= 2 * len(pairs)
    _check(lib.kfac_damp_invert(arr, len(pairs), float(gamma), int(bool(pi_split)), _ptr(info), _ptr(damp),
                                ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
           "kfac_damp_invert")
    return ws


# ------------------------------------------------------------ precondition

@dataclass
class PrecondItem:
    """out = G_inv @ grad @ A_inv for one layer (grad [dG, dA]); with w, also
    w -= eta * out in place (out may then be None)."""
    G_inv: torch.Tensor
    A_inv: torch.Tensor
    grad: torch.Tensor
    out: Optional[torch.Tensor]
    dG: Optional[int] = None
    dA: Optional[int] = None
    w: Optional[torch.Tensor] = None
    eta: float = 0.0


def _precond_descs(items: Sequence[PrecondItem]):
    arr = (PrecondDesc * max(len(items), 1))()
    for i, it in enumerate(items):
        dG = it.dG or it.grad.shape[0]
        dA = it.dA or it.grad.shape[1]
        if it.w is not None and it.w.dtype != torch.float32:
            raise TypeError("w must be fp32")
        arr[i] = PrecondDesc(dG, dA, it.G_inv.data_ptr(), _ld(it.G_inv), it.A_inv.data_ptr(), _ld(it.A_inv),
                             it.grad.data_ptr(), _ld(it.grad),
                             it.out.data_ptr() if it.out is not None else None,
                             _ld(it.out) if it.out is not None else 0,
                             it.w.data_ptr() if it.w is not None else None,
                             _ld(it.w) if it.w is not None else 0, float(it.eta))
    return arr


def _precond_dtype(items: Sequence[PrecondItem]) -> int:
    dts = {it.grad.dtype for it in items} | {it.A_inv.dtype for it in items} | {it.G_inv.dtype for it in items}
    if len(dts) == 1 and next(iter(dts)) in _DTYPES:
        return _DTYPES[next(iter(dts))]
    raise TypeError(f"operands must be all bf16, all fp16 or all fp32, got {dts}")


def kfac_precondition_workspace_size(items: Sequence[PrecondItem]) -> int:
    return int(load().kfac_precondition_workspace_size(_precond_descs(items), len(items),
                                                       _precond_dtype(items)))


def kfac_precondition(items: Sequence[PrecondItem], workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    lib = load()
    arr = _precond_descs(items)
    dt = _precond_dtype(items)
    need = int(lib.kfac_precondition_workspace_size(arr, len(items), dt))
    ws = _workspace(need, items[0].grad.device if items else "cuda", workspace)
    _check(lib.kfac_precondition(arr, len(items), dt, ws.data_ptr(), ws.numel() * ws.element_size(),
                                 _stream(stream)), "kfac_precondition")
    return ws


def kfac_precondition_noalloc(items: Sequence[PrecondItem], stream=None) -> None:
    """kfac_precondition with the library's fixed device scratch instead of a
    workspace: for callers that cannot allocate device memory (see kfac.h)."""
    lib = load()
    arr = _precond_descs(items)
    _check(lib.kfac_precondition_noalloc(arr, len(items), _precond_dtype(items), _stream(stream)),
           "kfac_precondition_noalloc")


# ------------------------------------------------------------ BN diagonal Fisher

@dataclass
class BnItem:
    x: torch.Tensor            # [n_samples, C] fp32
    F: torch.Tensor            # [C] fp32
    precond: torch.Tensor      # [C] fp32
    grad_mean: Optional[torch.Tensor] = None


def kfac_bn_diag_fisher(items: Sequence[BnItem], gamma: float, xi: float = 0.0, stream=None) -> None:
    lib = load()
    arr = (BnDesc * max(len(items), 1))()
    ns = items[0].x.shape[0] if items else 1
    for i, it in enumerate(items):
        assert it.x.dtype == torch.float32 and it.x.is_contiguous() and it.x.shape[0] == ns
        arr[i] = BnDesc(it.x.data_ptr(), it.x.shape[1], it.F.data_ptr(), _ptr(it.grad_mean),
                        it.precond.data_ptr())
    _check(lib.kfac_bn_diag_fisher(arr, len(items), ns, float(gamma), float(xi), _stream(stream)),
           "kfac_bn_diag_fisher")


# ------------------------------------------------------------ losses on logits

def memory_of(stream, device):
    """A context in which new tensors are the memory of `stream` (a torch stream, a raw handle, or
    None: the current one), and what fills them is enqueued there."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)  # (0 is the default stream, which has no external handle)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _scratch(nbytes: int, device, workspace: Optional[torch.Tensor], stream) -> torch.Tensor:
    """The caller's workspace, or a new one that may be dropped while a call on
    `stream` (an own stream, or None) still uses it.  It is that stream's memory: a
    block of the current stream's may still be in use there by earlier work."""
    if workspace is not None:
        return _workspace(nbytes, device, workspace)
    if stream is None:
        return torch.empty(nbytes if nbytes > 256 else 256, dtype=torch.uint8, device=device)
    with memory_of(stream, device):
        ws = _workspace(nbytes, device, None)
    ws.record_stream(torch.cuda.current_stream(device))  # the error word may be read there
    return ws


def _rowvec(t: Optional[torch.Tensor], n: int, name: str, dtype=torch.float32) -> Optional[int]:
    """Address of a dense vector of n values (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} dense values, got shape {tuple(t.shape)}")
    return t.data_ptr()


def _logits_args(logits: torch.Tensor, target: torch.Tensor, temperature: float, name: str = "target"):
    """The descriptor fields from dtype to temperature, the same for every call on logits."""
    dtype, tdtype = _DTYPES.get(logits.dtype), target.dtype
    if dtype is None:
        raise TypeError(f"unsupported logits dtype {logits.dtype}")
    if tdtype is not torch.int64 and tdtype is not torch.int32:
        raise TypeError(f"{name} must be int64 or int32, got {tdtype}")
    shape, stride = logits.shape, logits.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError("logits must be [rows, vocab] with unit column stride")
    rows, vocab = shape
    if target.numel() != rows or not target.is_contiguous():
        raise ValueError(f"{name} must be {rows} dense values, got shape {tuple(target.shape)}")
    return (dtype, logits.data_ptr(), stride[0] if rows > 1 else vocab, rows, vocab,
            target.data_ptr(), tdtype is torch.int32, temperature)


def _dlogits_args(logits: torch.Tensor, dlogits: Optional[torch.Tensor], name: str = "dlogits"):
    if dlogits is None:
        return None, 0
    shape, stride = dlogits.shape, dlogits.stride()
    if dlogits.dtype is not logits.dtype or shape != logits.shape:
        raise TypeError(f"{name} must have the logits' shape and dtype")
    if stride[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    return dlogits.data_ptr(), stride[0] if shape[0] > 1 else shape[1]


@dataclass
class TokenLogprob:
    """Log-probabilities of target [rows] under logits [rows, vocab] (bf16, fp16
    or fp32; target int64 or int32, negative: ignored), and optionally the
    rows' lse and entropy (fp32 [rows] each) and what the gradient needs of them
    (saved, fp32 [rows, 2])."""
    logits: torch.Tensor
    target: torch.Tensor
    logp: torch.Tensor
    lse: Optional[torch.Tensor] = None
    entropy: Optional[torch.Tensor] = None
    temperature: float = 1.0
    saved: Optional[torch.Tensor] = None


def kfac_token_logprob(item: TokenLogprob, stream=None) -> None:
    t = item
    n = t.logits.shape[0]
    d = LogprobDesc(*_logits_args(t.logits, t.target, t.temperature), _rowvec(t.logp, n, "logp"),
                    _rowvec(t.lse, n, "lse"), _rowvec(t.entropy, n, "entropy"), _rowvec(t.saved, 2 * n, "saved"))
    _check(load().kfac_token_logprob(ctypes.byref(d), _stream(stream)), "kfac_token_logprob")


@dataclass
class TokenLogprobGrad:
    """dlogits (the logits' shape and dtype) from the gradients of logp and,
    optionally, of the entropy; saved and entropy as kfac_token_logprob gave them."""
    logits: torch.Tensor
    target: torch.Tensor
    saved: torch.Tensor
    dlogp: torch.Tensor
    dlogits: torch.Tensor
    entropy: Optional[torch.Tensor] = None
    dentropy: Optional[torch.Tensor] = None
    temperature: float = 1.0


def kfac_token_logprob_grad(item: TokenLogprobGrad, stream=None) -> None:
    t = item
    n = t.logits.shape[0]
    d = LogprobGradDesc(*_logits_args(t.logits, t.target, t.temperature), _rowvec(t.saved, 2 * n, "saved"),
                        _rowvec(t.entropy, n, "entropy"), _rowvec(t.dlogp, n, "dlogp"),
                        _rowvec(t.dentropy, n, "dentropy"), *_dlogits_args(t.logits, t.dlogits))
    _check(load().kfac_token_logprob_grad(ctypes.byref(d), _stream(stream)), "kfac_token_logprob_grad")


@dataclass
class PolicyLoss:
    """Clipped policy loss with a KL term and an entropy bonus (formulas in
    kfac.h).  advantage: [rows], or [seqs] with seq_offsets int32 [seqs + 1].
    stats fp32 [5] receives the loss and the weighted sums of its policy term,
    the KL, the entropy and the clipped share; dlogits (optional) the gradient."""
    logits: torch.Tensor
    target: torch.Tensor
    advantage: torch.Tensor
    old_logp: torch.Tensor
    stats: torch.Tensor
    logp: Optional[torch.Tensor] = None
    dlogits: Optional[torch.Tensor] = None
    ref_logp: Optional[torch.Tensor] = None
    weight: Optional[torch.Tensor] = None
    seq_offsets: Optional[torch.Tensor] = None
    seq_mean: bool = False
    kl: Optional[torch.Tensor] = None
    entropy: Optional[torch.Tensor] = None
    clip_low: float = 0.2
    clip_high: float = 0.2
    kl_coef: float = 0.0
    entropy_coef: float = 0.0
    temperature: float = 1.0
    grad_scale: float = 1.0


def _policy_desc(t: PolicyLoss) -> PolicyDesc:
    n = t.logits.shape[0]
    seqs = 0 if t.seq_offsets is None else t.seq_offsets.numel() - 1
    return PolicyDesc(*_logits_args(t.logits, t.target, t.temperature),
                      _rowvec(t.advantage, n if t.seq_offsets is None else seqs, "advantage"),
                      _rowvec(t.old_logp, n, "old_logp"), _rowvec(t.ref_logp, n, "ref_logp"),
                      _rowvec(t.weight, n, "weight"), _rowvec(t.seq_offsets, seqs + 1, "seq_offsets", torch.int32),
                      seqs, bool(t.seq_mean), t.clip_low, t.clip_high, t.kl_coef, t.entropy_coef, t.grad_scale,
                      _rowvec(t.stats, 5, "stats"), _rowvec(t.logp, n, "logp"), _rowvec(t.kl, n, "kl"),
                      _rowvec(t.entropy, n, "entropy"), *_dlogits_args(t.logits, t.dlogits))


def kfac_policy_loss_workspace_size(item: PolicyLoss) -> int:
    return int(load().kfac_policy_loss_workspace_size(ctypes.byref(_policy_desc(item))))


def kfac_policy_loss(item: PolicyLoss, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Enqueue the loss and its gradient; returns the workspace used (its first
    int32 is the device error word: ERRW_TARGET, ERRW_NONFINITE)."""
    lib = load()
    d = _policy_desc(item)
    p = ctypes.byref(d)
    ws = _scratch(lib.kfac_policy_loss_workspace_size(p), item.logits.device, workspace, stream)
    _check(lib.kfac_policy_loss(p, ws.data_ptr(), ws.nbytes, _stream(stream)), "kfac_policy_loss")
    return ws


_PREF_KINDS = {"sigmoid": KFAC_PREF_SIGMOID, "hinge": KFAC_PREF_HINGE, "ipo": KFAC_PREF_IPO}


@dataclass
class PreferenceLoss:
    """Loss over pairs of sequences (formulas in kfac.h): sequences 2 b and
    2 b + 1 of seq_offsets (int32 [2 pairs + 1]) are the preferred and the other
    one of pair b.  loss fp32 [1]; seq_logp and ref_logp [2 pairs]; kind is
    "sigmoid", "hinge" or "ipo"."""
    logits: torch.Tensor
    target: torch.Tensor
    seq_offsets: torch.Tensor
    loss: torch.Tensor
    seq_logp: Optional[torch.Tensor] = None
    dlogits: Optional[torch.Tensor] = None
    ref_logp: Optional[torch.Tensor] = None
    pair_weight: Optional[torch.Tensor] = None
    pair_loss: Optional[torch.Tensor] = None
    token_logp: Optional[torch.Tensor] = None
    kind: str = "sigmoid"
    beta: float = 0.1
    label_smoothing: float = 0.0
    average: bool = False
    temperature: float = 1.0
    grad_scale: float = 1.0


def _preference_desc(t: PreferenceLoss) -> PreferenceDesc:
    n, m = t.logits.shape[0], t.seq_offsets.numel() - 1
    if m < 2 or m % 2:
        raise ValueError(f"seq_offsets must hold 2 pairs + 1 values, got {m + 1}")
    if t.kind not in _PREF_KINDS:
        raise ValueError(f"kind must be one of {sorted(_PREF_KINDS)}, got {t.kind!r}")
    return PreferenceDesc(*_logits_args(t.logits, t.target, t.temperature),
                          _rowvec(t.seq_offsets, m + 1, "seq_offsets", torch.int32), m // 2,
                          _rowvec(t.ref_logp, m, "ref_logp"), _rowvec(t.pair_weight, m // 2, "pair_weight"),
                          _PREF_KINDS[t.kind], bool(t.average), t.beta, t.label_smoothing, t.grad_scale,
                          _rowvec(t.loss, 1, "loss"), _rowvec(t.pair_loss, m // 2, "pair_loss"),
                          _rowvec(t.seq_logp, m, "seq_logp"), _rowvec(t.token_logp, n, "token_logp"),
                          *_dlogits_args(t.logits, t.dlogits))


def kfac_preference_loss_workspace_size(item: PreferenceLoss) -> int:
    return int(load().kfac_preference_loss_workspace_size(ctypes.byref(_preference_desc(item))))


def kfac_preference_loss(item: PreferenceLoss, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Enqueue the loss and its gradient; returns the workspace used (its first
    int32 is the device error word: ERRW_TARGET, ERRW_NONFINITE)."""
    lib = load()
    d = _preference_desc(item)
    p = ctypes.byref(d)
    ws = _scratch(lib.kfac_preference_loss_workspace_size(p), item.logits.device, workspace, stream)
    _check(lib.kfac_preference_loss(p, ws.data_ptr(), ws.nbytes, _stream(stream)), "kfac_preference_loss")
    return ws


# ------------------------------------------------------------ drafted tokens

@dataclass
class VerifyDraft:
    """Drafted tokens [rows] (int64 or int32) verified under the policy's logits [rows,
    vocab] (rules in kfac.h).  Sequence b of seq_offsets (int32 [seqs + 1]) holds its
    drafted tokens' rows and one more.  accepted int32 [seqs]; out_tokens [rows] of tokens'
    dtype (may be tokens): the tokens and -1 behind them; logp fp32 [rows].  draft: the scores
    [rows, vocab] of the logits' dtype that the tokens were drawn from (None: looked up),
    draft_saved their fp32 [rows, 2] from TokenLogprob.saved; uniform fp32 [rows], noise fp32
    [seqs, vocab].  greedy takes none of these."""
    logits: torch.Tensor
    tokens: torch.Tensor
    seq_offsets: torch.Tensor
    accepted: torch.Tensor
    out_tokens: torch.Tensor
    logp: Optional[torch.Tensor] = None
    draft: Optional[torch.Tensor] = None
    draft_saved: Optional[torch.Tensor] = None
    uniform: Optional[torch.Tensor] = None
    noise: Optional[torch.Tensor] = None
    greedy: bool = False
    temperature: float = 1.0
    draft_temperature: float = 1.0


def _verify_desc(t: VerifyDraft) -> VerifyDesc:
    seqs, saved, noise = t.seq_offsets.numel() - 1, t.draft_saved, t.noise
    dtype, logits, ld, n, vocab, tokens, i32, tau = _logits_args(t.logits, t.tokens, t.temperature, "tokens")
    draft, ld_draft = _dlogits_args(t.logits, t.draft, "draft")
    at, ld_noise = None, 0
    if noise is not None:
        if noise.dtype is not torch.float32:
            raise TypeError(f"noise must be fp32, got {noise.dtype}")
        if noise.shape != (seqs, vocab):
            raise ValueError(f"noise must be [{seqs}, {vocab}], got {tuple(noise.shape)}")
        ld_noise, unit = noise.stride()
        if unit != 1 and vocab > 1:
            raise ValueError("noise must have unit column stride")
        at, ld_noise = noise.data_ptr(), ld_noise if seqs > 1 else vocab
    return VerifyDesc(dtype, logits, ld, n, vocab, tokens, i32, tau,
                      _rowvec(t.seq_offsets, seqs + 1, "seq_offsets", torch.int32), seqs, draft, ld_draft,
                      _rowvec(saved, 2 * n, "draft_saved"), t.draft_temperature,
                      _rowvec(t.uniform, n, "uniform"), at, ld_noise, bool(t.greedy),
                      _rowvec(t.accepted, seqs, "accepted", torch.int32),
                      _rowvec(t.out_tokens, n, "out_tokens", t.tokens.dtype), _rowvec(t.logp, n, "logp"))


def kfac_verify_draft_workspace_size(item: VerifyDraft) -> int:
    return int(load().kfac_verify_draft_workspace_size(ctypes.byref(_verify_desc(item))))


def kfac_verify_draft(item: VerifyDraft, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Enqueue the verification; returns the workspace used (its first int32 is the device
    error word: ERRW_TARGET, ERRW_NONFINITE)."""
    lib = load()
    d = _verify_desc(item)
    p = ctypes.byref(d)
    ws = _scratch(lib.kfac_verify_draft_workspace_size(p), item.logits.device, workspace, stream)
    _check(lib.kfac_verify_draft(p, ws.data_ptr(), ws.nbytes, _stream(stream)), "kfac_verify_draft")
    return ws


# ------------------------------------------------------------ norm, clipping, weight step

@dataclass
class ClipTensor:
    """One tensor of kfac_clip_norm: x (and y, its dual under the metric, of x's
    dtype or, beside an fp32 x, 16-bit) are read; out = scale * x and w -= eta * scale * x are written where given.  All
    of one shape: dense, or 2-D with unit column stride.  out may be x."""
    x: torch.Tensor
    out: Optional[torch.Tensor] = None
    y: Optional[torch.Tensor] = None
    w: Optional[torch.Tensor] = None


def _clip_desc(t: ClipTensor) -> ClipDesc:
    x = t.x
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    ops = [o for o in (x, t.y, t.out, t.w) if o is not None]
    if any(o.shape != x.shape for o in ops):
        raise ValueError("x, y, out and w must have one shape")
    if t.y is not None and t.y.dtype is not x.dtype and (x.dtype is not torch.float32 or t.y.dtype not in _DTYPES):
        raise TypeError("y must have x's dtype, or be bf16 or fp16 beside an fp32 x")
    if t.w is not None and t.w.dtype is not torch.float32:
        raise TypeError("w must be fp32")
    if t.out is not None and t.out.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.out.dtype}")
    if all(o.is_contiguous() for o in ops):
        rows, cols = 1, x.numel()
        ld = lambda o: cols  # noqa: E731
    else:
        if x.dim() != 2 or any(o.shape[1] > 1 and o.stride(1) != 1 for o in ops):
            raise ValueError("tensors must be dense, or matrices with unit column stride")
        rows, cols = x.shape
        ld = lambda o: o.stride(0) if rows > 1 else cols  # noqa: E731
    a = [v for o in (x, t.y, t.out, t.w) for v in ((None, 0) if o is None else (o.data_ptr(), ld(o)))]
    dt = [_DTYPES[(x if o is None else o).dtype] for o in (x, t.y, t.out)]
    return ClipDesc(*a, rows, cols, *dt)


class ClipList:
    """A list of ClipTensor whose descriptors are made once: for callers that
    clip the same buffers at every step."""

    def __init__(self, tensors: Sequence[ClipTensor]):
        self.tensors = list(tensors)
        self.descs = (ClipDesc * max(len(self.tensors), 1))(*[_clip_desc(t) for t in self.tensors])
        self.device = self.tensors[0].x.device if self.tensors else torch.device("cuda")
        self.need = int(load().kfac_clip_norm_workspace_size(self.descs, len(self.tensors)))


def kfac_clip_norm_workspace_size(tensors) -> int:
    return (tensors if isinstance(tensors, ClipList) else ClipList(tensors)).need


def kfac_clip_norm(tensors, max_norm: float, norm: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                   eta: float = 0.0, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Enqueue norm, clipping and weight step over `tensors` (a sequence of
    ClipTensor, or a ClipList); norm and scale (fp32 [1]) receive the global
    norm and the factor applied.  Returns the workspace used (its first int32
    is the device error word: ERRW_NONFINITE)."""
    c = tensors if isinstance(tensors, ClipList) else ClipList(tensors)
    ws = _scratch(c.need, c.device, workspace, stream)
    _check(load().kfac_clip_norm(c.descs, len(c.tensors), max_norm, eta, _rowvec(norm, 1, "norm"),
                                 _rowvec(scale, 1, "scale"), ws.data_ptr(), ws.nbytes, _stream(stream)),
           "kfac_clip_norm")
    return ws
