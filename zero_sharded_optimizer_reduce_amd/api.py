"""Thin Python binding of libzero's C ABI (include/zero.h), same names.

Argument marshalling only: tensors are checked for device, dtype, layout and
size (the C ABI sees raw pointers and cannot), their data pointers and the
current HIP stream are passed through, and every computation runs in the HIP
kernels.  PyTorch provides device memory and streams.
"""
from __future__ import annotations

import ctypes as C
from typing import Mapping, Optional, Sequence

import numpy as np
import torch

from . import _lib
from ._lib import AdamHparams, MuonHparams, check, load

_BF16_LIKE = (torch.bfloat16, torch.int16, torch.uint16)
_FP32 = (torch.float32,)


_current_device = getattr(torch._C, "_cuda_getDevice", None)   # without torch.cuda's check that the runtime is up


def _stream(stream) -> int:
    if stream is None:
        # the handle itself: building a torch.cuda.Stream object takes 2.7 us, a
        # third of a small call
        return torch._C._cuda_getCurrentRawStream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on_device(t: torch.Tensor, what: str, dtypes) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what}: must be a device tensor, got {t.device}")
    if t.get_device() != _current_device():   # a device tensor: the runtime is up
        raise ValueError(f"{what}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: dtype {t.dtype} not in {dtypes}")


def _dev(t: torch.Tensor, what: str, dtypes) -> int:
    _on_device(t, what, dtypes)
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    return t.data_ptr()


def _dev_same(numel: int, wrong_size: str, *tensors) -> list:
    """The pointers of (tensor, name, dtypes), checked like _dev, without a call
    for each that passes: 0.2 instead of 0.35 us."""
    ptrs = []
    for t, what, dtypes in tensors:
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == _current_device()
                and t.dtype in dtypes and t.is_contiguous()):
            _dev(t, what, dtypes)
        if t.numel() != numel:
            raise ValueError(wrong_size)
        ptrs.append(t.data_ptr())
    return ptrs


def _dev_table(ts: Sequence[torch.Tensor], what: str, dtypes, numel: int, wrong_size: str) -> C.Array:
    """The pointers of equally long device tensors; their names are only formed
    for a refusal."""
    ptrs = []
    for k, t in enumerate(ts):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == _current_device()
                and t.dtype in dtypes and t.is_contiguous()):
            _dev(t, f"{what}[{k}]", dtypes)
        if t.numel() != numel:
            raise ValueError(wrong_size)
        ptrs.append(t.data_ptr())
    return (C.c_void_p * len(ptrs))(*ptrs)


def _ptrs(ptrs) -> C.Array:
    return (C.c_void_p * len(ptrs))(*ptrs)


def hparams(hp) -> AdamHparams:
    if isinstance(hp, AdamHparams):
        return hp
    return AdamHparams(float(hp["lr"]), float(hp["beta1"]), float(hp["beta2"]), float(hp["eps"]),
                       float(hp.get("weight_decay", 0.0)), int(hp["step"]))


# ------------------------------------------------------------ host metadata
def zero_adam_scalars_compute(hp) -> dict:
    out = _lib.AdamScalars()
    check(load().zero_adam_scalars_compute(C.byref(hparams(hp)), C.byref(out)), "zero_adam_scalars_compute")
    return {name: np.float32(getattr(out, name)) for name, _ in _lib.AdamScalars._fields_}


def zero_rank_weights(counts: Optional[Sequence[int]], n_ranks: int) -> np.ndarray:
    if counts is not None and len(counts) != n_ranks:
        raise ValueError("zero_rank_weights: len(counts) != n_ranks")
    if n_ranks < 1:
        raise ValueError("zero_rank_weights: n_ranks must be at least 1")
    out = (C.c_float * n_ranks)()
    arr = None if counts is None else (C.c_int64 * n_ranks)(*[int(c) for c in counts])
    check(load().zero_rank_weights(arr, n_ranks, out), "zero_rank_weights")
    return np.array(list(out), dtype=np.float32)


def zero_shard_layout(numels: Sequence[int], n_shards: int):
    arr = (C.c_int64 * max(1, len(numels)))(*[int(n) for n in numels])
    psi, pad, s = C.c_int64(), C.c_int64(), C.c_int64()
    check(load().zero_shard_layout(arr, len(numels), n_shards, C.byref(psi), C.byref(pad), C.byref(s)),
          "zero_shard_layout")
    return psi.value, pad.value, s.value


# ------------------------------------------------------------ device calls
def zero_reduce_scatter(rank_grads: Sequence[torch.Tensor], rank_weights, shards_out: Sequence[torch.Tensor],
                        accumulate: bool = False, stream=None) -> None:
    """Owner k's shard = sum_r w_r * float(rank_grads[r][k*S:(k+1)*S]) (rank order),
    or shard += that sum when accumulate.  rank_grads: BF16 (zero_reduce_scatter)
    or FP32 (zero_reduce_scatter_f32) device tensors of equal numel; shards_out:
    FP32 device tensors of numel/len(shards_out) each."""
    _reduce_scatter(rank_grads, rank_weights, shards_out, accumulate, stream, f32=False)


def zero_reduce_scatter_f32(rank_grads, rank_weights, shards_out, accumulate: bool = False, stream=None) -> None:
    _reduce_scatter(rank_grads, rank_weights, shards_out, accumulate, stream, f32=True)


def _reduce_scatter(rank_grads, rank_weights, shards_out, accumulate, stream, f32):
    name = "zero_reduce_scatter_f32" if f32 else "zero_reduce_scatter"
    n_ranks, n_shards = len(rank_grads), len(shards_out)
    if n_ranks < 1 or n_shards < 1:
        raise ValueError(f"{name}: need at least one rank and one shard")
    numel = rank_grads[0].numel()
    gp = [_dev(g, f"rank_grads[{r}]", (torch.float32,) if f32 else _BF16_LIKE) for r, g in enumerate(rank_grads)]
    if any(g.numel() != numel for g in rank_grads):
        raise ValueError("zero_reduce_scatter: rank contributions differ in size")
    if numel % n_shards:
        raise ValueError("zero_reduce_scatter: numel not divisible by the number of shards")
    op = [_dev(s, f"shards_out[{k}]", (torch.float32,)) for k, s in enumerate(shards_out)]
    if any(s.numel() != numel // n_shards for s in shards_out):
        raise ValueError("zero_reduce_scatter: each shard must hold numel/n_shards elements")
    w = np.ascontiguousarray(np.asarray(rank_weights, dtype=np.float32))
    if w.size != n_ranks:
        raise ValueError("zero_reduce_scatter: one weight per rank")
    check(getattr(load(), name)(_ptrs(gp), w.ctypes.data_as(_lib.FP), n_ranks, numel, _ptrs(op),
                                n_shards, int(bool(accumulate)), _stream(stream)), name)


def zero_adam_shard_step(master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor,
                         bf16_out: torch.Tensor, grad: torch.Tensor, hp, stream=None) -> None:
    """Fused Adam/AdamW owner update in place (master, m, v FP32; bf16_out written)."""
    n = master.numel()
    ptrs = [_dev(master, "master", (torch.float32,)), _dev(exp_avg, "exp_avg", (torch.float32,)),
            _dev(exp_avg_sq, "exp_avg_sq", (torch.float32,)), _dev(bf16_out, "bf16_out", _BF16_LIKE),
            _dev(grad, "grad", (torch.float32,))]
    if any(t.numel() != n for t in (exp_avg, exp_avg_sq, bf16_out, grad)):
        raise ValueError("zero_adam_shard_step: all buffers must have the same numel")
    h = hparams(hp)
    check(load().zero_adam_shard_step(*ptrs, n, C.byref(h), _stream(stream)), "zero_adam_shard_step")


def zero_adam_shard_step_scaled(master, exp_avg, exp_avg_sq, bf16_out, grad, grad_scale: torch.Tensor, hp,
                                stream=None) -> None:
    """zero_adam_shard_step on grad * grad_scale[0] (a one-element FP32 device
    tensor, e.g. the clip coefficient from zero_grad_norm_sq)."""
    n = master.numel()
    ptrs = [_dev(master, "master", (torch.float32,)), _dev(exp_avg, "exp_avg", (torch.float32,)),
            _dev(exp_avg_sq, "exp_avg_sq", (torch.float32,)), _dev(bf16_out, "bf16_out", _BF16_LIKE),
            _dev(grad, "grad", (torch.float32,)), _dev(grad_scale, "grad_scale", (torch.float32,))]
    if any(t.numel() != n for t in (exp_avg, exp_avg_sq, bf16_out, grad)) or grad_scale.numel() < 1:
        raise ValueError("zero_adam_shard_step_scaled: size mismatch")
    h = hparams(hp)
    check(load().zero_adam_shard_step_scaled(*ptrs, n, C.byref(h), _stream(stream)),
          "zero_adam_shard_step_scaled")


def _norm_args(name, shards, norm_sq_out, clip_coef_out):
    n = len(shards)
    if n < 1:
        raise ValueError(f"{name}: no shards")
    numel = shards[0].numel()
    sp = [_dev(t, f"shards[{k}]", (torch.float32,)) for k, t in enumerate(shards)]
    if any(t.numel() != numel for t in shards):
        raise ValueError(f"{name}: shards differ in size")
    op = _dev(norm_sq_out, "norm_sq_out", (torch.float64,))
    if norm_sq_out.numel() < 1:
        raise ValueError(f"{name}: norm_sq_out needs one element")
    cp = None
    if clip_coef_out is not None:
        cp = _dev(clip_coef_out, "clip_coef_out", (torch.float32,))
        if clip_coef_out.numel() < 1:
            raise ValueError(f"{name}: clip_coef_out needs one element")
    return _ptrs(sp), n, numel, op, cp


def zero_grad_norm_sq(shards: Sequence[torch.Tensor], workspace: torch.Tensor, norm_sq_out: torch.Tensor,
                      max_norm: float = 0.0, clip_coef_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """norm_sq_out[0] (FP64 device tensor) = sum of squares of all shards
    (deterministic order); clip_coef_out[0] (FP32) = min(1, max_norm/(norm+1e-6))
    when given.  workspace: FP64 device tensor of >= len(shards)*1024 elements."""
    sp, n, numel, op, cp = _norm_args("zero_grad_norm_sq", shards, norm_sq_out, clip_coef_out)
    wp = _dev(workspace, "workspace", (torch.float64,))
    check(load().zero_grad_norm_sq(sp, n, numel, wp, workspace.numel(), op, float(max_norm), cp,
                                   _stream(stream)), "zero_grad_norm_sq")


def zero_grad_norm_sq_no_alloc(shards: Sequence[torch.Tensor], norm_sq_out: torch.Tensor, max_norm: float = 0.0,
                               clip_coef_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """zero_grad_norm_sq with the partial sums in the library's own per-GPU
    array instead of a caller workspace: nothing is allocated.  Calls that
    overlap in time on one GPU race on that array."""
    sp, n, numel, op, cp = _norm_args("zero_grad_norm_sq_no_alloc", shards, norm_sq_out, clip_coef_out)
    check(load().zero_grad_norm_sq_no_alloc(sp, n, numel, op, float(max_norm), cp, _stream(stream)),
          "zero_grad_norm_sq_no_alloc")


def _fused_args(name, rank_grads, rank_weights, master, exp_avg, exp_avg_sq, bf16_out, grad_out, grad_acc):
    n_ranks, n_shards = len(rank_grads), len(master)
    if n_ranks < 1 or n_shards < 1:
        raise ValueError(f"{name}: need at least one rank and one owner")
    numel = rank_grads[0].numel()
    gp = [_dev(g, f"rank_grads[{r}]", _BF16_LIKE) for r, g in enumerate(rank_grads)]
    if any(g.numel() != numel for g in rank_grads):
        raise ValueError(f"{name}: rank contributions differ in size")
    if numel % n_shards:
        raise ValueError(f"{name}: numel not divisible by the number of owners")
    s = numel // n_shards
    tables = []
    for tname, ts, dt in (("master", master, (torch.float32,)), ("exp_avg", exp_avg, (torch.float32,)),
                          ("exp_avg_sq", exp_avg_sq, (torch.float32,)), ("bf16_out", bf16_out, _BF16_LIKE)):
        if len(ts) != n_shards or any(t.numel() != s for t in ts):
            raise ValueError(f"{name}: {tname} needs {n_shards} tensors of {s} elements")
        tables.append(_ptrs([_dev(t, f"{tname}[{k}]", dt) for k, t in enumerate(ts)]))
    go = None
    if grad_out is not None:
        if len(grad_out) != n_shards or any(t.numel() != s for t in grad_out):
            raise ValueError(f"{name}: grad_out needs one tensor per owner")
        go = _ptrs([_dev(t, f"grad_out[{k}]", (torch.float32,)) for k, t in enumerate(grad_out)])
    ga = None
    if grad_acc is not None:
        if len(grad_acc) != n_shards or any(t.numel() != s for t in grad_acc):
            raise ValueError(f"{name}: grad_acc needs one tensor per owner")
        ga = _ptrs([_dev(t, f"grad_acc[{k}]", (torch.float32,)) for k, t in enumerate(grad_acc)])
    w = np.ascontiguousarray(np.asarray(rank_weights, dtype=np.float32))
    if w.size != n_ranks:
        raise ValueError(f"{name}: one weight per rank")
    return (_ptrs(gp), w, n_ranks, numel, n_shards, tables, ga, go)


def zero_reduce_scatter_adam(rank_grads: Sequence[torch.Tensor], rank_weights, master, exp_avg, exp_avg_sq,
                             bf16_out, hp, grad_out=None, grad_acc=None, stream=None) -> None:
    """Fused reduce-scatter + owner Adam update: for each owner k, the reduced
    shard k of the rank contributions (plus grad_acc[k] when given) updates
    (master[k], exp_avg[k], exp_avg_sq[k]) and writes bf16_out[k]; grad_out
    (optional list) receives the gradient used.  Bit-identical to
    zero_reduce_scatter (accumulate mode with grad_acc) followed by
    zero_adam_shard_step on every owner."""
    gp, w, n_ranks, numel, n_shards, tables, ga, go = _fused_args(
        "zero_reduce_scatter_adam", rank_grads, rank_weights, master, exp_avg, exp_avg_sq, bf16_out, grad_out,
        grad_acc)
    h = hparams(hp)
    check(load().zero_reduce_scatter_adam(gp, w.ctypes.data_as(_lib.FP), n_ranks, numel, n_shards,
                                          *tables, ga, go, C.byref(h), _stream(stream)),
          "zero_reduce_scatter_adam")


# ------------------------------------------------------------ graph-capturable forms
ADAM_SCALARS_FLOATS = len(_lib.AdamScalars._fields_)


def adam_scalars_tensor(hp, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The step's scalars (zero_adam_scalars_compute) as a float32 tensor in the
    struct's field order, ready to be copied into the device struct that the
    _dev calls read.  out: an existing CPU float32 tensor to fill (e.g. pinned)."""
    sc = _lib.AdamScalars()
    check(load().zero_adam_scalars_compute(C.byref(hparams(hp)), C.byref(sc)), "zero_adam_scalars_compute")
    vals = [getattr(sc, f) for f, _ in _lib.AdamScalars._fields_]
    if out is None:
        return torch.tensor(vals, dtype=torch.float32)
    if out.device.type != "cpu" or out.dtype != torch.float32 or out.numel() < ADAM_SCALARS_FLOATS:
        raise ValueError(f"adam_scalars_tensor: out must be a CPU float32 tensor of >= {ADAM_SCALARS_FLOATS} elements")
    out.numpy()[:ADAM_SCALARS_FLOATS] = np.array(vals, dtype=np.float32)
    return out


def _scalars_dev(scalars_dev: torch.Tensor) -> int:
    ptr = _dev(scalars_dev, "scalars_dev", (torch.float32,))
    if scalars_dev.numel() < ADAM_SCALARS_FLOATS:
        raise ValueError(f"scalars_dev: needs {ADAM_SCALARS_FLOATS} float32 elements")
    return ptr


def zero_adam_shard_step_dev(master, exp_avg, exp_avg_sq, bf16_out, grad, scalars_dev: torch.Tensor,
                             grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """zero_adam_shard_step with the step's scalars read from scalars_dev (a
    device float32 tensor holding adam_scalars_tensor(hp)) when the kernel runs,
    so that a captured graph replays with new scalars; grad_scale as in
    zero_adam_shard_step_scaled, or None."""
    n = master.numel()
    ptrs = [_dev(master, "master", (torch.float32,)), _dev(exp_avg, "exp_avg", (torch.float32,)),
            _dev(exp_avg_sq, "exp_avg_sq", (torch.float32,)), _dev(bf16_out, "bf16_out", _BF16_LIKE),
            _dev(grad, "grad", (torch.float32,))]
    if any(t.numel() != n for t in (exp_avg, exp_avg_sq, bf16_out, grad)):
        raise ValueError("zero_adam_shard_step_dev: all buffers must have the same numel")
    gs = None
    if grad_scale is not None:
        gs = _dev(grad_scale, "grad_scale", (torch.float32,))
    check(load().zero_adam_shard_step_dev(*ptrs, gs, n, _scalars_dev(scalars_dev), _stream(stream)),
          "zero_adam_shard_step_dev")


def zero_reduce_scatter_adam_dev(rank_grads, rank_weights, master, exp_avg, exp_avg_sq, bf16_out,
                                 scalars_dev: torch.Tensor, grad_out=None, grad_acc=None, stream=None) -> None:
    """zero_reduce_scatter_adam with the step's scalars read from scalars_dev
    when the kernels run (see zero_adam_shard_step_dev)."""
    gp, w, n_ranks, numel, n_shards, tables, ga, go = _fused_args(
        "zero_reduce_scatter_adam_dev", rank_grads, rank_weights, master, exp_avg, exp_avg_sq, bf16_out,
        grad_out, grad_acc)
    check(load().zero_reduce_scatter_adam_dev(gp, w.ctypes.data_as(_lib.FP), n_ranks, numel, n_shards,
                                              *tables, ga, go, _scalars_dev(scalars_dev), _stream(stream)),
          "zero_reduce_scatter_adam_dev")


def zero_adam_scalars_fetch(ring_host: torch.Tensor, cursor_dev: torch.Tensor, scalars_dev: torch.Tensor,
                            stream=None) -> None:
    """One kernel on the stream: scalars_dev <- slot (cursor mod ring length)
    of ring_host, then cursor + 1.  ring_host: a pinned CPU float32 tensor of
    ring_len * ADAM_SCALARS_FLOATS elements (ring_len a power of two), one
    adam_scalars_tensor per slot; cursor_dev: a one-element int32 device tensor,
    zero before the first replay; scalars_dev: as for the _dev calls."""
    if ring_host.device.type != "cpu" or ring_host.dtype != torch.float32 or not ring_host.is_contiguous():
        raise ValueError("zero_adam_scalars_fetch: ring_host must be a contiguous CPU float32 tensor")
    if not ring_host.is_pinned():
        raise ValueError("zero_adam_scalars_fetch: ring_host must be pinned (pin_memory=True)")
    if ring_host.numel() == 0 or ring_host.numel() % ADAM_SCALARS_FLOATS:
        raise ValueError(f"zero_adam_scalars_fetch: ring_host must hold a multiple of {ADAM_SCALARS_FLOATS} floats")
    cur = _dev(cursor_dev, "cursor_dev", (torch.int32,))
    if cursor_dev.numel() != 1:
        raise ValueError("zero_adam_scalars_fetch: cursor_dev must have one element")
    check(load().zero_adam_scalars_fetch(ring_host.data_ptr(), ring_host.numel() // ADAM_SCALARS_FLOATS, cur,
                                         _scalars_dev(scalars_dev), _stream(stream)), "zero_adam_scalars_fetch")


def zero_all_gather_layer(shards: Sequence[torch.Tensor], full_view: torch.Tensor, stream=None) -> None:
    """full_view = concatenation of the shards' bytes in owner order."""
    n = len(shards)
    if n < 1:
        raise ValueError("zero_all_gather_layer: no shards")
    nbytes = shards[0].numel() * shards[0].element_size()
    sp = [_dev(s, f"shards[{k}]", (s.dtype,)) for k, s in enumerate(shards)]
    if any(s.numel() * s.element_size() != nbytes for s in shards):
        raise ValueError("zero_all_gather_layer: shards differ in size")
    vp = _dev(full_view, "full_view", (full_view.dtype,))
    if full_view.numel() * full_view.element_size() != n * nbytes:
        raise ValueError("zero_all_gather_layer: full_view must hold exactly n_shards*shard_bytes bytes")
    check(load().zero_all_gather_layer(_ptrs(sp), n, nbytes, vp, _stream(stream)), "zero_all_gather_layer")


# ------------------------------------------------------------ Muon step
# The quintic step's coefficients that raise small singular values fastest
# while keeping the others near 1, five times.
NS_COEFS = ((3.4445, -4.7750, 2.0315),) * 5


def muon_hparams(hp) -> MuonHparams:
    """lr, momentum, weight_decay (0) and nesterov (True) as the C struct."""
    if isinstance(hp, MuonHparams):
        return hp
    return MuonHparams(float(hp["lr"]), float(hp["momentum"]), float(hp.get("weight_decay", 0.0)),
                       int(bool(hp.get("nesterov", True))))


def _one_float(t: Optional[torch.Tensor], what: str):
    if t is None:
        return None
    ptr = _dev(t, what, (torch.float32,))
    if t.numel() < 1:
        raise ValueError(f"{what}: needs one element")
    return ptr


def zero_muon_momentum(momentum: torch.Tensor, direction_out: torch.Tensor, grad: torch.Tensor, hp,
                       grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """Momentum step of an owner's shard: momentum (FP32) in place, direction_out
    (BF16) written; grad_scale: a one-element FP32 device tensor that multiplies
    the gradient (the clip coefficient)."""
    n = momentum.numel()
    ptrs = _dev_same(n, "zero_muon_momentum: all buffers must have the same numel", (momentum, "momentum", _FP32),
                     (direction_out, "direction_out", _BF16_LIKE), (grad, "grad", _FP32))
    h = muon_hparams(hp)
    check(load().zero_muon_momentum(*ptrs, _one_float(grad_scale, "grad_scale"), n, C.byref(h), _stream(stream)),
          "zero_muon_momentum")


def zero_reduce_scatter_muon(rank_grads: Sequence[torch.Tensor], rank_weights, momentum: Sequence[torch.Tensor],
                             direction_out: Sequence[torch.Tensor], hp, grad_acc=None, stream=None) -> None:
    """Fused reduce-scatter + momentum step: for each owner k, the reduced shard
    k (plus grad_acc[k] when given) moves momentum[k] and writes
    direction_out[k].  Bit-identical to zero_reduce_scatter (accumulate mode
    with grad_acc) followed by zero_muon_momentum on every owner."""
    name = "zero_reduce_scatter_muon"
    n_ranks, n_shards = len(rank_grads), len(momentum)
    if n_ranks < 1 or n_shards < 1:
        raise ValueError(f"{name}: need at least one rank and one owner")
    numel = rank_grads[0].numel()
    grads = _dev_table(rank_grads, "rank_grads", _BF16_LIKE, numel, "zero_reduce_scatter_muon: rank contributions "
                                                                    "differ in size")
    if numel % n_shards:
        raise ValueError(f"{name}: numel not divisible by the number of owners")
    if len(direction_out) != n_shards or (grad_acc is not None and len(grad_acc) != n_shards):
        raise ValueError(f"{name}: one tensor per owner in each of momentum, direction_out and grad_acc")
    part, size = numel // n_shards, "zero_reduce_scatter_muon: an owner's tensors need numel / owners elements"
    m = _dev_table(momentum, "momentum", _FP32, part, size)
    u = _dev_table(direction_out, "direction_out", _BF16_LIKE, part, size)
    acc = None if grad_acc is None else _dev_table(grad_acc, "grad_acc", _FP32, part, size)
    w = rank_weights.tolist() if hasattr(rank_weights, "tolist") else rank_weights
    if len(w) != n_ranks:
        raise ValueError(f"{name}: one weight per rank")
    h = muon_hparams(hp)
    check(load().zero_reduce_scatter_muon(grads, (C.c_float * n_ranks)(*w), n_ranks, numel, n_shards, m, u, acc,
                                          C.byref(h), _stream(stream)), name)


def _stack(t: torch.Tensor, what: str, dtypes):
    """(pointer, matrices, rows, cols, row stride, matrix stride) of a 2-D or 3-D
    tensor whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dim() not in (2, 3):
        raise TypeError(f"{what}: expected a 2-D or 3-D torch.Tensor")
    _on_device(t, what, dtypes)
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        shape, stride = (1, *shape), (0, *stride)
    mats, rows, cols = shape
    if cols > 1 and stride[2] != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), mats, rows, cols, stride[1] if rows > 1 else cols, stride[0] if mats > 1 else 0


def zero_newton_schulz_workspace(g: torch.Tensor) -> torch.Tensor:
    """A device workspace for zero_newton_schulz on tensors of g's shape (2-D, or
    3-D: a stack of matrices)."""
    shape = tuple(g.shape) if g.dim() == 3 else (1, *g.shape)
    if len(shape) != 3:
        raise ValueError("zero_newton_schulz_workspace: expected a 2-D or 3-D tensor")
    n = C.c_int64()
    check(load().zero_newton_schulz_workspace(*shape, C.byref(n)), "zero_newton_schulz_workspace")
    return torch.empty(n.value, dtype=torch.uint8, device=g.device)


def zero_newton_schulz(g: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, coefs=NS_COEFS,
                       scale: float = 1.0, stream=None) -> None:
    """out (BF16) = scale * the Newton-Schulz orthogonalisation of each matrix of
    g (BF16 or FP32; [rows, cols] or [matrices, rows, cols], rows contiguous,
    other strides free).  coefs: one (a, b, c) per step."""
    ip, mats, rows, cols, irow, imat = _stack(g, "g", (torch.bfloat16, torch.float32))
    op, omats, orows, ocols, orow, omat = _stack(out, "out", (torch.bfloat16,))
    if (mats, rows, cols) != (omats, orows, ocols):
        raise ValueError("zero_newton_schulz: out must have g's shape")
    c = coefs.tolist() if hasattr(coefs, "tolist") else coefs
    if any(not hasattr(abc, "__len__") or len(abc) != 3 for abc in c):
        raise ValueError("zero_newton_schulz: coefs needs one (a, b, c) per step")
    flat = (C.c_float * (3 * len(c)))(*[v for abc in c for v in abc])
    wp = _dev(workspace, "workspace", (torch.uint8,))
    check(load().zero_newton_schulz(ip, _lib.ZERO_FP32 if g.dtype == torch.float32 else _lib.ZERO_BF16, irow, imat,
                                    op, orow, omat, mats, rows, cols, flat, len(c), float(scale), wp,
                                    workspace.numel(), _stream(stream)), "zero_newton_schulz")


def zero_muon_shard_step(master: torch.Tensor, bf16_out: torch.Tensor, update: torch.Tensor, hp,
                         lr_dev: Optional[torch.Tensor] = None, stream=None) -> None:
    """Owner update: master (FP32) -= lr * (update + wd * master), bf16_out
    written; lr_dev: a one-element FP32 device tensor read in place of hp's lr."""
    n = master.numel()
    ptrs = _dev_same(n, "zero_muon_shard_step: all buffers must have the same numel", (master, "master", _FP32),
                     (bf16_out, "bf16_out", _BF16_LIKE), (update, "update", _BF16_LIKE))
    h = muon_hparams(hp)
    check(load().zero_muon_shard_step(*ptrs, n, C.byref(h), _one_float(lr_dev, "lr_dev"), _stream(stream)),
          "zero_muon_shard_step")


# ------------------------------------------------------------ 8-bit activations, feed-forward block
ACT8_FORMATS = {"int8": _lib.ZERO_ACT8_INT8, "e4m3": _lib.ZERO_ACT8_E4M3}
FFN_ACTIVATIONS = {"silu": _lib.ZERO_FFN_SILU, "gelu": _lib.ZERO_FFN_GELU, "relu": _lib.ZERO_FFN_RELU}
_UINT8 = (torch.uint8,)
_BF16 = (torch.bfloat16,)
_ACT8_DTYPES = {torch.bfloat16: _lib.ZERO_BF16, torch.float32: _lib.ZERO_FP32}


def _choice(table: Mapping[str, int], name, what: str) -> int:
    if name not in table:
        raise ValueError(f"{what}: {name!r} is none of {', '.join(table)}")
    return table[name]


def _rows(t: torch.Tensor, what: str, dtypes):
    """(pointer, rows, cols, row stride) of a matrix whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise TypeError(f"{what}: expected a 2-D torch.Tensor")
    if not (t.is_cuda and t.get_device() == _current_device() and t.dtype in dtypes):
        _on_device(t, what, dtypes)
    rows, cols = t.shape
    row, col = t.stride()
    if cols > 1 and col != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), rows, cols, row if rows > 1 else cols


def _whole(device: int, dtypes, *matrices) -> list:
    """The pointers of contiguous (tensor, name, rows, cols), without a call for each
    that passes: a pass of the feed-forward block has up to sixteen."""
    ptrs = []
    for t, what, rows, cols in matrices:
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == device and t.dtype in dtypes
                and t.is_contiguous()):
            _dev(t, what, dtypes)
        if t.shape != (rows, cols):
            raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {(rows, cols)}")
        ptrs.append(t.data_ptr())
    return ptrs


def zero_act8_buffers(rows: int, cols: int, device="cuda"):
    """Buffers (codes, scales) of an 8-bit checkpoint of rows x cols values."""
    return (torch.empty(rows, cols, dtype=torch.uint8, device=device),
            torch.empty(rows, -(-cols // _lib.ZERO_ACT8_BLOCK), dtype=torch.uint8, device=device))


def zero_act8_save(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, format: str = "int8",
                   stream=None) -> None:
    """x (BF16 or FP32, [rows, cols], row stride free) as 8 bits a value and a power
    of two per 32 neighbours of a row; format "int8" or "e4m3"."""
    xp, rows, cols, row = _rows(x, "x", _ACT8_DTYPES)
    cp, sp = _whole(_current_device(), _UINT8, (codes, "codes", rows, cols), (scales, "scales", rows, (cols + 31) // 32))
    check(load().zero_act8_save(xp, _ACT8_DTYPES[x.dtype], row, rows, cols, _choice(ACT8_FORMATS, format, "format"), cp,
                                sp, _stream(stream)), "zero_act8_save")


def zero_act8_load(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, format: str = "int8",
                   stream=None) -> None:
    """out (BF16 or FP32, [rows, cols], row stride free) = the checkpoint's values."""
    op, rows, cols, row = _rows(out, "out", _ACT8_DTYPES)
    cp, sp = _whole(_current_device(), _UINT8, (codes, "codes", rows, cols), (scales, "scales", rows, (cols + 31) // 32))
    check(load().zero_act8_load(cp, sp, rows, cols, _choice(ACT8_FORMATS, format, "format"), op,
                                _ACT8_DTYPES[out.dtype], row, _stream(stream)), "zero_act8_load")


class FfnCheckpoint:
    """What a feed-forward block's forward pass keeps for its backward pass: x, x Wg^T
    and x Wu^T, each as the (codes, scales) of an 8-bit checkpoint."""

    def __init__(self, x, gate, up, format: str = "int8"):
        self.x, self.gate, self.up = tuple(x), tuple(gate), tuple(up)
        self.format = format
        _choice(ACT8_FORMATS, format, "format")

    @classmethod
    def empty(cls, tokens: int, model: int, hidden: int, format: str = "int8", device="cuda") -> "FfnCheckpoint":
        return cls(zero_act8_buffers(tokens, model, device), zero_act8_buffers(tokens, hidden, device),
                   zero_act8_buffers(tokens, hidden, device), format)

    def first(self, tokens: int) -> "FfnCheckpoint":
        """The first rows of these buffers, as a checkpoint of so many tokens."""
        return FfnCheckpoint(*([t[:tokens] for t in held] for held in (self.x, self.gate, self.up)), self.format)

    def buffers(self, tokens: int, model: int, hidden: int) -> _lib.FfnCheckpointBuffers:
        (xc, xs), (gc, gs), (uc, us) = self.x, self.gate, self.up
        mb, hb = (model + 31) // 32, (hidden + 31) // 32
        return _lib.FfnCheckpointBuffers(*_whole(
            _current_device(), _UINT8, (xc, "checkpoint.x codes", tokens, model), (xs, "checkpoint.x scales", tokens, mb),
            (gc, "checkpoint.gate codes", tokens, hidden), (gs, "checkpoint.gate scales", tokens, hb),
            (uc, "checkpoint.up codes", tokens, hidden), (us, "checkpoint.up scales", tokens, hb)),
            ACT8_FORMATS[self.format])


def zero_ffn_workspace(tokens: int, model: int, hidden: int, backward: bool = False, unaligned: bool = False,
                       device="cuda") -> torch.Tensor:
    """A device workspace for zero_ffn_forward or, with backward, zero_ffn_backward of up to
    `tokens` tokens.  unaligned: the weights' addresses are no multiples of 16 bytes."""
    n = C.c_int64()
    flags = (_lib.ZERO_FFN_BACKWARD if backward else 0) | (_lib.ZERO_FFN_UNALIGNED if unaligned else 0)
    check(load().zero_ffn_workspace(tokens, model, hidden, flags, C.byref(n)), "zero_ffn_workspace")
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def _hidden(w_gate: torch.Tensor) -> int:
    if not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 2:
        raise TypeError("w_gate: expected a 2-D torch.Tensor")
    return w_gate.shape[0]


def zero_ffn_forward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, y: torch.Tensor,
                     workspace: torch.Tensor, activation: str = "silu", checkpoint: Optional[FfnCheckpoint] = None,
                     stream=None) -> None:
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T, all BF16; x, y [tokens, model] with free row
    strides, w_gate and w_up [hidden, model], w_down [model, hidden].  activation: "silu", "gelu"
    (tanh) or "relu".  checkpoint: written, for zero_ffn_backward."""
    xp, tokens, model, xrow = _rows(x, "x", _BF16)
    yp, yrows, ycols, yrow = _rows(y, "y", _BF16)
    if yrows != tokens or ycols != model:
        raise ValueError("zero_ffn_forward: y must have x's shape")
    hidden = _hidden(w_gate)
    w = _whole(_current_device(), _BF16, (w_gate, "w_gate", hidden, model), (w_up, "w_up", hidden, model),
               (w_down, "w_down", model, hidden))
    held = None if checkpoint is None else C.byref(checkpoint.buffers(tokens, model, hidden))
    check(load().zero_ffn_forward(xp, xrow, tokens, model, hidden, *w, _choice(FFN_ACTIVATIONS, activation, "activation"),
                                  yp, yrow, held, _dev(workspace, "workspace", _UINT8), workspace.numel(),
                                  _stream(stream)), "zero_ffn_forward")


def zero_ffn_backward(dy: torch.Tensor, checkpoint: FfnCheckpoint, w_gate: torch.Tensor, w_up: torch.Tensor,
                      w_down: torch.Tensor, dx: Optional[torch.Tensor], d_gate: torch.Tensor, d_up: torch.Tensor,
                      d_down: torch.Tensor, workspace: torch.Tensor, activation: str = "silu", stream=None) -> None:
    """Gradients of zero_ffn_forward from its checkpoint: dx [tokens, model] (None: not
    wanted) and d_gate, d_up, d_down of the weights' shapes, all BF16, written."""
    dyp, tokens, model, dyrow = _rows(dy, "dy", _BF16)
    dxp, dxrow = None, model
    if dx is not None:
        dxp, dxrows, dxcols, dxrow = _rows(dx, "dx", _BF16)
        if dxrows != tokens or dxcols != model:
            raise ValueError("zero_ffn_backward: dx must have dy's shape")
    hidden = _hidden(w_gate)
    wg, wu, wd, *d = _whole(
        _current_device(), _BF16, (w_gate, "w_gate", hidden, model), (w_up, "w_up", hidden, model),
        (w_down, "w_down", model, hidden), (d_gate, "d_gate", hidden, model), (d_up, "d_up", hidden, model),
        (d_down, "d_down", model, hidden))
    held = checkpoint.buffers(tokens, model, hidden)
    check(load().zero_ffn_backward(dyp, dyrow, tokens, model, hidden, C.byref(held), wg, wu, wd,
                                   _choice(FFN_ACTIVATIONS, activation, "activation"), dxp, dxrow, *d,
                                   _dev(workspace, "workspace", _UINT8), workspace.numel(), _stream(stream)),
          "zero_ffn_backward")


def zero_last_path_vectorized() -> int:
    return int(load().zero_last_path_vectorized())


# ------------------------------------------------------------ offload engine
class ZeroOffload:
    """Two-slot host-offloaded gradient shard (zero_offload_* in include/zero.h).

    host_shard: pinned FP32 CPU tensor [shard_numel]; slot_contrib: two BF16
    device tensors [n_ranks*chunk_numel]; slot_f32: two FP32 device tensors
    [chunk_numel].  The tensors must outlive the handle."""

    def __init__(self, n_ranks: int, shard_numel: int, chunk_numel: int, host_shard: torch.Tensor,
                 slot_contrib: Sequence[torch.Tensor], slot_f32: Sequence[torch.Tensor]):
        if host_shard.device.type != "cpu" or host_shard.dtype != torch.float32 or not host_shard.is_contiguous():
            raise ValueError("host_shard: contiguous float32 CPU tensor required")
        if not host_shard.is_pinned():
            raise ValueError("host_shard: must be pinned host memory")
        if host_shard.numel() != shard_numel:
            raise ValueError("host_shard: numel != shard_numel")
        if len(slot_contrib) != 2 or len(slot_f32) != 2:
            raise ValueError("two slots required")
        cp = [_dev(t, f"slot_contrib[{s}]", _BF16_LIKE) for s, t in enumerate(slot_contrib)]
        fp = [_dev(t, f"slot_f32[{s}]", (torch.float32,)) for s, t in enumerate(slot_f32)]
        if any(t.numel() != n_ranks * chunk_numel for t in slot_contrib):
            raise ValueError("slot_contrib: numel must be n_ranks*chunk_numel")
        if any(t.numel() != chunk_numel for t in slot_f32):
            raise ValueError("slot_f32: numel must be chunk_numel")
        self._keep = (host_shard, tuple(slot_contrib), tuple(slot_f32))
        self.n_ranks, self.shard_numel, self.chunk_numel = n_ranks, shard_numel, chunk_numel
        self.n_chunks = -(-shard_numel // chunk_numel)
        h = C.c_void_p()
        check(load().zero_offload_create(n_ranks, shard_numel, chunk_numel, host_shard.data_ptr(),
                                         _ptrs(cp), _ptrs(fp), C.byref(h)), "zero_offload_create")
        self._h = h

    def chunk_len(self, c: int) -> int:
        return min(self.chunk_numel, self.shard_numel - c * self.chunk_numel)

    def reduce(self, chunk: int, micro_batch: int, rank_weights, stream=None) -> None:
        w = np.ascontiguousarray(np.asarray(rank_weights, dtype=np.float32))
        if w.size != self.n_ranks:
            raise ValueError("one weight per rank")
        check(load().zero_offload_stream(self._h, _lib.ZERO_OFFLOAD_REDUCE, chunk, micro_batch,
                                         w.ctypes.data_as(_lib.FP), None, None, None, None, None,
                                         _stream(stream)), "zero_offload_stream(REDUCE)")

    def adam(self, chunk: int, master, exp_avg, exp_avg_sq, bf16_out, hp, stream=None) -> None:
        ptrs = [_dev(master, "master", (torch.float32,)), _dev(exp_avg, "exp_avg", (torch.float32,)),
                _dev(exp_avg_sq, "exp_avg_sq", (torch.float32,)), _dev(bf16_out, "bf16_out", _BF16_LIKE)]
        if any(t.numel() != self.shard_numel for t in (master, exp_avg, exp_avg_sq, bf16_out)):
            raise ValueError("state tensors must cover the whole shard")
        h = hparams(hp)
        check(load().zero_offload_stream(self._h, _lib.ZERO_OFFLOAD_ADAM, chunk, 0, None, *ptrs,
                                         C.byref(h), _stream(stream)), "zero_offload_stream(ADAM)")

    def reduce_adam(self, chunk: int, micro_batch: int, rank_weights, master, exp_avg, exp_avg_sq, bf16_out, hp,
                    stream=None) -> None:
        """The last micro-batch of `chunk`: reduce, add to the host accumulation
        and update in one pass (no copy back to the host)."""
        w = np.ascontiguousarray(np.asarray(rank_weights, dtype=np.float32))
        if w.size != self.n_ranks:
            raise ValueError("one weight per rank")
        ptrs = [_dev(master, "master", (torch.float32,)), _dev(exp_avg, "exp_avg", (torch.float32,)),
                _dev(exp_avg_sq, "exp_avg_sq", (torch.float32,)), _dev(bf16_out, "bf16_out", _BF16_LIKE)]
        if any(t.numel() != self.shard_numel for t in (master, exp_avg, exp_avg_sq, bf16_out)):
            raise ValueError("state tensors must cover the whole shard")
        h = hparams(hp)
        check(load().zero_offload_stream(self._h, _lib.ZERO_OFFLOAD_REDUCE_ADAM, chunk, micro_batch,
                                         w.ctypes.data_as(_lib.FP), *ptrs, C.byref(h), _stream(stream)),
              "zero_offload_stream(REDUCE_ADAM)")

    def sync(self) -> None:
        check(load().zero_offload_sync(self._h), "zero_offload_sync")

    def close(self) -> None:
        if getattr(self, "_h", None):
            st = load().zero_offload_destroy(self._h)
            self._h = None
            check(st, "zero_offload_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def zero_offload_create(n_ranks, shard_numel, chunk_numel, host_shard, slot_contrib, slot_f32) -> ZeroOffload:
    return ZeroOffload(n_ranks, shard_numel, chunk_numel, host_shard, slot_contrib, slot_f32)


def zero_offload_stream(h: ZeroOffload, op: int, chunk: int, micro_batch: int = 0, rank_weights=None,
                        master=None, exp_avg=None, exp_avg_sq=None, bf16_out=None, hp=None, stream=None):
    if op == _lib.ZERO_OFFLOAD_REDUCE:
        return h.reduce(chunk, micro_batch, rank_weights, stream)
    if op == _lib.ZERO_OFFLOAD_REDUCE_ADAM:
        return h.reduce_adam(chunk, micro_batch, rank_weights, master, exp_avg, exp_avg_sq, bf16_out, hp, stream)
    return h.adam(chunk, master, exp_avg, exp_avg_sq, bf16_out, hp, stream)


def zero_offload_sync(h: ZeroOffload) -> None:
    h.sync()


def zero_offload_destroy(h: ZeroOffload) -> None:
    h.close()
