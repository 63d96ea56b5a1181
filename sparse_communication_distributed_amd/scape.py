"""ctypes binding of libscape.so (C ABI declared in include/scape.h).

Argument marshalling only: every step of the optimizer path runs in the HIP
library.  Tensors are torch device tensors (fp32 / uint8 blobs); streams are
torch streams (default: the current stream).  There is no fallback: if the
library is missing, loading raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
# SCAPE_LIB may name another build of the same library (same ABI).
LIB_PATH = os.environ.get("SCAPE_LIB") or os.path.join(_PKG, "libscape.so")

c_int64, c_int32, c_int, c_size_t = ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_size_t
c_float, c_void_p, c_char_p = ctypes.c_float, ctypes.c_void_p, ctypes.c_char_p

STATUS = {0: "SCAPE_OK", 1: "SCAPE_EINVAL", 2: "SCAPE_ESHAPE", 3: "SCAPE_EWORKSPACE", 4: "SCAPE_EHIP",
          5: "SCAPE_EMASK"}


class Dims(ctypes.Structure):
    _fields_ = [("n", c_int64), ("num_partitions", c_int32), ("num_workers", c_int32)]


class Betas(ctypes.Structure):
    _fields_ = [("beta1", c_float), ("beta2", c_float), ("eps", c_float), ("weight_decay", c_float)]


class MaskView(ctypes.Structure):
    _fields_ = [("bits", c_void_p), ("idx", c_void_p), ("tile_off", c_void_p), ("meta", c_void_p)]


class BiasState(ctypes.Structure):
    """scape_bias_state: beta^t products (binary64) and the fp32 reciprocals."""
    _fields_ = [("beta1_pow", ctypes.c_double), ("beta2_pow", ctypes.c_double), ("ibc1", c_float), ("ibc2", c_float)]


class Matrix(ctypes.Structure):
    """scape_matrix: rows ld elements apart, of one of the scape_dtype types."""
    _fields_ = [("data", c_void_p), ("ld", c_int64), ("dtype", c_int32)]


class ActView(ctypes.Structure):
    """scape_act_view: codes and scale bytes of an 8-bit checkpoint."""
    _fields_ = [("codes", c_void_p), ("scales", c_void_p)]


class ScapeError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {detail}")


# name -> (restype, argtypes); mirrors include/scape.h
_SIGS = {
    "scape_tile_elems": (c_int64, []),
    "scape_step_pass_count": (ctypes.c_int32, [ctypes.POINTER(Dims), c_int64]),
    "scape_mask_bytes": (c_size_t, [ctypes.POINTER(Dims), c_int64]),
    "scape_mask_slot": (c_int, [ctypes.POINTER(Dims), c_int64, c_void_p, c_int, ctypes.POINTER(MaskView)]),
    "scape_workspace_bytes": (c_size_t, [ctypes.POINTER(Dims), c_int64]),
    "scape_mask_topk": (c_int, [ctypes.POINTER(Dims), c_int64, c_void_p, MaskView, c_void_p, c_size_t, c_void_p]),
    "scape_compress": (c_int, [ctypes.POINTER(Dims), c_int64, c_void_p, c_void_p, MaskView, c_void_p, c_void_p]),
    "scape_reduce_sparse": (c_int, [ctypes.POINTER(Dims), c_int64, c_void_p, c_void_p, c_void_p]),
    "scape_adams_update": (c_int, [ctypes.POINTER(Dims), c_int64, c_void_p, c_void_p, c_void_p, c_void_p,
                                   MaskView, Betas, c_float, c_int64, c_void_p]),
    "scape_step": (c_int, [ctypes.POINTER(Dims), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                           c_int64, Betas, c_float, c_int64, c_void_p, c_size_t, c_void_p]),
    "scape_step_noalloc_max_bytes": (c_size_t, []),
    "scape_step_noalloc": (c_int, [ctypes.POINTER(Dims), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_int64, Betas, c_float, c_int64, c_void_p]),
    "scape_bias_state_at": (c_int, [Betas, c_int64, ctypes.POINTER(BiasState)]),
    "scape_step_graph": (c_int, [ctypes.POINTER(Dims), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_int64, Betas, c_float, c_int32, c_void_p, c_void_p, c_size_t, c_void_p]),
    "scape_mask_overlap": (c_int, [ctypes.POINTER(Dims), c_int64, MaskView, MaskView, c_void_p, c_void_p]),
    "scape_count_nonfinite": (c_int, [c_void_p, c_int64, c_void_p, c_void_p]),
    "scape_offload_stage_bytes": (c_size_t, [ctypes.POINTER(Dims), c_int64, c_int32]),
    "scape_step_offload": (c_int, [ctypes.POINTER(Dims), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_int64, Betas, c_float, c_int64, c_void_p, c_size_t, c_void_p, c_size_t, c_int32,
                                   c_void_p, c_void_p, c_void_p]),
    "scape_mask_union": (c_int, [ctypes.POINTER(Dims), c_int64, c_void_p, MaskView, c_void_p, c_void_p]),
    "scape_dense_adams_step": (c_int, [ctypes.POINTER(Dims), c_void_p, c_void_p, c_void_p, c_void_p, Betas, c_float,
                                       c_int64, c_void_p]),
    "scape_mask_check": (c_int, [ctypes.POINTER(Dims), c_int64, MaskView, c_void_p, c_void_p]),
    "scape_shard_partitions": (c_int, [ctypes.POINTER(Dims), c_int32, ctypes.POINTER(c_int32),
                                       ctypes.POINTER(c_int32)]),
    "scape_shard_select_initial": (c_int, [ctypes.POINTER(Dims), c_int64, c_int32, c_void_p, c_void_p, c_void_p,
                                           c_void_p, Betas, c_void_p, c_size_t, c_void_p]),
    "scape_shard_compress": (c_int, [ctypes.POINTER(Dims), c_int64, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, Betas, c_int64, c_void_p, c_size_t, c_void_p]),
    "scape_shard_update": (c_int, [ctypes.POINTER(Dims), c_int64, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_void_p, Betas, c_float, c_int64, c_void_p]),
    "scape_act_block": (c_int32, []),
    "scape_act_bytes": (c_size_t, [c_int64, c_int64]),
    "scape_act_slot": (c_int, [c_int64, c_int64, c_void_p, ctypes.POINTER(ActView)]),
    "scape_act_pack": (c_int, [c_int64, c_int64, Matrix, ActView, c_void_p]),
    "scape_act_unpack": (c_int, [c_int64, c_int64, ActView, c_void_p, Matrix, c_void_p]),
    "scape_rmsnorm_pack": (c_int, [c_int64, c_int64, Matrix, Matrix, c_void_p, c_float, Matrix, Matrix, ActView,
                                   c_void_p, c_void_p]),
    "scape_rmsnorm_workspace_bytes": (c_size_t, [c_int64, c_int64]),
    "scape_rmsnorm_backward": (c_int, [c_int64, c_int64, Matrix, ActView, c_void_p, c_void_p, Matrix, Matrix,
                                       c_void_p, c_int32, c_void_p, c_size_t, c_void_p]),
    "scape_wgrad_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, Matrix]),
    "scape_wgrad_splits": (c_int32, [c_int64, c_int64, c_int64, c_int32, ctypes.POINTER(c_int32),
                                     ctypes.POINTER(c_int32)]),
    "scape_wgrad": (c_int, [c_int64, c_int64, c_int64, Matrix, ActView, c_void_p, c_void_p, c_void_p, c_int32,
                            c_void_p, c_size_t, c_void_p]),
    "scape_status_string": (c_char_p, [c_int]),
    "scape_last_error": (c_char_p, []),
    "scape_profile_stages": (c_int, []),
    "scape_profile_stage_name": (c_char_p, [c_int]),
    "scape_profile_enable": (c_int, [c_int]),
    "scape_profile_collect": (c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(c_int64)]),
}

_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Loads libscape.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_communication_distributed_amd.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype, f.argtypes = res, args
        _lib = h
    return _lib


def exported_names() -> Tuple[str, ...]:
    return tuple(_SIGS)


def _check(status: int) -> None:
    if status != 0:
        raise ScapeError(status, lib().scape_last_error().decode())


def dims(n: int, P: int, K: int) -> Dims:
    return Dims(int(n), int(P), int(K))


def betas(beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0) -> Betas:
    return Betas(beta1, beta2, eps, weight_decay)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _need(t, name: str, numel: int, dtype: str = "float32", pinned: bool = False) -> None:
    """Checks a tensor argument before its address reaches the device: a
    host tensor, a wrong dtype or a short buffer would otherwise turn into a
    device memory fault.  None passes (the library reports null pointers)."""
    if t is None:
        return
    import torch
    if pinned:
        if t.is_cuda or not t.is_pinned():
            raise ValueError(f"{name} must be pinned host memory")
    elif not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if dtype is not None and t.dtype != getattr(torch, dtype):
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() * t.element_size() < numel * (t.element_size() if dtype is not None else 1):
        raise ValueError(f"{name} is too small: {t.numel()} elements of {t.element_size()} bytes, "
                         f"needs {numel}{'' if dtype is not None else ' bytes'}")


def _need_state(d: Dims, params, m, v, grads=None, e=None, e_pinned=False) -> None:
    n, K = d.n, d.num_workers
    _need(params, "params", n)
    _need(m, "m", n)
    _need(v, "v", n)
    _need(grads, "grads", K * n)
    _need(e, "e", K * n, pinned=e_pinned)


def _pk(d: Dims, k: int) -> int:
    return d.num_partitions * int(k)


def _stream(stream) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


# ------------------------------------------------------------------- layout


def tile_elems() -> int:
    return int(lib().scape_tile_elems())


def step_pass_count(d: Dims, k: int) -> int:
    """1 or K: the passes over the flat buffer a step makes (-1: invalid)."""
    return int(lib().scape_step_pass_count(ctypes.byref(d), k))


def mask_bytes(d: Dims, k: int) -> int:
    return int(lib().scape_mask_bytes(ctypes.byref(d), k))


def workspace_bytes(d: Dims, k: int) -> int:
    return int(lib().scape_workspace_bytes(ctypes.byref(d), k))


def mask_slot(d: Dims, k: int, blob, slot: int) -> MaskView:
    mv = MaskView()
    _check(lib().scape_mask_slot(ctypes.byref(d), k, _ptr(blob), slot, ctypes.byref(mv)))
    return mv


def mask_slot_tensors(d: Dims, k: int, blob, slot: int):
    """torch views (bits int64 [P*W], idx int32 [P*k], tile_off int32 [P*T])
    of one slot inside a uint8 blob tensor."""
    import torch
    mv = mask_slot(d, k, blob, slot)
    base = blob.data_ptr()
    P, n_p = d.num_partitions, d.n // d.num_partitions
    W = (n_p + 63) // 64
    T = (n_p + tile_elems() - 1) // tile_elems()

    def sub(ptr, count, dtype, size):
        off = ptr - base
        return blob[off:off + count * size].view(dtype)

    return (sub(mv.bits, P * W, torch.int64, 8), sub(mv.idx, P * k, torch.int32, 4),
            sub(mv.tile_off, P * T, torch.int32, 4))


def mask_slot_meta(d: Dims, k: int, blob, slot: int):
    """The slot's threshold record as an int32 view [3P] (k-th keys, the
    next capture bounds, then the selection's fault words)."""
    import torch
    mv = mask_slot(d, k, blob, slot)
    off = mv.meta - blob.data_ptr()
    return blob[off:off + 3 * d.num_partitions * 4].view(torch.int32)


def view_from_tensors(bits=None, idx=None, tile_off=None, meta=None) -> MaskView:
    return MaskView(_ptr(bits) or None, _ptr(idx) or None, _ptr(tile_off) or None, _ptr(meta) or None)


# --------------------------------------------------------------- components


def mask_topk(d: Dims, k: int, stat, out: MaskView, workspace, stream=None) -> None:
    _need(stat, "stat", d.n)
    _need(workspace, "workspace", workspace_bytes(d, k), dtype=None)
    _check(lib().scape_mask_topk(ctypes.byref(d), k, _ptr(stat), out, _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def compress(d: Dims, k: int, grads, e, cur: MaskView, b, stream=None) -> None:
    _need(grads, "grads", d.num_workers * d.n)
    _need(e, "e", d.num_workers * d.n)
    _need(b, "b", d.num_workers * _pk(d, k))
    _check(lib().scape_compress(ctypes.byref(d), k, _ptr(grads), _ptr(e), cur, _ptr(b), _stream(stream)))


def reduce_sparse(d: Dims, k: int, b, b_bar, stream=None) -> None:
    _need(b, "b", d.num_workers * _pk(d, k))
    _need(b_bar, "b_bar", _pk(d, k))
    _check(lib().scape_reduce_sparse(ctypes.byref(d), k, _ptr(b), _ptr(b_bar), _stream(stream)))


def adams_update(d: Dims, k: int, params, m, v, b_bar, cur: MaskView, bt: Betas, lr: float, step: int,
                 stream=None) -> None:
    _need_state(d, params, m, v)
    _need(b_bar, "b_bar", _pk(d, k))
    _check(lib().scape_adams_update(ctypes.byref(d), k, _ptr(params), _ptr(m), _ptr(v), _ptr(b_bar), cur,
                                    bt, lr, step, _stream(stream)))


def step(d: Dims, params, grads, m, v, e, mask_blob, k: int, bt: Betas, lr: float, step_no: int,
         workspace, stream=None) -> None:
    _need_state(d, params, m, v, grads, e)
    _need(mask_blob, "mask_blob", mask_bytes(d, k), dtype=None)
    _need(workspace, "workspace", workspace_bytes(d, k), dtype=None)
    _check(lib().scape_step(ctypes.byref(d), _ptr(params), _ptr(grads), _ptr(m), _ptr(v), _ptr(e),
                            _ptr(mask_blob), k, bt, lr, step_no, _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(stream)))


def step_noalloc_max_bytes() -> int:
    return int(lib().scape_step_noalloc_max_bytes())


def step_noalloc(d: Dims, params, grads, m, v, e, mask_blob, k: int, bt: Betas, lr: float, step_no: int,
                 stream=None) -> None:
    """scape_step_noalloc: scape_step with the library's static device
    scratch in place of a workspace (allocates nothing)."""
    _need_state(d, params, m, v, grads, e)
    _need(mask_blob, "mask_blob", mask_bytes(d, k), dtype=None)
    _check(lib().scape_step_noalloc(ctypes.byref(d), _ptr(params), _ptr(grads), _ptr(m), _ptr(v), _ptr(e),
                                    _ptr(mask_blob), k, bt, lr, step_no, _stream(stream)))


def bias_state_at(bt: Betas, steps_done: int) -> BiasState:
    out = BiasState()
    _check(lib().scape_bias_state_at(bt, steps_done, ctypes.byref(out)))
    return out


def bias_state_tensor(bt: Betas, steps_done: int, device):
    """scape_bias_state after `steps_done` steps, as a 24-byte device tensor."""
    import torch
    st = bias_state_at(bt, steps_done)
    host = torch.frombuffer(bytearray(bytes(st)), dtype=torch.uint8)
    return host.to(device)


def step_graph(d: Dims, params, grads, m, v, e, mask_blob, k: int, bt: Betas, lr: float, cur_slot: int,
               bias_state, workspace, stream=None) -> None:
    """scape_step_graph: one step t >= 2 with M_t in slot cur_slot and the
    bias state (device tensor of bias_state_tensor) advanced on the device;
    safe to record into a graph."""
    _need_state(d, params, m, v, grads, e)
    _need(mask_blob, "mask_blob", mask_bytes(d, k), dtype=None)
    _need(bias_state, "bias_state", ctypes.sizeof(BiasState), dtype=None)
    _need(workspace, "workspace", workspace_bytes(d, k), dtype=None)
    _check(lib().scape_step_graph(ctypes.byref(d), _ptr(params), _ptr(grads), _ptr(m), _ptr(v), _ptr(e),
                                  _ptr(mask_blob), k, bt, lr, cur_slot, _ptr(bias_state), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)))


def offload_stage_bytes(d: Dims, k: int, chunk_parts: int) -> int:
    return int(lib().scape_offload_stage_bytes(ctypes.byref(d), k, chunk_parts))


def step_offload(d: Dims, params, grads, m, v, e_host, mask_blob, k: int, bt: Betas, lr: float, step_no: int,
                 workspace, stage, chunk_parts: int, stream=None, copy_in=None, copy_out=None) -> None:
    """scape_step with e_host ([K][n] fp32, pinned host memory) staged
    through `stage` in chunks of chunk_parts partitions on two copy streams."""
    _need_state(d, params, m, v, grads, e_host, e_pinned=True)
    _need(mask_blob, "mask_blob", mask_bytes(d, k), dtype=None)
    _need(workspace, "workspace", workspace_bytes(d, k), dtype=None)
    _need(stage, "stage", offload_stage_bytes(d, k, chunk_parts), dtype=None)
    _check(lib().scape_step_offload(ctypes.byref(d), _ptr(params), _ptr(grads), _ptr(m), _ptr(v), _ptr(e_host),
                                    _ptr(mask_blob), k, bt, lr, step_no, _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _ptr(stage),
                                    stage.numel() * stage.element_size(), chunk_parts, _stream(stream),
                                    _stream(copy_in), _stream(copy_out)))


def mask_union(d: Dims, k: int, acc_bits, m: MaskView, count_out, stream=None) -> None:
    n_p = d.n // d.num_partitions
    _need(acc_bits, "acc_bits", d.num_partitions * ((n_p + 63) // 64) * 8, dtype=None)
    _need(count_out, "count_out", 8, dtype=None)
    _check(lib().scape_mask_union(ctypes.byref(d), k, _ptr(acc_bits), m, _ptr(count_out), _stream(stream)))


def dense_adams_step(d: Dims, params, grads, m, v, bt: Betas, lr: float, step_no: int, stream=None) -> None:
    _need_state(d, params, m, v, grads)
    _check(lib().scape_dense_adams_step(ctypes.byref(d), _ptr(params), _ptr(grads), _ptr(m), _ptr(v), bt, lr,
                                        step_no, _stream(stream)))


def mask_check(d: Dims, k: int, m: MaskView, result=None, stream=None) -> None:
    """scape_mask_check (synchronous): raises ScapeError (SCAPE_EMASK) if the
    mask breaks the partitioned top-k contract.  `result` is a device int32
    tensor of at least P entries (allocated here if None); it receives the
    per-partition reason bits."""
    import torch
    if result is None:
        result = torch.empty(d.num_partitions, dtype=torch.int32, device=torch.cuda.current_device())
    _need(result, "result", d.num_partitions, dtype="int32")
    _check(lib().scape_mask_check(ctypes.byref(d), k, m, _ptr(result), _stream(stream)))


# ---------------------------------------------------- one rank's share


def shard_partitions(d: Dims, rank: int):
    """(first, count): the partitions rank `rank` owns."""
    first, count = c_int32(), c_int32()
    _check(lib().scape_shard_partitions(ctypes.byref(d), rank, ctypes.byref(first), ctypes.byref(count)))
    return first.value, count.value


def shard_select_initial(d: Dims, k: int, rank: int, grads, e, m, mask_blob, bt: Betas, workspace,
                         stream=None) -> None:
    """scape_shard_select_initial: M_1 on the rank's partitions (slot 0);
    grads and e are the rank's rows [n]."""
    _need(grads, "grads", d.n)
    _need(e, "e", d.n)
    _need(m, "m", d.n)
    _need(mask_blob, "mask_blob", mask_bytes(d, k), dtype=None)
    _need(workspace, "workspace", workspace_bytes(d, k), dtype=None)
    _check(lib().scape_shard_select_initial(ctypes.byref(d), k, rank, _ptr(grads), _ptr(e), _ptr(m), _ptr(mask_blob),
                                            bt, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                            _stream(stream)))


def shard_compress(d: Dims, k: int, rank: int, grads, e, m, b, mask_blob, bt: Betas, step_no: int, workspace,
                   stream=None) -> None:
    """scape_shard_compress: the rank's rows (grads, e [n]) compressed at
    M_t into b [P*k]; M_{t+1} selected on the rank's partitions."""
    _need(grads, "grads", d.n)
    _need(e, "e", d.n)
    _need(m, "m", d.n)
    _need(b, "b", _pk(d, k))
    _need(mask_blob, "mask_blob", mask_bytes(d, k), dtype=None)
    _need(workspace, "workspace", workspace_bytes(d, k), dtype=None)
    _check(lib().scape_shard_compress(ctypes.byref(d), k, rank, _ptr(grads), _ptr(e), _ptr(m), _ptr(b),
                                      _ptr(mask_blob), bt, step_no, _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream)))


def shard_update(d: Dims, k: int, rank: int, params, m, v, b_bar, mask_blob, bt: Betas, lr: float, step_no: int,
                 stream=None) -> None:
    """scape_shard_update: AdamS at M_t on the rank's partitions from b_bar,
    the synchronised buffer of those partitions (count*k entries)."""
    _need_state(d, params, m, v)
    _need(b_bar, "b_bar", shard_partitions(d, rank)[1] * int(k))
    _need(mask_blob, "mask_blob", mask_bytes(d, k), dtype=None)
    _check(lib().scape_shard_update(ctypes.byref(d), k, rank, _ptr(params), _ptr(m), _ptr(v), _ptr(b_bar),
                                    _ptr(mask_blob), bt, lr, step_no, _stream(stream)))


def count_nonfinite(x, count_out, count=None, stream=None) -> None:
    """count_out (device u64 / int64 tensor of one element) += the number of
    NaN and +-inf values among the first `count` (default: all) fp32
    elements of x (device)."""
    c = x.numel() if count is None else int(count)
    _need(x, "x", max(c, 0))
    _need(count_out, "count_out", 8, dtype=None)
    _check(lib().scape_count_nonfinite(_ptr(x), c, _ptr(count_out), _stream(stream)))


def mask_overlap(d: Dims, k: int, a: MaskView, b: MaskView, count_out, stream=None) -> None:
    _need(count_out, "count_out", 8, dtype=None)
    _check(lib().scape_mask_overlap(ctypes.byref(d), k, a, b, _ptr(count_out), _stream(stream)))


# ------------------------------------- 8-bit activations, gradient rows

ACT_BLOCK = 32  # columns that share a scale (scape_act_block)


class ActCheckpoint:
    """An 8-bit activation checkpoint of a [rows][cols] matrix: ``codes``
    (int8 [rows][pitch], pitch = cols rounded up to 32) and ``scales`` (uint8
    [rows][pitch / 32]), contiguous tensors on one device."""

    __slots__ = ("codes", "scales", "rows", "cols", "device", "view")

    def __init__(self, codes, scales, cols: int):
        import torch
        for t, name in ((codes, "codes"), (scales, "scales")):
            if not torch.is_tensor(t):
                raise _no_tensor(t, name)
        self.codes, self.scales, self.cols = codes, scales, int(cols)
        nb = (self.cols + ACT_BLOCK - 1) // ACT_BLOCK
        if codes.dim() != 2 or scales.dim() != 2 or codes.dtype != torch.int8 or scales.dtype != torch.uint8:
            raise ValueError("codes must be int8 [rows][pitch] and scales uint8 [rows][pitch / 32]")
        self.rows = codes.shape[0]
        if self.cols < 1 or tuple(codes.shape) != (self.rows, nb * ACT_BLOCK) or tuple(scales.shape) != (self.rows, nb):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not fit {self.cols} columns")
        if not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        if not codes.is_cuda or scales.device != codes.device:
            raise ValueError("codes and scales must be device tensors of one device")
        self.device = codes.get_device()
        self.view = ActView(codes.data_ptr(), scales.data_ptr())


def act_bytes(rows: int, cols: int) -> int:
    return int(lib().scape_act_bytes(rows, cols))


def act_in(buffer, rows: int, cols: int) -> ActCheckpoint:
    """The checkpoint that lies inside `buffer`, a uint8 device tensor of at
    least act_bytes(rows, cols) bytes (256-byte aligned)."""
    import torch
    need = act_bytes(rows, cols)
    if need == 0:
        raise ScapeError(2, f"invalid shape rows={rows} cols={cols}")
    _need(buffer, "buffer", need, dtype="uint8")
    if buffer.data_ptr() % 256:
        raise ValueError("buffer must be 256-byte aligned")
    mv = ActView()
    _check(lib().scape_act_slot(rows, cols, buffer.data_ptr(), ctypes.byref(mv)))
    nb = (cols + ACT_BLOCK - 1) // ACT_BLOCK
    off = mv.scales - buffer.data_ptr()
    flat = buffer.view(-1)
    return ActCheckpoint(flat[:rows * nb * ACT_BLOCK].view(torch.int8).view(rows, nb * ACT_BLOCK),
                         flat[off:off + rows * nb].view(rows, nb), cols)


def act_alloc(rows: int, cols: int, device) -> ActCheckpoint:
    """A new checkpoint (contents undefined until packed)."""
    import torch
    need = act_bytes(rows, cols)
    if need == 0:
        raise ScapeError(2, f"invalid shape rows={rows} cols={cols}")
    return act_in(torch.empty(need, dtype=torch.uint8, device=device), rows, cols)


def _no_tensor(t, name: str) -> ValueError:
    return ValueError(f"{name} must be a tensor (got {type(t).__name__})")


_NO_MATRIX = Matrix(None, 0, 0)
_NO_ACT = ActView(None, None)
_DTYPES = None


def _dtype(t, name: str) -> int:
    """The scape_dtype of a torch dtype."""
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    dt = _DTYPES.get(t)
    if dt is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16 (got {t})")
    return dt


def _matrix(t, name: str, rows: int, cols: int, device: int) -> Matrix:
    """A [rows][cols] device tensor of fp32, bf16 or fp16 with consecutive
    elements in a row and rows that do not overlap; None: no matrix."""
    if t is None:
        return _NO_MATRIX
    try:
        at = t.get_device()  # -1: host memory
    except AttributeError:
        raise _no_tensor(t, name) from None
    if at != device:
        raise ValueError(f"{name} must be a tensor on device {device} (got {t.device})")
    dt = _dtype(t.dtype, name)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape ({rows}, {cols}) (got {tuple(t.shape)})")
    ld, one = t.stride()
    if cols > 1 and one != 1:
        raise ValueError(f"{name} must have consecutive elements in a row (stride {one})")
    if rows < 2:
        ld = cols
    elif ld < cols:
        raise ValueError(f"{name}: rows {ld} elements apart overlap (cols {cols})")
    return Matrix(t.data_ptr(), ld, dt)


def _vector(t, name: str, numel: int, device: int) -> Optional[int]:
    """Address of a contiguous fp32 device tensor of `numel` elements."""
    if t is None:
        return None
    try:
        at = t.get_device()
    except AttributeError:
        raise _no_tensor(t, name) from None
    import torch
    if at != device or t.dtype != torch.float32:
        raise ValueError(f"{name} must be a float32 tensor on device {device} (got {t.dtype} on {t.device})")
    if not t.is_contiguous() or t.numel() != numel:
        raise ValueError(f"{name} must be contiguous with {numel} elements (got {tuple(t.shape)})")
    return t.data_ptr()


def _checkpoint(a, name: str) -> ActCheckpoint:
    if not isinstance(a, ActCheckpoint):
        raise ValueError(f"{name} must be an ActCheckpoint (got {type(a).__name__})")
    return a


def _act(a, name: str, rows: int, cols: int, device: int) -> ActView:
    if a is None:
        return _NO_ACT
    _checkpoint(a, name)
    if a.device != device or a.rows != rows or a.cols != cols:
        raise ValueError(f"{name} must be a checkpoint of ({rows}, {cols}) on device {device} "
                         f"(got ({a.rows}, {a.cols}) on device {a.device})")
    return a.view


def _workspace(t, need: int, device: int):
    try:
        at = t.get_device()
    except AttributeError:
        raise _no_tensor(t, "workspace") from None
    if at != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on device {device}")
    have = t.numel() * t.element_size()
    if have < need:
        raise ValueError(f"workspace is too small: {have} bytes, needs {need}")
    if t.data_ptr() % 256:
        raise ValueError("workspace must be 256-byte aligned")
    return t.data_ptr(), have


def _device_of(t, name: str) -> int:
    try:
        cuda = t.is_cuda
    except AttributeError:
        raise _no_tensor(t, name) from None
    if not cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions (got {tuple(t.shape)})")
    return t.get_device()


_raw_stream = None  # device -> handle of its current stream


def _enqueue(device: int, stream, fn, *args) -> None:
    """Calls fn(*args, stream) with `device` current: on the given stream,
    which has to be that device's, or on the device's current one."""
    global _raw_stream
    import torch
    if stream is not None:
        if stream.device.index != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on device {device}")
        handle = stream.cuda_stream
    else:
        if _raw_stream is None:  # without the Stream object, a sixth of a small call's time
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda d: torch.cuda.current_stream(d).cuda_stream)
        handle = _raw_stream(device)
    if torch.cuda.current_device() == device:
        _check(fn(*args, handle))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, handle))


def act_pack(x, out: ActCheckpoint, stream=None) -> None:
    """out = the 8-bit checkpoint of x [rows][cols]."""
    dev = _device_of(x, "x")
    rows, cols = x.shape
    _enqueue(dev, stream, lib().scape_act_pack, rows, cols, _matrix(x, "x", rows, cols, dev),
             _act(out, "out", rows, cols, dev))


def act_unpack(a: ActCheckpoint, out, gain=None, stream=None) -> None:
    """out [rows][cols] = the checkpoint's values (times gain[cols])."""
    dev, rows, cols = _checkpoint(a, "a").device, a.rows, a.cols
    _enqueue(dev, stream, lib().scape_act_unpack, rows, cols, a.view, _vector(gain, "gain", cols, dev),
             _matrix(out, "out", rows, cols, dev))


def rmsnorm_pack(x, weight, eps: float, y=None, xhat: Optional[ActCheckpoint] = None, rstd=None, residual=None,
                 h=None, stream=None) -> None:
    """RMS norm of x + residual: y (times weight), the sum h, the reciprocal
    RMS rstd [rows], and xhat, the 8-bit checkpoint of the normalised rows
    before the weight.  Outputs that are None are left out."""
    dev = _device_of(x, "x")
    rows, cols = x.shape
    _enqueue(dev, stream, lib().scape_rmsnorm_pack, rows, cols, _matrix(x, "x", rows, cols, dev),
             _matrix(residual, "residual", rows, cols, dev), _vector(weight, "weight", cols, dev), eps,
             _matrix(h, "h", rows, cols, dev), _matrix(y, "y", rows, cols, dev), _act(xhat, "xhat", rows, cols, dev),
             _vector(rstd, "rstd", rows, dev))


def rmsnorm_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().scape_rmsnorm_workspace_bytes(rows, cols))


def rmsnorm_backward(dy, xhat: ActCheckpoint, rstd, weight, dh, dweight, workspace, dres=None,
                     accumulate: bool = False, stream=None) -> None:
    """Backward pass of rmsnorm_pack from its checkpoint: dh [rows][cols]
    (the gradient of x and of residual) and dweight [cols], set or (with
    accumulate) added to.  dres: the gradient that reaches h directly."""
    dev = _device_of(dy, "dy")
    rows, cols = dy.shape
    ws, have = _workspace(workspace, rmsnorm_workspace_bytes(rows, cols), dev)
    _enqueue(dev, stream, lib().scape_rmsnorm_backward, rows, cols, _matrix(dy, "dy", rows, cols, dev),
             _act(xhat, "xhat", rows, cols, dev), _vector(rstd, "rstd", rows, dev),
             _vector(weight, "weight", cols, dev), _matrix(dres, "dres", rows, cols, dev),
             _matrix(dh, "dh", rows, cols, dev), _vector(dweight, "dweight", cols, dev), 1 if accumulate else 0,
             ws, have)


def wgrad_workspace_bytes(rows: int, n_in: int, n_out: int, dy=None) -> int:
    """Bytes of workspace of wgrad with this dy [rows][out], or with any."""
    m = _NO_MATRIX if dy is None else _matrix(dy, "dy", rows, n_out, _device_of(dy, "dy"))
    return int(lib().scape_wgrad_workspace_bytes(rows, n_in, n_out, m))


def wgrad_splits(rows: int, n_in: int, n_out: int, dtype):
    """(splits, tile_out, tile_in): how wgrad divides its work for a dy of
    this torch dtype (splits -1: invalid size)."""
    m, n = c_int32(), c_int32()
    splits = lib().scape_wgrad_splits(rows, n_in, n_out, _dtype(dtype, "dtype"), ctypes.byref(m), ctypes.byref(n))
    return int(splits), m.value, n.value


def wgrad(dy, x: ActCheckpoint, dw, workspace, gain=None, dbias=None, accumulate: bool = False, stream=None) -> None:
    """Weight gradient dw [out][in] (and dbias [out]) of a linear layer from
    the gradient dy [rows][out] of its output and the checkpoint x [rows][in]
    of its input (times gain[in]); set or (with accumulate) added to.  dw and
    dbias may be parts of a row of the optimizer's gradients."""
    dev = _device_of(dy, "dy")
    rows, n_out = dy.shape
    n_in = _checkpoint(x, "x").cols
    m = _matrix(dy, "dy", rows, n_out, dev)
    ws, have = _workspace(workspace, int(lib().scape_wgrad_workspace_bytes(rows, n_in, n_out, m)), dev)
    if dw is None:
        raise ValueError("dw is needed")
    _enqueue(dev, stream, lib().scape_wgrad, rows, n_in, n_out, m,
             _act(x, "x", rows, n_in, dev), _vector(gain, "gain", n_in, dev), _vector(dw, "dw", n_out * n_in, dev),
             _vector(dbias, "dbias", n_out, dev), 1 if accumulate else 0, ws, have)


# ---------------------------------------------------------------- profiling


def profile_stage_names():
    L = lib()
    return [L.scape_profile_stage_name(i).decode() for i in range(L.scape_profile_stages())]


def profile_enable(on: bool) -> None:
    _check(lib().scape_profile_enable(1 if on else 0))


def profile_collect():
    """{stage: (total_ms, launches)} for the steps since the last collect."""
    L = lib()
    n = L.scape_profile_stages()
    ms = (ctypes.c_double * n)()
    cnt = (c_int64 * n)()
    _check(L.scape_profile_collect(ms, cnt))
    return {name: (ms[i], cnt[i]) for i, name in enumerate(profile_stage_names())}


# ---------------------------------------------------------------- optimizer


def choose_placement(current, candidates, run_steps, rounds: int = 2):
    """Physical placement of a large state tensor, chosen by measurement.

    The step pass streams every worker row of e in lockstep, and its rate
    depends on the physical memory behind e: some placements load the
    memory channels unevenly.  `current` is the tensor in use and
    `candidates` are separate allocations of its shape and dtype.
    run_steps(t) runs real optimizer steps with tensor t in current's role
    (on torch's current stream).  Each tensor takes the role in turn,
    `rounds` times, after receiving the role's contents by an exact copy, so
    the steps' results do not depend on the choice.  Returns the tensor that
    ran fastest (holding the contents) and each one's best time in ms; the
    caller drops the others."""
    import torch
    opts = [current] + list(candidates)
    times = [float("inf")] * len(opts)
    holder = 0
    for _ in range(rounds):
        for i, x in enumerate(opts):
            if i != holder:
                x.copy_(opts[holder])
                holder = i
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            run_steps(x)
            e1.record()
            e1.synchronize()
            times[i] = min(times[i], e0.elapsed_time(e1))
    best = min(range(len(opts)), key=times.__getitem__)
    if best != holder:
        opts[best].copy_(opts[holder])
    torch.cuda.synchronize()
    return opts[best], times


class ScapeOptimizer:
    """Device state of one SCAPE optimizer over a flat fp32 buffer.

    Holds params, m [n], the K error-feedback rows e [K][n], the two-slot
    mask blob and the workspace; ``step(grads)`` runs one fused step with
    grads [K][n] (fp32, device).  AdamS keeps no second moment (v_t is
    rebuilt every step); with ``store_v`` the step also writes the
    uncorrected v_t at the masked entries into ``v`` [n], else ``v`` is
    None.  With ``count_nonfinite`` each step first counts the non-finite
    values of its gradients on the device (``nonfinite_count()``)."""

    def __init__(self, params, P: int, K: int, k: int, beta1=0.9, beta2=0.95, eps=1e-8,
                 weight_decay=0.0, lr=1e-3, device=None, store_v: bool = True, count_nonfinite: bool = False):
        import torch
        self.n = params.numel()
        self.d = dims(self.n, P, K)
        self.k, self.P, self.K = int(k), int(P), int(K)
        self.bt = betas(beta1, beta2, eps, weight_decay)
        self.lr = float(lr)
        dev = params.device if device is None else device
        self.params = params.to(dev, torch.float32).contiguous()
        self.m = torch.zeros(self.n, dtype=torch.float32, device=dev)
        self.v = torch.zeros(self.n, dtype=torch.float32, device=dev) if store_v else None
        self.e = torch.zeros((K, self.n), dtype=torch.float32, device=dev)
        mb = mask_bytes(self.d, self.k)
        wb = workspace_bytes(self.d, self.k)
        if mb == 0 or wb == 0:
            raise ScapeError(2, f"invalid shape n={self.n} P={P} K={K} k={k}")
        self.mask = torch.zeros(mb, dtype=torch.uint8, device=dev)
        self.ws = torch.empty(wb, dtype=torch.uint8, device=dev)
        # debug switch: non-finite gradient values seen by the steps so far
        self.nonfinite = torch.zeros(1, dtype=torch.int64, device=dev) if count_nonfinite else None
        self.t = 0

    def step(self, grads, stream=None) -> None:
        t = self.t + 1
        if self.nonfinite is not None:
            count_nonfinite(grads, self.nonfinite, self.K * self.n, stream)
        step(self.d, self.params, grads, self.m, self.v, self.e, self.mask, self.k, self.bt, self.lr,
             t, self.ws, stream)
        self.t = t  # a rejected call leaves the step count unchanged

    def place_error_feedback(self, grads, candidates: int = 4, rounds: int = 2) -> dict:
        """Chooses the allocation that holds e (choose_placement): timed
        steps with `grads` run with e in its current allocation and in
        `candidates` new ones in turn, `rounds` times, and e stays in the
        fastest.  The optimizer's state (params, m, v, e, the masks and the
        step count) is saved first and restored afterwards, so training
        continues as if the call had not been made.  Needs device memory for
        the candidates and the saved state while it runs.  Returns
        {"step_ms": [...], "chosen": i}."""
        import torch
        saved = {name: getattr(self, name).clone() for name in ("params", "m", "v", "e", "mask")
                 if getattr(self, name) is not None}
        t0 = self.t
        cands = [torch.empty_like(self.e) for _ in range(candidates)]

        def run(x):
            self.e = x
            self.step(grads)

        chosen, times = choose_placement(self.e, cands, run, rounds)
        self.e = chosen
        for name, x in saved.items():
            getattr(self, name).copy_(x)
        self.t = t0
        torch.cuda.synchronize()
        del cands, chosen, saved
        torch.cuda.empty_cache()
        return {"step_ms": times, "chosen": times.index(min(times))}

    def nonfinite_count(self) -> int:
        """Non-finite gradient values the steps were given (NaN, +-inf),
        with the optimizer built with count_nonfinite=True; waits for the
        device."""
        if self.nonfinite is None:
            raise ValueError("the optimizer was built without count_nonfinite")
        return int(self.nonfinite.item())

    def check(self, which: str = "next", stream=None) -> None:
        """Validates mask M_{t+1} ("next") or M_t ("current") against the
        partitioned top-k contract (waits for the stream); raises on a
        violation."""
        s = (self.t & 1) if which == "next" else ((self.t - 1) & 1)
        mask_check(self.d, self.k, mask_slot(self.d, self.k, self.mask, s), stream=stream)

    def slot(self, which: str = "next"):
        """Mask views (bits, idx, tile_off): "next" = M_{t+1}, "current" = M_t."""
        s = (self.t & 1) if which == "next" else ((self.t - 1) & 1)
        return mask_slot_tensors(self.d, self.k, self.mask, s)
