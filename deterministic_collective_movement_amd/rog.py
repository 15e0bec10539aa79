"""ctypes binding of librog.so (include/rog.h): argument marshalling only.

Every byte is moved by the library's HIP kernels; this module turns torch
tensors into device pointers, byte counts and the current HIP stream, and
status codes into exceptions.  PyTorch provides device memory and streams.

Entry points keep the C names.  Tensor forms:

* ``rog_gather(srcs, out=None, stream=None)`` -> ``out`` (the same object);
* ``rog_gather_ex(srcs, out, path, stream=None)`` -> ``out``;
* ``rog_gather_many(batch, outs=None, stream=None)`` -> list of outputs;
* ``rog_plan(srcs, out, path=ROG_PATH_AUTO)`` -> dict (no GPU work);
* ``rog_reduce(srcs, out=None, stream=None)`` -> ``out``: the rank-ordered sum
  of W float32, bfloat16 or float16 tensors;
* ``rog_reduce_ex(srcs, out, path, stream=None)``, ``rog_reduce_plan(srcs, out, path)``;
* ``rog_reduce_many(batch, outs=None, stream=None)`` -> list of outputs (one
  launch);
* ``rog_reduce_scatter(inputs, rank, out=None, stream=None)`` -> ``out``: rank
  ``rank``'s share of a reduce-scatter, i.e. ``rog_reduce`` over shard
  ``rank`` of each input (views; nothing is copied).

* ``rog_logprob(shards, tokens=None, top_k=0, temperature=1.0, out=None, ...)``
  -> ``RogLogprob``: log probabilities of given tokens over W vocabulary shards,
  with entropy, log-sum-exp and the best alternatives;
* ``rog_logprob_grad(shards, tokens, lse, entropy, g_logp, g_entropy=None, ...)``
  -> the W shards' gradients;
* ``rog_policy_loss(logp, old_logp, advantage, weight=None, ...)`` ->
  ``RogPolicyLoss``: the clipped policy loss with its gradient;
* ``rog_logprob_plan(shards, top_k=0, form=...)`` -> dict (no GPU work).

* ``rog_linear_logprob(hidden, weights, tokens=None, temperature=1.0, out=None, ...)``
  -> ``RogLogprob``: the same from hidden states and W shards of head weights,
  without writing the logits;
* ``rog_linear_logprob_grad(hidden, weights, tokens, lse, entropy, g_logp, ...)``
  -> ``RogLinearGrad``: its gradient in the hidden states and the weights;
* ``rog_quantize_i8(x, out=None)`` -> ``RogQuantized``: rows in 8-bit integers;
* ``rog_linear_i8(q, scale, weights, weight_scales, dtype=..., out=None)`` -> W
  shards of logits of a head held in 8-bit integers;
* ``rog_linear_logprob_plan``, ``rog_linear_logprob_grad_plan`` -> dict (no GPU work).

Raw-pointer forms (``*_ptrs``) take integer device addresses, for callers that
manage their own memory.

Semantics follow RL-Align/RL-Kernel PR #491 ("perf(cuda): vectorize the
deterministic all-gather copy and right-size its single-block path"):
``all_gather(input, out=)`` returns ``out`` itself and hands offset views to
the kernel without copying them (author's replies to the size-test review).
The sum is the reduction of the same PR's deterministic all_reduce /
reduce_scatter ("Not in this PR"); its order and precision are stated in
include/rog.h.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
import struct
import threading
import warnings
from typing import List, NamedTuple, Optional, Sequence

import torch  # loads the process's HIP runtime before librog.so binds to it

from .build import BINDING_PATH, LIB_PATH

ROG_OK = 0
ROG_ERR_INVALID_ARGUMENT = 1
ROG_ERR_OVERLAP = 2
ROG_ERR_TOO_LARGE = 3
ROG_ERR_LAUNCH = 4

ROG_PATH_AUTO = 0
ROG_PATH_SINGLE_WG = 1
ROG_PATH_MULTI_WG = 2

ROG_PLAN_NT_LOADS = 1
ROG_PLAN_SHIFTED_LOADS = 2

ROG_KERNEL_NONE = 0
ROG_KERNEL_FLAT = 1
ROG_KERNEL_PEER = 2
ROG_KERNEL_REDUCE = 3

ROG_DTYPE_F32 = 0
ROG_DTYPE_BF16 = 1
ROG_DTYPE_F16 = 2

ROG_LOGPROB_AUTO = 0
ROG_LOGPROB_ROW = 1
ROG_LOGPROB_SPLIT = 2
ROG_LOGPROB_WAVE = 3

LOGPROB_FORM_NAMES = {ROG_LOGPROB_AUTO: "none", ROG_LOGPROB_ROW: "row", ROG_LOGPROB_SPLIT: "split",
                      ROG_LOGPROB_WAVE: "wave"}
PATH_NAMES = {ROG_PATH_AUTO: "auto", ROG_PATH_SINGLE_WG: "single_wg", ROG_PATH_MULTI_WG: "multi_wg"}
KERNEL_NAMES = {ROG_KERNEL_NONE: "none", ROG_KERNEL_FLAT: "flat", ROG_KERNEL_PEER: "peer",
                ROG_KERNEL_REDUCE: "reduce"}
DTYPES = {torch.float32: ROG_DTYPE_F32, torch.bfloat16: ROG_DTYPE_BF16, torch.float16: ROG_DTYPE_F16}


class RogError(RuntimeError):
    """A non-zero rog_status."""

    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class RogArgumentError(RogError, ValueError):
    pass


class rog_gather_desc(ctypes.Structure):
    _fields_ = [("srcs", ctypes.POINTER(ctypes.c_void_p)),
                ("out", ctypes.c_void_p),
                ("bytes_per_rank", ctypes.c_size_t)]


class rog_reduce_desc(ctypes.Structure):
    _fields_ = [("srcs", ctypes.POINTER(ctypes.c_void_p)),
                ("out", ctypes.c_void_p),
                ("count", ctypes.c_size_t)]


class rog_plan_info(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("kernel", ctypes.c_int32),
                ("grid", ctypes.c_uint32), ("block", ctypes.c_uint32),
                ("vec_ok_mask", ctypes.c_uint64), ("units", ctypes.c_uint64),
                ("peer_magic", ctypes.c_uint32), ("peer_sh1", ctypes.c_uint32),
                ("peer_sh2", ctypes.c_uint32), ("flags", ctypes.c_uint32)]


class rog_head_plan_info(ctypes.Structure):
    _fields_ = [("form", ctypes.c_int32), ("grid", ctypes.c_uint32), ("block", ctypes.c_uint32),
                ("blocks", ctypes.c_uint32), ("workspace_bytes", ctypes.c_uint64)]


class rog_linear_plan_info(ctypes.Structure):
    _fields_ = [("tile_columns", ctypes.c_uint32), ("tile_rows", ctypes.c_uint32), ("pieces", ctypes.c_uint32),
                ("launches", ctypes.c_uint32), ("workspace_bytes", ctypes.c_uint64)]


def _hip_runtimes_mapped() -> set:
    paths = set()
    with open("/proc/self/maps") as f:
        for line in f:
            parts = line.split()
            if len(parts) >= 6 and os.path.basename(parts[-1]).startswith("libamdhip64.so"):
                paths.add(os.path.realpath(parts[-1]))
    return paths


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "librog.so is not built (%s); run __graft_entry__.build() or "
            "python -m deterministic_collective_movement_amd.build" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    runtimes = _hip_runtimes_mapped()
    if len(runtimes) > 1:
        raise ImportError("two HIP runtimes are mapped (%s); librog.so must share torch's"
                          % ", ".join(sorted(runtimes)))
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    ptrs = ctypes.POINTER(ctypes.c_void_p)
    lib.rog_gather.argtypes = [ptrs, i32, sz, vp, vp]
    lib.rog_gather_ex.argtypes = [ptrs, i32, sz, vp, vp, i32]
    lib.rog_gather_many.argtypes = [ctypes.POINTER(rog_gather_desc), i32, i32, vp]
    lib.rog_plan.argtypes = [ptrs, i32, sz, vp, i32, ctypes.POINTER(rog_plan_info)]
    lib.rog_reduce.argtypes = [ptrs, i32, sz, i32, vp, vp]
    lib.rog_reduce_ex.argtypes = [ptrs, i32, sz, i32, vp, vp, i32]
    lib.rog_reduce_plan.argtypes = [ptrs, i32, sz, i32, vp, i32, ctypes.POINTER(rog_plan_info)]
    lib.rog_reduce_many.argtypes = [ctypes.POINTER(rog_reduce_desc), i32, i32, i32, vp]
    # host structures go in as packed bytes or by reference
    f32 = ctypes.c_float
    lib.rog_logprob_ex.argtypes = [vp, i32, sz, i32, f32, vp, i32, vp, vp, sz, vp, i32]
    lib.rog_logprob.argtypes = lib.rog_logprob_ex.argtypes[:-1]
    lib.rog_logprob_plan.argtypes = [vp, i32, sz, i32, i32, i32, vp]
    lib.rog_logprob_grad.argtypes = [vp, vp, i32, sz, i32, f32, vp, vp, vp, vp, vp, vp]
    lib.rog_policy_loss.argtypes = [vp, sz, vp, vp, vp, sz, vp]
    lib.rog_policy_loss_workspace_bytes.argtypes = [sz]
    lib.rog_policy_loss_workspace_bytes.restype = sz
    i64 = ctypes.c_int64
    lib.rog_linear_logprob.argtypes = [vp, i64, sz, i64, vp, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.rog_linear_logprob_plan.argtypes = [vp, i32, sz, i64, i32, i32, vp]
    lib.rog_linear_logprob_grad.argtypes = [vp, i64, sz, i64, vp, i32, i32, f32, vp, vp, vp, vp, vp, vp, i64, vp, vp, sz, vp]
    lib.rog_linear_logprob_grad_plan.argtypes = [vp, i32, sz, i64, i32, vp]
    lib.rog_quantize_i8.argtypes = [vp, i64, sz, i64, i32, vp, i64, vp, vp]
    lib.rog_linear_i8.argtypes = [vp, i64, vp, sz, i64, vp, i32, i32, vp, vp]
    for name in ("rog_linear_logprob", "rog_linear_logprob_plan", "rog_linear_logprob_grad", "rog_linear_logprob_grad_plan",
                 "rog_quantize_i8", "rog_linear_i8", "rog_logprob", "rog_logprob_ex", "rog_logprob_plan", "rog_logprob_grad", "rog_policy_loss"):
        getattr(lib, name).restype = i32
    for name in ("rog_max_top_k", "rog_logprob_max_split_rows"):
        getattr(lib, name).argtypes = []
        getattr(lib, name).restype = i32
    for name in ("rog_gather", "rog_gather_ex", "rog_gather_many", "rog_plan", "rog_reduce", "rog_reduce_ex",
                 "rog_reduce_plan", "rog_reduce_many"):
        getattr(lib, name).restype = i32
    for name in ("rog_single_wg_max_bytes", "rog_reduce_single_wg_max_bytes"):
        getattr(lib, name).argtypes = []
        getattr(lib, name).restype = sz
    for name in ("rog_max_peers", "rog_max_batch", "rog_max_batch_pointers", "rog_last_hip_error"):
        getattr(lib, name).argtypes = []
        getattr(lib, name).restype = i32
    lib.rog_status_string.argtypes = [i32]
    lib.rog_status_string.restype = ctypes.c_char_p
    return lib


_lib = _load()


def _load_binding():
    """The module that marshals ordinary calls (csrc/rog_binding.cpp), or None: it
    is built against one torch, and only saves a few microseconds of calls that
    this file makes as well.  The kernels are librog.so's either way."""
    if not os.path.exists(BINDING_PATH):
        return None
    try:
        spec = importlib.util.spec_from_file_location("_rog_binding", BINDING_PATH)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    except ImportError as e:
        warnings.warn("_rog_binding.so does not load (%s): calls go through ctypes, a few microseconds slower; "
                      "python -m deterministic_collective_movement_amd.build makes it anew" % e, RuntimeWarning)
        return None
    return mod


_binding = _load_binding()


def library_path() -> str:
    return LIB_PATH


def lib() -> ctypes.CDLL:
    return _lib


def _check(status: int, what: str) -> None:
    if status == ROG_OK:
        return
    name = _lib.rog_status_string(status).decode()
    if status == ROG_ERR_LAUNCH:
        raise RogError(status, "%s: %s (hipError_t %d)" % (what, name, _lib.rog_last_hip_error()))
    if status in (ROG_ERR_INVALID_ARGUMENT, ROG_ERR_OVERLAP, ROG_ERR_TOO_LARGE):
        raise RogArgumentError(status, "%s: %s" % (what, name))
    raise RogError(status, "%s: %s" % (what, name))


# ---------------------------------------------------------------------------
# Constants
# ---------------------------------------------------------------------------

def rog_single_wg_max_bytes() -> int:
    return int(_lib.rog_single_wg_max_bytes())


def rog_reduce_single_wg_max_bytes() -> int:
    return int(_lib.rog_reduce_single_wg_max_bytes())


def rog_max_peers() -> int:
    return int(_lib.rog_max_peers())


def rog_max_batch() -> int:
    return int(_lib.rog_max_batch())


def rog_max_batch_pointers() -> int:
    return int(_lib.rog_max_batch_pointers())


def rog_last_hip_error() -> int:
    return int(_lib.rog_last_hip_error())


def rog_max_top_k() -> int:
    return int(_lib.rog_max_top_k())


def rog_logprob_max_split_rows() -> int:
    return int(_lib.rog_logprob_max_split_rows())


def rog_policy_loss_workspace_bytes(n: int) -> int:
    return int(_lib.rog_policy_loss_workspace_bytes(n))


def rog_status_string(status: int) -> str:
    return _lib.rog_status_string(status).decode()


# ---------------------------------------------------------------------------
# Raw-pointer forms
# ---------------------------------------------------------------------------

def _ptr_array(addrs: Sequence[int]):
    return (ctypes.c_void_p * max(1, len(addrs)))(*addrs)


def rog_gather_ptrs(src_ptrs: Sequence[int], bytes_per_rank: int, out_ptr: int,
                    stream: int = 0, path: int = ROG_PATH_AUTO) -> None:
    """rog_gather_ex on raw device addresses; raises on a non-zero status."""
    st = _lib.rog_gather_ex(_ptr_array(src_ptrs), len(src_ptrs), bytes_per_rank,
                            ctypes.c_void_p(out_ptr), ctypes.c_void_p(stream), path)
    _check(st, "rog_gather")


def rog_plan_ptrs(src_ptrs: Sequence[int], bytes_per_rank: int, out_ptr: int,
                  path: int = ROG_PATH_AUTO) -> dict:
    """rog_plan on raw addresses (no HIP call); raises on a non-zero status."""
    info = rog_plan_info()
    st = _lib.rog_plan(_ptr_array(src_ptrs), len(src_ptrs), bytes_per_rank,
                       ctypes.c_void_p(out_ptr), path, ctypes.byref(info))
    _check(st, "rog_plan")
    return _plan_dict(info)


def rog_status_of_ptrs(src_ptrs: Optional[Sequence[int]], W: int, bytes_per_rank: int,
                       out_ptr: int, path: int = ROG_PATH_AUTO) -> int:
    """Status rog_plan returns for these arguments (``src_ptrs=None`` passes NULL)."""
    info = rog_plan_info()
    arr = None if src_ptrs is None else _ptr_array(src_ptrs)
    return int(_lib.rog_plan(arr, W, bytes_per_rank, ctypes.c_void_p(out_ptr), path,
                             ctypes.byref(info)))


def _plan_dict(info) -> dict:
    return {"path": PATH_NAMES[info.path], "kernel": KERNEL_NAMES[info.kernel],
            "grid": info.grid, "block": info.block, "vec_ok_mask": info.vec_ok_mask,
            "units": info.units, "peer_magic": info.peer_magic, "peer_sh1": info.peer_sh1,
            "peer_sh2": info.peer_sh2, "nt_loads": bool(info.flags & ROG_PLAN_NT_LOADS),
            "shifted_loads": bool(info.flags & ROG_PLAN_SHIFTED_LOADS)}


def rog_reduce_ptrs(src_ptrs: Sequence[int], count: int, dtype: int, out_ptr: int,
                    stream: int = 0, path: int = ROG_PATH_AUTO) -> None:
    """rog_reduce_ex on raw device addresses; raises on a non-zero status."""
    st = _lib.rog_reduce_ex(_ptr_array(src_ptrs), len(src_ptrs), count, dtype,
                            ctypes.c_void_p(out_ptr), ctypes.c_void_p(stream), path)
    _check(st, "rog_reduce")


def rog_reduce_plan_ptrs(src_ptrs: Optional[Sequence[int]], count: int, dtype: int, out_ptr: int,
                         path: int = ROG_PATH_AUTO, W: Optional[int] = None) -> dict:
    """rog_reduce_plan on raw addresses (no HIP call); raises on a non-zero status.
    ``src_ptrs=None`` passes NULL with the given W."""
    info = rog_plan_info()
    arr = None if src_ptrs is None else _ptr_array(src_ptrs)
    st = _lib.rog_reduce_plan(arr, len(src_ptrs) if W is None else W, count, dtype,
                              ctypes.c_void_p(out_ptr), path, ctypes.byref(info))
    _check(st, "rog_reduce_plan")
    return _plan_dict(info)


def rog_reduce_many_ptrs(batch_ptrs: Sequence[Sequence[int]], counts: Sequence[int],
                         out_ptrs: Sequence[int], W: int, dtype: int, stream: int = 0) -> None:
    """rog_reduce_many on raw addresses: tensor t sums the W sources batch_ptrs[t]."""
    n = len(out_ptrs)
    keep = [_ptr_array(p) for p in batch_ptrs]
    descs = (rog_reduce_desc * max(1, n))()
    for t in range(n):
        descs[t].srcs = ctypes.cast(keep[t], ctypes.POINTER(ctypes.c_void_p))
        descs[t].out = ctypes.c_void_p(out_ptrs[t])
        descs[t].count = counts[t]
    st = _lib.rog_reduce_many(descs, n, W, dtype, ctypes.c_void_p(stream))
    _check(st, "rog_reduce_many")


def rog_gather_many_ptrs(batch_ptrs: Sequence[Sequence[int]], sizes: Sequence[int],
                         out_ptrs: Sequence[int], W: int, stream: int = 0) -> None:
    """rog_gather_many on raw addresses: tensor t has W sources batch_ptrs[t]."""
    n = len(out_ptrs)
    keep = [_ptr_array(p) for p in batch_ptrs]
    descs = (rog_gather_desc * max(1, n))()
    for t in range(n):
        descs[t].srcs = ctypes.cast(keep[t], ctypes.POINTER(ctypes.c_void_p))
        descs[t].out = ctypes.c_void_p(out_ptrs[t])
        descs[t].bytes_per_rank = sizes[t]
    st = _lib.rog_gather_many(descs, n, W, ctypes.c_void_p(stream))
    _check(st, "rog_gather_many")


# ---------------------------------------------------------------------------
# Tensor forms
# ---------------------------------------------------------------------------

def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _check_tensor(t: torch.Tensor, what: str, device: torch.device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if not t.is_cuda:
        raise ValueError("%s must be on a GPU (got %s)" % (what, t.device))
    if t.get_device() != device.index:
        raise ValueError("%s is on %s, expected %s" % (what, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)


# torch's current stream of a device as a raw handle, without building a
# Stream object (a few microseconds per call otherwise).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, device) -> int:
    if stream is None:
        if _raw_stream is not None:
            return int(_raw_stream(device.index if device.index is not None else torch.cuda.current_device()))
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return int(stream.cuda_stream)
    return int(stream)


def _prepare(srcs: Sequence[torch.Tensor], out: Optional[torch.Tensor]):
    if len(srcs) == 0:
        raise ValueError("need at least one source tensor")
    _check_tensor(srcs[0], "srcs[0]", srcs[0].device if isinstance(srcs[0], torch.Tensor) else None)
    device = srcs[0].device
    idx = device.index
    S = _nbytes(srcs[0])
    for i, s in enumerate(srcs):
        # one pass of cheap checks; the full check names the first failure
        if not (isinstance(s, torch.Tensor) and s.is_cuda and s.get_device() == idx and s.is_contiguous()):
            _check_tensor(s, "srcs[%d]" % i, device)
        if s.numel() * s.element_size() != S:
            raise ValueError("every source must hold the same number of bytes")
    if out is None:
        out = torch.empty(len(srcs) * S, dtype=torch.uint8, device=device)
    _check_tensor(out, "out", device)
    if _nbytes(out) != len(srcs) * S:
        raise ValueError("out must hold exactly W*S = %d bytes (has %d)" % (len(srcs) * S, _nbytes(out)))
    return device, S, out


# The calling thread's current device index, without torch's lazy-init checks.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _on_device:
    """Make ``device`` the calling thread's current HIP device for the call (the
    library launches on the current device), restoring the previous one."""

    def __init__(self, device: torch.device):
        self.index = device.index if device.index is not None else _current_device()
        self.prev = None

    def __enter__(self):
        cur = _current_device()
        if cur != self.index:
            self.prev = cur
            torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        if self.prev is not None:
            torch.cuda.set_device(self.prev)


def rog_gather_ex(srcs: Sequence[torch.Tensor], out: Optional[torch.Tensor] = None,
                  path: int = ROG_PATH_AUTO, stream=None) -> torch.Tensor:
    """Rank-ordered gather of equal-size tensors into ``out`` with the path forced."""
    device, S, out = _prepare(srcs, out)
    with _on_device(device):
        rog_gather_ptrs([s.data_ptr() for s in srcs], S, out.data_ptr(),
                        _stream_handle(stream, device), path)
    return out


def rog_gather(srcs: Sequence[torch.Tensor], out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Rank-ordered gather: out[r*S:(r+1)*S] = bytes of srcs[r].  Returns ``out``."""
    return rog_gather_ex(srcs, out, ROG_PATH_AUTO, stream)


def rog_plan(srcs: Sequence[torch.Tensor], out: torch.Tensor, path: int = ROG_PATH_AUTO) -> dict:
    """The launch rog_gather_ex would make for these tensors (no GPU work)."""
    device, S, out = _prepare(srcs, out)
    return rog_plan_ptrs([s.data_ptr() for s in srcs], S, out.data_ptr(), path)


def rog_gather_many(batch: Sequence[Sequence[torch.Tensor]],
                    outs: Optional[Sequence[Optional[torch.Tensor]]] = None,
                    stream=None) -> List[torch.Tensor]:
    """Gather every tensor list ``batch[t]`` (W tensors each) into ``outs[t]``, one launch."""
    n = len(batch)
    if outs is None:
        outs = [None] * n
    if len(outs) != n:
        raise ValueError("one output per tensor")
    if n == 0:
        return []
    W = len(batch[0])
    if any(len(b) != W for b in batch):
        raise ValueError("every tensor of a batch has the same number of sources")
    device = batch[0][0].device
    ready, sizes = [], []
    for t in range(n):
        _, S, o = _prepare(batch[t], outs[t])
        if batch[t][0].device != device:
            raise ValueError("all tensors of a batch must be on one device")
        ready.append(o)
        sizes.append(S)
    with _on_device(device):
        rog_gather_many_ptrs([[s.data_ptr() for s in b] for b in batch], sizes,
                             [o.data_ptr() for o in ready], W, _stream_handle(stream, device))
    return ready


def _prepare_reduce(srcs: Sequence[torch.Tensor], out: Optional[torch.Tensor]):
    if len(srcs) == 0:
        raise ValueError("need at least one source tensor")
    device = srcs[0].device
    dtype = srcs[0].dtype
    if dtype not in DTYPES:
        raise ValueError("rog_reduce sums float32, bfloat16 or float16 tensors (got %s)" % dtype)
    n = srcs[0].numel()
    idx = device.index
    for i, s in enumerate(srcs):
        if not (isinstance(s, torch.Tensor) and s.is_cuda and s.get_device() == idx and s.is_contiguous()):
            _check_tensor(s, "srcs[%d]" % i, device)
        if s.dtype != dtype or s.numel() != n:
            raise ValueError("every source must have the dtype and element count of srcs[0]")
    if out is None:
        out = torch.empty(n, dtype=dtype, device=device)
    _check_tensor(out, "out", device)
    if out.dtype != dtype or out.numel() != n:
        raise ValueError("out must hold %d elements of %s" % (n, dtype))
    return device, n, DTYPES[dtype], out


def rog_reduce_ex(srcs: Sequence[torch.Tensor], out: Optional[torch.Tensor] = None,
                  path: int = ROG_PATH_AUTO, stream=None) -> torch.Tensor:
    """Rank-ordered sum of equal-shape tensors into ``out`` with the path forced."""
    device, n, dt, out = _prepare_reduce(srcs, out)
    with _on_device(device):
        rog_reduce_ptrs([s.data_ptr() for s in srcs], n, dt, out.data_ptr(),
                        _stream_handle(stream, device), path)
    return out


def rog_reduce(srcs: Sequence[torch.Tensor], out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """out[i] = rank-ordered binary32 sum of srcs[r][i], rounded to the tensors'
    dtype (float32, bfloat16 or float16).  ``out`` may be one of ``srcs`` (in
    place)."""
    return rog_reduce_ex(srcs, out, ROG_PATH_AUTO, stream)


def rog_reduce_plan(srcs: Sequence[torch.Tensor], out: torch.Tensor, path: int = ROG_PATH_AUTO) -> dict:
    """The launch rog_reduce_ex would make for these tensors (no GPU work)."""
    device, n, dt, out = _prepare_reduce(srcs, out)
    return rog_reduce_plan_ptrs([s.data_ptr() for s in srcs], n, dt, out.data_ptr(), path)


def rog_reduce_scatter(inputs: Sequence[torch.Tensor], rank: int, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Rank ``rank``'s share of a reduce-scatter over the W ``inputs``: each input
    holds W shards of n elements; out = rog_reduce over shard ``rank`` of every
    input (views into the inputs, no copy)."""
    W = len(inputs)
    if W == 0:
        raise ValueError("need at least one input")
    if not 0 <= rank < W:
        raise ValueError("rank must be in [0, %d)" % W)
    total = inputs[0].numel()
    if total % W:
        raise ValueError("each input must hold W equal shards (numel %% W == 0)")
    n = total // W
    for i, t in enumerate(inputs):
        _check_tensor(t, "inputs[%d]" % i, inputs[0].device)
    return rog_reduce([t.reshape(-1)[rank * n:(rank + 1) * n] for t in inputs], out, stream)


def rog_reduce_many(batch: Sequence[Sequence[torch.Tensor]],
                    outs: Optional[Sequence[Optional[torch.Tensor]]] = None,
                    stream=None) -> List[torch.Tensor]:
    """Rank-ordered sums of every tensor list ``batch[t]`` (W tensors each, one
    dtype for the batch) into ``outs[t]``, in one launch."""
    n = len(batch)
    if outs is None:
        outs = [None] * n
    if len(outs) != n:
        raise ValueError("one output per tensor")
    if n == 0:
        return []
    W = len(batch[0])
    if any(len(b) != W for b in batch):
        raise ValueError("every tensor of a batch has the same number of sources")
    device = batch[0][0].device
    ready, counts, dt0 = [], [], None
    for t in range(n):
        dev, count, dt, o = _prepare_reduce(batch[t], outs[t])
        if dev != device:
            raise ValueError("all tensors of a batch must be on one device")
        if dt0 is not None and dt != dt0:
            raise ValueError("all tensors of a batch must have one dtype")
        dt0 = dt
        ready.append(o)
        counts.append(count)
    with _on_device(device):
        rog_reduce_many_ptrs([[s.data_ptr() for s in b] for b in batch], counts,
                             [o.data_ptr() for o in ready], W, dt0, _stream_handle(stream, device))
    return ready


# ---------------------------------------------------------------------------
# The vocabulary side of a policy: token log probabilities, their gradient, the
# policy loss
# ---------------------------------------------------------------------------

class RogLogprob(NamedTuple):
    """rog_logprob's results; as ``out``, the tensors to write (None: not wanted)."""
    logp: Optional[torch.Tensor]        # [rows] float32
    entropy: Optional[torch.Tensor]     # [rows] float32
    lse: Optional[torch.Tensor]         # [rows] float32
    top_logp: Optional[torch.Tensor]    # [rows, top_k] float32
    top_ids: Optional[torch.Tensor]     # [rows, top_k] int64


class RogPolicyLoss(NamedTuple):
    """rog_policy_loss's results; as ``out``, the tensors to write."""
    stats: torch.Tensor                 # [4] float32: loss, sum w kl, sum w entropy, sum w [clipped]
    g_logp: Optional[torch.Tensor]      # [n] float32
    g_entropy: Optional[torch.Tensor]   # [n] float32


# The C structures of these calls as packed bytes, which cost less per call than
# ctypes structures: rog_logit_shard (address, row stride, width) and
# rog_grad_shard (address, row stride) once per shard, rog_logprob_out,
# rog_policy_in, rog_policy_params, rog_policy_out.
_PACK_SHARDS = [struct.Struct("=" + "Qqq" * w).pack for w in range(_lib.rog_max_peers() + 1)]
_PACK_GRADS = [struct.Struct("=" + "Qq" * w).pack for w in range(_lib.rog_max_peers() + 1)]
_pack_addresses5 = struct.Struct("=5Q").pack
_pack_addresses6 = struct.Struct("=6Q").pack
_pack_addresses3 = struct.Struct("=3Q").pack
_pack_floats5 = struct.Struct("=5f").pack
_MAX_TOP_K = int(_lib.rog_max_top_k())

# One workspace per stream, so that calls on different streams never share one;
# zero-filled when it is made, as the library asks, and left ready by every call.
# Threads that share a stream share it: a call is one launch, and launches on a
# stream do not overlap.  (The head's products are several: _with_scratch.)
_workspaces: dict = {}
_workspaces_lock = threading.Lock()
_NO_WORKSPACE = (None, 0)
_HERE = contextlib.nullcontext()       # the tensors' device is the current one
_OUT_NAMES = ("out.logp", "out.entropy", "out.lse", "out.top_logp", "out.top_ids")
_LOSS_NAMES = ("logp", "old_logp", "advantage", "weight", "ref_logp", "entropy", "out.g_logp", "out.g_entropy")


def rog_workspace(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """A zero-filled workspace of at least ``nbytes`` for calls on ``stream``
    (default: the current one), for callers that keep their own."""
    device = torch.device("cuda", _current_device()) if device is None else torch.device(device)
    with _made_on(stream, device):
        return torch.zeros(max(16, nbytes), dtype=torch.uint8, device=device)


def _made_on(stream, device: torch.device):
    """Where a call makes its outputs: on the stream that writes them, so that
    their memory is none that another stream's earlier work still uses."""
    if stream is None:
        return _HERE
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device))


def _own_workspace(nbytes: int, device: torch.device, stream, handle: int):
    """(address, bytes) of the stream's workspace, made or grown to hold ``nbytes``."""
    if nbytes == 0:
        return _NO_WORKSPACE
    if _capturing(stream, device):
        # a graph's replays may run beside eager calls on this stream: the graph gets its own, cleared in the graph
        t = rog_workspace(nbytes, device, stream)
        return t.data_ptr(), nbytes
    key = (device.index, handle)
    with _workspaces_lock:
        got = _workspaces.get(key)
        if got is None or got[1] < nbytes:
            # at least twice as large each time, and the smaller ones are kept: another
            # thread may be about to launch on this stream with one
            t = rog_workspace(max(nbytes, 1 << 20, 2 * got[1] if got else 0), device, stream)
            got = _workspaces[key] = (t.data_ptr(), t.numel(), t, got)
            if _binding is not None:
                _binding.workspace(device.index, handle, t.data_ptr(), t.numel())
    return got[:2]


_is_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing
_raw_stream_of = _raw_stream or (lambda device: torch.cuda.current_stream(device).cuda_stream)
if _binding is not None:
    _binding.bind(tuple(ctypes.cast(f, ctypes.c_void_p).value for f in (_lib.rog_logprob_ex, _lib.rog_logprob_grad, _lib.rog_policy_loss,
                                                                        _lib.rog_linear_logprob, _lib.rog_linear_logprob_grad,
                                                                        _lib.rog_quantize_i8, _lib.rog_linear_i8,
                                                                        _lib.rog_linear_logprob_plan, _lib.rog_linear_logprob_grad_plan)),
                  _lib.rog_max_peers(), _current_device, _raw_stream_of, _is_capturing)


def _capturing(stream, device: torch.device) -> bool:
    if stream is None:
        return _is_capturing()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return _is_capturing()


def _with_workspace(call, need, what: str, workspace, device: torch.device, stream, handle: int) -> None:
    """``call(address, bytes)`` with the caller's workspace or the stream's own.
    The library refuses one that is too small before it enqueues anything, so
    ``need()``, the bytes it asks for, is only looked up where the stream's own
    does not do."""
    if workspace is not None:
        _check_tensor(workspace, "workspace", device)
        _check(call(workspace.data_ptr(), _nbytes(workspace)), what)
        return
    # the stream's own, if it has one and this is no capture (of a stream that is
    # not the current one it takes a look at that stream)
    got = _workspaces.get((device.index, handle), _NO_WORKSPACE)
    if got[1] == 0 or not _capturing(stream, device):
        status = call(got[0], got[1])
        if status == ROG_OK:
            return
        if status != ROG_ERR_INVALID_ARGUMENT or got[1] >= need():
            _check(status, what)
    _check(call(*_own_workspace(need(), device, stream, handle)), what)


def _with_scratch(call, need, what: str, workspace, device: torch.device, stream) -> None:
    """``call(address, bytes)`` with the caller's workspace or one of the call's own,
    from torch's allocator.  For calls of several launches that hand data to each
    other through it: another thread's call on the same stream may come between
    two of them.  Once all are enqueued its memory goes back, for whatever is
    enqueued on this stream behind them."""
    if workspace is not None:
        _check_tensor(workspace, "workspace", device)
        _check(call(workspace.data_ptr(), _nbytes(workspace)), what)
        return
    nbytes = need()
    if nbytes == 0:
        _check(call(*_NO_WORKSPACE), what)
        return
    with _made_on(stream, device):
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _check(call(scratch.data_ptr(), nbytes), what)


def _vector_error(t, what: str, n: int, dtype: torch.dtype, device: torch.device):
    """The first thing wrong with what should be a contiguous vector of n elements."""
    _check_tensor(t, what, device)
    raise ValueError("%s must hold %d elements of %s (has %d of %s)" % (what, n, dtype, t.numel(), t.dtype))


def _addresses(tensors, names, n: int, dtype: torch.dtype, device: torch.device, idx: int) -> list:
    """Addresses of contiguous vectors of n elements (0 for None): one pass of
    cheap checks, the full ones name what is wrong."""
    got = []
    try:
        for t in tensors:
            if t is None:
                got.append(0)
            elif t.dtype is dtype and t.get_device() == idx and t.numel() == n and t.is_contiguous():
                got.append(t.data_ptr())
            else:
                break
        else:
            return got
    except AttributeError:
        pass
    _vector_error(tensors[len(got)], names[len(got)], n, dtype, device)


def _matrix_error(t, what: str, rows: int, dtype: torch.dtype, device: torch.device):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if not t.is_cuda:
        raise ValueError("%s must be on a GPU (got %s)" % (what, t.device))
    if t.get_device() != device.index:
        raise ValueError("%s is on %s, expected %s" % (what, t.device, device))
    if t.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (what, dtype, t.dtype))
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError("%s must be a matrix of %d rows (got %s)" % (what, rows, tuple(t.shape)))
    raise ValueError("%s must be contiguous within its rows (any row stride)" % what)


def _shard_bytes(shards):
    """(device, its index, rows, torch dtype, packed rog_logit_shard array) of W logits matrices."""
    if len(shards) == 0:
        raise ValueError("need at least one shard of logits")
    if len(shards) > rog_max_peers():
        raise ValueError("at most %d shards (got %d)" % (rog_max_peers(), len(shards)))
    first = shards[0]
    if not isinstance(first, torch.Tensor):
        raise TypeError("shards[0] must be a torch.Tensor")
    device, dtype = first.device, first.dtype
    if dtype not in DTYPES:
        raise ValueError("logits are float32, bfloat16 or float16 (got %s)" % dtype)
    if first.dim() != 2:
        raise ValueError("shards[0] must be a matrix (got %s)" % (tuple(first.shape),))
    rows, idx = first.size(0), first.get_device()
    if idx < 0:
        _matrix_error(first, "shards[0]", rows, dtype, device)
    vals = []
    for i, x in enumerate(shards):
        try:
            n, width = x.shape
            stride, step = x.stride()
            ok = n == rows and x.dtype is dtype and x.get_device() == idx and (step == 1 or width <= 1)
        except (AttributeError, ValueError):
            ok = False
        if not ok:
            _matrix_error(x, "shards[%d]" % i, rows, dtype, device)
        vals += (x.data_ptr(), stride, width)
    return device, idx, rows, dtype, _PACK_SHARDS[len(shards)](*vals)


def _logprob_plan(packed, W: int, rows: int, dtype: int, top_k: int, form: int) -> rog_head_plan_info:
    info = rog_head_plan_info()
    _check(_lib.rog_logprob_plan(packed, W, rows, dtype, top_k, form, ctypes.byref(info)), "rog_logprob_plan")
    return info


def _logprob_plan_dict(info) -> dict:
    return {"form": LOGPROB_FORM_NAMES[info.form], "grid": info.grid, "block": info.block, "blocks": info.blocks,
            "workspace_bytes": info.workspace_bytes}


def rog_logprob_plan(shards: Sequence[torch.Tensor], top_k: int = 0, form: int = ROG_LOGPROB_AUTO) -> dict:
    """The launch rog_logprob_ex would make for these logits (no GPU work)."""
    _, _, rows, dtype, packed = _shard_bytes(shards)
    return _logprob_plan_dict(_logprob_plan(packed, len(shards), rows, DTYPES[dtype], top_k, form))


def rog_logprob_plan_widths(widths: Sequence[int], rows: int, dtype: int, top_k: int = 0,
                            form: int = ROG_LOGPROB_AUTO) -> dict:
    """rog_logprob_plan from the shards' widths alone."""
    packed = struct.pack("=" + "Qqq" * len(widths), *(v for w in widths for v in (0, 0, w)))
    return _logprob_plan_dict(_logprob_plan(packed, len(widths), rows, dtype, top_k, form))


def rog_logprob_ex(shards: Sequence[torch.Tensor], tokens: Optional[torch.Tensor] = None, top_k: int = 0,
                   temperature: float = 1.0, out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None,
                   form: int = ROG_LOGPROB_AUTO) -> RogLogprob:
    """rog_logprob with the launch form forced (never changes the bits)."""
    if out is not None and workspace is None and stream is None:
        if type(out) is not RogLogprob:
            out = RogLogprob(*out)
        if _binding is not None and _binding.logprob(shards, tokens, top_k, temperature, out, form):
            return out
    device, idx, rows, dtype, packed = _shard_bytes(shards)
    if not 0 <= top_k <= _MAX_TOP_K:
        raise ValueError("top_k must be in [0, %d]" % _MAX_TOP_K)
    f32, i64 = torch.float32, torch.int64
    if out is None:
        new = lambda *shape, dtype=f32: torch.empty(*shape, dtype=dtype, device=device)  # noqa: E731
        with _made_on(stream, device):
            out = RogLogprob(new(rows) if tokens is not None else None, new(rows), new(rows),
                             new(rows, top_k) if top_k else None, new(rows, top_k, dtype=i64) if top_k else None)
    elif type(out) is not RogLogprob:
        out = RogLogprob(*out)
    addr = _addresses(out[:3], _OUT_NAMES, rows, f32, device, idx)
    if top_k:
        addr += _addresses(out[3:4], _OUT_NAMES[3:], rows * top_k, f32, device, idx)
        addr += _addresses(out[4:], _OUT_NAMES[4:], rows * top_k, i64, device, idx)
        outs = _pack_addresses5(*addr)
    elif out[3] is None and out[4] is None:
        outs = _pack_addresses5(*addr, 0, 0)
    else:
        raise ValueError("out.top_logp and out.top_ids need a top_k")
    tok = None if tokens is None else _addresses((tokens,), ("tokens",), rows, i64, device, idx)[0]
    W, dt = len(shards), DTYPES[dtype]
    with _on_device(device) if _current_device() != idx else _HERE:
        handle = _stream_handle(stream, device)
        _with_workspace(lambda ws, n: _lib.rog_logprob_ex(packed, W, rows, dt, temperature, tok, top_k, outs, ws, n, handle, form),
                        lambda: _logprob_plan(packed, W, rows, dt, top_k, form).workspace_bytes,
                        "rog_logprob", workspace, device, stream, handle)
    return out


def rog_logprob(shards: Sequence[torch.Tensor], tokens: Optional[torch.Tensor] = None, top_k: int = 0,
                temperature: float = 1.0, out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> RogLogprob:
    """Log probability of ``tokens[i]`` (int64; negative: the row is not scored)
    in row i of the logits whose columns are ``shards`` in rank order, with the
    row's entropy and log-sum-exp and its ``top_k`` best alternatives.

    ``shards``: W matrices [rows, width_r] of one dtype (float32, bfloat16 or
    float16), contiguous within rows, any row stride.  ``out``: a RogLogprob (or
    five tensors) to write, None for what is not wanted.

    The outputs have no gradient function, whatever the logits require:
    ``rog_logprob_grad`` gives the logits' gradients."""
    return rog_logprob_ex(shards, tokens, top_k, temperature, out, workspace, stream)


def rog_logprob_grad(shards: Sequence[torch.Tensor], tokens: torch.Tensor, lse: torch.Tensor, entropy: torch.Tensor,
                     g_logp: torch.Tensor, g_entropy: Optional[torch.Tensor] = None, temperature: float = 1.0,
                     out: Optional[Sequence[torch.Tensor]] = None, stream=None) -> List[torch.Tensor]:
    """Gradient of sum_i (g_logp[i] logp[i] + g_entropy[i] entropy[i]) in every
    shard, from rog_logprob's ``lse`` and ``entropy`` of the same logits, widths
    and temperature.  ``out``: W matrices to write; ``out[r]`` may be
    ``shards[r]`` (in place)."""
    if out is not None and stream is None and _binding is not None and _binding.grad(shards, tokens, lse, entropy, g_logp, g_entropy,
                                                                                     temperature, out):
        return out if isinstance(out, list) else list(out)
    device, idx, rows, dtype, packed = _shard_bytes(shards)
    if out is None:
        with _made_on(stream, device):
            out = [torch.empty(rows, x.shape[1], dtype=dtype, device=device) for x in shards]
    W = len(shards)
    if len(out) != W:
        raise ValueError("one gradient per shard")
    vals = []
    for i, g in enumerate(out):
        try:
            shape = g.shape
            stride, step = g.stride()
            ok = shape == shards[i].shape and g.dtype is dtype and g.get_device() == idx and (step == 1 or shape[1] <= 1)
        except (AttributeError, ValueError):
            ok = False
        if not ok:
            if isinstance(g, torch.Tensor) and g.dim() == 2 and g.shape != shards[i].shape:
                raise ValueError("out[%d] must have the shape of shards[%d]" % (i, i))
            _matrix_error(g, "out[%d]" % i, rows, dtype, device)
        vals += (g.data_ptr(), stride)
    if tokens is None or lse is None or entropy is None or g_logp is None:
        raise ValueError("tokens, lse, entropy and g_logp are needed")
    tok = _addresses((tokens,), ("tokens",), rows, torch.int64, device, idx)[0]
    vec = _addresses((lse, entropy, g_logp, g_entropy), ("lse", "entropy", "g_logp", "g_entropy"), rows, torch.float32,
                     device, idx)
    with _on_device(device) if _current_device() != idx else _HERE:
        _check(_lib.rog_logprob_grad(packed, _PACK_GRADS[W](*vals), W, rows, DTYPES[dtype], temperature, tok, *vec,
                                     _stream_handle(stream, device)), "rog_logprob_grad")
    return out if isinstance(out, list) else list(out)


def rog_policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantage: torch.Tensor,
                    weight: Optional[torch.Tensor] = None, ref_logp: Optional[torch.Tensor] = None,
                    entropy: Optional[torch.Tensor] = None, clip_low: float = 0.2, clip_high: float = 0.2,
                    kl_coef: float = 0.0, entropy_coef: float = 0.0, grad_scale: float = 1.0,
                    out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> RogPolicyLoss:
    """The clipped policy loss over n tokens (float32 vectors) with its gradients
    in ``logp`` and ``entropy``.  ``weight[i]`` is the token's weight in the sums
    (0: the token counts for nothing; None: 1 / n each).  The outputs have no
    gradient function: ``g_logp`` and ``g_entropy`` go to ``rog_logprob_grad``."""
    if out is not None and workspace is None and stream is None:
        if type(out) is not RogPolicyLoss:
            out = RogPolicyLoss(*out)
        if _binding is not None and _binding.loss(logp, old_logp, advantage, weight, ref_logp, entropy, clip_low, clip_high, kl_coef,
                                                  entropy_coef, grad_scale, out):
            return out
    if not isinstance(logp, torch.Tensor):
        raise TypeError("logp must be a torch.Tensor")
    device, n, f32, idx = logp.device, logp.numel(), torch.float32, logp.get_device()
    if idx < 0:
        _check_tensor(logp, "logp", device)
    if old_logp is None or advantage is None:
        raise ValueError("old_logp and advantage are needed")
    if out is None:
        with _made_on(stream, device):
            out = RogPolicyLoss(torch.empty(4, dtype=f32, device=device), torch.empty(n, dtype=f32, device=device),
                                torch.empty(n, dtype=f32, device=device) if entropy is not None else None)
    elif type(out) is not RogPolicyLoss:
        out = RogPolicyLoss(*out)
    addr = _addresses((logp, old_logp, advantage, weight, ref_logp, entropy, out[1], out[2]), _LOSS_NAMES, n, f32, device, idx)
    ins = _pack_addresses6(*addr[:6])
    outs = _pack_addresses3(_addresses(out[:1], ("out.stats",), 4, f32, device, idx)[0], *addr[6:])
    params = _pack_floats5(clip_low, clip_high, kl_coef, entropy_coef, grad_scale)
    with _on_device(device) if _current_device() != idx else _HERE:
        handle = _stream_handle(stream, device)
        _with_workspace(lambda ws, b: _lib.rog_policy_loss(ins, n, params, outs, ws, b, handle),
                        lambda: _lib.rog_policy_loss_workspace_bytes(n), "rog_policy_loss", workspace, device, stream, handle)
    return out


# ---------------------------------------------------------------------------
# The policy head's products: log probabilities from hidden states, their
# gradient, logits of 8-bit weights
# ---------------------------------------------------------------------------

class RogLinearGrad(NamedTuple):
    """rog_linear_logprob_grad's results; as ``out``, the tensors to write."""
    d_hidden: torch.Tensor              # [rows, dim]
    d_weights: List[torch.Tensor]       # W matrices [width, dim]


class RogQuantized(NamedTuple):
    """rog_quantize_i8's results; as ``out``, the tensors to write."""
    q: torch.Tensor                     # [rows, dim] int8
    scale: torch.Tensor                 # [rows] float32


_PACK_I8 = [struct.Struct("=" + "QqqQ" * w).pack for w in range(_lib.rog_max_peers() + 1)]
_PRODUCT_DTYPES = (torch.bfloat16, torch.float16)


def _row_matrix(t, what: str, rows: Optional[int], cols: Optional[int], dtype: torch.dtype, device: torch.device):
    """(address, row stride) of a matrix that is contiguous within its rows; None: any size."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if not t.is_cuda:
        raise ValueError("%s must be on a GPU (got %s)" % (what, t.device))
    if t.get_device() != device.index:
        raise ValueError("%s is on %s, expected %s" % (what, t.device, device))
    if t.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (what, dtype, t.dtype))
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError("%s must be a matrix of %s x %s (got %s)" % (what, "any" if rows is None else rows, "any" if cols is None else cols,
                                                                      tuple(t.shape)))
    stride, step = t.stride()
    if step != 1 and t.shape[1] > 1:
        raise ValueError("%s must be contiguous within its rows (any row stride)" % what)
    return t.data_ptr(), stride


def _head_bytes(hidden, what: str, weights, dtypes):
    """(device, its index, rows, dim, dtype, address and stride of the states, packed rog_weight_shard array)."""
    if not isinstance(hidden, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    device, dtype = hidden.device, hidden.dtype
    if dtype not in dtypes:
        raise ValueError("%s is %s (got %s)" % (what, " or ".join(str(d)[6:] for d in dtypes), dtype))
    at, stride = _row_matrix(hidden, what, None, None, dtype, device)
    rows, dim = hidden.shape
    if len(weights) == 0:
        raise ValueError("need at least one shard of weights")
    if len(weights) > rog_max_peers():
        raise ValueError("at most %d shards (got %d)" % (rog_max_peers(), len(weights)))
    vals = []
    for i, w in enumerate(weights):
        a, s = _row_matrix(w, "weights[%d]" % i, None, dim, dtype, device)
        vals += (a, s, w.shape[0])
    return device, hidden.get_device(), rows, dim, dtype, at, stride, _PACK_SHARDS[len(weights)](*vals)


def _linear_plan(call, what: str, *args) -> rog_linear_plan_info:
    info = rog_linear_plan_info()
    _check(call(*args, ctypes.byref(info)), what)
    return info


def _linear_plan_dict(info) -> dict:
    return {"tile": (info.tile_columns, info.tile_rows), "pieces": info.pieces, "launches": info.launches,
            "workspace_bytes": info.workspace_bytes}


def _widths_bytes(widths: Sequence[int]) -> bytes:
    return struct.pack("=" + "Qqq" * len(widths), *(v for w in widths for v in (0, 0, w)))


def rog_linear_logprob_plan(widths: Sequence[int], rows: int, dim: int, dtype: int = ROG_DTYPE_BF16, tokens: bool = True) -> dict:
    """The launches rog_linear_logprob would make for shards of these widths (no GPU work)."""
    return _linear_plan_dict(_linear_plan(_lib.rog_linear_logprob_plan, "rog_linear_logprob_plan", _widths_bytes(widths), len(widths), rows,
                                          dim, dtype, int(tokens)))


def rog_linear_logprob_grad_plan(widths: Sequence[int], rows: int, dim: int, dtype: int = ROG_DTYPE_BF16) -> dict:
    """The launches rog_linear_logprob_grad would make for shards of these widths (no GPU work)."""
    return _linear_plan_dict(_linear_plan(_lib.rog_linear_logprob_grad_plan, "rog_linear_logprob_grad_plan", _widths_bytes(widths),
                                          len(widths), rows, dim, dtype))


def rog_linear_logprob(hidden: torch.Tensor, weights: Sequence[torch.Tensor], tokens: Optional[torch.Tensor] = None,
                       temperature: float = 1.0, out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> RogLogprob:
    """``rog_logprob`` of the logits ``hidden @ cat(weights).T`` without writing them:
    log probability of ``tokens[i]`` (int64; negative: the row is not scored, and
    its state not used), entropy and log-sum-exp of every row.

    ``hidden``: [rows, dim] bfloat16 or float16; ``weights``: W shards
    [width_r, dim] of the same dtype in rank order; contiguous within rows, any
    row stride.  ``out``: a RogLogprob (or five tensors, the last two None) to
    write, None for what is not wanted.  The outputs have no gradient function:
    ``rog_linear_logprob_grad`` gives the gradients."""
    if out is not None and workspace is None and stream is None:
        if type(out) is not RogLogprob:
            out = RogLogprob(*out)
        if _binding is not None and _binding.linear_logprob(hidden, weights, tokens, temperature, out):
            return out
    device, idx, rows, dim, dtype, at, stride, packed = _head_bytes(hidden, "hidden", weights, _PRODUCT_DTYPES)
    f32 = torch.float32
    if out is None:
        new = lambda: torch.empty(rows, dtype=f32, device=device)  # noqa: E731
        with _made_on(stream, device):
            out = RogLogprob(new() if tokens is not None else None, new(), new(), None, None)
    elif type(out) is not RogLogprob:
        out = RogLogprob(*out)
    if out[3] is not None or out[4] is not None:
        raise ValueError("rog_linear_logprob gives no alternatives: out.top_logp and out.top_ids must be None")
    outs = _pack_addresses5(*_addresses(out[:3], _OUT_NAMES, rows, f32, device, idx), 0, 0)
    tok = None if tokens is None else _addresses((tokens,), ("tokens",), rows, torch.int64, device, idx)[0]
    W, dt = len(weights), DTYPES[dtype]
    with _on_device(device) if _current_device() != idx else _HERE:
        handle = _stream_handle(stream, device)
        _with_scratch(lambda ws, n: _lib.rog_linear_logprob(at, stride, rows, dim, packed, W, dt, temperature, tok, outs, ws, n, handle),
                      lambda: _linear_plan(_lib.rog_linear_logprob_plan, "rog_linear_logprob", packed, W, rows, dim, dt,
                                           int(tokens is not None)).workspace_bytes,
                      "rog_linear_logprob", workspace, device, stream)
    return out


def rog_linear_logprob_grad(hidden: torch.Tensor, weights: Sequence[torch.Tensor], tokens: torch.Tensor, lse: torch.Tensor,
                            entropy: torch.Tensor, g_logp: torch.Tensor, g_entropy: Optional[torch.Tensor] = None,
                            temperature: float = 1.0, out: Optional[Sequence] = None, workspace: Optional[torch.Tensor] = None,
                            stream=None) -> RogLinearGrad:
    """Gradient of sum_i (g_logp[i] logp[i] + g_entropy[i] entropy[i]) in the hidden
    states and in every shard's weights, from rog_linear_logprob's ``lse`` and
    ``entropy`` of the same states, weights and temperature.  Rows that are not
    scored get zeros, and so do the weights where there are no rows.  ``out``: a RogLinearGrad (or (d_hidden, W matrices)) to write."""
    if out is not None and workspace is None and stream is None:
        if type(out) is not RogLinearGrad:
            out = RogLinearGrad(out[0], list(out[1]))
        if _binding is not None and _binding.linear_grad(hidden, weights, tokens, lse, entropy, g_logp, g_entropy, temperature, out[0], out[1]):
            return out
    device, idx, rows, dim, dtype, at, stride, packed = _head_bytes(hidden, "hidden", weights, _PRODUCT_DTYPES)
    W = len(weights)
    if out is None:
        with _made_on(stream, device):
            out = RogLinearGrad(torch.empty(rows, dim, dtype=dtype, device=device),
                                [torch.empty(w.shape[0], dim, dtype=dtype, device=device) for w in weights])
    elif type(out) is not RogLinearGrad:
        out = RogLinearGrad(out[0], list(out[1]))
    if len(out.d_weights) != W:
        raise ValueError("one gradient per shard")
    d_at, d_stride = _row_matrix(out.d_hidden, "out.d_hidden", rows, dim, dtype, device)
    vals = []
    for i, g in enumerate(out.d_weights):
        vals += _row_matrix(g, "out.d_weights[%d]" % i, weights[i].shape[0], dim, dtype, device)
    if tokens is None or lse is None or entropy is None or g_logp is None:
        raise ValueError("tokens, lse, entropy and g_logp are needed")
    tok = _addresses((tokens,), ("tokens",), rows, torch.int64, device, idx)[0]
    vec = _addresses((lse, entropy, g_logp, g_entropy), ("lse", "entropy", "g_logp", "g_entropy"), rows, torch.float32, device, idx)
    grads, dt = _PACK_GRADS[W](*vals), DTYPES[dtype]
    with _on_device(device) if _current_device() != idx else _HERE:
        handle = _stream_handle(stream, device)
        _with_scratch(lambda ws, n: _lib.rog_linear_logprob_grad(at, stride, rows, dim, packed, W, dt, temperature, tok, *vec, d_at,
                                                                 d_stride, grads, ws, n, handle),
                      lambda: _linear_plan(_lib.rog_linear_logprob_grad_plan, "rog_linear_logprob_grad", packed, W, rows, dim,
                                           dt).workspace_bytes,
                      "rog_linear_logprob_grad", workspace, device, stream)
        if rows == 0:
            # the library enqueues nothing: a sum over no rows is zero
            with _made_on(stream, device):
                for g in out.d_weights:
                    g.detach().zero_()
    return out


def rog_quantize_i8(x: torch.Tensor, out: Optional[Sequence[torch.Tensor]] = None, stream=None) -> RogQuantized:
    """Rows of ``x`` (float32, bfloat16 or float16) in 8-bit integers with a scale
    each: ``scale = max(max |x| / 127, 2^-126)``, ``q = x / scale`` to the nearest,
    ties to even.  A row with a NaN or an infinity gets scale NaN and q 0.  For a
    head's weights the rows are its columns.  ``out``: a RogQuantized to write."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    device, dtype = x.device, x.dtype
    if dtype not in DTYPES:
        raise ValueError("x is float32, bfloat16 or float16 (got %s)" % dtype)
    at, stride = _row_matrix(x, "x", None, None, dtype, device)
    rows, dim = x.shape
    idx = x.get_device()
    if out is None:
        with _made_on(stream, device):
            out = RogQuantized(torch.empty(rows, dim, dtype=torch.int8, device=device), torch.empty(rows, dtype=torch.float32, device=device))
    elif type(out) is not RogQuantized:
        out = RogQuantized(*out)
    if stream is None and _binding is not None and _binding.quantize(x, out[0], out[1]):
        return out
    q_at, q_stride = _row_matrix(out.q, "out.q", rows, dim, torch.int8, device)
    s_at = _addresses(out[1:], ("out.scale",), rows, torch.float32, device, idx)[0]
    with _on_device(device) if _current_device() != idx else _HERE:
        _check(_lib.rog_quantize_i8(at, stride, rows, dim, DTYPES[dtype], q_at, q_stride, s_at, _stream_handle(stream, device)),
               "rog_quantize_i8")
    return out


def rog_linear_i8(q: torch.Tensor, scale: torch.Tensor, weights: Sequence[torch.Tensor], weight_scales: Sequence[torch.Tensor],
                  dtype: torch.dtype = torch.bfloat16, out: Optional[Sequence[torch.Tensor]] = None, stream=None) -> List[torch.Tensor]:
    """Logits of a head held in 8-bit integers, as shards that ``rog_logprob`` takes:
    ``out[r][i, j] = (q[i] . weights[r][j]) * scale[i] * weight_scales[r][j]``, the
    sum exact, the result rounded to ``dtype`` (float32, bfloat16 or float16; that of
    ``out`` where it is given).

    ``q``: [rows, dim] int8 and ``scale``: [rows] float32, as rog_quantize_i8 gives
    them; ``weights``: W shards [width_r, dim] int8; ``weight_scales``: W vectors
    [width_r] float32."""
    if out is not None and stream is None and _binding is not None and _binding.linear_i8(q, scale, weights, weight_scales, out):
        return out if isinstance(out, list) else list(out)
    device, idx, rows, dim, _, at, stride, _ = _head_bytes(q, "q", weights, (torch.int8,))
    W = len(weights)
    if out is None:
        if dtype not in DTYPES:
            raise ValueError("logits are float32, bfloat16 or float16 (got %s)" % dtype)
        with _made_on(stream, device):
            out = [torch.empty(rows, w.shape[0], dtype=dtype, device=device) for w in weights]
    elif len(out) and isinstance(out[0], torch.Tensor):
        dtype = out[0].dtype
        if dtype not in DTYPES:
            raise ValueError("logits are float32, bfloat16 or float16 (got %s)" % dtype)
    if len(out) != W or len(weight_scales) != W:
        raise ValueError("one vector of scales and one output per shard")
    s_at = _addresses((scale,), ("scale",), rows, torch.float32, device, idx)[0]
    if scale is None:
        raise ValueError("scale is needed")
    shards, outs = [], []
    for i, w in enumerate(weights):
        if weight_scales[i] is None:
            raise ValueError("weight_scales[%d] is needed" % i)
        shards += (w.data_ptr(), w.stride(0), w.shape[0],
                   _addresses(weight_scales[i:i + 1], ("weight_scales[%d]" % i,), w.shape[0], torch.float32, device, idx)[0])
        outs += _row_matrix(out[i], "out[%d]" % i, rows, w.shape[0], dtype, device)
    with _on_device(device) if _current_device() != idx else _HERE:
        _check(_lib.rog_linear_i8(at, stride, s_at, rows, dim, _PACK_I8[W](*shards), W, DTYPES[dtype], _PACK_GRADS[W](*outs),
                                  _stream_handle(stream, device)), "rog_linear_i8")
    return out if isinstance(out, list) else list(out)
