"""The gated recurrence (include/ssm.h, "Gated recurrence"): whole batches forward and backward, packed
prompts and single tokens on a cache of slots.

    y, last = ssm_gated_scan_fwd(x, a_gate, x_gate, a_param, a_bias, x_bias, z)
    y, last, saved = ssm_gated_scan_fwd_ckpt(x, a_gate, x_gate, a_param, a_bias, x_bias, z)
    grads = ssm_gated_scan_bwd_ckpt(x, a_gate, x_gate, a_param, dy, saved, a_bias, x_bias, z)
    y = ssm_gated_scan_packed_fwd(x, a_gate, x_gate, a_param, cu_seqlens, cache=states, cache_slots=slots)
    y = ssm_gated_update_cache(states, slots, x, a_gate, x_gate, a_param)

x, a_gate, x_gate, z and y share one dtype, float32 or bfloat16; a_param, a_bias, x_bias: (dim,) fp32.
Batches are (batch, seqlen, dim), contiguous; packed rows (total, dim) and tokens (batch, dim) may lie
apart (columns of a wider tensor).  Caches, slots and cu_seqlens are as in ``serving.py``.  A call
allocates only what it returns, and its workspace when none is passed in, both on the stream that it
runs on, so that calls may be captured into a graph.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import SSM_BF16, SSM_F32, GatedStrides, _check, load_library
from .serving import _cache, _dense, _indices, _optional, _packed, _refuse, _row_stride, _run


def _code(dtype: torch.dtype) -> int:
    if dtype is torch.bfloat16:
        return SSM_BF16
    if dtype is torch.float32:
        return SSM_F32
    raise TypeError(f"x must be float32 or bfloat16, got {dtype}")


def _param_ptrs(a_param, a_bias, x_bias, dim: int, dev: int):
    f = torch.float32
    return (_dense(a_param, "a_param", (dim,), f, dev), _optional(a_bias, "a_bias", (dim,), f, dev),
            _optional(x_bias, "x_bias", (dim,), f, dev))


@functools.lru_cache(maxsize=256)  # of the sizes alone, and a call into the library costs a microsecond
def _workspace_bytes(batch: int, seqlen: int, dim: int, code: int, backward: int) -> int:
    n = ctypes.c_int64(0)
    _check(load_library().ssm_gated_scan_workspace(batch, seqlen, dim, code, backward, ctypes.byref(n)))
    return n.value


def ssm_gated_scan_workspace(batch: int, seqlen: int, dim: int, dtype: torch.dtype, backward: bool = False) -> int:
    """Bytes of workspace of a forward or backward over a batch (packed prompts: one sequence of all rows)."""
    return _workspace_bytes(batch, seqlen, dim, _code(dtype), int(bool(backward)))


def _workspace(given: Optional[torch.Tensor], x: torch.Tensor, batch: int, seqlen: int, code: int, backward: int):
    """(the tensor, to be kept until the call is made, its address and size)"""
    if given is None:
        n = _workspace_bytes(batch, seqlen, x.shape[-1], code, backward)
        if n == 0:
            return None, None, 0
        given = x.new_empty(n, dtype=torch.uint8)
    return given, given.data_ptr(), given.numel()


def gated_checkpoint_shape(batch: int, seqlen: int, dim: int) -> Tuple[int, int]:
    """Shape of the checkpoints of ssm_gated_scan_fwd_ckpt: the state after every 64th row, of each sequence if
    there are several of 256 rows or more, else of the batch's rows."""
    return (batch * (seqlen // 64) if batch > 1 and seqlen >= 256 else batch * seqlen // 64, dim)


def _batch(x, a_gate, x_gate, a_param, a_bias, x_bias, z, initial_state):
    """(shape, device, code, pointers of the inputs) of a batch's call."""
    if x is None or x.dim() != 3:
        raise ValueError("x must be (batch, seqlen, dim)")
    batch, seqlen, dim = shape = x.shape
    dev, ty, code = x.get_device(), x.dtype, _code(x.dtype)
    f = torch.float32
    px, pa, pg = (_dense(t, n, shape, ty, dev) for t, n in ((x, "x"), (a_gate, "a_gate"), (x_gate, "x_gate")))
    pp, pab, pxb = _param_ptrs(a_param, a_bias, x_bias, dim, dev)
    pz = _optional(z, "z", shape, ty, dev)
    return shape, dev, code, (px, pa, pg, pp, pab, pxb, pz), _optional(initial_state, "initial_state", (batch, dim), f, dev)


def _forward(x, a_gate, x_gate, a_param, a_bias, x_bias, z, a_scale, initial_state, y, last_state, return_last_state,
             checkpoints, save, workspace, stream):
    lib = load_library()
    shape, dev, code, ptrs, h0 = _batch(x, a_gate, x_gate, a_param, a_bias, x_bias, z, initial_state)
    batch, seqlen, dim = shape
    f = torch.float32
    _optional(y, "y", shape, x.dtype, dev)
    _optional(last_state, "last_state", (batch, dim), f, dev)
    _optional(checkpoints, "checkpoints", gated_checkpoint_shape(batch, seqlen, dim), f, dev)
    if workspace is not None:
        _dense(workspace, "workspace", workspace.shape, torch.uint8, dev)

    def call(st):
        out = torch.empty_like(x) if y is None else y
        last = last_state
        if last is None and return_last_state:
            last = x.new_empty((batch, dim), dtype=f) if h0 is None else torch.empty_like(initial_state)
        saved = x.new_empty(gated_checkpoint_shape(batch, seqlen, dim), dtype=f) if checkpoints is None and save else checkpoints
        _keep, ws, n = _workspace(workspace, x, batch, seqlen, code, 0)
        _check(lib.ssm_gated_scan_fwd(batch, seqlen, dim, code, *ptrs, a_scale, h0, out.data_ptr(),
                                      None if last is None else last.data_ptr(),
                                      None if saved is None else saved.data_ptr(), ws, n, st))
        return out, last, saved

    return _run(call, dev, stream)


def ssm_gated_scan_fwd(x: torch.Tensor, a_gate: torch.Tensor, x_gate: torch.Tensor, a_param: torch.Tensor,
                       a_bias: Optional[torch.Tensor] = None, x_bias: Optional[torch.Tensor] = None,
                       z: Optional[torch.Tensor] = None, *, a_scale: float = 8.0,
                       initial_state: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                       last_state: Optional[torch.Tensor] = None, return_last_state: bool = True,
                       workspace: Optional[torch.Tensor] = None,
                       stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The gated recurrence over a batch (include/ssm.h: ssm_gated_scan_fwd).  x, a_gate, x_gate, z, y:
    (batch, seqlen, dim); initial_state, last_state: (batch, dim) fp32.  Returns (y, last_state); last_state
    is None when return_last_state is False and none was passed in.  workspace: a uint8 tensor of
    ssm_gated_scan_workspace bytes, allocated here when None."""
    return _forward(x, a_gate, x_gate, a_param, a_bias, x_bias, z, a_scale, initial_state, y, last_state,
                    return_last_state, None, False, workspace, stream)[:2]


def ssm_gated_scan_fwd_ckpt(x: torch.Tensor, a_gate: torch.Tensor, x_gate: torch.Tensor, a_param: torch.Tensor,
                            a_bias: Optional[torch.Tensor] = None, x_bias: Optional[torch.Tensor] = None,
                            z: Optional[torch.Tensor] = None, *, a_scale: float = 8.0,
                            initial_state: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                            last_state: Optional[torch.Tensor] = None, return_last_state: bool = True,
                            checkpoints: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor], torch.Tensor]:
    """ssm_gated_scan_fwd that also stores the state after every 64th row, for ssm_gated_scan_bwd_ckpt.
    Returns (y, last_state, checkpoints)."""
    return _forward(x, a_gate, x_gate, a_param, a_bias, x_bias, z, a_scale, initial_state, y, last_state,
                    return_last_state, checkpoints, True, workspace, stream)


def ssm_gated_scan_bwd_ckpt(x: torch.Tensor, a_gate: torch.Tensor, x_gate: torch.Tensor, a_param: torch.Tensor,
                            dy: torch.Tensor, checkpoints: torch.Tensor, a_bias: Optional[torch.Tensor] = None,
                            x_bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None, *,
                            a_scale: float = 8.0, initial_state: Optional[torch.Tensor] = None,
                            dlast_state: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            stream=None) -> dict:
    """Gradients of sum(dy y) + sum(dlast_state last_state) from the checkpoints of ssm_gated_scan_fwd_ckpt
    on the same inputs (include/ssm.h: ssm_gated_scan_bwd).  Returns a dict with dx, da_gate, dx_gate (x's
    dtype), da_param (fp32), and dz / da_bias / dx_bias / dinitial_state (None unless z / a_bias / x_bias /
    initial_state were given)."""
    lib = load_library()
    shape, dev, code, ptrs, h0 = _batch(x, a_gate, x_gate, a_param, a_bias, x_bias, z, initial_state)
    batch, seqlen, dim = shape
    f = torch.float32
    saved = _dense(checkpoints, "checkpoints", gated_checkpoint_shape(batch, seqlen, dim), f, dev)
    pdy = _dense(dy, "dy", shape, x.dtype, dev)
    dlast = _optional(dlast_state, "dlast_state", (batch, dim), f, dev)
    if workspace is not None:
        _dense(workspace, "workspace", workspace.shape, torch.uint8, dev)

    def call(st):
        out = {"dx": torch.empty_like(x), "da_gate": torch.empty_like(x), "dx_gate": torch.empty_like(x),
               "dz": None if z is None else torch.empty_like(x), "da_param": torch.empty_like(a_param),
               "da_bias": None if a_bias is None else torch.empty_like(a_bias),
               "dx_bias": None if x_bias is None else torch.empty_like(x_bias),
               "dinitial_state": None if initial_state is None else torch.empty_like(initial_state)}
        p = {k: None if t is None else t.data_ptr() for k, t in out.items()}
        _keep, ws, n = _workspace(workspace, x, batch, seqlen, code, 1)
        _check(lib.ssm_gated_scan_bwd(batch, seqlen, dim, code, *ptrs, a_scale, h0, saved, pdy, dlast, p["dx"],
                                      p["da_gate"], p["dx_gate"], p["da_param"], p["da_bias"], p["dx_bias"], p["dz"],
                                      p["dinitial_state"], ws, n, st))
        return out

    return _run(call, dev, stream)


def _row2(t: Optional[torch.Tensor], name: str, shape, dtype, device: int) -> int:
    """_row_stride of a matrix: elements between its rows."""
    if t is None or t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        _refuse(t, name, shape, dtype, device)
    row, one = t.stride()
    rows, width = shape
    if one == 1 and row >= width:
        return row
    return _row_stride(t, name, shape, dtype, device)


def _rows(x, a_gate, x_gate, a_param, a_bias, x_bias, z, y):
    """(shape, device, code, pointers of the inputs, strides) of a call on rows that may lie apart."""
    if x is None or x.dim() != 2:
        raise ValueError("x must be (rows, dim)")
    shape = x.shape
    dev, ty, code = x.get_device(), x.dtype, _code(x.dtype)
    strides = GatedStrides(_row2(x, "x", shape, ty, dev), _row2(a_gate, "a_gate", shape, ty, dev),
                           _row2(x_gate, "x_gate", shape, ty, dev), 0 if z is None else _row2(z, "z", shape, ty, dev),
                           0 if y is None else _row2(y, "y", shape, ty, dev))
    f, one = torch.float32, shape[1:]
    return shape, dev, code, (x.data_ptr(), a_gate.data_ptr(), x_gate.data_ptr(), _dense(a_param, "a_param", one, f, dev),
                              None if a_bias is None else _dense(a_bias, "a_bias", one, f, dev),
                              None if x_bias is None else _dense(x_bias, "x_bias", one, f, dev),
                              None if z is None else z.data_ptr()), strides


def ssm_gated_scan_packed_fwd(x: torch.Tensor, a_gate: torch.Tensor, x_gate: torch.Tensor, a_param: torch.Tensor,
                              cu_seqlens: torch.Tensor, a_bias: Optional[torch.Tensor] = None,
                              x_bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None, *,
                              a_scale: float = 8.0, cache: Optional[torch.Tensor] = None,
                              cache_slots: Optional[torch.Tensor] = None, has_initial: Optional[torch.Tensor] = None,
                              y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """The gated recurrence of every packed sequence (include/ssm.h: ssm_gated_scan_packed_fwd).  x, a_gate,
    x_gate, z, y: (total, dim); cache: (slots, dim) fp32 or bf16, or None.  Returns y; rows of no sequence
    are left as they were (as allocated)."""
    lib = load_library()
    shape, dev, code, ptrs, strides = _rows(x, a_gate, x_gate, a_param, a_bias, x_bias, z, y)
    total, dim = shape
    ref = _cache(cache, "cache", (dim,), dev) if cache is not None else None
    seqs = _packed(cu_seqlens, cache_slots, has_initial, total, ref, 0, dev)
    if workspace is not None:
        _dense(workspace, "workspace", workspace.shape, torch.uint8, dev)

    def call(st):
        out = x.new_empty((total, dim)) if y is None else y
        _keep, ws, n = _workspace(workspace, x, 1, total, code, 0)
        _check(lib.ssm_gated_scan_packed_fwd(seqs, dim, code, *ptrs, a_scale, out.data_ptr(), ref, strides, ws, n, st))
        return out

    return _run(call, dev, stream)


def ssm_gated_update_cache(cache: torch.Tensor, cache_slots: Optional[torch.Tensor], x: torch.Tensor,
                           a_gate: torch.Tensor, x_gate: torch.Tensor, a_param: torch.Tensor,
                           a_bias: Optional[torch.Tensor] = None, x_bias: Optional[torch.Tensor] = None,
                           z: Optional[torch.Tensor] = None, *, a_scale: float = 8.0,
                           y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of the gated recurrence on a cache (include/ssm.h: ssm_gated_update_cache).  cache: (slots,
    dim) fp32 or bf16, updated in place; x, a_gate, x_gate, z, y: (batch, dim).  Returns y."""
    lib = load_library()
    shape, dev, code, ptrs, strides = _rows(x, a_gate, x_gate, a_param, a_bias, x_bias, z, y)
    batch, dim = shape
    ref = _cache(cache, "cache", (dim,), dev)
    slots = _indices(cache_slots, "cache_slots", batch, dev, ref.slots)

    def call(st):
        out = x.new_empty((batch, dim)) if y is None else y
        _check(lib.ssm_gated_update_cache(batch, dim, code, ref, slots, *ptrs, a_scale, out.data_ptr(), strides, st))
        return out

    return _run(call, dev, stream)
