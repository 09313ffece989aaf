"""Serving calls of the binding: prompts packed one behind another, single tokens on a cache of
slots, and cached states set aside in 8 bits (include/ssm.h, "Serving").

    y = ssm_causal_conv1d_packed_fwd(x, weight, cu_seqlens, bias, cache=windows, cache_slots=slots)
    y = ssm_scan_packed_fwd(x, delta, A, B, C, cu_seqlens, D=D, z=z, cache=states, cache_slots=slots)
    y = ssm_causal_conv1d_update_cache(windows, slots, x, weight, bias)
    y = ssm_state_update_cache(states, slots, x, delta, A, B, C, D=D, z=z)
    y = ssm_ssd_state_update_cache(states, slots, x, dt, A, B, C, D=D, z=z)
    ssm_cache_store_q8(states, slots, codes, scales, entries)
    ssm_cache_load_q8(codes, scales, entries, states, slots)

Sequence s of a packed tensor is its rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1; cu_seqlens,
cache_slots and the entries are int32, has_initial bool or uint8, all on the tensors' device.
cache_slots None: sequence (entry) i has slot i.  A negative slot is the padding of a batch: a step
leaves that entry's row of y as it was, a prompt starts from zeros and stores no state.  Caches are
(slots, dim, dstate) and the like, fp32 or bf16, updated in place; x, delta, B, C, z, dt and y are
rows that may lie apart (columns of a wider tensor), each row contiguous.  A call allocates only
what it returns, and the packed scan its workspace when none is passed in; both on the stream that
it runs on, so that calls may be captured into a graph.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from . import SSM_BF16, SSM_F32, Cache, Packed, RowStrides, _check, _dtype_code, load_library

# A decode step's kernel takes a few microseconds, so the checks are written to cost little: devices
# are compared by index, and what is wrong is worked out only once something is.


# the current stream's handle; the public call makes a Stream object first, which takes a microsecond
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _refuse(t, name: str, shape, dtype, device: int) -> None:
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on the other tensors' device")
    raise ValueError(f"{name} must be contiguous")


def _dense(t: Optional[torch.Tensor], name: str, shape, dtype, device: int) -> int:
    """The address of a contiguous tensor of this shape, dtype and device."""
    if (t is None or t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous()):
        _refuse(t, name, shape, dtype, device)
    return t.data_ptr()


def _optional(t: Optional[torch.Tensor], name: str, shape, dtype, device: int) -> Optional[int]:
    return None if t is None else _dense(t, name, shape, dtype, device)


def _row_stride(t: Optional[torch.Tensor], name: str, shape, dtype, device: int) -> int:
    """Elements between the rows of t (0: contiguous or at most one), whose rows must be contiguous."""
    if t is None or t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        _refuse(t, name, shape, dtype, device)
    if t.is_contiguous():
        return 0
    stride = t.stride()
    width = 1
    for n, s in zip(reversed(shape[1:]), reversed(stride[1:])):
        if n > 1 and s != width:
            raise ValueError(f"the rows of {name} must be contiguous")
        width *= n
    if shape[0] <= 1:
        return 0
    if stride[0] < width:
        raise ValueError(f"the rows of {name} must not overlap")
    return stride[0]


def _cache(t: Optional[torch.Tensor], name: str, entry, device: int, dtype=None) -> Cache:
    """The cache's descriptor: (slots,) + entry, each slot contiguous."""
    if t is None:
        raise ValueError(f"{name} is required")
    shape = t.shape
    if shape[1:] != entry:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected (slots, {', '.join(map(str, entry))})")
    ty = t.dtype
    if ty is not dtype and (dtype is not None or ty not in (torch.float32, torch.bfloat16)):
        raise TypeError(f"{name} has dtype {ty}, expected {dtype or 'float32 or bfloat16'}")
    return Cache(t.data_ptr(), shape[0], _row_stride(t, name, shape, ty, device),
                 SSM_BF16 if ty is torch.bfloat16 else SSM_F32, 0)


def _indices(t: Optional[torch.Tensor], name: str, count: int, device: int, slots: int) -> Optional[int]:
    if t is None:
        if slots < count:
            raise ValueError(f"without {name} there must be at least {count} slots, not {slots}")
        return None
    return _dense(t, name, (count,), torch.int32, device)


def _packed(cu_seqlens, cache_slots, has_initial, total: int, ref: Optional[Cache], max_seqlen: int, device: int) -> Packed:
    if cu_seqlens is None or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold one more entry than there are sequences")
    nseq = cu_seqlens.numel() - 1
    cu = _dense(cu_seqlens, "cu_seqlens", (nseq + 1,), torch.int32, device)
    if ref is None:
        if cache_slots is not None or has_initial is not None:
            raise ValueError("cache_slots and has_initial need a cache")
        return Packed(total, nseq, max_seqlen, cu, None, None)
    slots = _indices(cache_slots, "cache_slots", nseq, device, ref.slots)
    if has_initial is not None:
        if has_initial.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"has_initial has dtype {has_initial.dtype}, expected bool or uint8")
        has_initial = _dense(has_initial, "has_initial", (nseq,), has_initial.dtype, device)
    return Packed(total, nseq, max_seqlen, cu, slots, has_initial)


@contextlib.contextmanager
def _other(device: int, stream):
    """The tensors' device current, and the given stream, where they are not already."""
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if not hasattr(stream, "cuda_stream"):
            stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                      else torch.cuda.default_stream(device))
        with torch.cuda.stream(stream):
            yield


def _run(call, device: int, stream):
    """call(stream handle) with the tensors' device current and, when one is given, on that stream: what
    it allocates then belongs to the stream that uses it."""
    if device < 0:
        raise ValueError("the tensors are on the host, expected a GPU")
    if stream is None and torch.cuda.current_device() == device:
        return call(_raw_stream(device))
    with _other(device, stream):
        return call(_raw_stream(device))


def ssm_causal_conv1d_packed_fwd(x: torch.Tensor, weight: torch.Tensor, cu_seqlens: torch.Tensor,
                                 bias: Optional[torch.Tensor] = None, silu: bool = True, *,
                                 cache: Optional[torch.Tensor] = None, cache_slots: Optional[torch.Tensor] = None,
                                 has_initial: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                                 stream=None) -> torch.Tensor:
    """The causal convolution of every packed sequence (include/ssm.h: ssm_causal_conv1d_packed_fwd).
    x, y: (total, dim); weight: (dim, width) fp32; bias: (dim,) fp32; cache: (slots, dim, width - 1) in
    x's dtype or None.  Returns y; rows of no sequence are left as they were (as allocated)."""
    lib = load_library()
    if x is None or weight is None or x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be (total, dim) and weight (dim, width)")
    total, dim = x.shape
    width = weight.shape[1]
    dev, dt, code = x.get_device(), x.dtype, _dtype_code(x)
    strides = RowStrides(x=_row_stride(x, "x", x.shape, dt, dev))
    w = _dense(weight, "weight", (dim, width), torch.float32, dev)
    b = _optional(bias, "bias", (dim,), torch.float32, dev)
    ref = _cache(cache, "cache", (dim, width - 1), dev, dt) if cache is not None else None
    seqs = _packed(cu_seqlens, cache_slots, has_initial, total, ref, 0, dev)
    if y is not None:
        strides.y = _row_stride(y, "y", x.shape, dt, dev)

    def call(st):
        out = x.new_empty((total, dim)) if y is None else y
        _check(lib.ssm_causal_conv1d_packed_fwd(seqs, dim, width, code, x.data_ptr(), w, b, int(bool(silu)),
                                                out.data_ptr(), ref, strides, st))
        return out

    return _run(call, dev, stream)


def ssm_scan_packed_workspace(total: int, sequences: int, max_seqlen: int, dim: int, dstate: int,
                              dtype: torch.dtype) -> int:
    """Bytes of workspace of ssm_scan_packed_fwd for these sizes, on the current device."""
    lib = load_library()
    n = ctypes.c_int64(0)
    _check(lib.ssm_scan_packed_workspace(Packed(total, sequences, max_seqlen, None, None, None), dim, dstate,
                                         SSM_BF16 if dtype == torch.bfloat16 else SSM_F32, ctypes.byref(n)))
    return n.value


def ssm_scan_packed_fwd(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                        cu_seqlens: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                        delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False, *,
                        cache: Optional[torch.Tensor] = None, cache_slots: Optional[torch.Tensor] = None,
                        has_initial: Optional[torch.Tensor] = None, max_seqlen: int = 0,
                        y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """The selective scan of every packed sequence (include/ssm.h: ssm_scan_packed_fwd).  x, delta, z, y:
    (total, dim); B, C: (total, dstate); A: (dim, dstate) fp32; D, delta_bias: (dim,) fp32; cache: (slots,
    dim, dstate) fp32 or bf16, or None.  max_seqlen (the longest sequence; 0: not known) only chooses the
    launch shape.  workspace: a uint8 tensor of ssm_scan_packed_workspace bytes, allocated here when None.
    Returns y; rows of no sequence are left as they were (as allocated)."""
    lib = load_library()
    if x is None or A is None or x.dim() != 2 or A.dim() != 2:
        raise ValueError("x must be (total, dim) and A (dim, dstate)")
    total, dim = x.shape
    dstate = A.shape[1]
    dev, dt, code = x.get_device(), x.dtype, _dtype_code(x)
    bc = (total, dstate)
    strides = RowStrides(_row_stride(x, "x", x.shape, dt, dev), _row_stride(delta, "delta", x.shape, dt, dev),
                         _row_stride(B, "B", bc, dt, dev), _row_stride(C, "C", bc, dt, dev),
                         0 if z is None else _row_stride(z, "z", x.shape, dt, dev),
                         0 if y is None else _row_stride(y, "y", x.shape, dt, dev))
    a = _dense(A, "A", (dim, dstate), torch.float32, dev)
    d = _optional(D, "D", (dim,), torch.float32, dev)
    bias = _optional(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    ref = _cache(cache, "cache", (dim, dstate), dev) if cache is not None else None
    seqs = _packed(cu_seqlens, cache_slots, has_initial, total, ref, int(max_seqlen), dev)
    if workspace is not None:
        _dense(workspace, "workspace", workspace.shape, torch.uint8, dev)

    def call(st):
        out = x.new_empty((total, dim)) if y is None else y
        ws = workspace
        if ws is None:
            n = ctypes.c_int64(0)
            _check(lib.ssm_scan_packed_workspace(seqs, dim, dstate, code, ctypes.byref(n)))
            ws = x.new_empty(n.value, dtype=torch.uint8) if n.value else None
        _check(lib.ssm_scan_packed_fwd(seqs, dim, dstate, code, x.data_ptr(), delta.data_ptr(), a, B.data_ptr(),
                                       C.data_ptr(), d, None if z is None else z.data_ptr(), bias,
                                       int(bool(delta_softplus)), out.data_ptr(), ref, strides,
                                       None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), st))
        return out

    return _run(call, dev, stream)


def ssm_causal_conv1d_update_cache(cache: Optional[torch.Tensor], cache_slots: Optional[torch.Tensor],
                                   x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                                   silu: bool = True, *, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of the convolution on a cache (include/ssm.h: ssm_causal_conv1d_update_cache).  cache:
    (slots, dim, width - 1) in x's dtype, updated in place; x, y: (batch, dim).  Returns y."""
    lib = load_library()
    if x is None or weight is None or x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be (batch, dim) and weight (dim, width)")
    batch, dim = x.shape
    width = weight.shape[1]
    dev, dt, code = x.get_device(), x.dtype, _dtype_code(x)
    strides = RowStrides(x=_row_stride(x, "x", x.shape, dt, dev))
    w = _dense(weight, "weight", (dim, width), torch.float32, dev)
    b = _optional(bias, "bias", (dim,), torch.float32, dev)
    ref = None
    if cache is not None or width != 1:
        ref = _cache(cache, "cache", (dim, width - 1), dev, dt)
    slots = _indices(cache_slots, "cache_slots", batch, dev, batch if ref is None else ref.slots)
    if y is not None:
        strides.y = _row_stride(y, "y", x.shape, dt, dev)

    def call(st):
        out = x.new_empty((batch, dim)) if y is None else y
        _check(lib.ssm_causal_conv1d_update_cache(batch, dim, width, code, ref, slots, x.data_ptr(), w, b,
                                                  int(bool(silu)), out.data_ptr(), strides, st))
        return out

    return _run(call, dev, stream)


def ssm_state_update_cache(cache: torch.Tensor, cache_slots: Optional[torch.Tensor], x: torch.Tensor,
                           delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                           D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                           delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False, *,
                           y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of the selective scan on a cache (include/ssm.h: ssm_state_update_cache).  cache: (slots,
    dim, dstate) fp32 or bf16, updated in place; x, delta, z, y: (batch, dim); B, C: (batch, dstate).
    Returns y."""
    lib = load_library()
    if x is None or A is None or x.dim() != 2 or A.dim() != 2:
        raise ValueError("x must be (batch, dim) and A (dim, dstate)")
    batch, dim = x.shape
    dstate = A.shape[1]
    dev, dt, code = x.get_device(), x.dtype, _dtype_code(x)
    bc = (batch, dstate)
    strides = RowStrides(_row_stride(x, "x", x.shape, dt, dev), _row_stride(delta, "delta", x.shape, dt, dev),
                         _row_stride(B, "B", bc, dt, dev), _row_stride(C, "C", bc, dt, dev),
                         0 if z is None else _row_stride(z, "z", x.shape, dt, dev),
                         0 if y is None else _row_stride(y, "y", x.shape, dt, dev))
    a = _dense(A, "A", (dim, dstate), torch.float32, dev)
    d = _optional(D, "D", (dim,), torch.float32, dev)
    bias = _optional(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    ref = _cache(cache, "cache", (dim, dstate), dev)
    slots = _indices(cache_slots, "cache_slots", batch, dev, ref.slots)

    def call(st):
        out = x.new_empty((batch, dim)) if y is None else y
        _check(lib.ssm_state_update_cache(batch, dim, dstate, code, ref, slots, x.data_ptr(), delta.data_ptr(), a,
                                          B.data_ptr(), C.data_ptr(), d, None if z is None else z.data_ptr(), bias,
                                          int(bool(delta_softplus)), out.data_ptr(), strides, st))
        return out

    return _run(call, dev, stream)


def ssm_ssd_state_update_cache(cache: torch.Tensor, cache_slots: Optional[torch.Tensor], x: torch.Tensor,
                               dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                               D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                               dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False, *,
                               y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of the Mamba-2 SSD layer on a cache (include/ssm.h: ssm_ssd_state_update_cache).  cache:
    (slots, nheads, headdim, dstate) fp32 or bf16, updated in place; x, z, y: (batch, nheads, headdim);
    dt: (batch, nheads); B, C: (batch, ngroups, dstate); A, D, dt_bias: (nheads,) fp32.  Returns y."""
    lib = load_library()
    if x is None or B is None or x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be (batch, nheads, headdim) and B (batch, ngroups, dstate)")
    batch, nheads, headdim = x.shape
    ngroups, dstate = B.shape[1], B.shape[2]
    dev, ty, code = x.get_device(), x.dtype, _dtype_code(x)
    strides = RowStrides(_row_stride(x, "x", x.shape, ty, dev), _row_stride(dt, "dt", (batch, nheads), ty, dev),
                         _row_stride(B, "B", B.shape, ty, dev), _row_stride(C, "C", (batch, ngroups, dstate), ty, dev),
                         0 if z is None else _row_stride(z, "z", x.shape, ty, dev),
                         0 if y is None else _row_stride(y, "y", x.shape, ty, dev))
    if B.shape[0] != batch:
        raise ValueError(f"B has shape {tuple(B.shape)}, expected {(batch, ngroups, dstate)}")
    a = _dense(A, "A", (nheads,), torch.float32, dev)
    d = _optional(D, "D", (nheads,), torch.float32, dev)
    bias = _optional(dt_bias, "dt_bias", (nheads,), torch.float32, dev)
    ref = _cache(cache, "cache", (nheads, headdim, dstate), dev)
    slots = _indices(cache_slots, "cache_slots", batch, dev, ref.slots)

    def call(st):
        out = x.new_empty((batch, nheads, headdim)) if y is None else y
        _check(lib.ssm_ssd_state_update_cache(batch, nheads, headdim, dstate, ngroups, code, ref, slots, x.data_ptr(),
                                              dt.data_ptr(), a, B.data_ptr(), C.data_ptr(), d,
                                              None if z is None else z.data_ptr(), bias, int(bool(dt_softplus)),
                                              out.data_ptr(), strides, st))
        return out

    return _run(call, dev, stream)


def _q8(cache, cache_slots, codes, scales, store_slots):
    """What a store or load needs, checked.  The cache's entries are (rows, dstate) or (nheads, headdim,
    dstate)."""
    if cache is None or cache.dim() not in (3, 4):
        raise ValueError("cache must be (slots, dim, dstate) or (slots, nheads, headdim, dstate)")
    if codes is None or codes.dim() != cache.dim():
        raise ValueError("codes must be (stored,) + a slot's shape")
    dev = cache.get_device()
    entry = tuple(cache.shape[1:])
    ref = _cache(cache, "cache", entry, dev)
    stored = codes.shape[0]
    q = _dense(codes, "codes", (stored,) + entry, torch.int8, dev)
    sc = _dense(scales, "scales", (stored,) + entry[:-1], torch.float32, dev)
    if cache_slots is None and store_slots is None:
        count = min(ref.slots, stored)
    else:
        count = (cache_slots if cache_slots is not None else store_slots).numel()
    slots = _indices(cache_slots, "cache_slots", count, dev, ref.slots)
    where = _indices(store_slots, "store_slots", count, dev, stored)
    rows = entry[0] if len(entry) == 2 else entry[0] * entry[1]
    return dev, ref, count, rows, entry[-1], stored, q, sc, slots, where


def ssm_cache_store_q8(cache: torch.Tensor, cache_slots: Optional[torch.Tensor], codes: torch.Tensor,
                       scales: torch.Tensor, store_slots: Optional[torch.Tensor] = None, *, stream=None) -> None:
    """Sets the states of cache_slots aside as int8 codes with one scale per row of dstate values, in the
    entries store_slots of codes and scales (include/ssm.h: ssm_cache_store_q8).  cache: (slots, dim,
    dstate) or (slots, nheads, headdim, dstate); codes: (stored,) + a slot's shape, int8; scales: the same
    without dstate, fp32.  Without either index pair i is slot i and entry i."""
    lib = load_library()
    dev, ref, count, rows, dstate, stored, q, sc, slots, where = _q8(cache, cache_slots, codes, scales, store_slots)
    _run(lambda st: _check(lib.ssm_cache_store_q8(count, rows, dstate, ref, slots, stored, q, sc, where, st)), dev, stream)


def ssm_cache_load_q8(codes: torch.Tensor, scales: torch.Tensor, store_slots: Optional[torch.Tensor],
                      cache: torch.Tensor, cache_slots: Optional[torch.Tensor] = None, *, stream=None) -> None:
    """Reads entries store_slots of codes and scales back into cache_slots of the cache (include/ssm.h:
    ssm_cache_load_q8); an entry may be read into several slots."""
    lib = load_library()
    dev, ref, count, rows, dstate, stored, q, sc, slots, where = _q8(cache, cache_slots, codes, scales, store_slots)
    _run(lambda st: _check(lib.ssm_cache_load_q8(count, rows, dstate, stored, q, sc, where, ref, slots, st)), dev, stream)
