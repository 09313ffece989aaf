"""Beam search on cached states (include/ssm.h, "Beam search"): the selection over beams and vocabulary,
and the reordering of the caches that follows it.

    parents, tokens, scores, _ = ssm_beam_select(logits, scores, beams)
    ssm_cache_reorder([states, windows], slots, parents)

logits: (batch, rows, vocab), float32 or bfloat16, one row per hypothesis (one of a prompt's end, `beams`
of later steps); scores: (batch, rows) fp32, the hypotheses' sums of log-probabilities so far.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple, Union

import torch

from . import SSM_BF16, SSM_F32, Entries, _check, load_library
from .serving import _dense, _row_stride, _run


def _code(dtype: torch.dtype) -> int:
    if dtype is torch.bfloat16:
        return SSM_BF16
    if dtype is torch.float32:
        return SSM_F32
    raise TypeError(f"logits must be float32 or bfloat16, got {dtype}")


@functools.lru_cache(maxsize=256)  # of the sizes alone, and a call into the library costs a microsecond
def _workspace_bytes(batch: int, rows: int, vocab: int, beams: int, code: int) -> int:
    n = ctypes.c_int64(0)
    _check(load_library().ssm_beam_select_workspace(batch, rows, vocab, beams, code, ctypes.byref(n)))
    return n.value


def ssm_beam_select(logits: torch.Tensor, scores: torch.Tensor, beams: int, *, finished: Optional[torch.Tensor] = None,
                    eos: int = -1, workspace: Optional[torch.Tensor] = None, stream=None
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """The `beams` best continuations of each sequence (include/ssm.h: ssm_beam_select).  logits: (batch, rows,
    vocab), each row contiguous; scores: (batch, rows) fp32; finished: (batch, rows) bool or None, whose rows
    continue with `eos` alone.  Returns parents and tokens (batch, beams) int32, scores (batch, beams) fp32 in
    falling order, and finished (batch, beams) bool (None without finished).  workspace: a uint8 tensor of
    ssm_beam_select_workspace bytes, allocated here when None."""
    lib = load_library()
    if logits is None or logits.dim() != 3:
        raise ValueError("logits must be (batch, rows, vocab)")
    batch, rows, vocab = logits.shape
    dev, code = logits.get_device(), _code(logits.dtype)
    sb, sr, sv = logits.stride()
    if vocab > 1 and sv != 1:
        raise ValueError("the rows of logits must be contiguous")
    if (batch > 1 and sb == 0) or (rows > 1 and sr == 0):
        raise ValueError("the rows of logits must not overlap")
    ps = _dense(scores, "scores", (batch, rows), torch.float32, dev)
    pf = None
    if finished is not None:
        if finished.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"finished has dtype {finished.dtype}, expected bool or uint8")
        pf = _dense(finished, "finished", (batch, rows), finished.dtype, dev)
    beams = int(beams)
    if workspace is not None:
        _dense(workspace, "workspace", workspace.shape, torch.uint8, dev)

    def call(st):
        size = _workspace_bytes(batch, rows, vocab, beams, code)  # (and refuses bad sizes before anything is allocated)
        if workspace is None:
            ws = logits.new_empty(size, dtype=torch.uint8)
        else:
            ws, size = workspace, workspace.numel()
        kept = (batch, beams)
        parents = logits.new_empty(kept, dtype=torch.int32)
        tokens = logits.new_empty(kept, dtype=torch.int32)
        out = logits.new_empty(kept, dtype=torch.float32)
        fin = None if pf is None else logits.new_empty(kept, dtype=torch.bool)
        # a stride of one row is any: given as that of contiguous ones
        _check(lib.ssm_beam_select(batch, rows, vocab, beams, code, logits.data_ptr(), sb if batch > 1 else 0,
                                   sr if rows > 1 else 0, ps, pf, int(eos), parents.data_ptr(), tokens.data_ptr(),
                                   out.data_ptr(), None if fin is None else fin.data_ptr(), ws.data_ptr(), size, st))
        return parents, tokens, out, fin

    return _run(call, dev, stream)


def ssm_beam_select_workspace(batch: int, rows: int, vocab: int, beams: int, dtype: torch.dtype) -> int:
    """Bytes of workspace of ssm_beam_select for these sizes."""
    return _workspace_bytes(batch, rows, vocab, beams, _code(dtype))


def ssm_cache_reorder(caches: Union[torch.Tensor, Sequence[torch.Tensor]], cache_slots: Optional[torch.Tensor],
                      parents: torch.Tensor, *, stream=None) -> None:
    """Beam i of sequence b takes, in every cache and in place, the entry of beam parents[b, i] of the same
    sequence (include/ssm.h: ssm_cache_reorder).  caches: one tensor or several, each (slots,) + any shape of
    any dtype with contiguous slots (states, windows, int8 codes and their scales); cache_slots, parents:
    (batch, beams) int32; without cache_slots beam i of sequence b has slot b * beams + i."""
    lib = load_library()
    if parents is None or parents.dim() != 2:
        raise ValueError("parents must be (batch, beams)")
    batch, beams = parents.shape
    dev = parents.get_device()
    pp = _dense(parents, "parents", (batch, beams), torch.int32, dev)
    pslots = None if cache_slots is None else _dense(cache_slots, "cache_slots", (batch, beams), torch.int32, dev)
    if caches is None:
        raise ValueError("caches is required")
    if isinstance(caches, torch.Tensor):
        caches = (caches,)
    table = (Entries * len(caches))()
    for k, c in enumerate(caches):
        if c is None or c.dim() < 1:
            raise ValueError(f"caches[{k}] must be (slots, ...)")
        es = c.element_size()
        stride = _row_stride(c, f"caches[{k}]", c.shape, c.dtype, dev)
        slots = c.shape[0]
        if pslots is None and slots < batch * beams:
            raise ValueError(f"without cache_slots there must be at least {batch * beams} slots, not {slots}")
        table[k] = Entries(c.data_ptr(), slots, stride * es, (c.numel() // slots if slots else 0) * es)
    _run(lambda st: _check(lib.ssm_cache_reorder(batch, beams, table, len(caches), pslots, pp, st)), dev, stream)
