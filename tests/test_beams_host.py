"""Beam search's entry points on the host: refusals before any HIP call, and the binding's own checks."""
import ctypes

import pytest
import torch

import selective_state_space_61_amd as ssm
from test_serving_host import BF16, F32, INVALID, MISALIGNED, OK, UNSUPPORTED, err, fake, lib  # noqa: F401

BIG = 1 << 40


def select(lib, batch=2, rows=3, vocab=100, beams=3, dtype=F32, logits=fake(0), sb=0, sr=0, scores=fake(1), fin=fake(2), eos=5,
           parents=fake(3), tokens=fake(4), out=fake(5), ofin=fake(6), ws=fake(7), nws=BIG):
    return lib.ssm_beam_select(batch, rows, vocab, beams, dtype, logits, sb, sr, scores, fin, eos, parents, tokens, out, ofin, ws,
                               nws, None)


def entries(*items):
    base = dict(data=fake(10), slots=8, slot_stride=0, bytes=64)
    table = (ssm.Entries * len(items))()
    for k, kw in enumerate(items):
        table[k] = ssm.Entries(**dict(base, **dict(dict(data=fake(10 + k)), **kw)))
    return table


def reorder(lib, batch=2, beams=4, caches=None, count=None, slots=fake(30), parents=fake(31)):
    caches = entries({}) if caches is None else caches
    return lib.ssm_cache_reorder(batch, beams, caches, len(caches) if count is None else count, slots, parents, None)


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(rows=0), dict(vocab=0), dict(beams=0), dict(vocab=1 << 31), dict(batch=1 << 31),
                                dict(rows=1, vocab=2, beams=3), dict(eos=-1), dict(eos=100), dict(sr=-1), dict(sb=-5),
                                dict(fin=None), dict(sr=1 << 62), dict(sb=1 << 62)])
def test_bad_sizes(lib, kw):  # noqa: F811
    assert select(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(rows=65), dict(beams=65),
                                dict(batch=(1 << 31) - 1, rows=64, vocab=(1 << 31) - 1)])
def test_unsupported(lib, kw):  # noqa: F811
    assert select(lib, **kw) == UNSUPPORTED


def test_missing_misaligned_and_overlapping(lib):  # noqa: F811
    for k in ("logits", "scores", "parents", "tokens", "out"):
        assert select(lib, **{k: None}) == INVALID and "NULL" in err(lib), k
    for kw in (dict(logits=fake(0, 2)), dict(logits=fake(0, 1), dtype=BF16), dict(scores=fake(1, 2)), dict(parents=fake(3, 1)),
               dict(ws=fake(7, 8))):
        assert select(lib, **kw) == MISALIGNED, kw
    for kw in (dict(parents=fake(0, 400)), dict(tokens=fake(3, 8)), dict(out=fake(1)), dict(ofin=fake(2)), dict(ws=fake(0))):
        assert select(lib, **kw) == INVALID and "overlap" in err(lib), kw
    for kw in (dict(ws=None), dict(nws=100)):
        assert select(lib, **kw) == INVALID and "workspace" in err(lib)
    assert select(lib, batch=0, logits=None) == OK


def test_workspace_sizes(lib):  # noqa: F811
    n = ctypes.c_int64(-1)
    assert lib.ssm_beam_select_workspace(2, 3, 50000, 4, BF16, ctypes.byref(n)) == OK and n.value > 0
    assert lib.ssm_beam_select_workspace(2, 3, 50000, 4, BF16, None) == INVALID
    assert lib.ssm_beam_select_workspace(2, 65, 50000, 4, BF16, ctypes.byref(n)) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(beams=0), INVALID), (dict(beams=65), UNSUPPORTED), (dict(count=-1), INVALID),
    (dict(caches=entries(dict(slots=-1))), INVALID), (dict(caches=entries(dict(bytes=-1))), INVALID),
    (dict(caches=entries(dict(slot_stride=63))), INVALID), (dict(caches=entries(dict(slots=1 << 31))), INVALID),
    (dict(caches=entries(dict(slot_stride=1 << 62))), INVALID), (dict(caches=entries({}, dict(data=None))), INVALID),
    (dict(parents=None), INVALID), (dict(parents=fake(31, 2)), MISALIGNED), (dict(slots=fake(30, 1)), MISALIGNED),
    (dict(parents=fake(10, 100)), INVALID), (dict(slots=fake(10)), INVALID),
    (dict(caches=entries(dict(slots=2, bytes=1 << 50))), UNSUPPORTED)])
def test_reorder_refusals(lib, kw, status):  # noqa: F811
    assert reorder(lib, **kw) == status


@pytest.mark.parametrize("order", [(0, 0), (0, 1, 2, 1), (3, 2, 1, 3), (5, 6, 5)])
def test_reorder_of_one_cache_twice(lib, order):  # noqa: F811
    caches = entries(*(dict(data=fake(10 + k)) for k in order))
    assert reorder(lib, caches=caches) == INVALID and "again" in err(lib)


def test_reorder_with_nothing_to_do(lib):  # noqa: F811
    assert reorder(lib, batch=0, parents=None) == OK and reorder(lib, beams=1, parents=None) == OK
    assert reorder(lib, count=0, parents=None) == OK
    assert reorder(lib, caches=entries(dict(slots=0, data=None), dict(bytes=0, data=None)), parents=None) == OK


# ---- the binding ---------------------------------------------------------------------------------------


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw,exc", [
    (dict(logits=t(2, 50)), ValueError), (dict(logits=None), ValueError), (dict(logits=t(2, 3, 50, dtype=torch.float16)), TypeError),
    (dict(logits=t(2, 50, 3).transpose(1, 2)), ValueError), (dict(logits=t(1, 1, 50).expand(2, 3, 50)), ValueError),
    (dict(scores=t(2, 4)), ValueError), (dict(scores=t(2, 3).double()), TypeError), (dict(scores=None), ValueError),
    (dict(finished=t(2, 3)), TypeError), (dict(finished=t(2, 2, dtype=torch.bool)), ValueError), (dict(workspace=t(5)), TypeError)])
def test_select_binding(kw, exc):
    with pytest.raises(exc):
        ssm.ssm_beam_select(**dict(dict(logits=t(2, 3, 50), scores=t(2, 3), beams=4), **kw))


@pytest.mark.parametrize("kw,exc", [
    (dict(parents=t(8, dtype=torch.int32)), ValueError), (dict(parents=t(2, 4)), TypeError), (dict(parents=None), ValueError),
    (dict(cache_slots=t(2, 3, dtype=torch.int32)), ValueError), (dict(cache_slots=t(2, 4, dtype=torch.int64)), TypeError),
    (dict(caches=None), ValueError), (dict(caches=[t(9, 5), None]), ValueError), (dict(caches=t(7, 5), cache_slots=None), ValueError),
    (dict(caches=t(5, 9).T), ValueError), (dict(caches=t()), ValueError), (dict(caches=t(1, 5).expand(9, 5)), ValueError)])
def test_reorder_binding(kw, exc):
    with pytest.raises(exc):
        ssm.ssm_cache_reorder(**dict(dict(caches=t(9, 5), cache_slots=t(2, 4, dtype=torch.int32),
                                          parents=t(2, 4, dtype=torch.int32)), **kw))


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="expected a GPU"):
        ssm.ssm_beam_select(t(2, 3, 50), t(2, 3), 4)
    with pytest.raises(ValueError, match="expected a GPU"):
        ssm.ssm_cache_reorder(t(9, 5), None, t(2, 4, dtype=torch.int32))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int8])
def test_no_workspace_for_types_that_the_call_refuses(dtype):
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssm.ssm_beam_select_workspace(2, 3, 50, 4, dtype)
