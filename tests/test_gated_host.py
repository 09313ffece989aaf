"""The gated recurrence's entry points on the host: every call here is refused (or has nothing to do)
before any HIP call, so no GPU is needed and the pointers are never dereferenced; and the binding's own
checks."""
import ctypes

import pytest
import torch

import selective_state_space_61_amd as ssm
from test_serving_host import BF16, F32, INVALID, MISALIGNED, OK, UNSUPPORTED, cache, err, fake, lib, packed  # noqa: F401

BIG = 1 << 40  # of workspace
GATES = dict(x=fake(0), ag=fake(1), xg=fake(2), param=fake(3), ab=fake(4), xb=fake(5), z=fake(6))


def inputs(kw):
    return [kw.pop(k, v) for k, v in GATES.items()], kw.pop("scale", 8.0)


def fwd(lib, batch=2, seqlen=300, dim=16, dtype=F32, h0=fake(7), y=fake(8), last=fake(9), saved=fake(10), ws=fake(11), nws=BIG,
        **kw):
    gates, scale = inputs(kw)
    return lib.ssm_gated_scan_fwd(batch, seqlen, dim, dtype, *gates, scale, h0, y, last, saved, ws, nws, None)


def bwd(lib, batch=2, seqlen=300, dim=16, dtype=F32, h0=fake(7), saved=fake(8), dy=fake(9), dlast=fake(10), dx=fake(11),
        dag=fake(12), dxg=fake(13), dparam=fake(14), dab=fake(15), dxb=fake(16), dz=fake(17), dh0=fake(18), ws=fake(19), nws=BIG,
        **kw):
    gates, scale = inputs(kw)
    return lib.ssm_gated_scan_bwd(batch, seqlen, dim, dtype, *gates, scale, h0, saved, dy, dlast, dx, dag, dxg, dparam, dab,
                                  dxb, dz, dh0, ws, nws, None)


def prompt(lib, seqs=None, dim=16, dtype=F32, y=fake(8), c="own", st=None, ws=fake(11), nws=BIG, **kw):
    gates, scale = inputs(kw)
    c = cache() if c == "own" else c
    return lib.ssm_gated_scan_packed_fwd(packed() if seqs is None else seqs, dim, dtype, *gates, scale, y, c, st, ws, nws, None)


def step(lib, batch=2, dim=16, dtype=F32, c="own", slots=fake(22), y=fake(8), st=None, **kw):
    gates, scale = inputs(kw)
    c = cache() if c == "own" else c
    return lib.ssm_gated_update_cache(batch, dim, dtype, c, slots, *gates, scale, y, st, None)


ALL = [fwd, bwd, prompt, step]


@pytest.mark.parametrize("call,kw", [(fwd, dict(batch=-1)), (fwd, dict(seqlen=-1)), (bwd, dict(dim=-2)), (prompt, dict(dim=-1)),
                                     (step, dict(batch=-1)), (step, dict(dim=-1)), (fwd, dict(batch=1 << 40, seqlen=1 << 40)),
                                     (prompt, dict(seqs=packed(total=-1))), (prompt, dict(seqs=packed(sequences=1 << 31)))])
def test_bad_sizes(lib, call, kw):  # noqa: F811
    assert call(lib, **kw) == INVALID


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("dtype", [-1, 2, 9])
def test_unknown_types(lib, call, dtype):  # noqa: F811
    assert call(lib, dtype=dtype) == UNSUPPORTED


@pytest.mark.parametrize("call,kw", [(fwd, dict(batch=1 << 16, seqlen=1 << 15, dim=1)), (fwd, dict(dim=1 << 23)),
                                     (step, dict(batch=1 << 31)), (step, dict(dim=1 << 23)), (prompt, dict(dim=1 << 23)),
                                     (fwd, dict(batch=1, seqlen=(1 << 31) - 1, dim=1 << 20))])
def test_too_large(lib, call, kw):  # noqa: F811
    assert call(lib, **kw) == UNSUPPORTED


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("scale", [-1.0, float("nan"), float("inf")])
def test_scales(lib, call, scale):  # noqa: F811
    assert call(lib, scale=scale) == INVALID and "a_scale" in err(lib)


@pytest.mark.parametrize("call,names", [(fwd, "x ag xg param y"), (bwd, "x ag xg param dy dx dag dxg dparam saved"),
                                        (prompt, "x ag xg param y"), (step, "x ag xg param y c")])
def test_missing_pointers(lib, call, names):  # noqa: F811
    for k in names.split():
        assert call(lib, **{k: None}) == INVALID and "NULL" in err(lib), k


def test_z_needs_its_gradient(lib):  # noqa: F811
    assert bwd(lib, dz=None) == INVALID and "dz" in err(lib)


@pytest.mark.parametrize("call,kw", [(fwd, dict(x=fake(0, 2))), (fwd, dict(dtype=BF16, ag=fake(1, 1))), (fwd, dict(param=fake(3, 2))),
                                     (fwd, dict(h0=fake(7, 1))), (fwd, dict(saved=fake(10, 2))), (fwd, dict(ws=fake(11, 8))),
                                     (bwd, dict(dy=fake(9, 1))), (bwd, dict(dab=fake(15, 2))), (bwd, dict(dh0=fake(18, 2))),
                                     (bwd, dict(ws=fake(19, 4))), (prompt, dict(xg=fake(2, 3))), (prompt, dict(xb=fake(5, 1))),
                                     (prompt, dict(seqs=packed(total=200, cu_seqlens=fake(21, 2)))), (step, dict(z=fake(6, 2))),
                                     (step, dict(slots=fake(22, 2))), (step, dict(c=cache(data=fake(20, 2))))])
def test_misaligned(lib, call, kw):  # noqa: F811
    assert call(lib, **kw) == MISALIGNED


@pytest.mark.parametrize("call,kw", [(fwd, dict(nws=64)), (fwd, dict(ws=None)), (bwd, dict(nws=100)), (bwd, dict(ws=None)),
                                     (bwd, dict(seqlen=5, ws=None)), (prompt, dict(seqs=packed(total=1000), nws=16))])
def test_workspaces(lib, call, kw):  # noqa: F811
    assert call(lib, **kw) == INVALID and "workspace" in err(lib)


@pytest.mark.parametrize("call,kw", [
    (fwd, dict(y=fake(0, 64))), (fwd, dict(last=fake(7))), (fwd, dict(saved=fake(8))), (fwd, dict(ws=fake(6))),
    (fwd, dict(last=fake(8))), (bwd, dict(dx=fake(9))), (bwd, dict(dag=fake(11))),
    (bwd, dict(dparam=fake(3))), (bwd, dict(dh0=fake(7))), (bwd, dict(ws=fake(8))), (bwd, dict(dz=fake(6))),
    (prompt, dict(y=fake(2))), (prompt, dict(x=fake(20))), (prompt, dict(y=fake(21))), (step, dict(y=fake(20))),
    (step, dict(slots=fake(20))), (step, dict(ag=fake(20, 32)))])
def test_overlaps(lib, call, kw):  # noqa: F811
    assert call(lib, **kw) == INVALID and "overlap" in err(lib)


@pytest.mark.parametrize("call", [prompt, step])
@pytest.mark.parametrize("name", ["x", "a_gate", "x_gate", "z", "y"])
def test_row_strides(lib, call, name):  # noqa: F811
    assert call(lib, st=ssm.GatedStrides(**{name: 15})) == INVALID and "row stride" in err(lib)
    assert call(lib, st=ssm.GatedStrides(**{name: -4})) == INVALID
    assert call(lib, st=ssm.GatedStrides(**{name: 1 << 62})) == INVALID
    if call is prompt:
        assert call(lib, st=ssm.GatedStrides(**{name: 1 << 23})) == UNSUPPORTED


@pytest.mark.parametrize("name", ["x", "a_gate", "x_gate", "z", "y"])
def test_one_row_has_no_stride(lib, name):  # noqa: F811
    """Whatever the distance to a row that is not there, a prompt of one row gets past the strides (here to the
    pointers)."""
    for n in (1 << 23, 1 << 40):
        st = ssm.GatedStrides(**{name: n})
        assert prompt(lib, seqs=packed(total=1, sequences=1), st=st, param=None) == INVALID and "NULL" in err(lib)
        assert prompt(lib, seqs=packed(total=2, sequences=1), st=st, param=None) == UNSUPPORTED


@pytest.mark.parametrize("call", [prompt, step])
@pytest.mark.parametrize("kw,status", [(dict(reserved=1), INVALID), (dict(slots=-1), INVALID), (dict(slots=1 << 31), INVALID),
                                       (dict(slot_stride=5), INVALID), (dict(data=None), INVALID), (dict(dtype=7), UNSUPPORTED)])
def test_bad_caches(lib, call, kw, status):  # noqa: F811
    assert call(lib, c=cache(**kw)) == status


def test_nothing_to_do(lib):  # noqa: F811
    none = dict(x=None, ag=None, xg=None, param=None, y=None)
    assert fwd(lib, batch=0, **none) == OK and fwd(lib, dim=0, **none) == OK and fwd(lib, seqlen=0, last=None, **none) == OK
    assert bwd(lib, dim=0, dparam=None) == OK
    assert prompt(lib, seqs=packed(total=0), **none) == OK and prompt(lib, seqs=packed(sequences=0), **none) == OK
    assert step(lib, batch=0, **none) == OK and step(lib, c=cache(slots=0, data=None), **none) == OK


def test_workspace_sizes(lib):  # noqa: F811
    def need(batch, seqlen, dim, backward=0, dtype=BF16):
        n = ctypes.c_int64(-1)
        assert lib.ssm_gated_scan_workspace(batch, seqlen, dim, dtype, backward, ctypes.byref(n)) == OK
        return n.value
    assert need(1, 64, 100) == 0 and need(0, 5, 100) == 0 and need(1, 64, 0) == 0
    assert need(1, 4000, 100) > 0 and need(1, 64, 100, 1) == 3 * 100 * 4
    assert need(4, 1000, 100) >= need(1, 4000, 100)  # sequences with tiles of their own
    assert lib.ssm_gated_scan_workspace(-1, 5, 5, F32, 0, ctypes.byref(ctypes.c_int64())) == INVALID
    assert lib.ssm_gated_scan_workspace(1, 5, 5, F32, 0, None) == INVALID
    assert lib.ssm_gated_scan_workspace(1, 5, 5, 3, 0, ctypes.byref(ctypes.c_int64())) == UNSUPPORTED


# ---- the binding ---------------------------------------------------------------------------------------


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def batch_args(**kw):
    return dict(dict(x=t(2, 6, 8), a_gate=t(2, 6, 8), x_gate=t(2, 6, 8), a_param=t(8)), **kw)


def row_args(**kw):
    return dict(dict(x=t(6, 8), a_gate=t(6, 8), x_gate=t(6, 8), a_param=t(8)), **kw)


BATCH = [("x", t(6, 8), ValueError), ("a_gate", t(2, 6, 7), ValueError), ("x_gate", t(2, 6, 8, dtype=torch.bfloat16), TypeError),
         ("a_param", t(8, dtype=torch.bfloat16), TypeError), ("a_param", t(9), ValueError), ("a_bias", t(1, 8), ValueError),
         ("x_bias", t(7), ValueError), ("z", t(2, 6, 9), ValueError), ("x", t(2, 8, 6).transpose(1, 2), ValueError),
         ("x", t(2, 6, 8, dtype=torch.float16), TypeError), ("initial_state", t(2, 9), ValueError),
         ("initial_state", t(2, 8, dtype=torch.bfloat16), TypeError), ("workspace", t(8), TypeError)]


@pytest.mark.parametrize("name,value,exc", BATCH + [("y", t(2, 6, 7), ValueError), ("last_state", t(3, 8), ValueError)])
def test_forward_binding(name, value, exc):
    for f in (ssm.ssm_gated_scan_fwd, ssm.ssm_gated_scan_fwd_ckpt):
        with pytest.raises(exc):
            f(**batch_args(**{name: value}))


@pytest.mark.parametrize("name,value,exc", BATCH + [("dy", t(2, 6, 7), ValueError), ("checkpoints", t(1, 8), ValueError),
                                                    ("dlast_state", t(2, 7), ValueError), ("checkpoints", None, ValueError)])
def test_backward_binding(name, value, exc):
    kw = batch_args(dy=t(2, 6, 8), checkpoints=t(0, 8))
    with pytest.raises(exc):
        ssm.ssm_gated_scan_bwd_ckpt(**dict(kw, **{name: value}))


@pytest.mark.parametrize("name,value,exc", [
    ("x", t(2, 6, 8), ValueError), ("a_gate", t(6, 7), ValueError), ("x_gate", None, ValueError), ("a_param", t(9), ValueError),
    ("cu_seqlens", t(3), TypeError), ("cu_seqlens", None, ValueError), ("z", t(6, 8).to(torch.bfloat16), TypeError),
    ("cache", t(4, 8, 1), ValueError), ("cache", t(4, 8, dtype=torch.float16), TypeError), ("cache", t(1, 8), ValueError),
    ("cache_slots", t(2, dtype=torch.int32), ValueError), ("has_initial", t(2, dtype=torch.bool), ValueError),
    ("x", t(8, 6).T, ValueError), ("y", t(1, 8).expand(6, 8), ValueError), ("workspace", t(8), TypeError)])
def test_packed_binding(name, value, exc):
    with pytest.raises(exc):
        ssm.ssm_gated_scan_packed_fwd(**row_args(**dict(dict(cu_seqlens=t(3, dtype=torch.int32)), **{name: value})))


@pytest.mark.parametrize("name,value,exc", [("cache", None, ValueError), ("cache", t(4, 9), ValueError), ("cache", t(3, 8), ValueError),
                                            ("cache_slots", t(6, dtype=torch.int64), TypeError), ("x_bias", t(9), ValueError),
                                            ("x", None, ValueError), ("y", t(6, 9), ValueError)])
def test_step_binding(name, value, exc):
    with pytest.raises(exc):
        ssm.ssm_gated_update_cache(**row_args(**dict(dict(cache=t(6, 8), cache_slots=None), **{name: value})))


def test_host_tensors_are_refused():
    for call in (lambda: ssm.ssm_gated_scan_fwd(**batch_args()), lambda: ssm.ssm_gated_update_cache(t(6, 8), None, **row_args()),
                 lambda: ssm.ssm_gated_scan_bwd_ckpt(**batch_args(dy=t(2, 6, 8), checkpoints=t(0, 8))),
                 lambda: ssm.ssm_gated_scan_packed_fwd(**row_args(cu_seqlens=t(3, dtype=torch.int32)))):
        with pytest.raises(ValueError, match="expected a GPU"):
            call()


def test_checkpoint_shapes():
    assert ssm.gated_checkpoint_shape(1, 2000, 7) == (31, 7) and ssm.gated_checkpoint_shape(3, 300, 7) == (12, 7)
    assert ssm.gated_checkpoint_shape(3, 200, 7) == (9, 7) and ssm.gated_checkpoint_shape(2, 5, 7) == (0, 7)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int8])
def test_no_workspace_for_types_that_the_calls_refuse(dtype):
    for backward in (False, True):
        with pytest.raises(TypeError, match="float32 or bfloat16"):
            ssm.ssm_gated_scan_workspace(2, 500, 64, dtype, backward)
