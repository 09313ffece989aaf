"""The serving entry points on the host: every call here is refused (or has nothing to do) before any
HIP call, so no GPU is needed and the pointers are never dereferenced; and the binding's own checks."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_61_amd as ssm
import serving_ref as R

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
F32, BF16 = 0, 1
P, GAP = 0x7F0000000000, 1 << 32


def fake(i, off=0):
    return P + i * GAP + off


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_61_amd import build as b
    if b.is_stale():
        b.build()
    return ssm.load_library()


def err(lib):
    return lib.ssm_last_error().decode()


def cache(**kw):
    f = dict(data=fake(20), slots=4, slot_stride=0, dtype=F32, reserved=0)
    f.update(kw)
    return ssm.Cache(*[f[k] for k in ("data", "slots", "slot_stride", "dtype", "reserved")])


def packed(**kw):
    f = dict(total=10, sequences=3, max_seqlen=0, cu_seqlens=fake(21), cache_slots=fake(22), has_initial=fake(23))
    f.update(kw)
    return ssm.Packed(*[f[k] for k in ("total", "sequences", "max_seqlen", "cu_seqlens", "cache_slots", "has_initial")])


def conv_packed(lib, seqs=None, dim=16, width=4, dtype=F32, x=fake(0), w=fake(1), b=fake(2), y=fake(3), c="own", st=None):
    c = cache(dtype=dtype) if c == "own" else c
    return lib.ssm_causal_conv1d_packed_fwd(packed() if seqs is None else seqs, dim, width, dtype, x, w, b, 1, y, c, st, None)


def scan_packed(lib, seqs=None, dim=16, dstate=16, dtype=F32, x=fake(0), delta=fake(1), A=fake(2), B=fake(3), C=fake(4),
                D=fake(5), z=fake(6), bias=fake(7), y=fake(8), c="own", st=None, ws=None, nws=0):
    c = cache() if c == "own" else c
    return lib.ssm_scan_packed_fwd(packed() if seqs is None else seqs, dim, dstate, dtype, x, delta, A, B, C, D, z, bias, 1,
                                   y, c, st, ws, nws, None)


def conv_step(lib, batch=2, dim=16, width=4, dtype=F32, c="own", slots=fake(22), x=fake(0), w=fake(1), b=fake(2),
              y=fake(3), st=None):
    c = cache(dtype=dtype) if c == "own" else c
    return lib.ssm_causal_conv1d_update_cache(batch, dim, width, dtype, c, slots, x, w, b, 1, y, st, None)


def scan_step(lib, batch=2, dim=16, dstate=16, dtype=F32, c="own", slots=fake(22), x=fake(0), delta=fake(1), A=fake(2),
              B=fake(3), C=fake(4), D=fake(5), z=fake(6), bias=fake(7), y=fake(8), st=None):
    c = cache() if c == "own" else c
    return lib.ssm_state_update_cache(batch, dim, dstate, dtype, c, slots, x, delta, A, B, C, D, z, bias, 1, y, st, None)


def ssd_step(lib, batch=2, heads=4, headdim=8, dstate=64, groups=2, dtype=BF16, c="own", slots=fake(22), x=fake(0),
             dt=fake(1), A=fake(2), B=fake(3), C=fake(4), D=fake(5), z=fake(6), bias=fake(7), y=fake(8), st=None):
    c = cache() if c == "own" else c
    return lib.ssm_ssd_state_update_cache(batch, heads, headdim, dstate, groups, dtype, c, slots, x, dt, A, B, C, D, z,
                                          bias, 1, y, st, None)


def store(lib, count=2, rows=8, dstate=16, c="own", slots=fake(22), stored=3, codes=fake(0), scales=fake(1), where=fake(23)):
    return lib.ssm_cache_store_q8(count, rows, dstate, cache() if c == "own" else c, slots, stored, codes, scales, where,
                                  None)


def load(lib, count=2, rows=8, dstate=16, c="own", slots=fake(22), stored=3, codes=fake(0), scales=fake(1), where=fake(23)):
    return lib.ssm_cache_load_q8(count, rows, dstate, stored, codes, scales, where, cache() if c == "own" else c, slots,
                                 None)


CALLS = [conv_packed, scan_packed, conv_step, scan_step, ssd_step]


@pytest.mark.parametrize("call", [conv_packed, scan_packed])
@pytest.mark.parametrize("kw", [dict(total=-1), dict(sequences=-1), dict(max_seqlen=-1), dict(total=1 << 31),
                                dict(sequences=1 << 31), dict(max_seqlen=1 << 31)])
def test_packed_sizes(lib, call, kw):
    assert call(lib, seqs=packed(**kw)) == INVALID and "2^31" in err(lib)


@pytest.mark.parametrize("call,kw", [(conv_packed, dict(dim=-1)), (scan_packed, dict(dim=-1)), (conv_step, dict(batch=-1)),
                                     (scan_step, dict(batch=-1)), (scan_step, dict(dim=-2)), (ssd_step, dict(heads=0)),
                                     (ssd_step, dict(batch=1 << 31)), (scan_packed, dict(dstate=-16)),
                                     (store, dict(count=-1)), (load, dict(stored=-1)),
                                     (store, dict(rows=1 << 62, dstate=1))])
def test_bad_sizes(lib, call, kw):
    assert call(lib, **kw) == INVALID


@pytest.mark.parametrize("call,kw", [(conv_packed, dict(width=5)), (conv_packed, dict(width=0)), (conv_step, dict(width=5)),
                                     (scan_packed, dict(dstate=3)), (scan_packed, dict(dstate=128)),
                                     (scan_step, dict(dstate=0)), (scan_step, dict(dstate=24)), (ssd_step, dict(dstate=8)),
                                     (ssd_step, dict(dstate=512)), (store, dict(dstate=48)), (load, dict(dstate=512)),
                                     (conv_packed, dict(dtype=2, c=None)), (scan_packed, dict(dtype=5)),
                                     (scan_step, dict(dtype=-1)), (ssd_step, dict(dtype=9)),
                                     (scan_step, dict(c=cache(dtype=7))), (store, dict(c=cache(dtype=7)))])
def test_unsupported(lib, call, kw):
    assert call(lib, **kw) == UNSUPPORTED


@pytest.mark.parametrize("call", CALLS + [store, load])
@pytest.mark.parametrize("kw,status", [(dict(reserved=1), INVALID), (dict(slots=-1), INVALID), (dict(slots=1 << 31), INVALID),
                                       (dict(slot_stride=5), INVALID), (dict(data=None), INVALID),
                                       (dict(data=fake(20, 1)), MISALIGNED), (dict(slot_stride=1 << 62), INVALID)])
def test_bad_caches(lib, call, kw, status):
    d = BF16 if call is ssd_step else F32
    assert call(lib, c=cache(dtype=F32 if call is not conv_packed and call is not conv_step else d, **kw)) == status


def test_the_window_has_the_inputs_type(lib):
    assert conv_packed(lib, dtype=BF16, c=cache(dtype=F32)) == INVALID and "dtype" in err(lib)
    assert conv_step(lib, dtype=F32, c=cache(dtype=BF16)) == INVALID


@pytest.mark.parametrize("call,name", [(c, n) for c, ns in (
    (conv_packed, ("x", "w", "y")), (scan_packed, ("x", "delta", "A", "B", "C", "y")), (conv_step, ("x", "w", "y")),
    (scan_step, ("x", "delta", "A", "B", "C", "y")), (ssd_step, ("x", "dt", "A", "B", "C", "y")),
    (store, ("codes", "scales")), (load, ("codes", "scales"))) for n in ns])
def test_null_required(lib, call, name):
    assert call(lib, **{name: None}) == INVALID and "NULL" in err(lib)


def test_null_structures(lib):
    assert lib.ssm_scan_packed_fwd(None, 16, 16, F32, *[fake(i) for i in range(8)], 1, fake(8), None, None, None, 0,
                                   None) == INVALID
    assert lib.ssm_causal_conv1d_packed_fwd(None, 16, 4, F32, fake(0), fake(1), None, 1, fake(2), None, None, None) == INVALID
    for call in (conv_step, scan_step, ssd_step, store, load):
        assert call(lib, c=None) == INVALID and "cache" in err(lib)
    assert scan_packed(lib, seqs=packed(cu_seqlens=None)) == INVALID
    assert lib.ssm_scan_packed_workspace(packed(), 16, 16, F32, None) == INVALID


@pytest.mark.parametrize("call,kw", [(conv_packed, dict(x=fake(0, 2))), (conv_packed, dict(w=fake(1, 2))),
                                     (scan_packed, dict(y=fake(8, 1), dtype=BF16)), (scan_packed, dict(A=fake(2, 2))),
                                     (scan_step, dict(z=fake(6, 2))), (scan_step, dict(slots=fake(22, 2))),
                                     (ssd_step, dict(B=fake(3, 1))), (ssd_step, dict(bias=fake(7, 2))),
                                     (conv_step, dict(b=fake(2, 1))), (store, dict(scales=fake(1, 2))),
                                     (load, dict(where=fake(23, 1))),
                                     (scan_packed, dict(seqs=packed(cu_seqlens=fake(21, 2))))])
def test_misaligned(lib, call, kw):
    assert call(lib, **kw) == MISALIGNED


@pytest.mark.parametrize("call,name", [(conv_packed, "x"), (scan_packed, "delta"), (scan_step, "B"), (ssd_step, "z"),
                                       (scan_packed, "y")])
def test_row_strides(lib, call, name):
    key = {"y": "y"}.get(name, name)
    width = {"B": 16, "z": 32}.get(name, 16)
    assert call(lib, st=ssm.RowStrides(**{key: width - 1})) == INVALID and "row stride" in err(lib)
    assert call(lib, st=ssm.RowStrides(**{key: -4})) == INVALID
    assert call(lib, st=ssm.RowStrides(**{key: 1 << 62})) == INVALID


@pytest.mark.parametrize("call,kw", [
    (conv_packed, dict(y=fake(0, 64))), (conv_packed, dict(y=fake(20))), (conv_packed, dict(x=fake(20))),
    (scan_packed, dict(y=fake(1))), (scan_packed, dict(y=fake(20, 64))), (scan_packed, dict(A=fake(20))),
    (scan_packed, dict(y=fake(21, 0))), (scan_step, dict(y=fake(0))), (scan_step, dict(B=fake(20))),
    (scan_step, dict(slots=fake(20))), (ssd_step, dict(y=fake(6))), (ssd_step, dict(y=fake(20))),
    (conv_step, dict(y=fake(0))), (store, dict(codes=fake(20))), (store, dict(scales=fake(0, 4))),
    (store, dict(where=fake(1))), (load, dict(codes=fake(20))), (load, dict(slots=fake(20)))])
def test_overlaps(lib, call, kw):
    assert call(lib, **kw) == INVALID and "overlap" in err(lib)


def test_a_strided_output_beside_its_input_is_judged_by_its_span(lib):
    # two columns of one tensor: their spans interleave
    st = ssm.RowStrides(x=32, y=32)
    assert conv_packed(lib, x=fake(0), y=fake(0, 64), st=st) == INVALID


def test_nothing_to_do(lib):
    none = dict(x=None, y=None)
    assert conv_packed(lib, seqs=packed(total=0), **none) == OK
    assert conv_packed(lib, seqs=packed(sequences=0)) == OK
    assert scan_packed(lib, seqs=packed(total=0), **none) == OK
    assert scan_packed(lib, dim=0) == OK
    assert scan_step(lib, batch=0, **none) == OK
    assert conv_step(lib, dim=0) == OK
    assert ssd_step(lib, batch=0) == OK
    for call in (conv_step, scan_step, ssd_step, store, load):
        assert call(lib, c=cache(slots=0, data=None)) == OK
    assert store(lib, count=0) == OK and load(lib, stored=0) == OK


def test_heads_and_groups(lib):
    assert ssd_step(lib, heads=4, groups=3) == INVALID and "divide" in err(lib)


# ---- the binding ---------------------------------------------------------------------------------------


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def good_scan():
    return dict(x=t(6, 8), delta=t(6, 8), A=t(8, 16), B=t(6, 16), C=t(6, 16), cu_seqlens=t(3, dtype=torch.int32))


@pytest.mark.parametrize("name,value,exc", [
    ("x", t(2, 6, 8), ValueError), ("delta", t(6, 7), ValueError), ("B", t(6, 8), ValueError),
    ("C", t(6, 16, dtype=torch.bfloat16), TypeError), ("A", t(8, 16, dtype=torch.bfloat16), TypeError),
    ("cu_seqlens", None, ValueError), ("cu_seqlens", t(3), TypeError), ("cu_seqlens", t(0, dtype=torch.int32), ValueError),
    ("cu_seqlens", t(1, 3, dtype=torch.int32), ValueError), ("x", t(8, 6).T, ValueError),
    ("z", t(6, 9), ValueError), ("z", t(1, 8).expand(6, 8), ValueError), ("D", t(9), ValueError),
    ("cache", t(4, 8, 15), ValueError), ("cache", t(4, 8, 16, dtype=torch.float16), TypeError),
    ("cache", t(1, 8, 16), ValueError), ("cache_slots", t(2, dtype=torch.int32), ValueError),
    ("has_initial", t(2, dtype=torch.bool), ValueError), ("workspace", t(8), TypeError), ("y", t(6, 8).int(), TypeError),
    ("x", t(6, 8, dtype=torch.float16), TypeError)])
def test_scan_binding(name, value, exc):
    kw = good_scan()
    kw[name] = value
    with pytest.raises(exc):
        ssm.ssm_scan_packed_fwd(**kw)


def test_cache_binding():
    kw = dict(good_scan(), cache=t(4, 8, 16), cache_slots=t(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        ssm.ssm_scan_packed_fwd(**kw)
    with pytest.raises(TypeError):
        ssm.ssm_scan_packed_fwd(**dict(good_scan(), cache=t(4, 8, 16), has_initial=t(2)))
    with pytest.raises(ValueError, match="must not overlap"):
        ssm.ssm_scan_packed_fwd(**dict(good_scan(), cache=t(1, 8, 16).expand(4, 8, 16)))


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="expected a GPU"):
        ssm.ssm_scan_packed_fwd(**good_scan())
    with pytest.raises(ValueError, match="expected a GPU"):
        ssm.ssm_causal_conv1d_update_cache(t(4, 8, 3), None, t(2, 8), t(8, 4))
    with pytest.raises(ValueError, match="expected a GPU"):
        ssm.ssm_cache_store_q8(t(4, 8, 16), None, t(2, 8, 16, dtype=torch.int8), t(2, 8))


@pytest.mark.parametrize("call", [
    lambda: ssm.ssm_causal_conv1d_packed_fwd(t(6, 8), t(8, 4), t(2, dtype=torch.int32), cache=t(3, 8, 4)),
    lambda: ssm.ssm_causal_conv1d_packed_fwd(t(6, 8), t(9, 4), t(2, dtype=torch.int32)),
    lambda: ssm.ssm_causal_conv1d_update_cache(None, None, t(2, 8), t(8, 4)),
    lambda: ssm.ssm_causal_conv1d_update_cache(t(1, 8, 3), None, t(2, 8), t(8, 4)),
    lambda: ssm.ssm_state_update_cache(t(1, 8, 16), None, t(2, 8), t(2, 8), t(8, 16), t(2, 16), t(2, 16)),
    lambda: ssm.ssm_state_update_cache(t(3, 8, 16), None, t(2, 8), t(2, 9), t(8, 16), t(2, 16), t(2, 16)),
    lambda: ssm.ssm_ssd_state_update_cache(t(3, 2, 8, 16), None, t(2, 2, 8), t(2, 3), t(2), t(2, 1, 16), t(2, 1, 16)),
    lambda: ssm.ssm_ssd_state_update_cache(t(3, 2, 9, 16), None, t(2, 2, 8), t(2, 2), t(2), t(2, 1, 16), t(2, 1, 16)),
    lambda: ssm.ssm_cache_store_q8(t(4, 8), None, t(2, 8, dtype=torch.int8), t(2)),
    lambda: ssm.ssm_cache_store_q8(t(4, 8, 16), t(3, dtype=torch.int32), t(2, 8, 16, dtype=torch.int8), t(2, 8)),
    lambda: ssm.ssm_cache_load_q8(t(2, 8, 15, dtype=torch.int8), t(2, 8), None, t(4, 8, 16))])
def test_other_bindings(call):
    with pytest.raises(ValueError):
        call()


def test_the_quantising_reference_rounds_to_the_nearest():
    """The 64-bit form that the GPU's codes are compared with: within half a scale, ties to even."""
    v = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 63.49999, 0.0]], np.float32)
    q, s = R.quantise(v)
    assert s[0] == 1.0 and q[0].tolist() == [127, 0, 2, 2, 0, -2, 63, 0]
    w = np.random.default_rng(0).standard_normal((200, 16)).astype(np.float32)
    q, s = R.quantise(w)
    assert np.all(np.abs(w.astype(np.float64) - q * s.astype(np.float64)[:, None]) <= s[:, None] * (0.5 + 1e-6))


def test_the_scan_reference_against_its_closed_form():
    """A constant step and no input: the state decays as exp(t dt A); the bound stays small."""
    L, n = 40, 4
    one = torch.ones(L, 3, dtype=torch.float64)
    A = -torch.arange(1, n + 1, dtype=torch.float64).repeat(3, 1)
    h0 = torch.full((3, n), 2.0, dtype=torch.float64)
    y, e, h, eh = R.scan_steps(0 * one, 0.01 * one, A, torch.ones(L, n, dtype=torch.float64),
                               torch.ones(L, n, dtype=torch.float64), None, None, None, False, h0)
    ref = 2.0 * torch.exp(0.01 * L * A)
    assert torch.allclose(h, ref, rtol=1e-12) and torch.allclose(y[-1], ref.sum(1), rtol=1e-12)
    assert (e < 2e-4).all() and (eh < 1e-4).all()
