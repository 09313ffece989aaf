"""Refusals of the serving calls beside those of test_serving_host.py: on the host, before any HIP call."""
import pytest
import torch

import selective_state_space_61_amd as ssm
from test_serving_host import BF16, INVALID, OK, cache, conv_step, err, lib  # noqa: F401


@pytest.mark.parametrize("kw,status", [(dict(reserved=1), INVALID), (dict(slots=-1), INVALID), (dict(slots=1 << 31), INVALID),
                                       (dict(slot_stride=-5), INVALID), (dict(dtype=7), INVALID), (dict(dtype=BF16), INVALID)])
def test_a_cache_of_width_one_is_checked(lib, kw, status):  # noqa: F811
    """Its slots say which entries are padding, so it is read although it holds no windows."""
    assert conv_step(lib, width=1, c=cache(**kw)) == status


def test_no_slots_or_no_cache_of_width_one(lib):  # noqa: F811
    assert conv_step(lib, width=1, c=cache(slots=0, data=None)) == OK  # every entry is padding
    assert conv_step(lib, width=1, c=None, x=None) == INVALID and "NULL" in err(lib)
    assert conv_step(lib, width=2, c=None) == INVALID and "cache" in err(lib)


# ---- the binding ---------------------------------------------------------------------------------------


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


CU = t(2, dtype=torch.int32)
CODES = t(4, 8, 16, dtype=torch.int8)
BINDINGS = [
    (ssm.ssm_causal_conv1d_packed_fwd, dict(x=t(6, 8), weight=t(8, 4), cu_seqlens=CU)),
    (ssm.ssm_scan_packed_fwd, dict(x=t(6, 8), delta=t(6, 8), A=t(8, 16), B=t(6, 16), C=t(6, 16), cu_seqlens=CU)),
    (ssm.ssm_causal_conv1d_update_cache, dict(cache=t(4, 8, 3), cache_slots=CU, x=t(2, 8), weight=t(8, 4))),
    (ssm.ssm_state_update_cache, dict(cache=t(4, 8, 16), cache_slots=CU, x=t(2, 8), delta=t(2, 8), A=t(8, 16), B=t(2, 16),
                                      C=t(2, 16))),
    (ssm.ssm_ssd_state_update_cache, dict(cache=t(4, 2, 8, 16), cache_slots=CU, x=t(2, 2, 8), dt=t(2, 2), A=t(2), B=t(2, 1, 16),
                                          C=t(2, 1, 16))),
    (ssm.ssm_cache_store_q8, dict(cache=t(4, 8, 16), cache_slots=CU, codes=CODES, scales=t(4, 8))),
    (ssm.ssm_cache_load_q8, dict(codes=CODES, scales=t(4, 8), store_slots=CU, cache=t(4, 8, 16)))]


@pytest.mark.parametrize("call,kw,name", [(f, kw, k) for f, kw in BINDINGS for k in kw if not k.endswith("_slots")])
def test_a_missing_tensor_is_named(call, kw, name):
    with pytest.raises(ValueError, match=rf"\b{name}\b"):
        call(**dict(kw, **{name: None}))


@pytest.mark.parametrize("codes", [t(dtype=torch.int8), t(4, dtype=torch.int8), t(4, 8, 16, 1, dtype=torch.int8)])
def test_codes_of_another_rank(codes):
    with pytest.raises(ValueError, match="codes"):
        ssm.ssm_cache_store_q8(t(4, 8, 16), None, codes, t(4, 8))
