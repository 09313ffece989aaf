"""Refusals of the serving calls beside those of test_serving_host.py: on the host, before any HIP call."""
import pytest

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
