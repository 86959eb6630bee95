"""hla_cache_evict into a cache whose memory overlaps the source's without being it (host check)."""
import ctypes

import pytest

from tests.test_abi_serving import P, fake_cache


@pytest.fixture(scope="module")
def hla():
    from gated_delta_rule_transitions_b200 import _hla
    from gated_delta_rule_transitions_b200 import build as b
    b.build()
    return _hla


def part(hla, cache, b0, nb):
    out = hla.HlaCache()
    assert hla.lib().hla_cache_slice(ctypes.byref(cache), b0, nb, ctypes.byref(out)) == hla.HLA_OK
    return out


@pytest.mark.parametrize("fmt", ["dense", "int8"])
def test_overlapping_slices_are_refused(hla, fmt):
    """Sequences 0, 1 of a cache into its sequences 1, 2, either way round: sequence 1 would be read
    and written at once."""
    cache = fake_cache(hla, hla.make_config(4, 2, 1, 64, 64, "bf16", cache_format=fmt), 4)
    c = hla.make_config(2, 2, 1, 64, 64, "bf16", cache_format=fmt)
    for a, b in ((0, 1), (1, 0), (2, 1)):
        src, dst = part(hla, cache, a, 2), part(hla, cache, b, 2)
        st = hla.lib().hla_cache_evict(ctypes.byref(c), ctypes.byref(src), ctypes.byref(dst), 3, 1, P, None)
        assert st == hla.HLA_ERR_INVALID_ARG and "overlap" in hla.last_error(), (a, b, st, hla.last_error())


@pytest.mark.parametrize("field", ["A", "rk", "buf_v", "n_chunks", "mass"])
def test_one_overlapping_array_is_refused(hla, field):
    c = hla.make_config(2, 2, 1, 64, 64, "bf16")
    src, dst = fake_cache(hla, c, 8), fake_cache(hla, c, 8, base=2 << 32)
    setattr(dst, field, getattr(src, field) + (4 if field == "n_chunks" else 16))
    st = hla.lib().hla_cache_evict(ctypes.byref(c), ctypes.byref(src), ctypes.byref(dst), 3, 1, P, None)
    assert st == hla.HLA_ERR_INVALID_ARG and "overlap" in hla.last_error()
