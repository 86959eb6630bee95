"""The weights that a cache's slices point at, on the host (hla_cache_slice launches nothing)."""
import gc
import weakref

import pytest
import torch

from tests.test_abi_serving import fake_cache


@pytest.fixture(scope="module")
def hla():
    from gated_delta_rule_transitions_b200 import _hla
    from gated_delta_rule_transitions_b200 import build as b
    b.build()
    return _hla


def tracked(hla, mass):
    c = hla.make_config(2, 2, 1, 64, 128, "bf16")
    cache = hla.Cache.__new__(hla.Cache)
    cache.struct, cache.cfg, cache.max_chunks, cache.mem = fake_cache(hla, c, 4, mass=False), c, 4, None
    cache.buffers, cache.mass = {}, mass
    cache.struct.mass = mass.data_ptr()
    return cache


def test_a_slice_keeps_the_weights_it_points_at(hla):
    """Tracking anew takes other memory; a slice made before still writes to the first."""
    cache = tracked(hla, torch.zeros(2, 2, 4))
    first, sub = weakref.ref(cache.mass), cache.slice(1, 1)
    assert sub.struct.mass == cache.mass.data_ptr() + 2 * 4 * 4
    cache.mass = torch.ones(2, 2, 4)
    cache.struct.mass = cache.mass.data_ptr()
    gc.collect()
    assert first() is not None
    del sub
    gc.collect()
    assert first() is None


def test_view_of_the_weights(hla):
    """The weights lie in memory of their own, not in the cache's block; tracked anew, not in the
    buffer that a cache over given tensors started with either."""
    cache = tracked(hla, torch.arange(16.0).view(2, 2, 4))
    cache.buffers["mass"] = torch.zeros(2, 2, 4)
    assert torch.equal(cache.view("mass", (2, 2, 4), torch.float32), cache.mass)
    cache.mem = torch.zeros(64, dtype=torch.uint8)
    assert torch.equal(cache.view("mass", (16,), torch.float32), torch.arange(16.0))


def test_tracking_stops(hla, monkeypatch):
    """untrack_mass: the C call with NULL; nothing is launched, the weights are let go."""
    cache = tracked(hla, torch.zeros(2, 2, 4))
    monkeypatch.setattr(hla.Cache, "device_index", 0)
    monkeypatch.setattr(hla, "_raw_stream", lambda d: 0)
    monkeypatch.setattr(hla, "_current_device", lambda: 0)
    cache.untrack_mass()
    assert cache.struct.mass is None and cache.mass is None
    assert cache.slice(0, 1).struct.mass is None
