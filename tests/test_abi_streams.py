"""Memory that the binding takes for a call comes from the call's own stream (the allocator hands
memory out in the order of the stream it is asked on: taken from another one, it may still be in
use there, or be handed on while the call's kernels run).  No GPU: library and allocator are fakes."""
import contextlib
import types

import pytest
import torch


class Stream:
    cuda_stream, device = 0x5500, torch.device("cuda", 0)


class Memory:
    """A tensor as far as the binding looks at one."""

    dtype, shape = torch.uint8, (1 << 30,)

    def __init__(self, stream):
        self.stream, self.recorded = stream, []

    def numel(self):
        return 1 << 30

    def element_size(self):
        return 1

    def data_ptr(self):
        return 0x100000

    def get_device(self):
        return 0

    def record_stream(self, s):
        self.recorded.append(s)


@pytest.fixture
def hla(monkeypatch):
    from gated_delta_rule_transitions_b200 import _hla
    from gated_delta_rule_transitions_b200 import build as b
    b.build()
    current, taken, calls = [], [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def empty(*a, **k):
        taken.append(Memory(current[-1] if current else None))
        return taken[-1]

    real = _hla.lib()
    sizes = {"hla_cache_bytes", "hla_prefill_workspace_bytes", "hla_decode_workspace_bytes", "gdn_workspace_bytes"}

    class Library:
        def __getattr__(self, name):
            return getattr(real, name) if name in sizes else lambda *a: calls.append((name, a[-1])) or 0

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "current")
    monkeypatch.setattr(_hla, "_current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(_hla, "lib", Library)
    monkeypatch.setattr(_hla, "_ptr", lambda t: None)
    monkeypatch.setattr(_hla, "_arg", lambda t, *a: None if t is None else t.data_ptr())
    monkeypatch.setattr(_hla, "_device", lambda *a: 0)
    return types.SimpleNamespace(m=_hla, taken=taken, calls=calls)


def test_transient_workspaces(hla):
    x, s = types.SimpleNamespace(device="cuda:0", shape=(64,), data_ptr=lambda: 0x100000), Stream()
    cfg = hla.m.make_config(1, 1, 128, 64, 128, "bf16", cache_format="int8")
    cache = types.SimpleNamespace(struct=hla.m.HlaCache(), max_chunks=4)
    hla.m.hla_prefill(cfg, x, x, x, x, x, x, stream=s)
    hla.m.hla_decode_step(cfg, cache, x, x, x, x, x, x, stream=s)
    hla.m.gdn_forward(hla.m.make_gdn_config(1, 1, 128, "bf16"), x, x, x, x, x, x, x, stream=s)
    assert [t.stream for t in hla.taken] == [s] * 3
    assert [getattr(c, "value", c) for _, c in hla.calls] == [s.cuda_stream] * 3


def test_kept_memory(hla):
    """A cache's memory and its weights are cleared on the call's stream: taken from it, and not
    given to another call while the stream that was current still uses them."""
    s = Stream()
    cache = hla.m.Cache(hla.m.make_config(1, 1, 1, 64, 128, "bf16"), 4, stream=s)
    mass = cache.track_mass(stream=s)
    assert hla.taken == [cache.mem, mass]
    for t in hla.taken:
        assert t.stream is s and t.recorded == ["current"]
    assert [getattr(c, "value", c) for _, c in hla.calls] == [s.cuda_stream] * 2


def test_calls_run_on_their_tensors_device(hla, monkeypatch):
    """Tensors on another device than the current one: the call runs there, on that device's
    current stream; a stream of a third device is refused."""
    now = [0]

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d
        yield
        now[0] = before

    ran = []
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(hla.m, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=100 + now[0]))
    monkeypatch.setattr(hla.m, "_raw_stream", lambda d: 100 + d)
    monkeypatch.setattr(hla.m, "_device", lambda *a: 1)
    real = hla.m.lib()

    class Library:
        def __getattr__(self, name):
            if "bytes" in name:
                return getattr(real, name)
            return lambda *a: ran.append((name, now[0], getattr(a[-1], "value", a[-1]))) or 0

    monkeypatch.setattr(hla.m, "lib", Library)
    x, ws = types.SimpleNamespace(device="cuda:1", shape=(64,), data_ptr=lambda: 0x100000), Memory(None)
    cfg = hla.m.make_config(1, 1, 128, 64, 128, "bf16")
    cache = types.SimpleNamespace(struct=hla.m.HlaCache(), max_chunks=4)
    hla.m.hla_prefill(cfg, x, x, x, x, x, x, workspace=ws)
    hla.m.hla_decode_step(cfg, cache, x, x, x, x, x, x, workspace=ws)
    hla.m.hla_decode_step_static(cfg, cache, x, x, x, x, x, x)
    hla.m.hla_routing(cfg, x, x, x, x)
    hla.m.hla_gate_support(cfg, x, x)
    hla.m.gdn_chunk_transitions(cfg, x, x, x, x, x, x)
    assert len(ran) == 6 and all(r[1:] == (1, 101) for r in ran), ran
    with pytest.raises(ValueError, match="stream is on"):
        hla.m.hla_decode_step(cfg, cache, x, x, x, x, x, x, workspace=ws, stream=Stream())
    monkeypatch.setattr(Memory, "get_device", lambda self: 1)
    hla.m.Cache(cfg, 4, device="cuda:1")
    assert ran[-1] == ("hla_cache_init", 1, 101)


def test_transposed_tensors_are_refused(monkeypatch):
    """As many elements and as many dimensions, in another order: not the tensor that was asked for.
    One of fewer or more dimensions is taken by its elements."""
    from gated_delta_rule_transitions_b200 import _hla

    class OnDevice(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0

    make = lambda *s: torch.zeros(*s).as_subclass(OnDevice)
    for shape in ((6, 4, 8), (192,), (24, 8), (6, 4, 8, 1)):
        t = make(*shape)
        assert _hla._arg(t, "x", torch.float32, (6, 4, 8), 0) == t.data_ptr()
    for shape in ((4, 6, 8), (8, 4, 6), (1, 24, 8)):
        with pytest.raises(ValueError, match="x: expected"):
            _hla._arg(make(*shape), "x", torch.float32, (6, 4, 8), 0)
    for shape in ((6, 4, 9), (191,), (0,)):
        with pytest.raises(ValueError, match="x: expected"):
            _hla._arg(make(*shape), "x", torch.float32, (6, 4, 8), 0)
