"""Argument checks of the carried-state gated delta rule, the 8-bit cache and the eviction
that need no GPU: sizes by the stated arithmetic, refusals on the host before any launch."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(0x100000)


@pytest.fixture(scope="module")
def hla():
    from gated_delta_rule_transitions_b200 import _hla
    from gated_delta_rule_transitions_b200 import build as b
    b.build()
    return _hla


def gdn(hla, **kw):
    base = dict(n_seq=2, H=4, d=128, dtype="bf16")
    base.update(kw)
    return hla.make_gdn_config(**base)


@pytest.mark.parametrize("kw,status,word", [
    (dict(n_seq=0), 1, "positive"), (dict(H=0), 1, "positive"), (dict(H=6, Hk=4), 1, "divide"),
    (dict(d=96), 2, "head dim"), (dict(n_slots=0), 1, "positive"), (dict(decay=2), 1, "decay_mode"),
    (dict(n_slots=1), 1, "no slots"), (dict(n_seq=1 << 20, H=1 << 10), 2, "too many"),
])
def test_gdn_config_refused(hla, kw, status, word):
    c = gdn(hla, **kw)
    L = hla.lib()
    assert L.gdn_step(ctypes.byref(c), P, P, P, P, P, None, P, P, None) == status
    assert word in hla.last_error()
    assert L.gdn_forward(ctypes.byref(c), P, P, P, P, P, P, 64, None, P, P, P, P, 1 << 40, None) == status
    assert word in hla.last_error()


def test_gdn_dk_dv_must_match(hla):
    c = gdn(hla)
    c.dv = 64
    assert hla.lib().gdn_step(ctypes.byref(c), P, P, P, P, P, None, P, P, None) == hla.HLA_ERR_UNSUPPORTED
    assert hla.gdn_workspace_bytes(c, 64) == 0


def test_gdn_pointers_refused(hla):
    c, L, bad = gdn(hla), hla.lib(), ctypes.c_void_p(0x100004)
    step = lambda *a: L.gdn_step(ctypes.byref(c), *a, None)
    for i, name in enumerate(("q", "k", "v", "alpha", "beta")):
        args = [P, P, P, P, P, None, P, P]
        args[i] = None
        assert step(*args) == hla.HLA_ERR_INVALID_ARG and f"{name} is NULL" in hla.last_error()
        args[i] = bad if i < 3 else ctypes.c_void_p(0x100002)  # alpha and beta: single values
        assert step(*args) == hla.HLA_ERR_INVALID_ARG and "aligned" in hla.last_error()
    assert step(P, P, P, P, P, None, None, P) == hla.HLA_ERR_INVALID_ARG and "state" in hla.last_error()
    assert step(P, P, P, P, P, ctypes.c_void_p(0x100002), P, P) == hla.HLA_ERR_INVALID_ARG
    fwd = lambda *a: L.gdn_forward(ctypes.byref(c), P, P, P, P, P, *a, None)
    assert fwd(P, 0, None, P, P, P, P, 1 << 40) == hla.HLA_ERR_INVALID_ARG and "T must" in hla.last_error()
    assert fwd(None, 64, None, P, P, P, P, 1 << 40) == hla.HLA_ERR_INVALID_ARG and "cu_seqlens" in hla.last_error()
    assert fwd(P, 64, None, bad, P, P, P, 1 << 40) == hla.HLA_ERR_INVALID_ARG and "state_in" in hla.last_error()
    assert fwd(P, 64, None, P, P, P, None, 1 << 40) == hla.HLA_ERR_INVALID_ARG and "workspace" in hla.last_error()
    need = hla.gdn_workspace_bytes(c, 64)
    assert need > 0
    assert fwd(P, 64, None, P, P, P, P, need - 1) == hla.HLA_ERR_WORKSPACE


def test_int8_cache_sizes_and_slices(hla):
    """An 8-bit cache holds two d x d code matrices and four float32 scales per closed chunk."""
    d = 128
    c = hla.make_config(3, 2, 1, 64, d, "bf16", cache_format="int8")
    per = hla.cache_bytes(c, 129) - hla.cache_bytes(c, 1)
    assert per == 3 * 2 * 128 * (2 * d * d + 16 + 4 * d)
    s = hla.HlaCache()
    s.B, s.H, s.C, s.d, s.dtype, s.max_chunks, s.format = 3, 2, 64, d, 1, 5, 2
    for i, f in enumerate(("A", "Bm", "df", "rk", "buf_k", "buf_v", "buf_qr", "buf_kr", "buf_alpha", "buf_beta",
                           "n_chunks", "m_partial", "mass")):
        setattr(s, f, (i + 1) << 32)
    out = hla.HlaCache()
    assert hla.lib().hla_cache_slice(ctypes.byref(s), 1, 2, ctypes.byref(out)) == hla.HLA_OK
    assert out.A == (1 << 32) + 2 * 5 * d * d and out.Bm == (2 << 32) + 2 * 5 * d * d
    assert out.df == (3 << 32) + 2 * 5 * 16 and out.mass == (13 << 32) + 2 * 5 * 4
    # the decode workspace also holds a closing chunk's two transitions
    dense = hla.make_config(3, 2, 1, 64, d, "bf16")
    assert hla.decode_workspace_bytes(c, 5) - hla.decode_workspace_bytes(dense, 5) == 2 * 3 * 2 * d * d * 2


def fake_cache(hla, c, mc, base=1 << 32, mass=True):
    s = hla.HlaCache()
    s.B, s.H, s.C, s.d, s.dtype, s.max_chunks, s.format = c.B, c.H, c.C, c.dk, c.dtype, mc, c.cache_format
    s.pool_window, s.decay_mode = c.pool_window, c.decay_mode
    for i, f in enumerate(("A", "Bm", "df", "rk", "buf_k", "buf_v", "buf_qr", "buf_kr", "buf_alpha", "buf_beta",
                           "n_chunks", "m_partial")):
        setattr(s, f, base + (i << 24))
    if mass:
        s.mass = base + (20 << 24)
    return s


def test_int8_cache_needs_its_scales(hla):
    c = hla.make_config(1, 1, 1, 64, 128, "bf16", cache_format="int8")
    s = fake_cache(hla, c, 4)
    s.df = None
    st = hla.lib().hla_decode_step(ctypes.byref(c), ctypes.byref(s), P, P, P, P, P, None, None, P, P, 1 << 30, None)
    assert st == hla.HLA_ERR_INVALID_ARG and "scales" in hla.last_error()


def test_evict_refusals(hla):
    c = hla.make_config(2, 2, 1, 64, 128, "bf16")
    ev = lambda a, b, keep, recent, kept=P: hla.lib().hla_cache_evict(ctypes.byref(c), ctypes.byref(a),
                                                                     ctypes.byref(b), keep, recent, kept, None)
    src = fake_cache(hla, c, 8)
    dst = fake_cache(hla, c, 4, base=2 << 32)
    assert ev(fake_cache(hla, c, 8, mass=False), dst, 4, 0) == hla.HLA_ERR_INVALID_ARG and "mass" in hla.last_error()
    for keep, recent, word in ((0, 0, "keep"), (5, 0, "keep"), (-1, 0, "keep"), (3, 4, "recent"), (3, -1, "recent")):
        assert ev(src, dst, keep, recent) == hla.HLA_ERR_INVALID_ARG and word in hla.last_error()
    assert ev(src, dst, 4, 0, None) == hla.HLA_ERR_INVALID_ARG and "kept_out" in hla.last_error()
    # some arrays shared, some not; or shared with another length
    half = fake_cache(hla, c, 8, base=2 << 32)
    half.rk = src.rk
    assert ev(src, half, 4, 0) == hla.HLA_ERR_INVALID_ARG and "shares" in hla.last_error()
    assert ev(src, fake_cache(hla, c, 4), 4, 0) == hla.HLA_ERR_INVALID_ARG and "shares" in hla.last_error()
    other = hla.make_config(2, 2, 1, 64, 128, "bf16", cache_format="int8")
    assert ev(src, fake_cache(hla, other, 4, base=2 << 32), 4, 0) == hla.HLA_ERR_INVALID_ARG


def test_tracked_prefill_needs_gates(hla):
    c = hla.make_config(1, 1, 256, 64, 128, "bf16")
    s = fake_cache(hla, c, 8)
    st = hla.lib().hla_prefill(ctypes.byref(c), P, P, P, P, P, None, None, None, P, None, None, None,
                               ctypes.byref(s), P, 1 << 40, None)
    assert st == hla.HLA_ERR_INVALID_ARG and "gates_out" in hla.last_error()


def test_gate_mass_and_track_refusals(hla):
    c = hla.make_config(1, 1, 256, 64, 128, "bf16")
    L = hla.lib()
    assert L.hla_gate_mass(ctypes.byref(c), None, P, None) == hla.HLA_ERR_INVALID_ARG
    assert L.hla_gate_mass(ctypes.byref(c), P, None, None) == hla.HLA_ERR_INVALID_ARG
    s = fake_cache(hla, c, 8)
    assert L.hla_cache_track_mass(ctypes.byref(s), ctypes.c_void_p(0x1001), None) == hla.HLA_ERR_INVALID_ARG
    assert L.hla_cache_track_mass(ctypes.byref(s), None, None) == hla.HLA_OK and not s.mass
    assert L.hla_cache_track_mass(ctypes.byref(hla.HlaCache()), P, None) == hla.HLA_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors_and_foreign_buffers(hla):
    c = gdn(hla, n_seq=1, H=1, d=64, dtype="f32")
    x, a, S = torch.zeros(1, 1, 64), torch.zeros(1, 1), torch.zeros(1, 1, 64, 64)
    with pytest.raises(ValueError, match="CUDA"):
        hla.gdn_step(c, x, x, x, a, a, S, x)
    cc = hla.make_config(1, 1, 1, 64, 64, "f32", cache_format="int8")
    with pytest.raises(ValueError, match="expected the buffers"):
        hla.Cache.from_tensors(cc, 2, A=S)
    with pytest.raises(hla.HlaError):
        hla.Cache.from_tensors(cc, 0)
