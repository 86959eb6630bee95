"""Gate mass and eviction of cached chunks against plain references: what moves is bit for
bit what was there, who stays is decided by (weight descending, index ascending)."""
import pytest
import torch

import hla_synth as syn
from tests import _parity as P
from tests import _serving as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hla():
    import gated_delta_rule_transitions_b200 as m
    m.lib()
    return m._hla


@pytest.mark.parametrize("B,H,T,C,thr", [(1, 1, 1, 64, 0.0), (2, 3, 64, 64, 0.0), (1, 2, 65, 64, 0.05),
                                         (2, 2, 64 * 33, 64, 0.3), (1, 5, 128 * 40 + 77, 128, 0.05),
                                         (1, 3, 256 * 130 + 1, 256, 0.0), (3, 1, 64 * 97, 64, 0.99)])
def test_gate_mass(hla, B, H, T, C, thr):
    """Column sums of weighted gates: at most N terms, each lane's added in sequence, so off
    by at most (N / 16 + 24) 2^-24 of the sum (all terms are positive)."""
    N = -(-T // C)
    gen = torch.Generator().manual_seed(N)
    g = torch.sigmoid(2 * torch.randn(B, H, N, N, generator=gen) - 1)
    g[torch.triu(torch.ones(N, N, dtype=bool)).expand(B, H, N, N)] = float("nan")  # never read
    cfg = hla.make_config(B, H, T, C, 128, "bf16", skip_threshold=thr)
    out = torch.full((B, H, N), 9.0, device="cuda")
    hla.hla_gate_mass(cfg, g.cuda(), out)
    w = torch.tensor([min(C, T - i * C) for i in range(N)], dtype=torch.float64)
    x = torch.where(torch.tril(torch.ones(N, N, dtype=bool), -1), g, 0.0).double()
    if thr > 0:
        x = x * (x >= torch.tensor(thr, dtype=torch.float32).double())
    ref = (w[:, None] * x).sum(2)
    assert bool(((out.cpu().double() - ref).abs() <= (N / 16 + 24) * 2.0 ** -24 * ref).all())
    again = torch.empty_like(out)
    hla.hla_gate_mass(cfg, g.cuda(), again)
    assert torch.equal(again, out)


FIELDS = {"dense": ("A", "Bm"), "int8": ("A", "Bm", "df"), "factored": ("Kf", "Wf", "Uf", "df")}


def make_cache(hla, gen, cfg, mc, n, fmt):
    """A cache over tensors of random contents, n[b] closed chunks."""
    B, H, C, d = cfg.B, cfg.H, cfg.C, cfg.dk
    dt = R.BF16 if cfg.dtype == 1 else R.F32
    reps = C // cfg.pool_window if cfg.pool_window else 1
    r = lambda *s: torch.randn(*s, generator=gen)
    t = {"rk": r(B, H, mc, reps, d), "buf_beta": r(B, H, C), "mass": torch.floor(r(B, H, mc).abs() * 4) / 4,
         "buf_alpha": r(B, H, C, d) if cfg.decay_mode else r(B, H, C),
         "n_chunks": torch.tensor(n, dtype=torch.int32), "m_partial": torch.arange(B, dtype=torch.int32) + 3}
    for f in ("buf_k", "buf_v", "buf_qr", "buf_kr"):
        t[f] = r(B, H, C, d).to(dt)
    if fmt == "factored":
        t.update({f: r(B, H, mc, C, d).to(dt) for f in ("Kf", "Wf", "Uf")}, df=r(B, H, mc, C + 4))
    elif fmt == "int8":
        t.update({f: torch.randint(-127, 128, (B, H, mc, d, d), generator=gen, dtype=torch.int8) for f in ("A", "Bm")},
                 df=r(B, H, mc, 4))
    else:
        t.update({f: r(B, H, mc, d, d).to(dt) for f in ("A", "Bm")})
    return t, hla.Cache.from_tensors(cfg, mc, **{k: v.cuda() for k, v in t.items()})


@pytest.mark.parametrize("fmt,dtype,d,C,window,decay", [
    ("dense", "bf16", 128, 64, 0, "scalar"), ("dense", "f32", 64, 64, 16, "scalar"),
    ("dense", "bf16", 64, 128, 0, "channel"), ("int8", "bf16", 128, 64, 0, "scalar"),
    ("int8", "f32", 64, 256, 32, "channel"), ("factored", "bf16", 128, 64, 0, "scalar"),
])
@pytest.mark.parametrize("n,keep,recent", [([10], 6, 2), ([0, 1, 7], 3, 3), ([9, 5, 9], 5, 0), ([20, 19], 1, 1),
                                           ([20, 3], 19, 4), ([4], 8, 0), ([300], 290, 7)])
def test_evict(hla, fmt, dtype, d, C, window, decay, n, keep, recent):
    B, H = len(n), 3
    gen = torch.Generator().manual_seed(sum(n) + keep)
    cfg = hla.make_config(B, H, 1, C, d, dtype, cache_format=fmt, pool_window=window, decay=decay)
    mc = max(max(n) + 1, keep)
    t, src = make_cache(hla, gen, cfg, mc, n, fmt)
    t["mass"][0, 0, :3] = torch.tensor([float("nan"), -0.0, 0.0])[:min(3, mc)]
    src.buffers["mass"].copy_(t["mass"])
    _, dst = make_cache(hla, gen, cfg, keep, [0] * B, fmt)
    before = {k: v.cpu() for k, v in dst.buffers.items()}
    kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
    kept2 = torch.empty_like(kept)
    hla.hla_cache_evict(cfg, src, dst, keep, recent, kept)
    torch.cuda.synchronize()
    assert all(torch.equal(src.buffers[f].cpu().nan_to_num(3.5), t[f].nan_to_num(3.5)) for f in t)  # src untouched
    hla.hla_cache_evict(cfg, src, src, keep, recent, kept2)
    assert torch.equal(kept, kept2)
    for c, moved in ((dst, True), (src, False)):
        got = {k: v.cpu() for k, v in c.buffers.items()}
        for b in range(B):
            for h in range(H):
                ref = R.evict_reference(t["mass"][b, h], n[b], keep, recent)
                assert kept[b, h].tolist() == ref + [-1] * (keep - len(ref))
                for f in FIELDS[fmt] + ("rk", "mass"):
                    assert torch.equal(got[f][b, h, :len(ref)].nan_to_num(3.5), t[f][b, h, ref].nan_to_num(3.5)), f
                    rest = (before if moved else t)[f][b, h, len(ref):]
                    if moved or len(ref) == n[b]:
                        assert torch.equal(got[f][b, h, len(ref):].nan_to_num(3.5), rest.nan_to_num(3.5)), f
            assert int(got["n_chunks"][b]) == min(n[b], keep)
        for f in ("buf_k", "buf_v", "buf_qr", "buf_kr", "buf_alpha", "buf_beta", "m_partial"):
            assert torch.equal(got[f], t[f]), f


def test_evict_untracked_target_and_slices(hla):
    """A target without weights, and one sequence of a batch through slices."""
    gen = torch.Generator().manual_seed(2)
    cfg = hla.make_config(3, 2, 1, 64, 64, "f32")
    t, src = make_cache(hla, gen, cfg, 9, [9, 8, 9], "dense")
    one = hla.make_config(1, 2, 1, 64, 64, "f32")
    tensors = {k: v.cuda() for k, v in make_cache(hla, gen, one, 4, [0], "dense")[0].items() if k != "mass"}
    dst = hla.Cache.from_tensors(one, 4, **tensors)
    kept = torch.empty(1, 2, 4, dtype=torch.int32, device="cuda")
    hla.hla_cache_evict(one, src.slice(1, 1), dst, 4, 1, kept)
    for h in range(2):
        ref = R.evict_reference(t["mass"][1, h], 8, 4, 1)
        assert kept[0, h].tolist() == ref
        assert torch.equal(dst.buffers["A"].cpu()[0, h], t["A"][1, h, ref])


@pytest.mark.parametrize("dtype,d,fmt,mode,window", [
    ("bf16", 128, "dense", "routed", 0), ("bf16", 128, "factored", "routed", 0), ("bf16", 128, "int8", "routed", 0),
    ("f32", 64, "dense", "routed", 0), ("f32", 64, "int8", "one", 0), ("bf16", 128, "dense", "routed", 32),
])
def test_mass_through_prefill_and_decode(hla, dtype, d, fmt, mode, window):
    """A tracked cache: the prompt's gate mass, then every step's gates, a closing chunk
    starting at zero; the outputs are those of an untracked cache."""
    w = syn.PREFILL_0P8B.with_(B=2, H=2, T=64 * 6 + 60, d=d, dtype=dtype, thr=0.05, gate_mode=mode, window=window)
    inp = P.to_cuda(P.gpu_inputs(w))
    cfg = hla.make_config(2, 2, w.T, 64, d, dtype, mode, w.tau, w.bias, w.thr, cache_format=fmt, pool_window=window)
    N = w.N
    gates = torch.empty(2, 2, N, N, device="cuda")
    caches, outs = [], []
    for tracked in (True, False):
        c = hla.Cache(cfg, 8)
        if tracked:
            mass = c.track_mass()
        o = torch.empty_like(inp["q"])
        hla.hla_prefill(cfg, inp["q"], inp["k"], inp["v"], inp["alpha"], inp["beta"], o, q_route=inp["q_route"],
                        k_route=inp["k_route"], gates_out=gates, cache=c)
        caches.append(c)
        outs.append([o])
    ref = torch.empty(2, 2, N, device="cuda")
    hla.hla_gate_mass(cfg, gates, ref)
    want = mass.clone()
    assert torch.equal(mass[:, :, :N - 1], ref[:, :, :N - 1])
    want[:, :, :N - 1] = ref[:, :, :N - 1]
    dcfg = hla.make_config(2, 2, 1, 64, d, dtype, mode, w.tau, w.bias, w.thr, cache_format=fmt, pool_window=window)
    want = want.cpu().double()
    for tok in syn.make_decode_tokens(w.with_(B=2), 7):
        tok = {k: v.cuda() for k, v in tok.items()}
        val = R.cache_values(caches[0], dcfg) if fmt != "factored" else None
        for c, o in zip(caches, outs):
            out = torch.empty_like(tok["q"])
            hla.hla_decode_step(dcfg, c, tok["q"], tok["k"], tok["v"], tok["alpha"], tok["beta"], out)
            o.append(out)
        if val is not None:
            host = {k: v.cpu() for k, v in tok.items()}
            g = R.decode_reference(val, dcfg, host)[1]
            if mode == "one":
                for b in range(2):
                    g[b, :, :int(val["n"][b])] = 1.0
            want = want + g
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    if fmt != "factored":
        # gates by the binary32 recipe against 64 bits: a few 2^-24 each, summed in float32
        err = (mass.cpu().double() - want).abs() / want.clamp(min=1.0)
        assert float(err[:, :, :7].max()) <= 2e-5
    assert hla.hla_device_status() == (0, 0)


@pytest.mark.parametrize("fmt", ["dense", "int8"])
def test_prefill_evict_decode_together(hla, fmt):
    """As they are used together: a prompt into a tracked cache, its chunks cut down into a
    smaller cache, tokens decoded across a chunk's end, an eviction in place, more tokens.
    Each step is compared with its definition from the values that the cache holds."""
    B, H, d, C = 2, 2, 128, 64
    w = syn.PREFILL_0P8B.with_(B=B, H=H, T=64 * 9 + 61)
    inp = P.to_cuda(P.gpu_inputs(w))
    cfg = hla.make_config(B, H, w.T, C, d, "bf16", "routed", w.tau, w.bias, 0.0, cache_format=fmt)
    dcfg = hla.make_config(B, H, 1, C, d, "bf16", "routed", w.tau, w.bias, 0.0, cache_format=fmt)
    big, small = hla.Cache(cfg, 9), hla.Cache(dcfg, 7)
    mass = big.track_mass()
    small_mass = small.track_mass()
    gates = torch.empty(B, H, w.N, w.N, device="cuda")
    o = torch.empty_like(inp["q"])
    hla.hla_prefill(cfg, inp["q"], inp["k"], inp["v"], inp["alpha"], inp["beta"], o, q_route=inp["q_route"],
                    k_route=inp["k_route"], gates_out=gates, cache=big)
    kept = torch.empty(B, H, 6, dtype=torch.int32, device="cuda")
    hla.hla_cache_evict(dcfg, big, small, 6, 2, kept)
    a, b_ = R.cache_values(big, dcfg), R.cache_values(small, dcfg)
    for b in range(B):
        for h in range(H):
            ref = R.evict_reference(mass[b, h].cpu(), 9, 6, 2)
            assert kept[b, h].tolist() == ref
            assert torch.equal(b_["A"][b, h, :6], a["A"][b, h, ref]) and torch.equal(b_["rk"][b, h, :6], a["rk"][b, h, ref])
            assert torch.equal(small_mass[b, h, :6].cpu(), mass[b, h, ref].cpu())
    assert b_["n"].tolist() == [6, 6] and b_["m"].tolist() == [61, 61]
    kept2 = torch.empty(B, H, 5, dtype=torch.int32, device="cuda")
    for i, tok in enumerate(syn.make_decode_tokens(w, 6)):
        if i == 4:  # 7 closed chunks now: the cache is full, make room
            assert R.cache_values(small, dcfg)["n"].tolist() == [7, 7]
            hla.hla_cache_evict(dcfg, small, small, 5, 1, kept2)
            assert R.cache_values(small, dcfg)["n"].tolist() == [5, 5]
        val = R.cache_values(small, dcfg)
        ref, _ = R.decode_reference(val, dcfg, tok)
        t = {k: v.cuda() for k, v in tok.items()}
        out = torch.empty_like(t["q"])
        hla.hla_decode_step(dcfg, small, t["q"], t["k"], t["v"], t["alpha"], t["beta"], out)
        # float32 arithmetic on the stored values: the output's own rounding is what shows
        assert R.rel(out.cpu(), ref) <= 2.0 ** -8 + 1e-4
    assert hla.hla_device_status() == (0, 0)


def test_caches_on_another_device_are_refused(hla):
    import types
    c = hla.make_config(1, 1, 1, 64, 64, "f32")
    cache = hla.Cache(c, 2)
    cache.track_mass()
    away = types.SimpleNamespace(device_index=1, struct=cache.struct)
    kept = torch.empty(1, dtype=torch.int32, device="cuda:0")
    for src, dst, name in ((away, cache, "src"), (cache, away, "dst")):
        with pytest.raises(ValueError, match=name):
            hla.hla_cache_evict(c, src, dst, 1, 0, kept)
