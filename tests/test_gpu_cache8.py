"""The 8-bit chunk cache: what the prefill and the decode close store, and decode steps from
it, against the definition in 64 bits on the stored values.

A stored entry is off by at most half a scale (the codes round to nearest); the scale itself
is one float32 division of a float32 difference, so two more 2^-24 of the largest entry.  A
decode step works in float32 on the stored values: the bf16 output's own rounding (2^-8) and
1e-4 for float32 sums of d terms over at most ten chunks (10 (128 / 4 + 8) 2^-24 = 2.4e-5)."""
import pytest
import torch

import hla_synth as syn
from tests import _parity as P
from tests import _serving as R

pytestmark = pytest.mark.gpu

CASES = [("bf16", 128, 64, 0, "scalar"), ("bf16", 128, 128, 0, "scalar"), ("bf16", 128, 256, 32, "scalar"),
         ("f32", 64, 64, 0, "scalar"), ("f32", 128, 64, 16, "channel"), ("bf16", 128, 64, 0, "channel"),
         ("bf16", 64, 64, 0, "scalar")]


@pytest.fixture(scope="module")
def hla():
    import gated_delta_rule_transitions_b200 as m
    m.lib()
    return m._hla


def check_codes(val8, exact, nc, d):
    """Stored values against the transitions they stand for (dense cache, 64 bits)."""
    sc = val8["scales"]
    eye = torch.eye(d, dtype=torch.float64)
    A, B = exact["A"][:, :, :nc], exact["B"][:, :, :nc]
    mean = A.diagonal(dim1=-2, dim2=-1).mean(-1)
    assert bool(((sc[:, :, :nc, 0] - mean).abs() <= 16 * 2.0 ** -24 * A.abs().amax((-1, -2))).all())
    off = (A - sc[:, :, :nc, 0, None, None] * eye).abs().amax((-1, -2))
    big = A.abs().amax((-1, -2))
    slack = 4 * 2.0 ** -24
    assert bool(((sc[:, :, :nc, 1] * 127 - off).abs() <= slack * big).all())
    assert bool(((sc[:, :, :nc, 2] * 127 - B.abs().amax((-1, -2))).abs() <= slack * B.abs().amax((-1, -2))).all())
    ea = (val8["A"][:, :, :nc] - A).abs().amax((-1, -2))
    eb = (val8["B"][:, :, :nc] - B).abs().amax((-1, -2))
    assert bool((ea <= 0.5 * sc[:, :, :nc, 1] + 2 * slack * big).all())
    assert bool((eb <= 0.5 * sc[:, :, :nc, 2] * (1 + 128 * slack)).all())
    assert bool((sc[:, :, :nc, 3] == 0).all())


@pytest.mark.parametrize("dtype,d,C,window,decay", CASES)
@pytest.mark.parametrize("m0", [0, 61])
def test_prefill_close_and_decode(hla, dtype, d, C, window, decay, m0):
    B, H, nc = 2, 2, 4
    w = syn.PREFILL_0P8B.with_(B=B, H=H, T=C * nc + (C - 3 if m0 else 0), d=d, dtype=dtype, C=C, window=window,
                               decay=decay)
    inp = P.to_cuda(P.gpu_inputs(w))
    mk = lambda T, fmt: hla.make_config(B, H, T, C, d, dtype, "routed", w.tau, w.bias, 0.0, cache_format=fmt,
                                        pool_window=window, decay=decay)
    caches, outs = {}, {}
    for fmt in ("dense", "int8"):
        caches[fmt] = hla.Cache(mk(w.T, fmt), nc + 2)
        outs[fmt] = torch.empty_like(inp["q"])
        hla.hla_prefill(mk(w.T, fmt), inp["q"], inp["k"], inp["v"], inp["alpha"], inp["beta"], outs[fmt],
                        q_route=inp["q_route"], k_route=inp["k_route"], cache=caches[fmt])
    assert torch.equal(outs["dense"], outs["int8"])
    check_codes(R.cache_values(caches["int8"], mk(1, "int8")), R.cache_values(caches["dense"], mk(1, "dense")), nc, d)
    tol = (2.0 ** -8 if dtype == "bf16" else 0.0) + 1e-4
    for tok in syn.make_decode_tokens(w, 5):
        t = {k: v.cuda() for k, v in tok.items()}
        ref, _ = R.decode_reference(R.cache_values(caches["int8"], mk(1, "int8")), mk(1, "int8"), tok)
        for fmt in ("dense", "int8"):
            out = torch.empty_like(t["q"])
            hla.hla_decode_step(mk(1, fmt), caches[fmt], t["q"], t["k"], t["v"], t["alpha"], t["beta"], out)
        assert R.rel(out.cpu(), ref) <= tol
    end = nc + (1 if m0 else 0)
    v8, vd = R.cache_values(caches["int8"], mk(1, "int8")), R.cache_values(caches["dense"], mk(1, "dense"))
    assert v8["n"].tolist() == [end] * B and torch.equal(v8["m"], vd["m"])
    check_codes(v8, vd, end, d)  # the chunk that the decode steps closed among them
    assert torch.equal(v8["rk"][:, :, :end], vd["rk"][:, :, :end])
    assert hla.hla_device_status() == (0, 0)


def random_cache(hla, gen, cfg, mc, n, m, dtype):
    B, H, C, d = cfg.B, cfg.H, cfg.C, cfg.dk
    r = lambda *s: torch.randn(*s, generator=gen)
    qa = torch.randint(-127, 128, (B, H, mc, d, d), generator=gen, dtype=torch.int8)
    qb = torch.randint(-127, 128, (B, H, mc, d, d), generator=gen, dtype=torch.int8)
    sc = torch.zeros(B, H, mc, 4)
    sc[..., 0] = 0.5 * torch.rand(B, H, mc, generator=gen)
    # spectral norm of the codes is near 2 sqrt(d) 73: keep A_j a contraction
    sc[..., 1] = 0.2 / (2 * d ** 0.5 * 73) * torch.rand(B, H, mc, generator=gen)
    sc[..., 2] = 0.01 * torch.rand(B, H, mc, generator=gen)
    t = {"A": qa, "Bm": qb, "df": sc, "rk": r(B, H, mc, 1, d), "buf_alpha": torch.rand(B, H, C, generator=gen),
         "buf_beta": torch.rand(B, H, C, generator=gen), "n_chunks": torch.tensor(n, dtype=torch.int32),
         "m_partial": torch.tensor(m, dtype=torch.int32)}
    for f in ("buf_k", "buf_v", "buf_qr", "buf_kr"):
        x = r(B, H, C, d)
        t[f] = (x / x.norm(dim=-1, keepdim=True) if f == "buf_k" else x).to(R.DT[dtype])
    return t, hla.Cache.from_tensors(cfg, mc, **{k: v.cuda() for k, v in t.items()})


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("n,m,thr", [([0], [0], 0.0), ([1], [5], 0.0), ([2, 0, 3], [62, 0, 7], 0.0),
                                     ([70, 65], [1, 30], 0.3), ([64], [0], 0.999), ([200], [10], 0.0)])
def test_decode_from_given_codes(hla, dtype, d, n, m, thr):
    """Random full-range codes: no chunk, one, ragged counts, all skipped, many."""
    gen = torch.Generator().manual_seed(sum(n) + d)
    B, H, mc = len(n), 2, max(n) + 1
    cfg = hla.make_config(B, H, 1, 64, d, dtype, "routed", 1.0, -1.0, thr, cache_format="int8")
    t, cache = random_cache(hla, gen, cfg, mc, n, m, dtype)
    tok = dict(zip(("q", "k", "v", "alpha", "beta"), R.tokens(gen, B, H, H, d, R.DT[dtype])))
    ref, _ = R.decode_reference(R.cache_values(cache, cfg), cfg, tok)
    g = {a: b.contiguous().cuda() for a, b in tok.items()}
    out = torch.empty_like(g["q"])
    hla.hla_decode_step(cfg, cache, g["q"], g["k"], g["v"], g["alpha"], g["beta"], out)
    tol = (2.0 ** -8 if dtype == "bf16" else 0.0) + max(n) * (d / 4 + 8) * 2.0 ** -24 + 1e-5
    assert R.rel(out.cpu(), ref) <= tol
    after = R.cache_values(cache, cfg)
    assert after["n"].tolist() == n and after["m"].tolist() == [x + 1 for x in m]


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_zero_tiny_and_bad_values(hla, dtype, d):
    """A query of zeros; a chunk of all zeros (scale 0); tiny and huge states; a chunk with a
    NaN shows in the output of its head alone."""
    gen = torch.Generator().manual_seed(1)
    B, H, mc = 1, 4, 5
    cfg = hla.make_config(B, H, 1, 64, d, dtype, "routed", 1.0, 0.0, 0.0, cache_format="int8")
    t, cache = random_cache(hla, gen, cfg, mc, [4], [0], dtype)
    sc = t["df"]
    sc[0, 1, 2] = 0.0                       # head 1: a chunk that was all zeros
    sc[0, 2, :, 2] *= 1e-30                 # head 2: tiny writes
    sc[0, 3, 1, 2] = float("nan")           # head 3: a chunk that held a NaN
    cache.buffers["df"].copy_(sc)
    q, k, v, al, be = R.tokens(gen, B, H, H, d, R.DT[dtype])
    q[0, 0] = 0
    tok = {"q": q, "k": k, "v": v, "alpha": al, "beta": torch.zeros_like(be)}
    ref, _ = R.decode_reference(R.cache_values(cache, cfg), cfg, tok)
    g = {a: b.contiguous().cuda() for a, b in tok.items()}
    out = torch.empty_like(g["q"])
    hla.hla_decode_step(cfg, cache, g["q"], g["k"], g["v"], g["alpha"], g["beta"], out)
    out = out.cpu()
    assert torch.equal(out[0, 0], torch.zeros_like(out[0, 0]))
    tol = (2.0 ** -8 if dtype == "bf16" else 0.0) + 1e-4
    assert R.rel(out[0, 1], ref[0, 1]) <= tol and R.rel(out[0, 2], ref[0, 2]) <= tol
    assert bool(out[0, 3].isnan().all())


def test_static_scratch_and_capture(hla):
    """hla_decode_step_static on an 8-bit cache, and a captured step replayed: the bits of the
    workspace call."""
    gen = torch.Generator().manual_seed(6)
    B, H, d = 1, 2, 128
    cfg = hla.make_config(B, H, 1, 64, d, "bf16", "routed", 1.0, -1.0, 0.0, cache_format="int8")
    toks = [R.tokens(gen, B, H, H, d, R.BF16) for _ in range(4)]
    outs = []
    for how in ("workspace", "static", "graph"):
        t, cache = random_cache(hla, torch.Generator().manual_seed(7), cfg, 6, [4], [61], "bf16")
        buf = [x.cuda() for x in toks[0]]
        out, got = torch.empty(B, H, d, dtype=R.BF16, device="cuda"), []
        ws = torch.empty(hla.decode_workspace_bytes(cfg, 6), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        if how == "graph":
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                hla.hla_decode_step(cfg, cache, *buf, out, workspace=ws)
        for tok in toks:
            for x, y in zip(buf, tok):
                x.copy_(y)
            if how == "workspace":
                hla.hla_decode_step(cfg, cache, *buf, out, workspace=ws)
            elif how == "static":
                hla.hla_decode_step_static(cfg, cache, *buf, out)
            else:
                graph.replay()
            torch.cuda.synchronize()
            got.append(out.clone())
        assert cache.buffers["n_chunks"].tolist() == [5]
        outs.append(torch.stack(got))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
