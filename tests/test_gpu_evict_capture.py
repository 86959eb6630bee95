"""A tracked cache's step, eviction in place and gate mass captured into one graph and replayed, and on
a stream of their own: the bits of the eager calls."""
import pytest
import torch

from tests import _serving as R
from tests.test_gpu_evict import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hla():
    import gated_delta_rule_transitions_b200 as m
    m.lib()
    return m._hla


@pytest.mark.parametrize("fmt,dtype,d", [("dense", "bf16", 128), ("int8", "bf16", 128), ("factored", "bf16", 128),
                                         ("int8", "f32", 64), ("dense", "f32", 64)])
def test_captured_step_and_eviction(hla, fmt, dtype, d):
    B, H, mc, keep, recent = 2, 2, 9, 5, 2
    cfg = hla.make_config(B, H, 1, 64, d, dtype, "routed", 1.0, -1.0, 0.05, cache_format=fmt)
    mcfg = hla.make_config(B, H, 64 * 7 + 3, 64, d, dtype, skip_threshold=0.05)
    gates = torch.sigmoid(torch.randn(B, H, 8, 8, generator=torch.Generator().manual_seed(3))).cuda()
    toks = [R.tokens(torch.Generator().manual_seed(20 + i), B, H, H, d, R.DT[dtype]) for i in range(3)]
    results = []
    for how in ("eager", "graph", "stream"):
        t, cache = make_cache(hla, torch.Generator().manual_seed(4), cfg, mc, [8, 6], fmt)
        cache.buffers["m_partial"].copy_(torch.tensor([62, 61], dtype=torch.int32))
        cache.buffers["mass"].abs_()
        for f in ("buf_alpha", "buf_beta"):
            cache.buffers[f].sigmoid_()
        for f in ("A", "Bm", "Kf", "Wf", "Uf", "buf_k"):
            if f in cache.buffers and cache.buffers[f].dtype != torch.int8:
                cache.buffers[f].mul_(0.05)
        if fmt == "factored":
            cache.buffers["df"].sigmoid_()
        elif fmt == "int8":
            cache.buffers["df"].abs_().mul_(1e-3)
        buf, o = [x.contiguous().cuda() for x in toks[0]], torch.empty(B, H, d, dtype=R.DT[dtype], device="cuda")
        kept = torch.full((B, H, keep), -7, dtype=torch.int32, device="cuda")
        mass = torch.empty(B, H, 8, device="cuda")
        ws = torch.empty(hla.decode_workspace_bytes(cfg, mc), dtype=torch.uint8, device="cuda")

        def once():
            hla.hla_decode_step(cfg, cache, *buf, o, workspace=ws)
            hla.hla_cache_evict(cfg, cache, cache, keep, recent, kept)
            hla.hla_gate_mass(mcfg, gates, mass)

        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        if how == "graph":
            with torch.cuda.graph(graph):
                once()
        seen = []
        for tok in toks:
            for x, y in zip(buf, tok):
                x.copy_(y)
            torch.cuda.synchronize()
            if how == "graph":
                graph.replay()
            elif how == "stream":
                with torch.cuda.stream(side):
                    once()
            else:
                once()
            torch.cuda.synchronize()
            seen += [o.clone(), kept.clone(), mass.clone()] + [cache.buffers[f].clone() for f in sorted(cache.buffers)]
        # a chunk closes in each sequence, and the cache is cut down to `keep` in every call
        assert cache.buffers["n_chunks"].tolist() in ([6, 5], [5, 5])
        assert bool(o.isfinite().all())
        results.append(seen)
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
    assert hla.hla_device_status() == (0, 0)
