"""Gate mass where its wide tiles run (from 19 tiles of 256 columns up on 148 SMs), and the weight
that a factored cache keeps, against plain sums in 64 bits."""
import math

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


# N a multiple of four (16-byte loads) and not; less than a tile, some tiles and a part, enough heads
# for one, two and more CTAs a tile; N = 1 and 2
@pytest.mark.parametrize("B,H,T,C,thr", [
    (2, 16, 64 * 128, 64, 0.0), (1, 20, 64 * 255, 64, 0.05), (5, 8, 64 * 258 - 3, 64, 0.3), (1, 25, 64 * 600, 64, 0.05),
    (1, 19, 128 * 513 - 100, 128, 0.0), (19, 8, 256 * 66 + 1, 256, 0.99), (32, 10, 65, 64, 0.0), (32, 10, 64, 64, 0.0),
    (1, 7, 64 * 1027, 64, 0.05), (2, 80, 64 * 300, 64, 0.05)])
def test_gate_mass_many_heads(hla, B, H, T, C, thr):
    """All terms are positive.  A lane adds at most N / 8 of them in sequence (its warp's rows), then
    at most 64 partial sums: off by at most (N / 8 + 64) 2^-24 of the sum."""
    N = -(-T // C)
    gen = torch.Generator().manual_seed(N + H)
    g = torch.sigmoid(2 * torch.randn(B, H, N, N, generator=gen) - 1)
    live = torch.tril(torch.ones(N, N, dtype=bool), -1)
    w = torch.tensor([min(C, T - i * C) for i in range(N)], dtype=torch.float64)
    x = torch.where(live, g, 0.0).double()
    if thr > 0:
        x = x * (x >= torch.tensor(thr, dtype=torch.float32).double())
    ref = torch.einsum("i,bhij->bhj", w, x)
    dev = torch.where(live, g, float("nan")).cuda()  # the others are never read
    cfg = hla.make_config(B, H, T, C, 128, "bf16", skip_threshold=thr)
    out, again = torch.full((B, H, N), 9.0, device="cuda"), torch.empty(B, H, N, device="cuda")
    hla.hla_gate_mass(cfg, dev, out)
    assert bool(((out.cpu().double() - ref).abs() <= (N / 8 + 64) * 2.0 ** -24 * ref).all())
    hla.hla_gate_mass(cfg, dev, again)
    assert torch.equal(again, out)


def test_mass_of_a_prompt_of_many_heads(hla):
    """A prompt of 25 heads into a tracked cache: the gates' column sums, row pitch and length of
    the cache's own array."""
    w = syn.PREFILL_0P8B.with_(B=1, H=25, T=64 * 9 + 5, thr=0.05)
    inp = P.to_cuda(P.gpu_inputs(w))
    cfg = hla.make_config(1, 25, w.T, 64, w.d, w.dtype, "routed", w.tau, w.bias, w.thr)
    cache = hla.Cache(cfg, 13)
    mass = cache.track_mass(torch.full((1, 25, 13), 5.0, device="cuda"))
    gates = torch.empty(1, 25, w.N, w.N, device="cuda")
    hla.hla_prefill(cfg, inp["q"], inp["k"], inp["v"], inp["alpha"], inp["beta"], torch.empty_like(inp["q"]),
                    q_route=inp["q_route"], k_route=inp["k_route"], gates_out=gates, cache=cache)
    g = gates.cpu().double().tril(-1)
    g = g * (g >= torch.tensor(w.thr, dtype=torch.float32).double())
    rows = torch.tensor([min(64, w.T - 64 * i) for i in range(w.N)], dtype=torch.float64)
    ref = torch.einsum("i,bhij->bhj", rows, g)[:, :, :9]
    got = mass.cpu().double()
    assert bool(((got[:, :, :9] - ref).abs() <= 24 * 2.0 ** -24 * ref).all())
    assert torch.equal(got[:, :, 9:], torch.zeros(1, 25, 4, dtype=torch.float64))


def test_mass_of_a_factored_cache(hla):
    """The factored cache's weight through decode steps: gates from its key pools in 64 bits.  A gate's
    binary32 recipe is off by a few 2^-24 (128 terms of a dot product of size below 8: at most
    128 x 8 x 2^-24 = 6e-5 in the exponent, a quarter of that in the gate), summed over seven steps."""
    B, H, d, nc = 2, 2, 128, 6
    w = syn.PREFILL_0P8B.with_(B=B, H=H, T=64 * nc + 60, thr=0.05)
    inp = P.to_cuda(P.gpu_inputs(w))
    mk = lambda T: hla.make_config(B, H, T, 64, d, "bf16", "routed", w.tau, w.bias, w.thr, cache_format="factored")
    cache = hla.Cache(mk(w.T), nc + 2)
    mass = cache.track_mass()
    gates = torch.empty(B, H, w.N, w.N, device="cuda")
    hla.hla_prefill(mk(w.T), inp["q"], inp["k"], inp["v"], inp["alpha"], inp["beta"], torch.empty_like(inp["q"]),
                    q_route=inp["q_route"], k_route=inp["k_route"], gates_out=gates, cache=cache)
    want, thr = mass.cpu().double(), float(torch.tensor(w.thr, dtype=torch.float32))
    unsure = torch.zeros_like(want, dtype=torch.bool)  # a gate next to the threshold decides
    for tok in syn.make_decode_tokens(w, 7):
        n = cache.view("n_chunks", (B,), torch.int32).tolist()
        m = cache.view("m_partial", (B,), torch.int32).tolist()
        rk = cache.view("rk", (B, H, nc + 2, d), torch.float32).cpu().double()
        qr = cache.view("buf_qr", (B, H, 64, d), torch.bfloat16).cpu().double()
        for b in range(B):
            pool = torch.cat([qr[b, :, :m[b]], tok["q"][b].double()[:, None]], 1)
            rq = w.tau * torch.log(torch.exp(pool / w.tau).mean(1))
            g = torch.sigmoid(torch.einsum("hjd,hd->hj", rk[b, :, :n[b]], rq) / math.sqrt(d) + w.bias)
            want[b, :, :n[b]] += torch.where(g >= thr, g, 0.0)
            unsure[b, :, :n[b]] |= (g - thr).abs() <= 2e-5
            if m[b] + 1 == 64:
                want[b, :, n[b]] = 0.0
        t = {k: v.cuda() for k, v in tok.items()}
        hla.hla_decode_step(mk(1), cache, t["q"], t["k"], t["v"], t["alpha"], t["beta"], torch.empty_like(t["q"]))
    assert cache.view("n_chunks", (B,), torch.int32).tolist() == [nc + 1] * B
    err = (mass.cpu().double() - want).abs() / want.clamp(min=1.0)
    err = torch.where(unsure, 0.0, err)[:, :, :nc + 1]
    assert not bool(unsure.all()) and float(err.max()) <= 7 * 1.5e-5
    assert float(mass[:, :, :nc].min()) > 0.0
    assert hla.hla_device_status() == (0, 0)
