"""Decode over the 8-bit cache with a query of wide range, whose largest entry no chunk reads: the
products run on x in fixed point relative to its largest entry, with a half unit of at most 2^-30 of
it.

float32 outputs: the others lie 2^-7 below, so they are off by 2^-23 of themselves at most and an
output by 2^-23 / sqrt(d) of its size and the roundings of joining digits, scales and chunks (a few
2^-24 each: 16 allowed).  bf16 outputs: 2^-18 below, off by 2^-12, and the output's own 2^-8 / 2."""
import pytest
import torch

from tests import _serving as R
from tests.test_gpu_cache8 import random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hla():
    import gated_delta_rule_transitions_b200 as m
    m.lib()
    return m._hla


@pytest.mark.parametrize("dtype,d,below,tol", [("f32", 64, 2.0 ** -7, 18 * 2.0 ** -24), ("f32", 128, 2.0 ** -7, 18 * 2.0 ** -24),
                                               ("bf16", 64, 2.0 ** -18, 2.0 ** -9 + 2.0 ** -12),
                                               ("bf16", 128, 2.0 ** -18, 2.0 ** -9 + 2.0 ** -12)])
@pytest.mark.parametrize("scale", [1.0, 1.9, 2.0 ** -60, 2.0 ** 60])
def test_small_entries_beside_a_large_one(hla, dtype, d, below, tol, scale):
    gen = torch.Generator().manual_seed(d)
    B, H, n = 1, 2, 3
    cfg = hla.make_config(B, H, 1, 64, d, dtype, "one", cache_format="int8")
    t, cache = random_cache(hla, gen, cfg, n + 1, [n], [0], dtype)
    t["df"][..., 0], t["df"][..., 1] = 1.0, 0.0         # A_j = I: every chunk sees the same x
    t["Bm"][..., 7] = 0                                  # and none reads entry 7
    for f in ("df", "Bm"):
        cache.buffers[f].copy_(t[f])
    q = (scale * below * (0.5 + torch.rand(B, H, d, generator=gen))).to(R.DT[dtype])
    q[..., 7] = scale
    _, k, v, _, _ = R.tokens(gen, B, H, H, d, R.DT[dtype])
    al, be = torch.ones(B, H), torch.zeros(B, H)
    x = q.double()
    ref = torch.zeros(B, H, d, dtype=torch.float64)
    for j in range(n):
        ref += t["df"][:, :, j, 2, None].double() * (t["Bm"][:, :, j].double() @ x[..., None])[..., 0]
    out = torch.empty(B, H, d, dtype=R.DT[dtype], device="cuda")
    hla.hla_decode_step(cfg, cache, *(a.cuda() for a in (q, k, v, al, be)), out)
    assert R.rel(out.cpu(), ref) <= tol


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_digits_at_their_ends(hla, dtype, d):
    """Powers of two, their neighbours below, negative ones, zeros, the smallest and the largest: one
    entry at a time is read (codes of one row of the identity).

    The unit is 2^(e - 30) with big >= 127/128 2^e, so half of it is at most 2^-31 128/127 big.  It is
    a power of two: an entry whose last place is worth a unit or more is exact.  bf16 entries down to
    2^-22 big are; float32 ones (last place 2^-24 of the power of two above) from 2^-6 big up, and
    between 2^-7 and 2^-6 big the last place can be half a unit: off by that at most."""
    B, H, n = 1, 1, 1
    cfg = hla.make_config(B, H, 1, 64, d, dtype, "one", cache_format="int8")
    t, cache = random_cache(hla, torch.Generator().manual_seed(1), cfg, n + 1, [n], [0], dtype)
    t["df"][:] = torch.tensor([1.0, 0.0, 1.0, 0.0])
    t["Bm"][:] = torch.eye(d).to(torch.int8)
    for f in ("df", "Bm"):
        cache.buffers[f].copy_(t[f])
    top = 1 - torch.finfo(R.DT[dtype]).eps / 2
    for big in (1.0, top, 2.0 ** -90, 2.0 ** 100, top * 2.0 ** 120, 0.0):
        q = torch.zeros(B, H, d)
        q[..., 0], q[..., 1], q[..., 2], q[..., 3] = big, -big, big * 2.0 ** -7, -top * big * 2.0 ** -6
        q[..., 4], q[..., 5] = big / 256 * 3, -big / 2
        q = q.to(R.DT[dtype])
        k, z = torch.zeros_like(q), torch.zeros(B, H)
        out = torch.empty_like(q, device="cuda")
        cache.buffers["m_partial"].zero_()
        hla.hla_decode_step(cfg, cache, *(a.cuda() for a in (q, k, k, z + 1, z)), out)
        off = (out.cpu().double() - q.double()).abs()
        assert float(off.max()) <= (0.0 if dtype == "bf16" else 2.0 ** -31 * 128 / 127 * big), big
        assert bool((off[q.abs().double() >= 2.0 ** -6 * big] == 0).all()), big
