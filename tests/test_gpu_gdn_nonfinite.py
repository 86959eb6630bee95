"""A NaN or an infinity among a sequence's tokens, by chunks and by rows alike: what the rule makes
finite from the same inputs is right, what it does not is not finite here either.  So nothing that
comes before a bad token is touched by it, a bad query spoils its own output alone, a bad value
its own row of the state alone, the others spoil all from their token on."""
import pytest
import torch

from tests import _serving as R

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def hla():
    import gated_delta_rule_transitions_b200 as m
    m.lib()
    return m._hla


def check(got, ref, tol, what):
    got, ref = got.cpu().double(), ref.double()
    good = ref.isfinite()
    assert torch.equal(got.isfinite(), good), what
    if bool(good.any()):
        assert R.rel(got[good], ref[good]) <= tol, what


def run(hla, x, lens, S0, Hk, H, d, dtype, channel):
    cu, n = torch.tensor([0] + lens).cumsum(0).to(torch.int32), len(lens)
    cfg = hla.make_gdn_config(n, H, d, dtype, Hk=Hk, decay="channel" if channel else "scalar")
    S, o = S0.cuda(), torch.full((sum(lens), H, d), 7.0, dtype=R.DT[dtype], device="cuda")
    hla.gdn_forward(cfg, *(t.cuda() for t in x), cu.cuda(), o, state_in=S, state_out=S)
    ro, rS = R.gdn_reference(*x, [(int(cu[i]), int(cu[i + 1])) for i in range(n)], S0)
    # float32 sums of d terms, 64 tokens of them (what is older has decayed); the output's rounding
    tol = 64 * (d / 8 + 8) * 2.0 ** -24
    for h in range(H):
        check(o[:, h], ro[:, h], tol + R.half_step(R.DT[dtype]), f"outputs of head {h}")
        check(S[:, h], rS[:, h], tol, f"states of head {h}")
    assert hla.hla_device_status() == (0, 0)


FORMS = [("bf16", 128, False), ("f32", 128, False), ("bf16", 64, False), ("f32", 64, True)]


@pytest.mark.parametrize("dtype,d,channel", FORMS)
@pytest.mark.parametrize("what,value", [(w, x) for w in ("q", "k", "v", "alpha", "beta") for x in (NAN, INF, -INF)
                                        if (w, x) != ("alpha", -INF)])  # (no decay)
@pytest.mark.parametrize("at", [0, 1, 37, 63, 64, 100, 149])
def test_one_bad_number(hla, dtype, d, channel, what, value, at):
    gen = torch.Generator().manual_seed(at + d)
    H, lens = 3, [150]
    x = R.tokens(gen, 150, H, H, d, R.DT[dtype], channel)
    t = x[("q", "k", "v", "alpha", "beta").index(what)]
    t[(at, 1) + ((5,) if t.dim() == 3 else ())] = value  # one number of head 1
    run(hla, x, lens, torch.randn(1, H, d, d, generator=gen), H, H, d, dtype, channel)


@pytest.mark.parametrize("lens,H", [([90, 200], 2), ([130, 70, 90], 8), ([100] * 6, 8), ([1] * 20 + [300, 40, 64], 2)],
                         ids=["16", "32", "64", "shared"])
def test_many_bad_numbers(hla, lens, H):
    """Bad values in several columns, tokens and heads, bad queries, a bad key near the end of some
    sequences, one bad number in a state: 16, 32 and 64 value columns per CTA, and a shared batch."""
    gen = torch.Generator().manual_seed(len(lens))
    n, T, d, dtype = len(lens), sum(lens), 128, "bf16"
    q, k, v, al, be = x = R.tokens(gen, T, H, H, d, R.BF16)
    pick = lambda m: int(torch.randint(m, (1,), generator=gen))
    for _ in range(12):
        v[pick(T), pick(H), pick(d)] = (NAN, INF, -INF)[pick(3)]
        q[pick(T), pick(H), pick(d)] = (NAN, INF)[pick(2)]
    ends = torch.tensor(lens).cumsum(0).tolist()
    for i in range(0, n, 3):
        k[max(ends[i] - 9, ends[i] - lens[i]), pick(H), pick(d)] = NAN
        be[ends[i] - 1, pick(H)] = INF
    al[ends[-1] - 5, 0] = NAN
    S0 = torch.randn(n, H, d, d, generator=gen)
    S0[n // 2, 1, 17, 3] = NAN
    S0[n // 2, 0, 100, 3] = INF
    run(hla, x, lens, S0, H, H, d, dtype, False)


def test_keys_whose_products_overflow(hla):
    """Finite keys of length 1e25: the products of two of them are beyond float32, in the state as
    in the triangular system; what comes before the second is not touched."""
    gen = torch.Generator().manual_seed(2)
    H, d, T = 2, 128, 128
    x = R.tokens(gen, T, H, H, d, R.BF16)
    x[1][[70, 90], 1] *= 1e25
    x[4][70:91, 1] = 1.0
    S0 = torch.zeros(1, H, d, d)
    cfg = hla.make_gdn_config(1, H, d, "bf16")
    S, o = S0.cuda(), torch.empty(T, H, d, dtype=R.BF16, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32)
    hla.gdn_forward(cfg, *(t.cuda() for t in x), cu.cuda(), o, state_in=S, state_out=S)
    ro, rS = R.gdn_reference(*x, [(0, T)], S0)
    tol = 64 * (d / 8 + 8) * 2.0 ** -24
    assert R.rel(o[:70].cpu(), ro[:70]) <= tol + 2.0 ** -8
    assert R.rel(o[:, 0].cpu(), ro[:, 0]) <= tol + 2.0 ** -8 and R.rel(S[:, 0].cpu(), rS[:, 0]) <= tol
    assert not bool(o[90:, 1].isfinite().any()) and not bool(S[:, 1].isfinite().any())
