"""How exactly the chunked gated delta rule (bf16, d = 128) computes, against its definition in
64 bits, on ordinary tokens (unit keys, decays near one).

States.  Four products stand between a state and the next (K S^T, T R, U^T K and those of the
inverse inside T).  Their factors go in as three bf16 parts (exact but for products of parts of
3 x 2^-24) or as two tf32 numbers (2^-20.5 with the product of the remainders), and the sums of 64
or 128 terms in float32 add some 2^-21: each is off by at most 2^-20 of the size of its terms.
Independent errors add as their root: 2 x 2^-20 = 2^-19, and a chunk's decay forgets what came
before.  Leaving out the third part of a factor leaves out up to 2^-16 of it, always towards zero:
more than this bound allows.

Outputs.  One product more (G R) and the sum: sqrt(5) 2^-20 = 2^-18.8 before the rounding to bf16.
An error e turns the rounding of x with a probability of |e| / ulp(x), and then by ulp(x) <= 2^-7
|x|: against the rounded definition the mean square is at most E|e| ulp(x), the relative L2 at most
sqrt(2^-18.8 2^-7) = 2^-12.9."""
import pytest
import torch

from tests import _serving as R

pytestmark = pytest.mark.gpu

STATE_TOL = 2.0 ** -19
OUT_TOL = 2.0 ** -12.9


@pytest.fixture(scope="module")
def hla():
    import gated_delta_rule_transitions_b200 as m
    m.lib()
    return m._hla


# 16, 32 and 64 value columns per CTA; the last one shares its batch with single tokens
@pytest.mark.parametrize("lens,Hk,H", [([1000, 500], 2, 4), ([320, 257, 448], 4, 8), ([200] * 6, 8, 8),
                                       ([1] * 30 + [700, 65, 100], 4, 4)], ids=["16", "32", "64", "shared"])
def test_states_and_outputs_to_float32(hla, lens, Hk, H):
    gen = torch.Generator().manual_seed(len(lens) * 100 + H)
    n, T, d = len(lens), sum(lens), 128
    x = R.tokens(gen, T, Hk, H, d, R.BF16)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    S0 = 0.3 * torch.randn(n, H, d, d, generator=gen)
    S, o = S0.cuda(), torch.empty(T, H, d, dtype=R.BF16, device="cuda")
    hla.gdn_forward(hla.make_gdn_config(n, H, d, "bf16", Hk=Hk), *(t.cuda() for t in x), cu.cuda(), o, state_in=S,
                    state_out=S)
    bounds = [(int(cu[i]), int(cu[i + 1])) for i in range(n)]
    ro, rS = R.gdn_reference(*x, bounds, S0)
    errs = [R.rel(S[i].cpu(), rS[i]) for i in range(n)]
    out = R.rel(o.cpu(), ro.to(R.BF16))
    print(f"states {max(errs):.2e} of {STATE_TOL:.2e}, outputs {out:.2e} of {OUT_TOL:.2e}")
    assert max(errs) <= STATE_TOL
    assert out <= OUT_TOL
    assert hla.hla_device_status() == (0, 0)
