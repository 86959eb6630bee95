"""The fixed scratch of hla_decode_step_static and the 8-bit cache (host checks, nothing launched):
beside the lists and gates it holds a closing chunk's two d x d matrices per (sequence, head)."""
import ctypes
import os

import pytest

from tests.test_abi_serving import P, fake_cache

SCRATCH = 8 << 20


@pytest.fixture(scope="module")
def hla():
    from gated_delta_rule_transitions_b200 import _hla
    from gated_delta_rule_transitions_b200 import build as b
    b.build()
    return _hla


def config(hla, B, H, fmt, d=128, dtype="bf16"):
    return hla.make_config(B, H, 1, 64, d, dtype, cache_format=fmt)


@pytest.mark.parametrize("d,dtype,pairs", [(128, "bf16", 127), (128, "f32", 63), (64, "bf16", 508), (64, "f32", 254)])
def test_pairs_that_fit(hla, d, dtype, pairs):
    es = 2 if dtype == "bf16" else 4
    up = lambda n: -(-n // 256) * 256
    for n, mc in ((pairs, 14), (pairs + 4, 1)):
        need = hla.decode_workspace_bytes(config(hla, n, 1, "int8", d, dtype), mc)
        assert need == 2 * up(n * mc * 4) + up(n * 4) + 2 * up(n * d * d * es)
        assert (need <= SCRATCH) == (n == pairs)
    assert hla.decode_workspace_bytes(config(hla, pairs + 4, 1, "dense", d, dtype), 14) <= SCRATCH


def test_refusal_gives_the_8_bit_term(hla):
    """8 sequences x 16 heads: a dense cache fits, an 8-bit one is refused, and told why."""
    c = config(hla, 8, 16, "int8")
    cache = fake_cache(hla, c, 4)
    st = hla.lib().hla_decode_step_static(ctypes.byref(c), ctypes.byref(cache), P, P, P, P, P, None, None, P, None)
    assert st == hla.HLA_ERR_WORKSPACE
    assert "8-bit" in hla.last_error() and "two d x d" in hla.last_error()
    d = config(hla, 1024, 16, "dense")
    cache = fake_cache(hla, d, 400)
    st = hla.lib().hla_decode_step_static(ctypes.byref(d), ctypes.byref(cache), P, P, P, P, P, None, None, P, None)
    assert st == hla.HLA_ERR_WORKSPACE and "8-bit" not in hla.last_error()


def test_header_gives_the_8_bit_term():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "hla.h")) as f:
        text = " ".join(f.read().replace("\n *", " ").split())
    for call in ("hla_decode_step -- ", "hla_decode_step_static -- "):
        part = text[text.index(call):].split("*/")[0]
        assert "closing chunk's" in part, call
