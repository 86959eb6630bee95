"""The gated delta rule with a carried state (gdn_step, gdn_forward) against its definition
in 64 bits.

Tolerances.  Every token's update of a state row is a float32 dot product of d terms and a
rank-one correction: with d / 8 terms in sequence and a handful of operations more it is off
by less than (d / 8 + 8) 2^-24 of the row's size, and the rule contracts what it carries, so
T tokens add up to at most min(T, 64) such errors (alpha averages 0.95: an error's weight
after 64 tokens is below 4 %).  For the tensor-core form (bf16, d = 128) 2e-5 is asked for:
with each factor of its products as two bf16 numbers, each product is off by at most 2 x 2^-17
relative, at most six products stand between a state and the next, which makes 12 x 2^-17 =
9.2e-5 for one chunk if every error pointed the same way, and rounding errors of independent
elements add as their root (the kernels take three parts).  An output is rounded once to its type on top."""
import pytest
import torch

from tests import _serving as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hla():
    import gated_delta_rule_transitions_b200 as m
    m.lib()
    return m._hla


def state_tol(T, d, dtype, chunked):
    f32 = min(T, 64) * (d / 8 + 8) * 2.0 ** -24
    return max(f32, 2e-5) if chunked else f32


def cuda(*xs):
    return [x.cuda() for x in xs]


@pytest.mark.parametrize("n,Hk,H,d,dtype,channel", [
    (1, 1, 1, 128, "bf16", False), (1, 16, 16, 128, "bf16", False), (5, 2, 6, 128, "f32", False),
    (3, 1, 3, 64, "bf16", True), (40, 4, 16, 128, "bf16", True), (41, 8, 8, 64, "f32", False),
    (2, 2, 2, 128, "f32", True), (70, 2, 4, 64, "f32", True),
])
def test_step(hla, n, Hk, H, d, dtype, channel):
    gen = torch.Generator().manual_seed(n * 1000 + H)
    dt = R.DT[dtype]
    q, k, v, al, be = R.tokens(gen, n, Hk, H, d, dt, channel)
    S0 = 0.3 * torch.randn(n, H, d, d, generator=gen)
    cfg = hla.make_gdn_config(n, H, d, dtype, Hk=Hk, decay="channel" if channel else "scalar")
    S, o = S0.cuda(), torch.zeros(n, H, d, dtype=dt, device="cuda")
    hla.gdn_step(cfg, *cuda(q, k, v, al, be), S, o)
    ro, rS = R.gdn_reference(q, k, v, al, be, [(i, i + 1) for i in range(n)], S0)
    tol = state_tol(1, d, dt, False)
    assert R.rel(S.cpu(), rS) <= tol
    assert R.rel(o.cpu(), ro) <= tol + R.half_step(dt)
    assert hla.hla_device_status() == (0, 0)


LENS = [[1], [63], [64], [65], [130], [1, 0, 64, 3, 127, 128, 129, 0, 40], [0, 5], [333, 2], [200] * 3]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("Hk,H,d,dtype,channel", [
    (2, 4, 128, "bf16", False), (1, 1, 128, "bf16", False), (2, 2, 128, "bf16", True), (1, 3, 64, "bf16", False),
    (2, 2, 128, "f32", False), (1, 2, 64, "f32", True),
])
def test_forward(hla, lens, Hk, H, d, dtype, channel):
    gen = torch.Generator().manual_seed(sum(lens) * 7 + H)
    dt, T, n = R.DT[dtype], sum(lens) + 3, len(lens)  # three rows belong to no sequence
    q, k, v, al, be = R.tokens(gen, T, Hk, H, d, dt, channel)
    # what stands behind the last sequence is no number
    for x in (q, k, v, al, be):
        x[sum(lens):] = float("nan")
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    slots = torch.randperm(n + 2, generator=gen)[:n].to(torch.int32)
    S0 = 0.3 * torch.randn(n + 2, H, d, d, generator=gen)
    cfg = hla.make_gdn_config(n, H, d, dtype, Hk=Hk, n_slots=n + 2, decay="channel" if channel else "scalar")
    o = torch.full((T, H, d), 7.0, dtype=dt, device="cuda")
    Sin, Sout = S0.cuda(), torch.full((n + 2, H, d, d), 5.0, device="cuda")
    dev = cuda(q, k, v, al, be, cu)
    hla.gdn_forward(cfg, *dev, o, state_in=Sin, state_out=Sout, slots=slots.cuda())
    bounds = [(int(cu[i]), int(cu[i + 1])) for i in range(n)]
    ro, rS = R.gdn_reference(q, k, v, al, be, bounds, S0[slots.long()])
    tol = state_tol(max(lens), d, dt, dtype == "bf16" and d == 128 and not channel)
    got = Sout.cpu()
    for i, s in enumerate(slots.tolist()):
        if lens[i] == 0:
            assert torch.equal(got[s], S0[s])
        else:
            assert R.rel(got[s], rS[i]) <= tol, (i, lens[i])
    other = [s for s in range(n + 2) if s not in slots.tolist()]
    assert torch.equal(got[other], torch.full_like(got[other], 5.0))
    end = sum(lens)
    for i, (a, e) in enumerate(bounds):
        if e > a:
            assert R.rel(o[a:e].cpu(), ro[a:e]) <= tol + R.half_step(dt), (i, lens[i])
    assert torch.equal(o[end:].cpu(), torch.full_like(o[end:].cpu(), 7.0))
    # in place, twice: the same bits both times
    again = []
    for _ in range(2):
        S, o2 = S0.cuda(), torch.full_like(o, 7.0)
        hla.gdn_forward(cfg, *dev, o2, state_in=S, state_out=S, slots=slots.cuda())
        again.append((S, o2))
        assert torch.equal(S[slots.long()], Sout[slots.long()]) and torch.equal(o2, o)
    assert torch.equal(again[0][0], again[1][0])
    assert hla.hla_device_status() == (0, 0)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_zero_state_and_no_state_out(hla, dtype, d):
    gen = torch.Generator().manual_seed(3)
    dt, T, H = R.DT[dtype], 150, 2
    args = cuda(*R.tokens(gen, T, H, H, d, dt))
    cu = torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    cfg = hla.make_gdn_config(2, H, d, dtype)
    zero = torch.zeros(2, H, d, d, device="cuda")
    o1, o2, S = torch.empty_like(args[2]), torch.empty_like(args[2]), torch.empty_like(zero)
    hla.gdn_forward(cfg, *args, cu, o1, state_in=zero, state_out=S)
    hla.gdn_forward(cfg, *args, cu, o2)
    assert torch.equal(o1, o2)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("bf16", 64)])
def test_split_prompt_and_steps_agree_with_one_call(hla, dtype, d):
    """A prompt in pieces (state carried by the caller), then token by token: the same
    states as in one call."""
    gen = torch.Generator().manual_seed(11)
    dt, T, H = R.DT[dtype], 229, 3
    q, k, v, al, be = cuda(*R.tokens(gen, T, H, H, d, dt))
    cfg = hla.make_gdn_config(1, H, d, dtype)
    bounds = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    o, S = torch.empty_like(v), torch.zeros(1, H, d, d, device="cuda")
    hla.gdn_forward(cfg, q, k, v, al, be, bounds(T), o, state_in=S, state_out=S)
    o2, S2 = torch.empty_like(v), torch.zeros(1, H, d, d, device="cuda")
    for a, e in ((0, 100), (100, 101), (101, 220)):
        part = o2[a:e].contiguous()
        hla.gdn_forward(cfg, *(x[a:e].contiguous() for x in (q, k, v, al, be)), bounds(e - a), part, state_in=S2,
                        state_out=S2)
        o2[a:e] = part
    for t in range(220, T):
        hla.gdn_step(cfg, *(x[t:t + 1].contiguous() for x in (q, k, v, al, be)), S2, o2[t:t + 1])
    tol = 2 * state_tol(T, d, dt, dtype == "bf16" and d == 128)
    assert R.rel(S2, S) <= tol
    assert R.rel(o2, o) <= tol + 2 * R.half_step(dt)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_padding_bad_slots_and_bad_bounds_are_left_out(hla, dtype, d):
    """Slots below zero are padding; a slot out of range or twice, and bounds outside the
    tokens, leave their sequence out and are reported; the others are not touched by it."""
    gen = torch.Generator().manual_seed(5)
    dt, H, n = R.DT[dtype], 2, 6
    q, k, v, al, be = R.tokens(gen, n, H, H, d, dt)
    S0 = torch.randn(4, H, d, d, generator=gen)
    slots = torch.tensor([2, -1, 0, 2, 9, 1], dtype=torch.int32)  # 3: slot twice, 4: out of range
    cfg = hla.make_gdn_config(n, H, d, dtype, n_slots=4)
    S, o = S0.cuda(), torch.full((n, H, d), 7.0, dtype=dt, device="cuda")
    hla.gdn_step(cfg, *cuda(q, k, v, al, be), S, o, slots=slots.cuda())
    st, code = hla.hla_device_status()
    assert st == hla.HLA_ERR_INVALID_ARG and code == 16
    good = [0, 2, 5]
    ro, rS = R.gdn_reference(*(x[good] for x in (q, k, v, al, be)), [(i, i + 1) for i in range(3)],
                             S0[slots[good].long()])
    tol = state_tol(1, d, dt, False)
    assert R.rel(S.cpu()[slots[good].long()], rS) <= tol and torch.equal(S.cpu()[3], S0[3])
    assert R.rel(o.cpu()[good], ro) <= tol + R.half_step(dt)
    assert torch.equal(o.cpu()[[1, 3, 4]], torch.full((3, H, d), 7.0, dtype=dt))
    # bounds: the second sequence's run backwards, the third's leave the tokens
    T = 200
    q, k, v, al, be = R.tokens(gen, T, H, H, d, dt)
    cu = torch.tensor([0, 120, 90, 150, 300], dtype=torch.int32)
    cfg = hla.make_gdn_config(4, H, d, dtype)
    S, o = S0.cuda(), torch.full((T, H, d), 7.0, dtype=dt, device="cuda")
    hla.gdn_forward(cfg, *cuda(q, k, v, al, be, cu), o, state_in=S, state_out=S)
    st, code = hla.hla_device_status()
    assert st == hla.HLA_ERR_INVALID_ARG and code == 16
    ro, rS = R.gdn_reference(q, k, v, al, be, [(0, 120)], S0[:1])
    tol = state_tol(120, d, dt, dtype == "bf16" and d == 128)
    assert R.rel(S.cpu()[:1], rS) <= tol and torch.equal(S.cpu()[[1, 3]], S0[[1, 3]])
    assert R.rel(o.cpu()[:90], ro[:90]) <= tol + R.half_step(dt)
    assert torch.equal(o.cpu()[150:], torch.full((50, H, d), 7.0, dtype=dt))
    assert hla.hla_device_status() == (0, 0)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_extreme_decays_and_writes(hla, dtype, d):
    """Decays of exactly one, exactly zero and far below; writes of zero and one."""
    gen = torch.Generator().manual_seed(8)
    dt, T, H = R.DT[dtype], 140, 2
    q, k, v, al, be = R.tokens(gen, T, H, H, d, dt)
    al[::3], be[::5], be[1::5] = 1.0, 0.0, 1.0
    al[40], al[41], al[100, 0], al[130] = 0.0, 1e-30, 1e-3, 0.5
    cu = torch.tensor([0, T], dtype=torch.int32)
    S0 = torch.randn(1, H, d, d, generator=gen)
    cfg = hla.make_gdn_config(1, H, d, dtype)
    S, o = S0.cuda(), torch.empty(T, H, d, dtype=dt, device="cuda")
    hla.gdn_forward(cfg, *cuda(q, k, v, al, be, cu), o, state_in=S, state_out=S)
    ro, rS = R.gdn_reference(q, k, v, al, be, [(0, T)], S0)
    tol = state_tol(T, d, dt, dtype == "bf16" and d == 128)
    assert R.rel(S.cpu(), rS) <= tol and R.rel(o.cpu(), ro) <= tol + R.half_step(dt)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_repeated_keys(hla, dtype, d):
    """Every token writes to the same key (the triangular system at its stiffest)."""
    gen = torch.Generator().manual_seed(9)
    dt, T, H = R.DT[dtype], 192, 1
    q, k, v, al, be = R.tokens(gen, T, H, H, d, dt)
    k[:] = k[:1]
    be[:] = 0.95
    al[:] = 0.999
    cu = torch.tensor([0, T], dtype=torch.int32)
    S0 = torch.randn(1, H, d, d, generator=gen)
    cfg = hla.make_gdn_config(1, H, d, dtype)
    S, o = S0.cuda(), torch.empty(T, H, d, dtype=dt, device="cuda")
    hla.gdn_forward(cfg, *cuda(q, k, v, al, be, cu), o, state_in=S, state_out=S)
    ro, rS = R.gdn_reference(q, k, v, al, be, [(0, T)], S0)
    tol = state_tol(T, d, dt, dtype == "bf16" and d == 128)
    assert R.rel(S.cpu(), rS) <= tol and R.rel(o.cpu(), ro) <= tol + R.half_step(dt)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_captured_and_side_stream(hla, dtype, d):
    """Captured into a graph and replayed on new inputs, and on a stream of its own."""
    gen = torch.Generator().manual_seed(21)
    dt, T, H = R.DT[dtype], 300, 2
    toks = [cuda(*R.tokens(gen, T, H, H, d, dt)) for _ in range(2)]
    cu = torch.tensor([0, 130, 300], dtype=torch.int32, device="cuda")
    cfg = hla.make_gdn_config(2, H, d, dtype)
    ws = torch.empty(hla.gdn_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")

    def eager(tok):
        S, o = torch.zeros(2, H, d, d, device="cuda"), torch.empty_like(tok[2])
        hla.gdn_forward(cfg, *tok, cu, o, state_out=S, workspace=ws)
        o1 = torch.empty_like(tok[2][:2])
        hla.gdn_step(cfg, *(x[:2].contiguous() for x in tok), S, o1)
        return o, S, o1

    want = [eager(t) for t in toks]
    torch.cuda.synchronize()
    buf = [x.clone() for x in toks[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = eager(buf)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = eager(buf)
    for i in (1, 0):
        for b, x in zip(buf, toks[i]):
            b.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))


def test_two_calls_on_two_streams(hla):
    """Two calls at once, each with a workspace and states of its own."""
    gen = torch.Generator().manual_seed(4)
    T, H, d = 700, 4, 128
    cfg = hla.make_gdn_config(1, H, d, "bf16")
    toks = [cuda(*R.tokens(gen, T, H, H, d, R.BF16)) for _ in range(2)]
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")

    def call(tok, stream=None):
        S, o = torch.zeros(1, H, d, d, device="cuda"), torch.empty_like(tok[2])
        ws = torch.empty(hla.gdn_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for _ in range(3):
            hla.gdn_forward(cfg, *tok, cu, o, state_out=S, workspace=ws, stream=stream)
        return o, S, ws

    want = [call(t) for t in toks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [call(t, s) for t, s in zip(toks, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("n,H,Hk", [(24, 4, 2), (7, 4, 4), (3, 16, 8), (40, 8, 8)])
def test_many_sequences_of_mixed_lengths(hla, n, H, Hk):
    """The chunked form over one to many CTAs per SM (16, 32 and 64 value columns per CTA,
    longest sequences first), padded entries and a slot twice among them."""
    gen = torch.Generator().manual_seed(n)
    lens = [int(x) for x in torch.randint(1, 260, (n,), generator=gen)]
    lens[0], lens[n // 2] = 300, 0
    T, d = sum(lens), 128
    q, k, v, al, be = R.tokens(gen, T, Hk, H, d, R.BF16)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    slots = torch.randperm(n, generator=gen).to(torch.int32)
    slots[1] = -1
    if n > 10:
        slots[9] = slots[4]
    live = [i for i in range(n) if i != 1 and not (n > 10 and i == 9)]
    S0 = torch.randn(n, H, d, d, generator=gen)
    cfg = hla.make_gdn_config(n, H, d, "bf16", Hk=Hk, n_slots=n)
    S, o = S0.cuda(), torch.full((T, H, d), 7.0, dtype=R.BF16, device="cuda")
    hla.gdn_forward(cfg, *cuda(q, k, v, al, be, cu), o, state_in=S, state_out=S, slots=slots.cuda())
    bounds = [(int(cu[i]), int(cu[i + 1])) for i in live]
    ro, rS = R.gdn_reference(q, k, v, al, be, bounds, S0[slots[live].long()])
    tol = state_tol(300, d, R.BF16, True)
    got, o = S.cpu(), o.cpu()
    for i, (a, e) in enumerate(bounds):
        assert R.rel(got[int(slots[live[i]])], rS[i]) <= tol, i
        if e > a:
            assert R.rel(o[a:e], ro[a:e]) <= tol + R.half_step(R.BF16), i
    for i in set(range(n)) - set(live):
        assert torch.equal(o[int(cu[i]):int(cu[i + 1])], torch.full_like(o[int(cu[i]):int(cu[i + 1])], 7.0))
    st, code = hla.hla_device_status()
    assert code == (16 if n > 10 else 0)


MIXED = [[1] * 40 + [300], [1] * 31 + [200, 0, 65], [36, 37, 32, 33, 64, 65, 1, 128, 0, 31, 97, 38],
         [40] * 12, [30] * 20, [700] + [2] * 70, [1] * 511 + [129], [1] * 512 + [30000 // 16], [5, 400] * 9]


@pytest.mark.parametrize("lens", MIXED, ids=lambda x: f"{len(x)}x{max(x)}")
def test_prompts_among_short_sequences(hla, lens):
    """Batches that rows and chunks share: a prompt among single tokens, lengths on either side
    of the kernels' border, all short, all long, as many sequences as are ranked and one more;
    two calls and a step between them in place on one workspace, the second call replayed."""
    gen = torch.Generator().manual_seed(len(lens))
    n, T, d = len(lens), sum(lens), 128
    H, Hk = (4, 2) if n < 100 else (1, 1)
    cfg = hla.make_gdn_config(n, H, d, "bf16", Hk=Hk)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    S0 = torch.randn(n, H, d, d, generator=gen)
    parts = [R.tokens(gen, T, Hk, H, d, R.BF16), R.tokens(gen, n, Hk, H, d, R.BF16), R.tokens(gen, T, Hk, H, d, R.BF16)]
    dev, S = [cuda(*p) for p in parts], S0.cuda()
    outs = [torch.full((p[2].shape[0] + 3, H, d), 7.0, dtype=R.BF16, device="cuda") for p in parts]
    cud, ws = cu.cuda(), torch.empty(hla.gdn_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    fwd = lambda i: hla.gdn_forward(cfg, *dev[i], cud, outs[i][:T], state_in=S, state_out=S, workspace=ws)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd(0)
        S.copy_(S0)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        fwd(2)
    fwd(0)
    hla.gdn_step(cfg, *dev[1], S, outs[1][:n])
    graph.replay()
    torch.cuda.synchronize()
    assert hla.hla_device_status() == (0, 0)
    bounds = [(int(cu[i]), int(cu[i + 1])) for i in range(n)]
    ref = S0
    for p, o, b in zip(parts, outs, (bounds, [(i, i + 1) for i in range(n)], bounds)):
        ro, ref = R.gdn_reference(*p, b, ref)
        o = o.cpu()
        for i, (a, e) in enumerate(b):
            if e > a:
                assert R.rel(o[a:e], ro[a:e]) <= 2 * state_tol(max(lens), d, R.BF16, True) + R.half_step(R.BF16), i
        assert torch.equal(o[b[-1][1]:], torch.full_like(o[b[-1][1]:], 7.0))
    tol = 3 * state_tol(max(lens), d, R.BF16, True)
    for i in range(n):
        assert R.rel(S[i].cpu(), ref[i]) <= tol, i


def test_bad_bounds_in_a_shared_batch(hla):
    """Bounds that run backwards or leave the tokens among prompts and single tokens: their
    sequences are left out and reported, the others are worked on."""
    gen = torch.Generator().manual_seed(9)
    T, H, d = 400, 2, 128
    cu = torch.tensor([0, 1, 101, 102, 99, 140, 240, 241, 2 ** 30, 2 ** 30 + 50, 300, 301], dtype=torch.int32)
    n = len(cu) - 1
    q, k, v, al, be = R.tokens(gen, T, H, H, d, R.BF16)
    S0 = torch.randn(n, H, d, d, generator=gen)
    S, o = S0.cuda(), torch.full((T, H, d), 7.0, dtype=R.BF16, device="cuda")
    hla.gdn_forward(hla.make_gdn_config(n, H, d, "bf16"), *cuda(q, k, v, al, be, cu), o, state_in=S, state_out=S)
    st, code = hla.hla_device_status()
    assert st == hla.HLA_ERR_INVALID_ARG and code == 16
    S = S.cpu()
    for i in (0, 1, 5, 6, 10):
        a, e = int(cu[i]), int(cu[i + 1])
        ro, rS = R.gdn_reference(q, k, v, al, be, [(a, e)], S0[i:i + 1])
        assert R.rel(S[i], rS[0]) <= state_tol(100, d, R.BF16, True), i
    for i in (3, 7, 8, 9):
        assert torch.equal(S[i], S0[i])
    assert torch.equal(o[301:].cpu(), torch.full((99, H, d), 7.0, dtype=R.BF16))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("lens", [[100, 70, 200], [3, 1, 300, 1, 40, 5, 90, 36]], ids=str)
def test_nan_of_one_sequence_stays_there(hla, lens, dtype, d):
    """Tokens and state of every other sequence are NaN: the rest does not see them, though
    tiles of 64 tokens reach over a sequence's end."""
    gen, dt, H = torch.Generator().manual_seed(3), R.DT[dtype], 2
    n, T = len(lens), sum(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    x = R.tokens(gen, T, H, H, d, dt)
    S0 = torch.randn(n, H, d, d, generator=gen)
    for i in range(1, n, 2):
        for t in x:
            t[int(cu[i]):int(cu[i + 1])] = float("nan")
        S0[i] = float("nan")
    S, o = S0.cuda(), torch.empty(T, H, d, dtype=dt, device="cuda")
    hla.gdn_forward(hla.make_gdn_config(n, H, d, dtype), *cuda(*x, cu), o, state_in=S, state_out=S)
    assert hla.hla_device_status() == (0, 0)
    tol = state_tol(max(lens), d, dt, dtype == "bf16" and d == 128)
    for i in range(n):
        a, e = int(cu[i]), int(cu[i + 1])
        if i % 2:
            assert bool(S[i].isnan().all()) and bool(o[a:e].isnan().all())
        else:
            ro, rS = R.gdn_reference(*x, [(a, e)], S0[i:i + 1])
            assert R.rel(S[i].cpu(), rS[0]) <= tol and R.rel(o[a:e].cpu(), ro[a:e]) <= tol + R.half_step(dt)


def test_agrees_with_the_gated_composition_of_weight_one(hla):
    """HLA with every gate one is the rule itself: the prompt's outputs by gdn_forward and by
    hla_prefill, then tokens by gdn_step from the state and by hla_decode_step over the cached
    transitions, both to the composition's own bar (bf16 transitions: relative L2 2e-2)."""
    import hla_synth as syn
    w = syn.GDN_REDUCTION.with_(B=1, H=2, T=64 * 5 + 9)
    inp = {k: v.cuda() for k, v in syn.make_gdn_inputs(w).items()}
    H, d = 2, 128
    mk = lambda T: hla.make_config(1, H, T, 64, d, "bf16", "one")
    cache = hla.Cache(mk(w.T), 8)
    o1, o2 = torch.empty_like(inp["q"]), torch.empty_like(inp["q"])
    hla.hla_prefill(mk(w.T), inp["q"], inp["k"], inp["v"], inp["alpha"], inp["beta"], o1, cache=cache)
    cfg = hla.make_gdn_config(1, H, d, "bf16")
    S = torch.zeros(1, H, d, d, device="cuda")
    cu = torch.tensor([0, w.T], dtype=torch.int32, device="cuda")
    rows = {k: inp[k][0].contiguous() for k in inp}
    hla.gdn_forward(cfg, rows["q"], rows["k"], rows["v"], rows["alpha"], rows["beta"], cu, o2[0], state_in=S,
                    state_out=S)
    for h in range(H):
        assert R.rel(o1[0, :, h], o2[0, :, h]) <= 2e-2
    for tok in syn.make_decode_tokens(w, 3):
        t = {k: v.cuda() for k, v in tok.items()}
        a, b = torch.empty_like(t["q"]), torch.empty_like(t["q"])
        hla.hla_decode_step(mk(1), cache, t["q"], t["k"], t["v"], t["alpha"], t["beta"], a)
        hla.gdn_step(cfg, t["q"], t["k"], t["v"], t["alpha"], t["beta"], S, b)
        for h in range(H):
            assert R.rel(a[0, h], b[0, h]) <= 2e-2
    assert hla.hla_device_status() == (0, 0)


def test_binding_refuses_wrong_sizes_and_types(hla):
    gen = torch.Generator().manual_seed(1)
    q, k, v, al, be = cuda(*R.tokens(gen, 2, 1, 2, 64, R.BF16))
    cfg = hla.make_gdn_config(2, 2, 64, "bf16", Hk=1)
    S, o = torch.zeros(2, 2, 64, 64, device="cuda"), torch.empty_like(v)
    with pytest.raises(ValueError, match="q: expected"):
        hla.gdn_step(cfg, v, k, v, al, be, S, o)
    with pytest.raises(TypeError, match="state"):
        hla.gdn_step(cfg, q, k, v, al, be, S.bfloat16(), o)
    with pytest.raises(ValueError, match="contiguous"):
        hla.gdn_step(cfg, q, k, v.transpose(0, 1).contiguous().transpose(0, 1), al, be, S, o)
    with pytest.raises(TypeError, match="slots"):
        hla.gdn_step(cfg, q, k, v, al, be, S, o, slots=torch.zeros(2, device="cuda"))
    ws = torch.empty(128, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    with pytest.raises(hla.HlaError, match="workspace"):
        hla.gdn_forward(cfg, q, k, v, al, be, cu, o, workspace=ws)
