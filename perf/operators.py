"""Measured cases of the serving operators: the gated delta rule with a carried state
(recurrent step, ragged chunked forward), the decode step over a chunk cache held in
8 bits, and the eviction of cached chunks by accumulated gate weight.

`own` false: every operator in plain torch operations, in float32 (float64 where
float32 loses what matters).  `own` true: the framework's calls on the same inputs.
"""
import math

import torch

own = False

F64, F32, I32 = torch.float64, torch.float32, torch.int32


# ---- cases ---------------------------------------------------------------------------


def listed():
    return [
        # one user of a chat model: a single token through one layer, where latency counts
        {"name": "step one sequence", "op": "step", "n": 1, "Hk": 16, "H": 16, "d": 128, "dtype": "bf16",
         "decay": "scalar", "pad": 0},
        # the 64-sequence decode batch of the repository's own benchmark, on recurrent states
        {"name": "step 64 sequences", "op": "step", "n": 64, "Hk": 16, "H": 16, "d": 128, "dtype": "bf16",
         "decay": "scalar", "pad": 0},
        # a padded batch of an odd size with shared key heads, float32 and a decay per channel
        {"name": "step 37 padded f32", "op": "step", "n": 37, "Hk": 2, "H": 6, "d": 64, "dtype": "f32",
         "decay": "channel", "pad": 5},
        # a scheduler's mixed batch: fresh prompts, continued ones, single tokens, an empty entry
        {"name": "forward ragged", "op": "forward", "lens": "1,63,0,64,65,129,200,7,333,1", "Hk": 8, "H": 16,
         "d": 128, "dtype": "bf16"},
        # a few sequences of the native delta-rule workload (4 x 4096 tokens, 16 heads)
        {"name": "forward 4 x 4096", "op": "forward", "lens": "4096,4096,4096,4096", "Hk": 16, "H": 16, "d": 128,
         "dtype": "bf16"},
        # one long prompt (16384 tokens, 16 heads): little parallel work, a long axis
        {"name": "forward 16384", "op": "forward", "lens": "16384", "Hk": 16, "H": 16, "d": 128, "dtype": "bf16"},
        # one sequence with a short context over the 8-bit chunk cache
        {"name": "decode8 one sequence", "op": "decode8", "B": 1, "H": 16, "n": 37, "C": 64, "d": 128,
         "dtype": "bf16", "bias": -2.0, "thr": 0.0},
        # a middling batch whose gates skip most chunks
        {"name": "decode8 8 sparse", "op": "decode8", "B": 8, "H": 16, "n": 500, "C": 64, "d": 128,
         "dtype": "bf16", "bias": -4.0, "thr": 0.05},
        # the 64 x 32768-token decode of the repository's benchmark, every chunk active
        {"name": "decode8 64 x 512 chunks", "op": "decode8", "B": 64, "H": 16, "n": 512, "C": 64, "d": 128,
         "dtype": "bf16", "bias": -2.0, "thr": 0.0},
        # gate weight of every chunk after a long prompt (131072 tokens, 32 heads)
        {"name": "mass 2048 chunks", "op": "mass", "B": 1, "H": 32, "T": 131072, "C": 64, "thr": 0.05},
        # a small cache trimmed while one sequence decodes
        {"name": "evict one sequence", "op": "evict", "B": 1, "H": 16, "n": 29, "keep": 21, "recent": 4, "d": 128,
         "dtype": "bf16"},
        # sixteen 32768-token caches cut down to their serving budget
        {"name": "evict 16 sequences", "op": "evict", "B": 16, "H": 16, "n": 512, "keep": 384, "recent": 32,
         "d": 128, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["step", "forward", "decode8", "mass", "evict"])
    if op == "step":
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 2, 3])
        n = _log_int(rng, 1, max(1, 4096 // H))
        return {"op": op, "n": n, "Hk": Hk, "H": H, "d": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "f32"]),
                "decay": rng.choice(["scalar", "channel"]), "pad": rng.randint(0, min(n - 1, 7))}
    if op == "forward":
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 2])
        dtype, d = rng.choice([("bf16", 128), ("bf16", 128), ("f32", 64), ("bf16", 64), ("f32", 128)])
        most = 8192 if dtype == "bf16" and d == 128 else 2048
        lens = [_log_int(rng, 1, most) for _ in range(_log_int(rng, 1, 24))]
        while len(lens) > 1 and (sum(lens) * H > 262144 or max(lens) * len(lens) * H > 1048576):
            lens.remove(max(lens))
        if rng.random() < 0.3:
            lens.insert(rng.randint(0, len(lens)), 0)
        return {"op": op, "lens": ",".join(map(str, lens)), "Hk": Hk, "H": H, "d": d, "dtype": dtype}
    if op == "decode8":
        d, dtype = rng.choice([(128, "bf16"), (128, "bf16"), (64, "bf16"), (64, "f32"), (128, "f32")])
        H = rng.choice([1, 2, 4, 8, 16, 32])
        n = _log_int(rng, 1, 700)
        B = _log_int(rng, 1, max(1, min(48, 131072 // (H * n))))
        # a threshold only where the output's type does not show a gate next to it
        thr = rng.choice([0.0, 0.05]) if dtype == "bf16" else 0.0
        return {"op": op, "B": B, "H": H, "n": n, "C": rng.choice([64, 64, 128, 256]), "d": d, "dtype": dtype,
                "bias": rng.choice([-4.0, -2.0, 0.0]), "thr": thr}
    if op == "mass":
        T = _log_int(rng, 100, 131072)
        return {"op": op, "B": rng.choice([1, 2, 3]), "H": rng.choice([1, 2, 4, 8]), "T": T,
                "C": rng.choice([64, 128, 256]), "thr": rng.choice([0.0, 0.05, 0.3])}
    n = _log_int(rng, 2, 600)
    H = rng.choice([1, 2, 4, 8, 16])
    keep = rng.randint(1, n)
    return {"op": op, "B": _log_int(rng, 1, max(1, min(16, 65536 // (H * n)))), "H": H, "n": n, "keep": keep,
            "recent": rng.randint(0, min(keep, 16)), "d": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "f32"])}


# ---- inputs --------------------------------------------------------------------------


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else F32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _tokens(g, rows, Hk, H, d, dtype, channel):
    """Queries and keys of unit length, values, decays near one and write strengths."""
    q = _unit(_randn(g, rows, Hk, d)).to(dtype)
    k = _unit(_randn(g, rows, Hk, d)).to(dtype)
    v = _randn(g, rows, H, d).to(dtype)
    shape = (rows, H, d) if channel else (rows, H)
    alpha = torch.exp(-torch.nn.functional.softplus(_randn(g, *shape) - 3.0))
    return q, k, v, alpha, torch.sigmoid(_randn(g, rows, H))


def _chunk_pool(g, count, d):
    """Transitions (A, B) of `count` chunks of 64 tokens, by the token rule."""
    A = torch.eye(d, device="cuda").repeat(count, 1, 1)
    B = torch.zeros(count, d, d, device="cuda")
    _, k, v, alpha, beta = _tokens(g, 64, count, count, d, F32, False)
    for t in range(64):
        kt, a, b = k[t][:, None, :], alpha[t][:, None, None], beta[t][:, None, None]
        A = a * (A - b * (A * kt).sum(-1, keepdim=True) * kt)
        B = a * (B - b * (B * kt).sum(-1, keepdim=True) * kt) + b * v[t][:, :, None] * kt
    return A, B


def _codes8(X):
    """8-bit codes of [count, d, d] matrices, one scale each."""
    s = X.abs().amax((1, 2)) / 127.0
    return torch.round(X / s[:, None, None]).to(torch.int8), s


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "op": case["op"]}
    {"step": _prepare_step, "forward": _prepare_forward, "decode8": _prepare_decode8, "mass": _prepare_mass,
     "evict": _prepare_evict}[case["op"]](case, g, s)
    return s


def _prepare_step(case, g, s):
    n, H, d = case["n"], case["H"], case["d"]
    s["q"], s["k"], s["v"], s["alpha"], s["beta"] = _tokens(g, n, case["Hk"], H, d, _dtype(case),
                                                            case["decay"] == "channel")
    slots = torch.randperm(n + 3, generator=g, device="cuda")[:n].to(I32)
    if case["pad"]:
        slots[n - case["pad"]:] = -1  # entries that fill the batch up
    s["slots"] = slots
    s["state"] = 0.3 * _randn(g, n + 3, H, d, d)
    s["o"] = torch.zeros_like(s["v"])
    if own:
        from gated_delta_rule_transitions_b200 import _hla as hla
        s["hla"] = hla
        s["cfg"] = hla.make_gdn_config(n, H, d, case["dtype"], Hk=case["Hk"], n_slots=n + 3, decay=case["decay"])


def _prepare_forward(case, g, s):
    lens = [int(x) for x in case["lens"].split(",")]
    n, T, H, d = len(lens), sum(lens), case["H"], case["d"]
    s["q"], s["k"], s["v"], s["alpha"], s["beta"] = _tokens(g, T, case["Hk"], H, d, _dtype(case), False)
    s["cu"] = torch.tensor([0] + lens, dtype=I32, device="cuda").cumsum(0, dtype=I32)
    s["longest"] = max(lens)
    s["state_in"] = 0.3 * _randn(g, n, H, d, d)
    s["state_out"] = torch.zeros_like(s["state_in"])
    s["o"] = torch.zeros_like(s["v"])
    if own:
        from gated_delta_rule_transitions_b200 import _hla as hla
        s["hla"] = hla
        s["cfg"] = hla.make_gdn_config(n, H, d, case["dtype"], Hk=case["Hk"], n_slots=n)
        s["ws"] = torch.empty(max(hla.gdn_workspace_bytes(s["cfg"], T), 256), dtype=torch.uint8, device="cuda")


def _prepare_decode8(case, g, s):
    B, H, n, C, d = case["B"], case["H"], case["n"], case["C"], case["d"]
    dt, mc = _dtype(case), case["n"] + 1
    A, Bm = _chunk_pool(g, 128, d)
    a = A.diagonal(dim1=1, dim2=2).mean(1)
    qa, sa = _codes8(A - a[:, None, None] * torch.eye(d, device="cuda"))
    qb, sb = _codes8(Bm)
    pick = torch.randint(128, (B, H, mc), generator=g, device="cuda")
    s["A8"] = qa.view(torch.int64)[pick].view(torch.int8)
    s["B8"] = qb.view(torch.int64)[pick].view(torch.int8)
    s["scales"] = torch.stack([a, sa, sb, torch.zeros_like(a)], 1)[pick].contiguous()
    s["rk"] = _randn(g, B, H, mc, 1, d)
    for name in ("buf_v", "buf_kr"):
        s[name] = _randn(g, B, H, C, d).to(dt)
    s["buf_k"] = _unit(_randn(g, B, H, C, d)).to(dt)
    centre = _randn(g, B, H, 1, d)
    s["buf_qr"] = (centre + 0.3 * _randn(g, B, H, C, d)).to(dt)
    s["buf_alpha"] = torch.exp(-torch.nn.functional.softplus(_randn(g, B, H, C) - 3.0))
    s["buf_beta"] = torch.sigmoid(_randn(g, B, H, C))
    b = torch.arange(B, device="cuda")
    # sequences of different lengths; no chunk closes in the pass
    s["counters0"] = torch.stack([(n - b * 5 % 8).clamp(min=0), (17 + 7 * b) % (C - 1)]).to(I32)
    s["counters"] = s["counters0"].clone()
    q, k, v, alpha, beta = _tokens(g, B, H, H, d, dt, False)
    s["q"], s["k"], s["v"], s["alpha"], s["beta"] = q, k, v, alpha, beta
    s["q_route"] = (centre[:, :, 0] + 0.3 * _randn(g, B, H, d)).to(dt)
    s["k_route"] = _randn(g, B, H, d).to(dt)
    s["o"] = torch.zeros_like(q)
    if own:
        from gated_delta_rule_transitions_b200 import _hla as hla
        s["hla"] = hla
        s["cfg"] = hla.make_config(B, H, 1, C, d, case["dtype"], bias=case["bias"], skip_threshold=case["thr"],
                                   cache_format="int8")
        s["cache"] = hla.Cache.from_tensors(s["cfg"], mc, A=s["A8"], Bm=s["B8"], df=s["scales"], rk=s["rk"],
                                            buf_k=s["buf_k"], buf_v=s["buf_v"], buf_qr=s["buf_qr"],
                                            buf_kr=s["buf_kr"], buf_alpha=s["buf_alpha"], buf_beta=s["buf_beta"],
                                            n_chunks=s["counters"][0], m_partial=s["counters"][1])
        s["ws"] = torch.empty(max(hla.decode_workspace_bytes(s["cfg"], mc), 256), dtype=torch.uint8, device="cuda")


def _prepare_mass(case, g, s):
    B, H, T, C = case["B"], case["H"], case["T"], case["C"]
    N = -(-T // C)
    # sigmoids around a bias: most weights small, a few near one; zero where j >= i
    gates = torch.sigmoid(1.5 * _randn(g, B, H, N, N) - 2.5)
    s["gates"] = gates.tril_(-1)
    s["mass"] = torch.zeros(B, H, N, device="cuda")
    if own:
        from gated_delta_rule_transitions_b200 import _hla as hla
        s["hla"] = hla
        s["cfg"] = hla.make_config(B, H, T, C, 128, "bf16", skip_threshold=case["thr"])


def _prepare_evict(case, g, s):
    B, H, n, keep, d = case["B"], case["H"], case["n"], case["keep"], case["d"]
    dt, C = _dtype(case), 64
    A, Bm = _chunk_pool(g, 64, d)
    pick = torch.randint(64, (B, H, n), generator=g, device="cuda")
    s["A"], s["Bm"] = A.to(dt)[pick], Bm.to(dt)[pick]
    s["rk"] = _randn(g, B, H, n, 1, d)
    # weights with a long tail, many of them equal
    s["mass"] = torch.floor(64.0 * _rand(g, B, H, n) ** 4) / 4.0
    b = torch.arange(B, device="cuda")
    s["n_chunks"] = (n - b * 3 % max(1, n // 4)).to(I32)
    s["m_partial"] = ((17 + 7 * b) % C).to(I32)
    for name in ("buf_k", "buf_v", "buf_qr", "buf_kr"):
        s[name] = _randn(g, B, H, C, d).to(dt)
    s["buf_alpha"], s["buf_beta"] = _rand(g, B, H, C), _rand(g, B, H, C)
    out = {"A": (keep, d, d), "Bm": (keep, d, d), "rk": (keep, 1, d), "mass": (keep,)}
    s["out"] = {k: torch.zeros(B, H, *v, dtype=s[k].dtype, device="cuda") for k, v in out.items()}
    for name in ("n_chunks", "m_partial", "buf_k", "buf_v", "buf_qr", "buf_kr", "buf_alpha", "buf_beta"):
        s["out"][name] = torch.zeros_like(s[name])
    s["out"]["kept"] = torch.zeros(B, H, keep, dtype=I32, device="cuda")
    if own:
        from gated_delta_rule_transitions_b200 import _hla as hla
        s["hla"] = hla
        s["cfg"] = hla.make_config(B, H, 1, C, d, case["dtype"])
        names = ("A", "Bm", "rk", "mass", "n_chunks", "m_partial", "buf_k", "buf_v", "buf_qr", "buf_kr",
                 "buf_alpha", "buf_beta")
        s["src"] = hla.Cache.from_tensors(s["cfg"], n, **{k: s[k] for k in names})
        s["dst"] = hla.Cache.from_tensors(s["cfg"], keep, **{k: s["out"][k] for k in names})


# ---- one pass ------------------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return {"step": _plain_step, "forward": _plain_forward, "decode8": _plain_decode8, "mass": _plain_mass,
            "evict": _plain_evict}[s["op"]](s)


def _own(s):
    hla, op = s["hla"], s["op"]
    if op == "step":
        hla.gdn_step(s["cfg"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["state"], s["o"], slots=s["slots"])
        return {"o": s["o"], "state": s["state"]}
    if op == "forward":
        hla.gdn_forward(s["cfg"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["cu"], s["o"],
                        state_in=s["state_in"], state_out=s["state_out"], workspace=s["ws"])
        return {"o": s["o"], "state": s["state_out"]}
    if op == "decode8":
        # a draft token is tried out: the open chunk starts from where it stood
        s["counters"].copy_(s["counters0"])
        hla.hla_decode_step(s["cfg"], s["cache"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["o"],
                            q_route=s["q_route"], k_route=s["k_route"], workspace=s["ws"])
        return _decode8_outputs(s)
    if op == "mass":
        hla.hla_gate_mass(s["cfg"], s["gates"], s["mass"])
        return {"mass": s["mass"]}
    hla.hla_cache_evict(s["cfg"], s["src"], s["dst"], s["case"]["keep"], s["case"]["recent"], s["out"]["kept"])
    return s["out"]


def _decode8_outputs(s):
    return {k: s[k] for k in ("o", "counters", "buf_k", "buf_v", "buf_qr", "buf_kr", "buf_alpha", "buf_beta")}


def _plain_step(s):
    rep = s["case"]["H"] // s["case"]["Hk"]
    q = s["q"].float().repeat_interleave(rep, 1)
    k = s["k"].float().repeat_interleave(rep, 1)
    n = s["case"]["n"] - s["case"]["pad"]
    at = s["slots"][:n].long()
    S = s["state"][at]
    alpha = s["alpha"][:n]
    S = S * (alpha[:, :, None, :] if alpha.dim() == 3 else alpha[:, :, None, None])
    u = s["beta"][:n, :, None] * (s["v"][:n].float() - (S @ k[:n, :, :, None])[..., 0])
    S = S + u[..., None] * k[:n, :, None, :]
    s["state"][at] = S
    s["o"][:n] = (S @ q[:n, :, :, None])[..., 0].to(s["o"].dtype)
    return {"o": s["o"], "state": s["state"]}


def _plain_forward(s):
    """Chunks of 64 tokens: all that does not need the state for every chunk at once,
    then one round of products per chunk."""
    case, cu, C = s["case"], s["cu"].long(), 64
    H, d, rep, T = case["H"], case["d"], case["H"] // case["Hk"], s["v"].shape[0]
    nc = -(-s["longest"] // C)
    t = torch.arange(nc * C, device="cuda")
    ok = t < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(ok, cu[:-1, None] + t, torch.zeros_like(t))
    n = ok.shape[0]

    def rows(x):  # [n, H, nc, C, ...] in float32, zero behind a sequence's end
        y = x[at].float() * ok.view(n, -1, *[1] * (x.dim() - 1))
        if y.shape[2] != H:
            y = y.repeat_interleave(rep, 2)
        return y.view(n, nc, C, *y.shape[2:]).transpose(2, 3).transpose(1, 2)

    q, k, v, beta = rows(s["q"]), rows(s["k"]), rows(s["v"]), rows(s["beta"])
    log_a = torch.where(ok[..., None], torch.log(s["alpha"][at].double()), 0.0)
    ell = log_a.view(n, nc, C, H).permute(0, 3, 1, 2).cumsum(-1)
    gamma = ell.exp().float()
    left = (ell[..., -1:] - ell).exp().float()
    decay = (ell[..., :, None] - ell[..., None, :]).tril().exp().float().tril()
    L = (beta[..., :, None] * decay * (k @ k.transpose(-1, -2))).tril(-1)
    # (I + L)^-1 = (I - L)(I + L^2)(I + L^4)...(I + L^32), since L^64 = 0
    eye = torch.eye(C, device="cuda")
    inv, P = eye - L, L
    for _ in range(5):
        P = P @ P
        inv = inv + inv @ P
    Tm = inv * beta[..., None, :]
    W, U = Tm @ (gamma[..., None] * k), Tm @ v
    QK = decay * (q @ k.transpose(-1, -2))
    qg, kl = gamma[..., None] * q, left[..., None] * k
    S = s["state_in"]
    o = torch.empty(n, H, nc, C, d, device="cuda")
    for c in range(nc):
        St = S.transpose(-1, -2)
        X = U[:, :, c] - W[:, :, c] @ St
        o[:, :, c] = qg[:, :, c] @ St + QK[:, :, c] @ X
        S = gamma[:, :, c, -1, None, None] * S + X.transpose(-1, -2) @ kl[:, :, c]
    s["state_out"].copy_(S)
    full = torch.empty(T + 1, H, d, dtype=s["o"].dtype, device="cuda")
    full[torch.where(ok, at, T)] = o.reshape(n, H, nc * C, d).transpose(1, 2).to(full.dtype)
    s["o"].copy_(full[:T])
    return {"o": s["o"], "state": s["state_out"]}


def _plain_decode8(s):
    case = s["case"]
    B, H, d = case["B"], case["H"], case["d"]
    b = torch.arange(B, device="cuda")
    n, m = s["counters0"].long()
    # append the token to the open chunk
    for buf, x in (("buf_k", "k"), ("buf_v", "v"), ("buf_qr", "q_route"), ("buf_kr", "k_route"),
                   ("buf_alpha", "alpha"), ("buf_beta", "beta")):
        s[buf][b, :, m] = s[x]
    s["counters"].copy_(s["counters0"])
    s["counters"][1] += 1
    # the open chunk, right to left: x = A_p q and y = B_p q
    x, y = s["q"].float(), torch.zeros(B, H, d, device="cuda")
    for t in range(case["C"] - 2, -1, -1):
        live = (t <= m).view(B, 1, 1)
        k, v = s["buf_k"][:, :, t].float(), s["buf_v"][:, :, t].float()
        w = s["buf_beta"][:, :, t, None] * (k * x).sum(-1, keepdim=True)
        y = torch.where(live, y + w * v, y)
        x = torch.where(live, s["buf_alpha"][:, :, t, None] * (x - w * k), x)
    # gates of the closed chunks, in 64 bits: a gate next to the threshold decides
    seen = (torch.arange(case["C"], device="cuda") <= m[:, None]).view(B, 1, -1, 1)
    rq = torch.where(seen, s["buf_qr"].double(), -torch.inf)
    rq = torch.logsumexp(rq, 2) - torch.log((m + 1).double()).view(B, 1, 1)
    z = (s["rk"][:, :, :, 0].double() @ rq[..., None])[..., 0] / math.sqrt(d) + case["bias"]
    gate = torch.sigmoid(z)
    keep = torch.arange(case["n"] + 1, device="cuda") < n.view(B, 1, 1)
    if case["thr"] > 0:
        keep = keep & (gate >= case["thr"])
    gate = torch.where(keep, gate, 0.0).float()
    for j in range(case["n"] - 1, -1, -1):
        g, sc = gate[:, :, j, None], s["scales"][:, :, j]
        bx = (s["B8"][:, :, j].float() @ x[..., None])[..., 0]
        ax = (s["A8"][:, :, j].float() @ x[..., None])[..., 0]
        y = y + g * sc[..., 2:3] * bx
        x = (1.0 - g) * x + g * (sc[..., 0:1] * x + sc[..., 1:2] * ax)
    s["o"].copy_(y)
    return _decode8_outputs(s)


def _plain_mass(s):
    case, g = s["case"], s["gates"]
    N = g.shape[-1]
    w = (case["T"] - case["C"] * torch.arange(N, device="cuda")).clamp(max=case["C"]).float()
    if case["thr"] > 0:
        g = torch.where(g >= case["thr"], g, 0.0)
    s["mass"].copy_((w @ g).view_as(s["mass"]))
    return {"mass": s["mass"]}


def _plain_evict(s):
    case, out = s["case"], s["out"]
    B, H, n, keep, recent = case["B"], case["H"], case["n"], case["keep"], case["recent"]
    j = torch.arange(n, device="cuda")
    nb = s["n_chunks"].long().view(B, 1, 1)
    score = torch.where(j >= nb - recent, torch.inf, s["mass"])
    score = torch.where(j < nb, score, -torch.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(best < nb, best, n).sort(-1).values
    ok = best < n
    at = best.clamp(max=n - 1)
    out["kept"].copy_(torch.where(ok, best, -1))
    for name in ("A", "Bm", "rk", "mass"):
        x = s[name].view(B, H, n, -1)
        y = out[name].view(B, H, keep, -1)
        y.copy_(torch.where(ok[..., None], torch.gather(x, 2, at[..., None].expand(-1, -1, -1, x.shape[-1])), y))
    out["n_chunks"].copy_(s["n_chunks"].clamp(max=keep))
    for name in ("m_partial", "buf_k", "buf_v", "buf_qr", "buf_kr", "buf_alpha", "buf_beta"):
        out[name].copy_(s[name])
    return out


# ---- what a pass cannot do without ---------------------------------------------------


def work(case):
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    op = case["op"]
    if op == "step":
        n, Hk, H, d = case["n"] - case["pad"], case["Hk"], case["H"], case["d"]
        a = 4 * (d if case["decay"] == "channel" else 1)
        return {"bytes": n * (H * (8 * d * d + 2 * d * es + a + 4) + 2 * Hk * d * es), "flops": 7 * n * H * d * d}
    if op == "forward":
        lens = [int(x) for x in case["lens"].split(",")]
        T, Hk, H, d = sum(lens), case["Hk"], case["H"], case["d"]
        return {"bytes": T * (2 * Hk * d * es + 2 * H * d * es + 8 * H) + len(lens) * H * 8 * d * d,
                "flops": 7 * T * H * d * d}
    if op == "decode8":
        B, H, n, d, C = case["B"], case["H"], case["n"], case["d"], case["C"]
        # share of chunks whose gate passes: scores are near N(bias, 1.04)
        share = 1.0
        if case["thr"] > 0:
            cut = (math.log(case["thr"] / (1 - case["thr"])) - case["bias"]) / 1.04
            share = 0.5 * math.erfc(cut / math.sqrt(2))
        chunks = B * H * n
        return {"bytes": chunks * (4 * d + share * (2 * d * d + 16)) + B * H * (C // 2) * (3 * d * es + 8),
                "flops": chunks * (2 * d + share * 4 * d * d)}
    if op == "mass":
        N = -(-case["T"] // case["C"])
        return {"bytes": case["B"] * case["H"] * (N * (N - 1) // 2 + N) * 4,
                "flops": case["B"] * case["H"] * N * (N - 1)}
    B, H, n, keep, d = case["B"], case["H"], case["n"], case["keep"], case["d"]
    return {"bytes": B * H * (2 * keep * (2 * d * d * es + 4 * d + 4) + 4 * n + 2 * 64 * (4 * d * es + 8)),
            "flops": B * H * n}


# ---- the definitions in 64 bits ------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "forward": _exact_forward, "decode8": _exact_decode8, "mass": _exact_mass,
            "evict": _exact_evict}[case["op"]](case, s)


def _token(S, q, k, v, a, b):
    """One token of the rule on [.., H, dv, dk] states in 64 bits."""
    S = S * a
    S = S + torch.einsum("...hv,...hk->...hvk", b[..., None] * (v - torch.einsum("...hvk,...hk->...hv", S, k)), k)
    return S, torch.einsum("...hvk,...hk->...hv", S, q)


def _exact_step(case, s):
    n, rep = case["n"] - case["pad"], case["H"] // case["Hk"]
    state, o = s["state"].double(), s["o"].double()
    at = s["slots"][:n].long()
    q, k = (s[x][:n].double().repeat_interleave(rep, 1) for x in ("q", "k"))
    a = s["alpha"][:n].double()
    a = a[:, :, None, :] if a.dim() == 3 else a[:, :, None, None]
    state[at], o[:n] = _token(state[at], q, k, s["v"][:n].double(), a, s["beta"][:n].double())
    return {"o": o, "state": state}


def _exact_forward(case, s):
    rep, cu = case["H"] // case["Hk"], s["cu"].tolist()
    o, S = s["o"].double(), s["state_in"].double()
    q, k, v, a, b = (s[x].double() for x in ("q", "k", "v", "alpha", "beta"))
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    for t in range(s["longest"]):
        who = [i for i in range(len(cu) - 1) if cu[i] + t < cu[i + 1]]
        row = torch.tensor([cu[i] + t for i in who], device="cuda")
        seq = torch.tensor(who, device="cuda")
        new, out = _token(S[seq], q[row], k[row], v[row], a[row][..., None, None], b[row])
        S[seq] = new
        o[row] = out
    return {"o": o, "state": S}


def _exact_decode8(case, s):
    B, H, n, d = case["B"], case["H"], case["n"], case["d"]
    nb, mb = s["counters0"].tolist()
    out = {k: v.clone() for k, v in _decode8_outputs(s).items()}
    out["counters"] = s["counters0"] + torch.tensor([[0], [1]], dtype=I32, device="cuda")
    for buf, x in (("buf_k", "k"), ("buf_v", "v"), ("buf_qr", "q_route"), ("buf_kr", "k_route"),
                   ("buf_alpha", "alpha"), ("buf_beta", "beta")):
        for i in range(B):
            out[buf][i, :, mb[i]] = s[x][i]
    # forward form: compose the gated transitions, then the open chunk's tokens
    gates = []
    for i in range(B):
        m = mb[i] + 1
        rq = out["buf_qr"][i, :, :m].double().exp().mean(1).log()
        g = 1.0 / (1.0 + torch.exp(-(s["rk"][i, :, :, 0].double() * rq[:, None]).sum(-1) / d ** 0.5 - case["bias"]))
        g[:, nb[i]:] = 0.0
        if case["thr"] > 0:
            g[g < case["thr"]] = 0.0
        gates.append(g)
    gates = torch.stack(gates)
    S = torch.zeros(B, H, d, d, dtype=F64, device="cuda")
    eye = torch.eye(d, dtype=F64, device="cuda")
    for j in range(n):
        sc = s["scales"][:, :, j].double()[..., None]
        A = sc[:, :, 0:1] * eye + sc[:, :, 1:2] * s["A8"][:, :, j].double()
        g = gates[:, :, j, None, None]
        S = S + g * (S @ A + sc[:, :, 2:3] * s["B8"][:, :, j].double() - S)
    o = torch.zeros(B, H, d, dtype=F64, device="cuda")
    for i in range(B):
        Si = S[i]
        for t in range(mb[i] + 1):
            Si, o[i] = _token(Si, s["q"][i].double(), out["buf_k"][i, :, t].double(), out["buf_v"][i, :, t].double(),
                              out["buf_alpha"][i, :, t].double()[:, None, None], out["buf_beta"][i, :, t].double())
    out["o"] = o
    return {k: v.double() if v.is_floating_point() else v for k, v in out.items()}


def _exact_mass(case, s):
    g = s["gates"]
    mass = torch.zeros(g.shape[:3], dtype=F64, device="cuda")
    for i in range(g.shape[2]):
        row = g[:, :, i, :i].double()
        if case["thr"] > 0:
            row = row * (g[:, :, i, :i] >= case["thr"])
        mass[:, :, :i] += min(case["C"], case["T"] - i * case["C"]) * row
    return {"mass": mass}


def _exact_evict(case, s):
    if case["B"] * case["H"] * case["keep"] * case["d"] ** 2 > 1 << 28:
        return None
    out = {k: v.clone() for k, v in s["out"].items()}
    mass, nb = s["mass"].tolist(), s["n_chunks"].tolist()
    for i in range(case["B"]):
        n = nb[i]
        for h in range(case["H"]):
            kept = list(range(n))
            if n > case["keep"]:
                old = sorted(range(n - case["recent"]), key=lambda j: (-mass[i][h][j], j))
                kept = sorted(old[:case["keep"] - case["recent"]]) + list(range(n - case["recent"], n))
            at = torch.tensor(kept, device="cuda", dtype=torch.long)
            out["kept"][i, h] = -1
            out["kept"][i, h, :len(kept)] = at.to(I32)
            for name in ("A", "Bm", "rk", "mass"):
                out[name][i, h, :len(kept)] = s[name][i, h, at]
        out["n_chunks"][i] = min(n, case["keep"])
    for name in ("m_partial", "buf_k", "buf_v", "buf_qr", "buf_kr", "buf_alpha", "buf_beta"):
        out[name] = s[name]
    return {k: v.double() if v.is_floating_point() else v for k, v in out.items()}
