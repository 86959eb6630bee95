"""Plain 64-bit references of the serving operators (carried-state gated delta rule, decode
over a chunk cache from its stored values, eviction), shared by their tests."""
import math

import torch

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DT = {"bf16": BF16, "f32": F32}


def half_step(dtype):
    """Largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def rel(got, ref):
    got, ref = got.double(), ref.double()
    return float((got - ref).norm() / ref.norm().clamp(min=1e-300))


def tokens(gen, rows, Hk, H, d, dtype, channel=False):
    """Unit-length queries and keys, values, decays near one, write strengths (CPU)."""
    r = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    q, k = unit(r(rows, Hk, d)).to(dtype), unit(r(rows, Hk, d)).to(dtype)
    v = r(rows, H, d).to(dtype)
    alpha = torch.exp(-torch.nn.functional.softplus(r(rows, H, d) - 3.0 if channel else r(rows, H) - 3.0))
    return q, k, v, alpha, torch.sigmoid(r(rows, H))


def rule(S, q, k, v, a, b):
    """One token on states [.., dv, dk]; a: [..] or [.., dk]; everything in 64 bits."""
    S = S * (a[..., None, :] if a.dim() == S.dim() - 1 else a[..., None, None])
    u = b[..., None] * (v - (S @ k[..., None])[..., 0])
    S = S + u[..., None] * k[..., None, :]
    return S, (S @ q[..., None])[..., 0]


def gdn_reference(q, k, v, alpha, beta, bounds, S0):
    """(o, states): sequence i is rows bounds[i][0] .. bounds[i][1] - 1, S0 [n, H, dv, dk]."""
    H, rep = v.shape[1], v.shape[1] // q.shape[1]
    q, k = (x.double().repeat_interleave(rep, 1) for x in (q, k))
    v, alpha, beta = v.double(), alpha.double(), beta.double()
    o, S = torch.zeros(v.shape, dtype=F64), S0.double().clone()
    for i, (a, e) in enumerate(bounds):
        for t in range(a, e):
            S[i], o[t] = rule(S[i], q[t], k[t], v[t], alpha[t], beta[t])
    return o, S


def cache_values(cache, cfg):
    """Host copies (64 bits) of what a dense or 8-bit cache holds: A, B, rk, n, m, buffers."""
    B, H, C, d, mc = cfg.B, cfg.H, cfg.C, cfg.dk, cache.max_chunks
    reps = C // cfg.pool_window if cfg.pool_window else 1
    dt = BF16 if cfg.dtype == 1 else F32
    get = lambda f, shape, t: (cache.buffers[f].view(*shape) if cache.mem is None else cache.view(f, shape, t)).cpu()
    out = {}
    if cfg.cache_format == 2:
        sc = get("df", (B, H, mc, 4), F32).double()
        eye = torch.eye(d, dtype=F64)
        out["A"] = (sc[..., 0, None, None] * eye
                    + sc[..., 1, None, None] * get("A", (B, H, mc, d, d), torch.int8).double())
        out["B"] = sc[..., 2, None, None] * get("Bm", (B, H, mc, d, d), torch.int8).double()
        out["scales"] = sc
    else:
        out["A"] = get("A", (B, H, mc, d, d), dt).double()
        out["B"] = get("Bm", (B, H, mc, d, d), dt).double()
    out["rk"] = get("rk", (B, H, mc, reps, d), F32).double()
    for f in ("buf_k", "buf_v", "buf_qr", "buf_kr"):
        out[f] = get(f, (B, H, C, d), dt).double()
    out["buf_alpha"] = get("buf_alpha", (B, H, C, d) if cfg.decay_mode else (B, H, C), F32).double()
    out["buf_beta"] = get("buf_beta", (B, H, C), F32).double()
    out["n"] = get("n_chunks", (B,), torch.int32)
    out["m"] = get("m_partial", (B,), torch.int32)
    return out


def decode_reference(val, cfg, tok):
    """(o, gates [B, H, mc]) of one decode step from the cache's values before it."""
    B, H, d = cfg.B, cfg.H, cfg.dk
    o = torch.zeros(B, H, d, dtype=F64)
    gates = torch.zeros(val["rk"].shape[:3], dtype=F64)
    qr = tok.get("q_route", tok["q"])
    for b in range(B):
        n, m = int(val["n"][b]), int(val["m"][b])
        for h in range(H):
            pool = torch.cat([val["buf_qr"][b, h, :m], qr[b, h].double()[None]])
            rq = cfg.tau * torch.log(torch.exp(pool / cfg.tau).mean(0))
            S = torch.zeros(d, d, dtype=F64)
            for j in range(n):
                t = (val["rk"][b, h, j] @ rq) / math.sqrt(d)
                g = torch.sigmoid(torch.logsumexp(t, 0) + cfg.bias)
                if cfg.skip_threshold > 0 and g < cfg.skip_threshold:
                    continue
                gates[b, h, j] = g
                S = S + g * (S @ val["A"][b, h, j] + val["B"][b, h, j] - S)
            for t in range(m):
                S, _ = rule(S, torch.zeros(d, dtype=F64), val["buf_k"][b, h, t], val["buf_v"][b, h, t],
                            val["buf_alpha"][b, h, t], val["buf_beta"][b, h, t])
            _, o[b, h] = rule(S, tok["q"][b, h].double(), tok["k"][b, h].double(), tok["v"][b, h].double(),
                              tok["alpha"][b, h].double(), tok["beta"][b, h].double())
    return o, gates


def evict_reference(mass, n, keep, recent):
    """The chunks that one (sequence, head) keeps."""
    if n <= keep:
        return list(range(n))
    w = [(-math.inf if math.isnan(float(x)) else float(x)) for x in mass[:n]]
    old = sorted(range(n - recent), key=lambda j: (-w[j], j))
    return sorted(old[:keep - recent]) + list(range(n - recent, n))
