"""Plain 64-bit forms of the prompt-side operators, with error bounds.

Each function returns the exact results and, beside them, the sum of the
absolute values of the terms behind each result ("mag"): a rounding of relative size u
somewhere in the sum moves the result by at most u * mag."""
import math

import torch

F64 = torch.float64
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype) -> float:
    """Relative error of one rounding to `dtype` (half a unit of the last place)."""
    return torch.finfo(dtype).eps / 2


# Relative error allowed to a chain of fp32 operations on the longest sums used
# here (under 512 terms, each at most half a step off).
FP32_CHAIN = 512 * 2.0 ** -24


def silu(v):
    return v * torch.sigmoid(v)


def dt_of(dt, bias, softplus, N, H):
    if dt is None:
        return torch.ones(N, H, dtype=F64)
    v = dt.to(F64) + (bias.to(F64) if bias is not None else 0)
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs())) if softplus else v


def linear_attention(state, A, x, B, C, dt, slots, seqs, *, load=None, D=None, dt_bias=None, z=None, softplus=True,
                     pad=-1):
    """Token by token.  seqs: list of (first row, rows).  Returns y and its mag
    [N, H, dim] (NaN in rows that are not computed), the pool and its mag."""
    N, H, dim = x.shape
    hpg = H // B.shape[1]
    d = dt_of(dt, dt_bias, softplus, N, H)
    xs, Bs, Cs = x.to(F64), B.to(F64).repeat_interleave(hpg, 1), C.to(F64).repeat_interleave(hpg, 1)
    y = torch.full((N, H, dim), math.nan, dtype=F64)
    ym = y.clone()
    pool, pm = state.to(F64).clone(), state.to(F64).abs()
    for i, (a, n) in enumerate(seqs):
        s = int(slots[i])
        if s == pad or not 0 <= s < state.shape[0]:
            continue
        S = pool[s].clone() if load is None or int(load[i]) else torch.zeros_like(pool[s])
        M = S.abs()
        for t in range(a, a + n):
            e = torch.exp(d[t] * A.to(F64))[:, None, None]
            dx = (d[t][:, None] * xs[t])[:, :, None]
            S = e * S + dx * Bs[t][:, None, :]
            M = e * M + dx.abs() * Bs[t].abs()[:, None, :]
            y[t] = (S * Cs[t][:, None, :]).sum(-1)
            ym[t] = (M * Cs[t].abs()[:, None, :]).sum(-1)
        pool[s], pm[s] = S, M
    if D is not None:
        y = y + D.to(F64)[:, None] * xs
        ym = ym + (D.to(F64)[:, None] * xs).abs()
    if z is not None:
        y, ym = y * silu(z.to(F64)), ym * silu(z.to(F64)).abs()
    return y, ym, pool, pm


def y_bound(y, ym, dtype):
    """One rounding of each term's factor (16-bit inputs) and of the result, and the fp32 chain."""
    u = half_step(dtype) if dtype != torch.float32 else 0.0
    return half_step(dtype) * y.abs() + (u * 1.01 + FP32_CHAIN) * ym + torch.finfo(dtype).tiny


def state_bound(pool, pm, dtype, chunks=1):
    return half_step(dtype) * pool.abs() + (FP32_CHAIN + 4 * chunks * 2.0 ** -24) * pm + torch.finfo(dtype).tiny


def paged_attention(q, kc, vc, table, seqs, kv, *, scale=None, window=0, sinks=0):
    """q [N, Hq, D], caches [P, ps, Hkv, D], seqs (first row, rows) and kv lengths.
    Returns out, sum p|v|, lse and the relative error that fp32 scores give the weights."""
    N, Hq, D = q.shape
    P, ps, Hkv, _ = kc.shape
    g = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((N, Hq, D), math.nan, dtype=F64)
    mag, lse, err = out.clone(), torch.full((N, Hq), math.nan, dtype=F64), torch.zeros(N, Hq, dtype=F64)
    for s, (a, n) in enumerate(seqs):
        L = min(int(kv[s]), table.shape[1] * ps)
        j = torch.arange(L)
        page = table[s, j // ps].long()
        ok = (page >= 0) & (page < P)
        rows = (torch.where(ok, page, 0), j % ps)
        K, V = kc[rows].to(F64), vc[rows].to(F64)      # [L, Hkv, D]
        for t in range(n):
            pos = int(kv[s]) - n + t
            see = ok & (j <= pos)
            if window:
                see &= (j > pos - window) | (j < sinks)
            if not bool(see.any()):
                out[a + t], mag[a + t], lse[a + t] = 0, 0, -math.inf
                continue
            Ks, Vs = K[see].repeat_interleave(g, 1), V[see].repeat_interleave(g, 1)
            qt = q[a + t].to(F64)
            sc = (Ks * qt).sum(-1) * scale                  # [L', Hq]
            m = sc.amax(0)
            p = torch.exp(sc - m)
            tot = p.sum(0)
            p = p / tot
            out[a + t] = (p[..., None] * Vs).sum(0)
            mag[a + t] = (p[..., None] * Vs.abs()).sum(0)
            lse[a + t] = m + torch.log(tot)
            # D-term fp32 dot products and the rounding of the scaled score
            err[a + t] = ((Ks * qt).abs().sum(-1) * scale).amax(0) * (D + 4) * 2.0 ** -24
    return out, mag, lse, err


def out_bound(out, mag, err, dtype):
    u = half_step(dtype) if dtype != torch.float32 else 0.0
    return half_step(dtype) * out.abs() + (u * 1.01 + FP32_CHAIN + 2 * err[..., None]) * mag + torch.finfo(dtype).tiny


def block_norm(y, residual, *, z=None, post=None, pre=None, cs=None, rs=1.0, groups=1, eps=1e-5):
    """residual_out, normed and the sizes of their terms."""
    R, C = y.shape
    u = y.to(F64)
    if z is not None:
        u = u * silu(z.to(F64))
    if post is not None:
        g = u.view(R, groups, -1)
        u = (g / torch.sqrt((g * g).mean(-1, keepdim=True) + eps)).view(R, C) * post.to(F64)
    v = rs * u * (cs.to(F64) if cs is not None else 1.0)
    r = residual.to(F64) + v
    rm = residual.to(F64).abs() + v.abs()
    inv = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    w = pre.to(F64) if pre is not None else torch.ones(C, dtype=F64)
    return r, rm, r * inv * w, rm * inv * w.abs()


def norm_bound(v, m, dtype):
    return half_step(dtype) * v.abs() + FP32_CHAIN * m + torch.finfo(dtype).tiny


def check(got, want, bound, what):
    got = got.detach().cpu().to(F64)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got) & ~nan, torch.zeros_like(nan)), f"{what}: NaN where there is a value"
    off = ((got - want).abs() / bound)[~nan]
    assert not off.numel() or float(off.max()) <= 1, f"{what}: {float(off.max()):.3g} times the bound"
