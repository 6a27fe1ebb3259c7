"""Plain 64-bit forms of the causal convolution, the selective scan, rotary positions and the page pool,
with error bounds (operators_ref.py's conventions: a value, and the sum of the sizes of its terms)."""
import math

import torch

from operators_ref import F64, check, half_step, silu  # noqa: F401

STEP = 2.0 ** -24          # half a step of an fp32 operation


def act(v, m, on):
    """silu and its terms: its slope is below 1.1, and its exponential's argument is rounded."""
    return (silu(v), 1.1 * m) if on else (v, m)


def conv(x, weight, state, slots, seqs, *, bias=None, load=None, on=True, pad=-1):
    """seqs: (first row, rows).  y, its terms [N, C] (NaN where not computed) and the pool."""
    W = weight.shape[0]
    y = torch.full(x.shape, math.nan, dtype=F64)
    ym, pool = y.clone(), state.clone()
    for i, (a, n) in enumerate(seqs):
        s = int(slots[i])
        if s == pad or not 0 <= s < state.shape[0]:
            continue
        old = state[s] if load is None or int(load[i]) else torch.zeros_like(state[s])
        col = torch.cat((old, x[a:a + n]))
        for t in range(n):
            terms = weight.to(F64) * col[t:t + W].to(F64)
            b = bias.to(F64) if bias is not None else torch.zeros(x.shape[1], dtype=F64)
            y[a + t], ym[a + t] = act(terms.sum(0) + b, terms.abs().sum(0) + b.abs(), on)
        pool[s] = col[col.shape[0] - (W - 1):]
    return y, ym, pool


def conv_bound(y, ym, dtype):
    """One rounding of the result; 5 sums and products and at most 16 half steps for silu (exponential, reciprocal,
    products), whose argument's rounding is relative to its size (inputs here stay below 16)."""
    return half_step(dtype) * y.abs() + 64 * STEP * ym + torch.finfo(dtype).tiny


def scan(state, A, x, B, C, dt, slots, seqs, *, load=None, D=None, bias=None, z=None, softplus=True, pad=-1):
    """Token by token.  y, its terms, the pool and its terms."""
    N, Ch = x.shape
    per = Ch // B.shape[1]
    v = dt.to(F64) + (bias.to(F64) if bias is not None else 0)
    d = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs())) if softplus else v
    xs, Bs, Cs, A = x.to(F64), B.to(F64).repeat_interleave(per, 1), C.to(F64).repeat_interleave(per, 1), A.to(F64)
    y = torch.full((N, Ch), math.nan, dtype=F64)
    ym, pool, pm = y.clone(), state.to(F64).clone(), state.to(F64).abs()
    for i, (a, n) in enumerate(seqs):
        s = int(slots[i])
        if s == pad or not 0 <= s < state.shape[0]:
            continue
        h = pool[s].clone() if load is None or int(load[i]) else torch.zeros_like(pool[s])
        m = h.abs()
        for t in range(a, a + n):
            e = torch.exp(d[t][:, None] * A)
            u = (d[t] * xs[t])[:, None] * Bs[t]
            h, m = e * h + u, e * m + u.abs()
            y[t], ym[t] = (h * Cs[t]).sum(-1), (m * Cs[t].abs()).sum(-1)
        pool[s], pm[s] = h, m
    if D is not None:
        y, ym = y + D.to(F64) * xs, ym + (D.to(F64) * xs).abs()
    if z is not None:
        y, ym = y * silu(z.to(F64)), ym * silu(z.to(F64)).abs()
    return y, ym, pool, pm


def scan_chain(tokens, dstate):
    """Half steps on a sum of terms that went through `tokens` steps: at most 4 a step (the exponential, whose
    argument's rounding costs less than 2 of them where a term has not vanished, the product and the sum),
    a step size of 16 and its product, one each for dstate products and sums of the readout, 16 for the gate."""
    return (4 * tokens + dstate + 64) * STEP


def scan_bound(v, m, dtype, chain):
    return half_step(dtype) * v.abs() + chain * m + torch.finfo(dtype).tiny


def turned(t, pos, freq, inter, factor):
    """t [N, H, D] turned by pos [N]; the terms' sizes beside it."""
    half, r = freq.shape[0], t.to(F64).clone()
    first = torch.arange(half) * 2 if inter else torch.arange(half)
    second = first + 1 if inter else first + half
    ang = pos.to(F64)[:, None] * freq.to(F64)
    c, s = (factor * torch.cos(ang))[:, None], (factor * torch.sin(ang))[:, None]
    a, b, m = t[..., first].to(F64), t[..., second].to(F64), torch.zeros_like(r)
    r[..., first], r[..., second] = a * c - b * s, a * s + b * c
    m[..., first] = m[..., second] = abs(factor) * (a.abs() + b.abs())
    return r, m


def turned_bound(r, m, dtype):
    """Sines and cosines: the turns' rounding (2 pi / 2 half steps of 1), 4 half steps of the functions, one of the
    factor; a product and a sum each."""
    return half_step(dtype) * r.abs() + 12 * STEP * m + torch.finfo(dtype).tiny


class Pool:
    """The page pool on the host: lists, call by call.  caches: any object with copy(src, dst, tokens)."""

    def __init__(self, table, kv_len, ref, page):
        self.table, self.kv, self.ref, self.page = [list(r) for r in table], list(kv_len), list(ref), page
        self.copies = []                  # (from, to, tokens or None for a whole page)

    def held(self, r):
        return -(-self.kv[r] // self.page)

    def free(self):
        return [p for p, n in enumerate(self.ref) if n <= 0]

    def extend(self, rows, add):
        free, asked, status, seen = self.free(), 0, [], set()
        old = list(self.kv)
        for r, n in zip(rows, add):
            bad = not 0 <= r < len(self.table) or r in seen or n < 0 or old[r] + n > len(self.table[r]) * self.page
            if 0 <= r < len(self.table):
                seen.add(r)
            if bad:
                status.append(2)
                continue
            last = self.table[r][self.held(r) - 1] if old[r] % self.page else -1
            if n > 0 and last >= 0 and self.ref[last] > 1:
                status.append(3)
                continue
            need = -(-(old[r] + n) // self.page) - self.held(r)
            asked += need
            if need and asked > len(free):
                status.append(1)
                continue
            for k in range(need):
                p = free[asked - need + k]
                self.table[r][self.held(r) + k] = p
                self.ref[p] = 1
            self.kv[r] += n
            status.append(0)
        return status

    def fork(self, src, dst, lengths):
        free, asked, status, seen = self.free(), 0, [], set()
        old = list(self.kv)
        for s, d, n in zip(src, dst, lengths):
            bad = not 0 <= d < len(self.table) or d in seen
            if 0 <= d < len(self.table):
                seen.add(d)
            if bad or not 0 <= s < len(self.table) or (n is not None and n < 0) or old[d] != 0:
                status.append(2)
                continue
            n = old[s] if n is None else min(n, old[s])
            full, rest = divmod(n, self.page)
            asked += rest > 0
            if rest and asked > len(free):
                status.append(1)
                continue
            for k in range(full):
                self.table[d][k] = self.table[s][k]
                self.ref[self.table[s][k]] += 1
            if rest:
                p = free[asked - 1]
                self.table[d][full] = p
                self.ref[p] = 1
                self.copies.append((self.table[s][full], p, rest))
            self.kv[d] = n
            status.append(0)
        return status

    def release(self, rows, lengths=None):
        for i, r in enumerate(rows):
            keep = 0 if lengths is None else lengths[i]
            if not 0 <= r < len(self.table) or keep < 0 or keep >= self.kv[r]:
                continue
            for k in range(-(-keep // self.page), self.held(r)):
                self.ref[self.table[r][k]] -= 1
                self.table[r][k] = -1
            self.kv[r] = keep

    def compact(self):
        live = sum(n > 0 for n in self.ref)
        holes = [p for p in range(live) if self.ref[p] <= 0]
        new = dict(zip([p for p in range(live, len(self.ref)) if self.ref[p] > 0], holes))
        for p, q in new.items():
            self.ref[q], self.ref[p] = self.ref[p], 0
            self.copies.append((p, q, None))
        for r in range(len(self.table)):
            for k in range(self.held(r)):
                self.table[r][k] = new.get(self.table[r][k], self.table[r][k])
        return live

    def apply(self, cache):
        """The copies so far on a cache [pages, page, ...] (in order)."""
        for s, d, n in self.copies:
            cache[d, :n] = cache[s, :n]
        return cache
