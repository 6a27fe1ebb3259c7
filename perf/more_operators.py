"""Timing cases and plain forms of the operators in front of the cores of a hybrid decoder and of its page pool.

Four operators, each in the layout the library takes it:
  conv    short causal convolution of each channel over ragged prompts, or of one new token per request
  scan    selective state-space scan (a step size for each channel, a decay for each channel and state)
          over ragged prompts, or of one new token per request
  rotary  rotary positions of new queries and keys, the keys and values appended to a paged cache
  pages   pages of a cache: branches of requests (release, fork, extend), and packing the pool (compact)

`own` selects between the plain form (elementary torch operations in 32 bits, angles and step sizes in 64) and the
library's entry points.  `exact` is each definition once more in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # the mixer of a small model reads a chat-sized prompt: latency counts
        dict(name="conv_prompt_short", op="conv", step=False, S=1, L=97, even=True, C=1024, W=4, it="bf16", resume=False),
        # the packed x, B and C of a large mixer (256 heads of 64, 8 groups of 128) over a batch of ragged prompts
        dict(name="conv_batch", op="conv", step=False, S=12, L=2011, even=False, C=18432, W=4, it="bf16", resume=True),
        # one decoding step of a full batch of the same mixer
        dict(name="conv_step", op="conv", step=True, S=256, L=1, even=True, C=18432, W=4, it="bf16", resume=True),
        # scan: a chat-sized prompt on a small model, a long document on one shard, a ragged batch, a decoding step
        dict(name="scan_prompt_short", op="scan", step=False, S=1, L=97, even=True, C=1024, N=16, G=1, it="bf16", st="f32", z=True, resume=False),
        dict(name="scan_document", op="scan", step=False, S=1, L=16384, even=True, C=4096, N=16, G=1, it="bf16", st="f32", z=True, resume=True),
        dict(name="scan_batch", op="scan", step=False, S=12, L=2011, even=False, C=8192, N=16, G=1, it="bf16", st="f32", z=True, resume=True),
        dict(name="scan_step", op="scan", step=True, S=256, L=1, even=True, C=8192, N=16, G=1, it="f16", st="f32", z=True, resume=True),
        # rotary: the tokens of a decoding batch far into their contexts, frequencies scaled for them
        dict(name="rotary_decode", op="rotary", S=64, Q=1, L=131071, even=False, Hq=32, Hkv=8, D=128, rot=128, inter=False, page=16, it="bf16", scaled=True),
        # chunks of ragged prompts, half of each head in interleaved pairs
        dict(name="rotary_prompt", op="rotary", S=6, Q=4001, L=9001, even=False, Hq=32, Hkv=8, D=128, rot=64, inter=True, page=48, it="f16", scaled=False),
        # pages: branches of a few requests of a small model, and of a batch of a larger one
        dict(name="pages_branch_few", op="pages", kind="branch", parents=1, forks=4, tokens=133, caches=8, page=16, Hkv=2, D=64, it="bf16"),
        dict(name="pages_branch_batch", op="pages", kind="branch", parents=16, forks=128, tokens=3001, caches=32, page=16, Hkv=8, D=128, it="bf16"),
        # a pool that loses half of its requests, is packed and filled up again, twice
        dict(name="pages_pack", op="pages", kind="pack", parents=32, forks=0, tokens=510, caches=32, page=16, Hkv=8, D=128, it="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "rotary", "pages"])
    it = rng.choice(["bf16", "f16"])
    if op == "conv":
        step, C = rng.random() < 0.4, 8 * _log(rng, 8, 2304)
        S = _log(rng, 1, 256 if step else 12)
        return dict(op=op, step=step, S=S, L=1 if step else _log(rng, 1, min(16384, 200000000 // (S * C) + 1)),
                    even=step or rng.random() < 0.3, C=C, W=rng.choice([2, 3, 4, 4]), it=it, resume=rng.random() < 0.5)
    if op == "scan":
        step, N, G = rng.random() < 0.4, rng.choice([16, 16, 32, 64]), rng.choice([1, 1, 2])
        C = 16 * G * _log(rng, 4, 512 // G)
        S = _log(rng, 1, 256 if step else 12)
        return dict(op=op, step=step, S=S, L=1 if step else _log(rng, 1, min(16384, 1000000000 // (S * C * N) + 1)),
                    even=step or rng.random() < 0.3, C=C, N=N, G=G, it=it, st=rng.choice(["f32", "bf16", "f16"]),
                    z=rng.random() < 0.7, resume=rng.random() < 0.5)
    if op == "rotary":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        S = _log(rng, 1, 64)
        L = _log(rng, 1, 131072 // S)
        return dict(op=op, S=S, Q=1 if rng.random() < 0.4 else _log(rng, 1, min(L, 16384 // S)), L=L, even=rng.random() < 0.3,
                    Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, D=D, rot=rng.choice([16, 32, D // 2, D - 16, D]),
                    inter=rng.random() < 0.5, page=rng.choice([16, 24, 48, 64, 256]), it=it, scaled=rng.random() < 0.5)
    kind, page = rng.choice(["branch", "pack"]), rng.choice([16, 24, 64])
    Hkv, D, caches = rng.choice([1, 2, 8]), rng.choice([64, 128]), 2 * _log(rng, 1, 16)
    parents = _log(rng, 1, 16) if kind == "branch" else 2 * _log(rng, 1, 16)
    return dict(op=op, kind=kind, parents=parents, forks=_log(rng, 1, 128) if kind == "branch" else 0,
                tokens=_log(rng, 1, min(3000, 1000000000 // (parents * caches * Hkv * D * 2))), caches=caches, page=page,
                Hkv=Hkv, D=D, it=it)


def _lengths(S, L, even):
    """Ragged lengths from 1 to L, spread evenly (the first is L)."""
    return [L if even or i == 0 else max(1, int(L * ((i * 0.6180339887498949) % 1.0))) for i in range(S)]


def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return s


def _loads(case):
    """1: a later chunk of a prompt, which continues from its slot's state; 0: a new prompt."""
    return [1 if case["resume"] and i % 3 != 2 else 0 for i in range(case["S"])]


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return _prepare[case["op"]](case, g)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _prepare_conv(case, g):
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)          # noqa: E731
    it, S, C, W = DTYPES[case["it"]], case["S"], case["C"], case["W"]
    lens = _lengths(S, case["L"], case["even"])
    return dict(case=case, x=rn(sum(lens), C).to(it), weight=rn(W, C) / math.sqrt(W), bias=0.1 * rn(C),
                state=rn(S, W - 1, C).to(it), y=torch.zeros(sum(lens), C, dtype=it, device=DEV),
                slots=torch.randperm(S, generator=g, device=DEV).int(), seq_start=_i32(_starts(lens)),
                load_state=_i32(_loads(case)))


def _prepare_scan(case, g):
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)          # noqa: E731
    ru = lambda *s: torch.rand(s, generator=g, device=DEV)           # noqa: E731
    it, S, C, N, G = DTYPES[case["it"]], case["S"], case["C"], case["N"], case["G"]
    lens = _lengths(S, case["L"], case["even"])
    T = sum(lens)
    return dict(case=case, state=rn(S, C, N).to(DTYPES[case["st"]]), A=-(1 + ru(C, N)) * torch.arange(1, N + 1, device=DEV) * 0.6,
                D=0.5 + ru(C), dt_bias=torch.log(torch.expm1(0.001 + 0.099 * ru(C))), x=rn(T, C).to(it),
                dt=(rn(T, C) * 0.3).to(it), z=rn(T, C).to(it) if case["z"] else None,
                B=rn(T, G, N).to(it), C=(rn(T, G, N) / math.sqrt(N)).to(it), y=torch.zeros(T, C, dtype=it, device=DEV),
                slots=torch.randperm(S, generator=g, device=DEV).int(), seq_start=_i32(_starts(lens)),
                load_state=_i32(_loads(case)))


def _frequencies(case):
    """Frequencies of the pairs; scaled: those with few turns in the trained length are slowed down 8 times, the
    fast ones stay, and between the two the slowing grows evenly."""
    half = case["rot"] // 2
    f = [10000.0 ** (-i / half) for i in range(half)]
    if not case["scaled"]:
        return f, 1.0
    turns = [8192 * v / (2 * math.pi) for v in f]
    keep = [min(1.0, max(0.0, (t - 1.0) / 31.0)) for t in turns]
    return [v * (k + (1 - k) / 8.0) for v, k in zip(f, keep)], 0.1 * math.log(8.0) + 1.0


def _prepare_rotary(case, g):
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)          # noqa: E731
    it, S, D, page = DTYPES[case["it"]], case["S"], case["D"], case["page"]
    kv = _lengths(S, case["L"], case["even"])
    ql = [min(case["Q"], n) for n in kv]
    per = (case["L"] + page - 1) // page
    # the pages that this call's tokens fall on are there; older ones are on pages of their own, which nobody reads
    first = [(n - q) // page for n, q in zip(kv, ql)]
    count = [(n + page - 1) // page - f for n, f in zip(kv, first)]
    need, N = sum(count), sum(ql)
    table = torch.full((S, per), -1, dtype=torch.int32, device=DEV)
    order, at = torch.randperm(need, generator=g, device=DEV).int(), 0
    for i in range(S):
        table[i, first[i]:first[i] + count[i]] = order[at:at + count[i]]
        at += count[i]
    freq, factor = _frequencies(case)
    return dict(case=case, q=rn(N, case["Hq"], D).to(it), k_new=rn(N, case["Hkv"], D).to(it), v_new=rn(N, case["Hkv"], D).to(it),
                k_cache=rn(need, page, case["Hkv"], D).to(it), v_cache=rn(need, page, case["Hkv"], D).to(it), page_table=table,
                seq_start=_i32(_starts(ql)), kv_len=_i32(kv), q_out=torch.zeros(N, case["Hq"], D, dtype=it, device=DEV),
                inv_freq=torch.tensor(freq, dtype=torch.float64).float().to(DEV), factor=factor)


def _page_counts(case):
    """(pages a parent holds, rows of the table, pages of the pool)"""
    held = (case["tokens"] + case["page"] - 1) // case["page"]
    rows = case["parents"] + case["forks"]
    return held, rows, held * case["parents"] + 2 * case["forks"] + 3


def _prepare_pages(case, g):
    it, ps = DTYPES[case["it"]], case["page"]
    held, rows, pool = _page_counts(case)
    caches = torch.randn(case["caches"], pool, ps, case["Hkv"], case["D"], generator=g, device=DEV, dtype=torch.float32).to(it)
    table = torch.full((rows, held + 1), -1, dtype=torch.int32, device=DEV)
    ref = torch.zeros(pool, dtype=torch.int32, device=DEV)
    half = case["parents"] // 2
    parts = [range(case["parents"])] if case["kind"] == "branch" else [range(half), range(half, case["parents"])]
    at = 0
    for part in parts:                     # the first half of a pack case holds the lower pages
        n = len(part) * held
        order = (at + torch.randperm(n, generator=g, device=DEV)).int()
        table[part[0]:part[0] + len(part), :held] = order.view(len(part), held)
        at += n
    ref[:at] = 1
    kv = [case["tokens"]] * case["parents"] + [0] * case["forks"]
    st = dict(case=case, caches=caches, page_table=table, kv_len=_i32(kv), page_ref=ref)
    st["cache_ptrs"] = torch.tensor([c.data_ptr() for c in caches], dtype=torch.int64, device=DEV)
    if case["kind"] == "branch":
        st["src"] = _i32([i % case["parents"] for i in range(case["forks"])])
        st["dst"] = _i32([case["parents"] + i for i in range(case["forks"])])
        # branches start at accepted prefixes, some of the whole request, some of a part of it
        st["length"] = _i32([max(1, case["tokens"] - (i * 7) % case["tokens"] if i % 2 else case["tokens"]) for i in range(case["forks"])])
        st["add"] = _i32([1 + i % ps for i in range(case["forks"])])
        st["status"] = torch.zeros(2, case["forks"], dtype=torch.int32, device=DEV)
    else:
        st["parts"] = [_i32(list(p)) for p in parts]
        st["add"] = [torch.full((len(p),), case["tokens"], dtype=torch.int32, device=DEV) for p in parts]
        st["status"] = torch.zeros(2, half, dtype=torch.int32, device=DEV)
        st["live"] = torch.zeros(2, dtype=torch.int32, device=DEV)
    return st


_prepare = {"conv": _prepare_conv, "scan": _prepare_scan, "rotary": _prepare_rotary, "pages": _prepare_pages}


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _own_conv(st):
    import replayssm_persistent_rssm_amd as rp
    if st["case"]["step"]:
        rp.rssm_causal_conv_step(st["x"], st["weight"], st["y"], st["state"], st["slots"], bias=st["bias"])
    else:
        rp.rssm_causal_conv(st["x"], st["weight"], st["y"], st["state"], st["slots"], st["seq_start"], bias=st["bias"],
                            load_state=st["load_state"])
    return st["y"], st["state"]


def _own_scan(st):
    import replayssm_persistent_rssm_amd as rp
    args = (st["state"], st["A"], st["x"], st["B"], st["C"], st["dt"], st["y"], st["slots"])
    kw = dict(D=st["D"], dt_bias=st["dt_bias"], z=st["z"])
    if st["case"]["step"]:
        rp.rssm_selective_scan_step(*args, **kw)
    else:
        rp.rssm_selective_scan(*args, st["seq_start"], max_seq_len=st["case"]["L"], load_state=st["load_state"], **kw)
    return st["y"], st["state"]


def _own_rotary(st):
    import replayssm_persistent_rssm_amd as rp
    rp.rssm_rotary_append(st["q"], st["q_out"], st["k_cache"], st["v_cache"], st["k_new"], st["v_new"], st["page_table"],
                          st["seq_start"], st["kv_len"], st["inv_freq"], interleaved=st["case"]["inter"], factor=st["factor"])
    return st["q_out"], st["k_cache"], st["v_cache"]


def _own_pages(st):
    import replayssm_persistent_rssm_amd as rp
    c, table, kv, ref = st["case"], st["page_table"], st["kv_len"], st["page_ref"]
    ps = c["page"]
    token = c["Hkv"] * c["D"] * SIZE[c["it"]]
    kw = dict(page_size=ps, page_bytes=ps * token)
    if c["kind"] == "branch":
        rp.rssm_page_release(table, kv, ref, st["dst"], page_size=ps)
        rp.rssm_page_fork(st["cache_ptrs"], table, kv, ref, st["src"], st["dst"], st["status"][0], lengths=st["length"],
                          token_bytes=token, **kw)
        rp.rssm_page_extend(table, kv, ref, st["dst"], st["add"], st["status"][1], page_size=ps)
        return table, kv, ref, st["status"], st["caches"]
    for i, rows in enumerate(st["parts"]):
        rp.rssm_page_release(table, kv, ref, rows, page_size=ps)
        rp.rssm_page_compact(st["cache_ptrs"], table, kv, ref, st["live"][i:i + 1], **kw)
        rp.rssm_page_extend(table, kv, ref, rows, st["add"][i], st["status"][i], page_size=ps)
    return table, kv, ref, st["status"], st["live"], st["caches"]


_own = {"conv": _own_conv, "scan": _own_scan, "rotary": _own_rotary, "pages": _own_pages}


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_conv(st):
    c, x = st["case"], st["x"].float()
    W, S, C = c["W"], c["S"], c["C"]
    starts = st["seq_start"].long()
    lens = starts[1:] - starts[:-1]
    slots = st["slots"].long()
    old = st["state"][slots].float()                                   # [S, W-1, C]
    if not c["step"]:
        old = torch.where(st["load_state"].bool().view(S, 1, 1), old, 0)
    n = torch.arange(x.shape[0], device=DEV)
    seq = torch.searchsorted(starts[1:].contiguous(), n, right=True)
    at = n - starts[seq]                                               # place inside the sequence
    y = st["bias"] + st["weight"][W - 1] * x
    for k in range(W - 1):
        back = W - 1 - k
        before = torch.where((at >= back)[:, None], x[(n - back).clamp(min=0)], old[seq, (at - back + W - 1).clamp(max=W - 2)])
        y = y + st["weight"][k] * before
    for k in range(W - 1):                                             # the last W - 1 inputs of each sequence
        p = lens - (W - 1) + k
        row = torch.where((p >= 0)[:, None], x[(starts[:-1] + p).clamp(min=0)], old[torch.arange(S, device=DEV), (p + W - 1).clamp(max=W - 2)])
        st["state"][slots, k] = row.to(st["state"].dtype)
    st["y"].copy_(_silu(y))
    return st["y"], st["state"]


def _softplus64(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_scan(st, Q=64):
    """Blocks of Q tokens side by side: each block's own end and decay, the starts of the blocks one after the
    other, then the outputs of all blocks from their starts."""
    c = st["case"]
    S, C, N, G, L = c["S"], c["C"], c["N"], c["G"], c["L"]
    slots = st["slots"].long()
    starts = st["seq_start"].long()
    first = st["state"][slots].float()
    if not c["step"]:
        first = torch.where(st["load_state"].bool().view(S, 1, 1), first, 0)
    Q = min(Q, L)
    nb = (L + Q - 1) // Q
    pos = torch.arange(nb * Q, device=DEV)
    live = pos[None] < (starts[1:] - starts[:-1])[:, None]             # [S, nb * Q]
    idx = torch.where(live, starts[:-1, None] + pos[None], 0).view(S, nb, Q)
    live = live.view(S, nb, Q)
    groups = lambda t: t.float()[:, :, :, None, :].expand(S, nb, G, C // G, N).reshape(S, nb, C, N)    # noqa: E731

    def token(q):
        """Step size (0 past the end), input times step size, B and C of token q of every block."""
        i, on = idx[:, :, q], live[:, :, q, None]
        d = torch.where(on, _softplus64(st["dt"][i].double() + st["dt_bias"].double()).float(), 0)
        return d, d * st["x"][i].float(), groups(st["B"][i]), groups(st["C"][i])

    h = torch.zeros(S, nb, C, N, device=DEV)
    total = torch.zeros(S, nb, C, device=DEV, dtype=torch.float64)
    if nb > 1:
        for q in range(Q):
            d, dx, B, _ = token(q)
            h = torch.exp(d[..., None] * st["A"]) * h + dx[..., None] * B
            total += d
    into, at = torch.empty_like(h), first
    for b in range(nb):
        into[:, b] = at
        if nb > 1:
            at = torch.exp(total[:, b, :, None] * st["A"].double()).float() * at + h[:, b]
    h = into
    y = torch.empty(st["x"].shape, device=DEV)
    for q in range(Q):
        d, dx, B, Ct = token(q)
        h = torch.exp(d[..., None] * st["A"]) * h + dx[..., None] * B
        on = live[:, :, q]
        y[idx[:, :, q][on]] = (h * Ct).sum(-1)[on]
    y += st["D"] * st["x"].float()
    if st["z"] is not None:
        y *= _silu(st["z"].float())
    st["state"][slots] = h[:, nb - 1].to(st["state"].dtype)
    st["y"].copy_(y)
    return st["y"], st["state"]


def _plain_rotary(st):
    c, page = st["case"], st["case"]["page"]
    starts = st["seq_start"].long()
    n = torch.arange(st["q"].shape[0], device=DEV)
    seq = torch.searchsorted(starts[1:].contiguous(), n, right=True)
    pos = st["kv_len"].long()[seq] - starts[1:][seq] + n
    angle = pos.double()[:, None] * st["inv_freq"].double()
    cos, sin = (torch.cos(angle) * st["factor"]).float()[:, None], (torch.sin(angle) * st["factor"]).float()[:, None]
    half = c["rot"] // 2

    def turn(t):
        t = t.float()
        r = t[..., :c["rot"]]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :half], r[..., half:])
        u, v = a * cos - b * sin, a * sin + b * cos
        r = torch.stack((u, v), -1).flatten(-2) if c["inter"] else torch.cat((u, v), -1)
        return torch.cat((r, t[..., c["rot"]:]), -1)

    st["q_out"].copy_(turn(st["q"]))
    pg = st["page_table"].long()[seq, pos // page]
    st["k_cache"][pg, pos % page] = turn(st["k_new"]).to(st["k_cache"].dtype)
    st["v_cache"][pg, pos % page] = st["v_new"]
    return st["q_out"], st["k_cache"], st["v_cache"]


def _pages_of(n, page):
    return (n + page - 1) // page


def _plain_release(table, kv, ref, rows, page):
    held = _pages_of(kv[rows].long(), page)
    r = rows.long()
    old = table[r]
    on = torch.arange(table.shape[1], device=DEV)[None] < held[:, None]
    ref.index_add_(0, torch.where(on, old, 0).flatten().long(), -on.flatten().int())
    table[r] = torch.where(on, torch.full_like(old, -1), old)
    kv[r] = 0


def _plain_take(ref, need):
    """For each item its place in the list of free pages, lowest first, and whether its pages are there."""
    free = torch.sort((ref != 0).int(), stable=True).indices
    end = need.cumsum(0)
    return free, end - need, (need == 0) | (end <= (ref == 0).sum())


def _plain_extend(table, kv, ref, rows, add, status, page):
    r = rows.long()
    have, want = _pages_of(kv[r].long(), page), _pages_of(kv[r].long() + add, page)
    free, at, ok = _plain_take(ref, want - have)
    j = torch.arange(table.shape[1], device=DEV)[None]
    new = (j >= have[:, None]) & (j < want[:, None]) & ok[:, None]
    pick = free[torch.where(new, at[:, None] + j - have[:, None], 0)]
    table[r] = torch.where(new, pick.int(), table[r])
    ref.index_add_(0, torch.where(new, pick, 0).flatten(), new.flatten().int())
    kv[r] += torch.where(ok, add, 0)
    status.copy_((~ok).int())


def _plain_pages(st):
    c, table, kv, ref, page = st["case"], st["page_table"], st["kv_len"], st["page_ref"], st["case"]["page"]
    j = torch.arange(table.shape[1], device=DEV)[None]
    if c["kind"] == "branch":
        src, dst = st["src"].long(), st["dst"].long()
        _plain_release(table, kv, ref, st["dst"], page)
        length = torch.minimum(st["length"], kv[src])
        full, rest = length.long() // page, length.long() % page
        free, at, ok = _plain_take(ref, (rest > 0).long())
        shared = (j < full[:, None]) & ok[:, None]
        own_page = free[at.clamp(max=ref.shape[0] - 1)]
        old = table[src]
        copied = ((rest > 0) & ok)[:, None] & (j == full[:, None])
        table[dst] = torch.where(shared, old, torch.where(copied, own_page[:, None].int(), table[dst]))
        ref.index_add_(0, torch.where(shared, old, 0).flatten().long(), shared.flatten().int())
        ref.index_add_(0, own_page, ((rest > 0) & ok).int())
        kv[dst] = torch.where(ok, length, 0)
        st["status"][0] = (~ok).int()
        # the filled tokens of the last page, cache by cache
        source = old.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long().clamp(min=0)
        some = torch.nonzero((rest > 0) & ok)[:, 0]
        source, target = source[some], own_page[some]
        filled = (torch.arange(page, device=DEV)[None] < rest[some, None])[:, :, None, None]
        for cache in st["caches"]:
            cache[target] = torch.where(filled, cache[source], cache[target])
        _plain_extend(table, kv, ref, st["dst"], st["add"], st["status"][1], page)
        return table, kv, ref, st["status"], st["caches"]
    P = ref.shape[0]
    number = torch.arange(P, device=DEV)
    for i, rows in enumerate(st["parts"]):
        _plain_release(table, kv, ref, rows, page)
        used = ref > 0
        live = used.sum()
        high, hole = used & (number >= live), ~used & (number < live)
        to = torch.sort((~hole).int(), stable=True).indices        # holes first, in order
        new = torch.where(high, to[(high.cumsum(0) - 1).clamp(min=0)], number)
        moved = torch.nonzero(high)[:, 0]
        source = number.clone()
        source[new[moved]] = moved                                 # page that each page's content comes from
        for cache in st["caches"]:
            cache.copy_(cache[source])
        ref.copy_(torch.where(hole, ref[source], torch.where(high, 0, ref)))
        on = j < _pages_of(kv.long(), page)[:, None]
        table.copy_(torch.where(on, new[torch.where(on, table, 0).long()].int(), table))
        st["live"][i] = live
        _plain_extend(table, kv, ref, rows, st["add"][i], st["status"][i], page)
    return table, kv, ref, st["status"], st["live"], st["caches"]


_plain = {"conv": _plain_conv, "scan": _plain_scan, "rotary": _plain_rotary, "pages": _plain_pages}


# --------------------------------------------------------------------------
# The work of one pass
# --------------------------------------------------------------------------
def work(case):
    if case["op"] == "conv":
        e, n = SIZE[case["it"]], sum(_lengths(case["S"], case["L"], case["even"]))
        loads = case["S"] if case["step"] else sum(_loads(case))
        b = 2 * n * case["C"] * e + (case["S"] + loads) * (case["W"] - 1) * case["C"] * e + (case["W"] + 1) * case["C"] * 4
        return {"bytes": b, "flops": n * case["C"] * (2 * case["W"] + 4)}
    if case["op"] == "scan":
        e, n, C, N = SIZE[case["it"]], sum(_lengths(case["S"], case["L"], case["even"])), case["C"], case["N"]
        loads = case["S"] if case["step"] else sum(_loads(case))
        b = n * C * e * (4 if case["z"] else 3) + 2 * n * case["G"] * N * e + (case["S"] + loads) * C * N * SIZE[case["st"]]
        # of each state element: the decay's argument and exponential (2), update (3) and readout (2)
        return {"bytes": b + C * (N + 2) * 4, "flops": n * C * (7 * N + 10)}
    if case["op"] == "rotary":
        e = SIZE[case["it"]]
        n = sum(min(case["Q"], m) for m in _lengths(case["S"], case["L"], case["even"]))
        return {"bytes": n * case["D"] * e * (2 * case["Hq"] + 4 * case["Hkv"]),
                "flops": n * 3 * case["rot"] * (case["Hq"] + case["Hkv"])}
    ps, token = case["page"], case["Hkv"] * case["D"] * SIZE[case["it"]]
    held, rows, pool = _page_counts(case)
    meta = rows * (held + 1) * 4 + 2 * pool * 4
    if case["kind"] == "branch":
        rest = sum(max(1, case["tokens"] - (i * 7) % case["tokens"] if i % 2 else case["tokens"]) % ps for i in range(case["forks"]))
        return {"bytes": 2 * rest * token * case["caches"] + meta, "flops": 0}
    moved = 2 * (case["parents"] // 2) * held
    return {"bytes": 2 * moved * ps * token * case["caches"] + 4 * meta, "flops": 0}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "rotary": _exact_rotary, "pages": _exact_pages}[case["op"]](st, case)


def _exact_conv(st, case):
    """Sequence by sequence: its earlier inputs and its own in one column, weighted sums along it."""
    W, starts = case["W"], st["seq_start"].tolist()
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device=DEV)
    pool = st["state"].double()
    for s, slot in enumerate(st["slots"].tolist()):
        a, b = starts[s], starts[s + 1]
        old = pool[slot] if case["step"] or int(st["load_state"][s]) else torch.zeros_like(pool[slot])
        col = torch.cat((old, st["x"][a:b].double()))
        v = (col.unfold(0, W, 1) * st["weight"].double().T).sum(-1) + st["bias"].double()
        y[a:b] = v * torch.sigmoid(v)
        pool[slot] = col[-(W - 1):]
    return y, pool


def _exact_scan(st, case):
    """Token by token, the sequences side by side, longest first."""
    lens = _lengths(case["S"], case["L"], case["even"])
    starts, per = _starts(lens), case["C"] // case["G"]
    dt = torch.nn.functional.softplus(st["dt"].double() + st["dt_bias"].double(), threshold=1e9)
    A, pool = st["A"].double(), st["state"].double()
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device=DEV)
    slots = st["slots"].tolist()
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    h = torch.stack([pool[slots[i]] if case["step"] or int(st["load_state"][i]) else torch.zeros_like(pool[0]) for i in order])
    t = 0
    while t < lens[order[0]]:
        rows = [i for i in order if lens[i] > t]
        k, until = len(rows), min(lens[i] for i in rows)
        at = torch.tensor([starts[i] for i in rows], device=DEV) + t
        part = h[:k].clone()
        while t < until:
            d = dt[at]
            part.mul_(torch.exp(d[..., None] * A))
            part.addcmul_((d * st["x"][at].double())[..., None], st["B"][at].double().repeat_interleave(per, 1))
            y[at] = (part * st["C"][at].double().repeat_interleave(per, 1)).sum(-1)
            t, at = t + 1, at + 1
        h[:k] = part
    y += st["D"].double() * st["x"].double()
    if st["z"] is not None:
        y *= st["z"].double() * torch.sigmoid(st["z"].double())
    for k, i in enumerate(order):
        pool[slots[i]] = h[k]
    return y, pool


def _exact_rotary(st, case):
    """Each pair as a complex number times factor * exp(i position frequency), sequence by sequence."""
    kc, vc, starts = st["k_cache"].double(), st["v_cache"].double(), st["seq_start"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    f, half, page = st["inv_freq"].double(), case["rot"] // 2, case["page"]
    first = torch.arange(half, device=DEV) * 2 if case["inter"] else torch.arange(half, device=DEV)
    second = first + 1 if case["inter"] else first + half

    def turn(t, pos):
        r = t.double().clone()
        w = st["factor"] * torch.exp(1j * pos.double()[:, None] * f)[:, None]
        p = torch.complex(t.double()[..., first], t.double()[..., second]) * w
        r[..., first], r[..., second] = p.real, p.imag
        return r

    for s, n in enumerate(st["kv_len"].tolist()):
        a, b = starts[s], starts[s + 1]
        pos = torch.arange(n - (b - a), n, device=DEV)
        pages = st["page_table"][s].long()[pos // page]
        out[a:b] = turn(st["q"][a:b], pos)
        kc[pages, pos % page] = turn(st["k_new"][a:b], pos)
        vc[pages, pos % page] = st["v_new"][a:b].double()
    return out, kc, vc


def _exact_pages(st, case):
    """The bookkeeping on the host, call by call; the caches follow the list of copies."""
    ps, table, kv, ref = case["page"], st["page_table"].tolist(), st["kv_len"].tolist(), st["page_ref"].tolist()
    caches, status, lives = st["caches"].clone(), st["status"].tolist(), []
    count = lambda n: -(-n // ps)                                    # noqa: E731

    def release(rows):
        for r in rows:
            for k in range(count(kv[r])):
                ref[table[r][k]] -= 1
                table[r][k] = -1
            kv[r] = 0

    def extend(rows, add):
        asked, there, result = 0, ref.count(0), []
        free = [p for p, n in enumerate(ref) if n == 0]
        for r, n in zip(rows, add):
            need = count(kv[r] + n) - count(kv[r])
            asked += need
            result.append(int(need > 0 and asked > there))
            if not result[-1]:
                for k in range(need):
                    page = free[asked - need + k]
                    table[r][count(kv[r]) + k] = page
                    ref[page] = 1
                kv[r] += n
        return result

    if case["kind"] == "branch":
        src, dst = st["src"].tolist(), st["dst"].tolist()
        release(dst)
        free, used, was = [p for p, n in enumerate(ref) if n == 0], 0, list(kv)
        for i, (s, d, n) in enumerate(zip(src, dst, st["length"].tolist())):
            n = min(n, was[s])
            full, rest = divmod(n, ps)
            used += rest > 0
            status[0][i] = int(rest > 0 and used > len(free))
            if status[0][i]:
                continue
            for k in range(full):
                table[d][k] = table[s][k]
                ref[table[s][k]] += 1
            if rest:
                page = free[used - 1]
                table[d][full] = page
                ref[page] = 1
                caches[:, page, :rest] = caches[:, table[s][full], :rest]
            kv[d] = n
        status[1] = extend(dst, st["add"].tolist())
        return tuple(torch.tensor(v, dtype=torch.int32) for v in (table, kv, ref, status)) + (caches.double(),)
    for i, rows in enumerate(st["parts"]):
        release(rows.tolist())
        live = sum(n > 0 for n in ref)
        lives.append(live)
        holes = [p for p in range(live) if ref[p] == 0]
        new = dict(zip([p for p in range(live, len(ref)) if ref[p] > 0], holes))
        for old, page in new.items():
            ref[page], ref[old] = ref[old], 0
        if new:
            caches[:, list(new.values())] = caches[:, list(new)]
        for r, n in enumerate(kv):
            for k in range(count(n)):
                table[r][k] = new.get(table[r][k], table[r][k])
        status[i] = extend(rows.tolist(), st["add"][i].tolist())
    return tuple(torch.tensor(v, dtype=torch.int32) for v in (table, kv, ref, status, lives)) + (caches.double(),)
