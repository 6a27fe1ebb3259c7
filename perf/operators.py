"""Timing cases and plain forms of the prompt-side operators of a Mamba-2 hybrid decoder.

Four operators, each in the layout the library takes it:
  chunk   linear attention with a decay for each head over ragged prompts (chunked form)
  step    the same recurrence for one new token per request
  attend  append of a chunk of new tokens to a paged key/value cache, and their causal
          attention over it (optionally a sliding window plus first tokens that stay visible)
  norm    gate, norm, residual scale and add after a block, and the norm before the next one

`own` selects between the plain form (elementary torch operations in 32 bits, angles and long
sums in 64) and the library's entry points.  `exact` is each definition once more in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
DIM, DSTATE = 64, 128        # the library's compiled state tile
EPS = 1e-5


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # a chat-sized prompt on a small model: latency counts
        dict(name="chunk_prompt_short", op="chunk", S=1, L=97, even=True, H=8, hpg=4, it="bf16", st="f32", z=True, resume=False),
        # one long document on one shard of a model: few heads, a long sequence axis
        dict(name="chunk_document", op="chunk", S=1, L=16384, even=True, H=64, hpg=8, it="bf16", st="bf16", z=True, resume=True),
        # a batch of ragged prompts at the full head count, some of them later chunks of a prompt
        dict(name="chunk_batch", op="chunk", S=12, L=2011, even=False, H=256, hpg=32, it="bf16", st="f32", z=True, resume=True),
        # single-token decoding of one request, and of a full batch of the large shape
        dict(name="step_one", op="step", S=1, H=256, hpg=32, it="bf16", st="bf16", z=True),
        dict(name="step_batch", op="step", S=256, H=256, hpg=32, it="bf16", st="bf16", z=True),
        # a mid-size batch with an fp32 state and fp16 activations
        dict(name="step_f16", op="step", S=37, H=64, hpg=8, it="f16", st="f32", z=False),
        # decoding against a paged cache: a ragged batch, and one request with a very long context
        dict(name="attend_decode_batch", op="attend", S=64, Q=1, L=8192, even=False, Hq=32, Hkv=8, D=128, page=16, it="bf16", window=0, sinks=0),
        dict(name="attend_decode_long", op="attend", S=1, Q=1, L=131071, even=True, Hq=32, Hkv=4, D=128, page=64, it="bf16", window=0, sinks=0),
        # a chunk of a long prompt over what the cache already holds
        dict(name="attend_prompt", op="attend", S=1, Q=2048, L=16384, even=True, Hq=32, Hkv=8, D=128, page=16, it="bf16", window=0, sinks=0),
        # ragged chunks under a sliding window with first tokens kept
        dict(name="attend_window", op="attend", S=5, Q=731, L=9001, even=False, Hq=16, Hkv=16, D=64, page=48, it="f16", window=1024, sinks=4),
        # a prefill batch's rows, and a decode batch's rows with grouped norm
        dict(name="norm_prompt", op="norm", rows=16384, C=8192, groups=1, it="bf16", rt="f32", z=False, post=True),
        dict(name="norm_decode", op="norm", rows=7, C=4096, groups=8, it="bf16", rt="bf16", z=True, post=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "step", "attend", "norm"])
    it = rng.choice(["bf16", "f16"])
    if op in ("chunk", "step"):
        hpg = rng.choice([1, 4, 8, 32])
        H = hpg * _log(rng, 1, 8)
        c = dict(op=op, H=H, hpg=hpg, it=it, st=rng.choice(["f32", "bf16", "f16"]), z=rng.random() < 0.5)
        if op == "step":
            return dict(c, S=_log(rng, 1, 256))
        S = _log(rng, 1, 12)
        return dict(c, S=S, L=_log(rng, 1, min(16384, 3000000 // (S * H) + 1)), even=rng.random() < 0.3,
                    resume=rng.random() < 0.5)
    if op == "attend":
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 8])
        S = _log(rng, 1, 64)
        L = _log(rng, 1, 131072 // S)
        Q = 1 if rng.random() < 0.4 else min(L, _log(rng, 1, 2048))
        Q = max(1, min(Q, 900000000 // (S * L * Hq)))
        w = rng.random() < 0.4
        return dict(op=op, S=S, Q=Q, L=L, even=rng.random() < 0.3, Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128]),
                    page=rng.choice([16, 24, 48, 64, 256]), it=it, window=_log(rng, 16, 4096) if w else 0,
                    sinks=rng.randint(0, 8) if w else 0)
    g = rng.choice([1, 1, 4, 8])
    return dict(op=op, rows=_log(rng, 1, 16384), C=g * 8 * _log(rng, 8, 1024 // g), groups=g, it=it,
                rt=rng.choice(["f32", "bf16", "f16"]) if it == "f16" else rng.choice(["f32", "bf16"]),
                z=rng.random() < 0.5, post=rng.random() < 0.7)


def _lengths(S, L, even):
    """Ragged lengths from 1 to L, spread evenly (the first is L)."""
    return [L if even or i == 0 else max(1, int(L * ((i * 0.6180339887498949) % 1.0))) for i in range(S)]


def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return s


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _recurrent_inputs(case, g, N):
    H, G, it = case["H"], case["H"] // case["hpg"], DTYPES[case["it"]]
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)          # noqa: E731
    ru = lambda *s: torch.rand(s, generator=g, device=DEV)           # noqa: E731
    sd = 1.0 / math.sqrt(DSTATE)
    return dict(
        state=rn(case["S"], H, DIM, DSTATE).to(DTYPES[case["st"]]),
        A=-torch.exp(ru(H) * math.log(16.0)), D=0.5 + ru(H),
        dt_bias=torch.log(torch.expm1(0.001 + 0.099 * ru(H))),
        x=rn(N, H, DIM).to(it), B=(rn(N, G, DSTATE) * sd).to(it), C=(rn(N, G, DSTATE) * sd).to(it),
        dt=rn(N, H) * 0.3, z=rn(N, H, DIM).to(it) if case["z"] else None,
        y=torch.zeros(N, H, DIM, dtype=it, device=DEV),
        slots=torch.randperm(case["S"], generator=g, device=DEV).int())


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    st = dict(case=case, op=case["op"])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)          # noqa: E731
    if case["op"] == "step":
        st.update(_recurrent_inputs(case, g, case["S"]))
    elif case["op"] == "chunk":
        lens = _lengths(case["S"], case["L"], case["even"])
        st.update(_recurrent_inputs(case, g, sum(lens)))
        st["seq_start"] = i32(_starts(lens))
        # 1: a later chunk of a prompt, which continues from its slot's state; 0: a new prompt
        st["load_state"] = i32([1 if case["resume"] and i % 3 != 2 else 0 for i in range(case["S"])])
    elif case["op"] == "attend":
        it, S, D, page = DTYPES[case["it"]], case["S"], case["D"], case["page"]
        kv = _lengths(S, case["L"], case["even"])
        ql = [min(case["Q"], n) for n in kv]
        per = (case["L"] + page - 1) // page
        need = sum((n + page - 1) // page for n in kv)
        table = torch.randint(0, need, (S, per), generator=g, device=DEV).int()
        order, at = torch.randperm(need, generator=g, device=DEV).int(), 0
        for i, n in enumerate(kv):
            k = (n + page - 1) // page
            table[i, :k] = order[at:at + k]
            at += k
        N = sum(ql)
        st.update(q=rn(N, case["Hq"], D).to(it), k_new=rn(N, case["Hkv"], D).to(it), v_new=rn(N, case["Hkv"], D).to(it),
                  k_cache=rn(need, page, case["Hkv"], D).to(it), v_cache=rn(need, page, case["Hkv"], D).to(it),
                  page_table=table, seq_start=i32(_starts(ql)), kv_len=i32(kv),
                  out=torch.zeros(N, case["Hq"], D, dtype=it, device=DEV), max_q=max(ql), max_kv=max(kv))
    else:
        it, rt, R, C = DTYPES[case["it"]], DTYPES[case["rt"]], case["rows"], case["C"]
        st.update(y=rn(R, C).to(it), z=rn(R, C).to(it) if case["z"] else None, residual=(rn(R, C) * 2).to(rt),
                  post_weight=1 + 0.1 * rn(C) if case["post"] else None, pre_weight=1 + 0.1 * rn(C),
                  channel_scale=0.5 + 0.1 * rn(C), residual_out=torch.empty(R, C, dtype=rt, device=DEV),
                  normed=torch.empty(R, C, dtype=it, device=DEV))
    return st


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(st):
    return (_own if own else _plain)[st["op"]](st)


def _own_chunk(st):
    import replayssm_persistent_rssm_amd as rp
    rp.rssm_linear_attention(st["state"], st["A"], st["x"], st["B"], st["C"], st["dt"], st["y"], st["slots"],
                             st["seq_start"], max_seq_len=st["case"]["L"], load_state=st["load_state"], D=st["D"],
                             dt_bias=st["dt_bias"], z=st["z"])
    return st["y"], st["state"]


def _own_step(st):
    import replayssm_persistent_rssm_amd as rp
    rp.rssm_linear_attention_step(st["state"], st["A"], st["x"], st["B"], st["C"], st["dt"], st["y"], st["slots"],
                                  D=st["D"], dt_bias=st["dt_bias"], z=st["z"])
    return st["y"], st["state"]


def _own_attend(st):
    import replayssm_persistent_rssm_amd as rp
    c = st["case"]
    rp.rssm_paged_append(st["k_cache"], st["v_cache"], st["k_new"], st["v_new"], st["page_table"], st["seq_start"],
                         st["kv_len"])
    rp.rssm_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["page_table"], st["seq_start"], st["kv_len"],
                            st["out"], max_seq_len=st["max_q"], max_kv_len=st["max_kv"], window=c["window"],
                            sinks=c["sinks"])
    return st["out"], st["k_cache"], st["v_cache"]


def _own_norm(st):
    import replayssm_persistent_rssm_amd as rp
    rp.rssm_block_norm(st["y"], st["residual"], st["residual_out"], st["normed"], z=st["z"],
                       post_weight=st["post_weight"], pre_weight=st["pre_weight"], channel_scale=st["channel_scale"],
                       residual_scale=0.7, groups=st["case"]["groups"], eps=EPS)
    return st["residual_out"], st["normed"]


_own = {"chunk": _own_chunk, "step": _own_step, "attend": _own_attend, "norm": _own_norm}


def _softplus64(st):
    v = st["dt"].double() + st["dt_bias"].double()
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_step(st):
    c = st["case"]
    S, H, G = c["S"], c["H"], c["H"] // c["hpg"]
    dt = _softplus64(st).float()
    slots = st["slots"].long()
    x = st["x"].float()
    S0 = st["state"][slots].float().view(S, G, c["hpg"], DIM, DSTATE)
    a = torch.exp(dt * st["A"]).view(S, G, c["hpg"], 1, 1)
    dx = (dt[:, :, None] * x).view(S, G, c["hpg"], DIM, 1)
    S1 = a * S0 + dx * st["B"].float().view(S, G, 1, 1, DSTATE)
    y = (S1 * st["C"].float().view(S, G, 1, 1, DSTATE)).sum(-1).view(S, H, DIM) + st["D"][:, None] * x
    if st["z"] is not None:
        y = y * _silu(st["z"].float())
    st["state"][slots] = S1.view(S, H, DIM, DSTATE).to(st["state"].dtype)
    st["y"].copy_(y)
    return st["y"], st["state"]


def _plain_chunk(st, Q=64):
    """Chunks of Q tokens: products inside a chunk, and a decay-weighted sum of the chunks' states before it."""
    c = st["case"]
    S, H, G, L = c["S"], c["H"], c["H"] // c["hpg"], c["L"]
    nc = (L + Q - 1) // Q
    starts = st["seq_start"].long()
    pos = torch.arange(nc * Q, device=DEV)
    live = pos[None] < (starts[1:] - starts[:-1])[:, None]                       # [S, nc*Q]
    idx = torch.where(live, starts[:-1, None] + pos[None], 0)
    pick = lambda t: torch.where(live.view(S, -1, *([1] * (t.dim() - 1))), t[idx], 0)   # noqa: E731
    dt = pick(_softplus64(st))                                                   # [S, nc*Q, H], 0 past the end
    la = (dt * st["A"].double()).view(S, nc, Q, H).cumsum(2).transpose(2, 3)      # [S, nc, H, Q]
    dt = dt.float().view(S, nc, Q, H).transpose(2, 3)
    x = pick(st["x"]).float().view(S, nc, Q, H, DIM).transpose(2, 3)             # [S, nc, H, Q, DIM]
    B = pick(st["B"]).float().view(S, nc, Q, G, DSTATE).transpose(2, 3)          # [S, nc, G, Q, DSTATE]
    C = pick(st["C"]).float().view(S, nc, Q, G, DSTATE).transpose(2, 3)
    heads = lambda t: t[:, :, :, None].expand(S, nc, G, c["hpg"], Q, t.shape[-1]).reshape(S, nc, H, Q, t.shape[-1])  # noqa: E731
    i = torch.arange(Q, device=DEV)
    decay = torch.exp(torch.where(i[:, None] >= i[None], (la[..., :, None] - la[..., None, :]).float(), -math.inf))
    M = heads(torch.matmul(C, B.transpose(-1, -2))) * decay * dt[..., None, :]
    y = torch.matmul(M, x)
    del M, decay
    end = la[..., -1]                                                            # [S, nc, H]
    w = torch.exp((end[..., None] - la).float()) * dt
    own_state = torch.matmul((x * w[..., None]).transpose(-1, -2), heads(B))     # [S, nc, H, DIM, DSTATE]
    T = torch.cat([torch.zeros_like(end[:, :1]), end.cumsum(1)], 1).transpose(1, 2)   # [S, H, nc+1]
    k = torch.arange(nc + 1, device=DEV)
    E = torch.exp(torch.where(k[:, None] >= k[None], (T[..., :, None] - T[..., None, :]), -math.inf)).float()
    slots = st["slots"].long()
    first = torch.where(st["load_state"].bool().view(S, 1, 1, 1), st["state"][slots].float(), 0).view(S, H, 1, -1)
    # chunk k starts from the initial state (as a chunk before the first) and the states of chunks before k
    before = torch.matmul(E, torch.cat([first, own_state.transpose(1, 2).reshape(S, H, nc, -1)], 2))
    del own_state
    into = before[:, :, :nc].reshape(S, H, nc, DIM, DSTATE).transpose(1, 2)
    y += torch.matmul(heads(C), into.transpose(-1, -2)) * torch.exp(la.float())[..., None]
    y = y.transpose(2, 3).reshape(S, nc * Q, H, DIM)[live] + st["D"][:, None] * st["x"].float()
    if st["z"] is not None:
        y = y * _silu(st["z"].float())
    st["state"][slots] = before[:, :, nc].reshape(S, H, DIM, DSTATE).to(st["state"].dtype)
    st["y"].copy_(y)
    return st["y"], st["state"]


def _places(st):
    """(sequence, position) of each new token."""
    starts = st["seq_start"].long()
    n = torch.arange(st["q"].shape[0], device=DEV)
    seq = torch.searchsorted(starts[1:].contiguous(), n, right=True)
    return seq, st["kv_len"].long()[seq] - starts[1:][seq] + n


def _plain_attend(st):
    c = st["case"]
    S, Hq, Hkv, D, page, L, Q = c["S"], c["Hq"], c["Hkv"], c["D"], c["page"], st["max_kv"], st["max_q"]
    seq, pos = _places(st)
    table = st["page_table"].long()
    pg = table[seq, pos // page]
    st["k_cache"][pg, pos % page] = st["k_new"]
    st["v_cache"][pg, pos % page] = st["v_new"]
    j = torch.arange(L, device=DEV)
    has = j[None] < st["kv_len"][:, None]
    rows = torch.where(has, table[:, j // page], 0) * page + (j % page)[None]          # [S, L]
    take = lambda t: t.view(-1, Hkv, D)[rows].float().transpose(1, 2)                  # noqa: E731  [S, Hkv, L, D]
    K, V = take(st["k_cache"]), take(st["v_cache"])
    within = pos - (st["kv_len"].long() - (st["seq_start"][1:] - st["seq_start"][:-1]).long())[seq]
    q = torch.zeros(S, Q, Hq, D, device=DEV)
    q[seq, within] = st["q"].float()
    at = torch.full((S, Q), -1, device=DEV)
    at[seq, within] = pos
    q = q.view(S, Q, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D)   # rows: (head in group, token)
    s = torch.matmul(q, K.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(S, Hkv, Hq // Hkv, Q, L)
    seen = j[None, None] <= at[..., None]
    if c["window"]:
        seen &= (j[None, None] > at[..., None] - c["window"]) | (j < c["sinks"])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(torch.isinf(m), 0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, Hkv, -1, L), V).view(S, Hkv, -1, Q, D) / torch.where(total > 0, total, 1)
    st["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(S, Q, Hq, D)[seq, within])
    return st["out"], st["k_cache"], st["v_cache"]


def _plain_norm(st):
    R, C, g = st["y"].shape[0], st["y"].shape[1], st["case"]["groups"]
    u = st["y"].float()
    if st["z"] is not None:
        u = u * _silu(st["z"].float())
    if st["post_weight"] is not None:
        u = u.view(R, g, C // g)
        u = (u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)).view(R, C) * st["post_weight"]
    r = st["residual"].float() + 0.7 * st["channel_scale"] * u
    n = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * st["pre_weight"]
    st["residual_out"].copy_(r)
    st["normed"].copy_(n)
    return st["residual_out"], st["normed"]


_plain = {"chunk": _plain_chunk, "step": _plain_step, "attend": _plain_attend, "norm": _plain_norm}


# --------------------------------------------------------------------------
# The work of one pass
# --------------------------------------------------------------------------
def work(case):
    if case["op"] in ("chunk", "step"):
        H, G, e = case["H"], case["H"] // case["hpg"], SIZE[case["it"]]
        lens = _lengths(case["S"], case["L"], case["even"]) if case["op"] == "chunk" else [1] * case["S"]
        N = sum(lens)
        loads = sum(1 for i in range(case["S"]) if case["op"] == "step" or (case["resume"] and i % 3 != 2))
        tile = H * DIM * DSTATE
        b = tile * SIZE[case["st"]] * (case["S"] + loads)
        b += N * (H * DIM * e * (3 if case["z"] else 2) + 2 * G * DSTATE * e + H * 4) + 12 * H
        return {"bytes": b, "flops": N * tile * 5}      # decay, update (2) and readout (2) of each state element
    if case["op"] == "attend":
        e, D, w = SIZE[case["it"]], case["D"], case["window"]
        kv = _lengths(case["S"], case["L"], case["even"])
        b = f = 0
        for n in kv:
            q = min(case["Q"], n)
            pairs = sum(_visible(p, w, case["sinks"]) for p in range(n - q, n))
            rows = n if not w else min(n, min(w + q - 1, n) + case["sinks"])
            b += 2 * rows * case["Hkv"] * D * e + 2 * q * case["Hkv"] * D * e + 2 * q * case["Hq"] * D * e
            f += 4 * pairs * case["Hq"] * D
        return {"bytes": b, "flops": f}
    e, r, n = SIZE[case["it"]], SIZE[case["rt"]], case["rows"] * case["C"]
    return {"bytes": n * (e * (3 if case["z"] else 2) + 2 * r) + case["C"] * 4 * (3 if case["post"] else 2), "flops": 12 * n}


def _visible(pos, window, sinks):
    if not window:
        return pos + 1
    low = max(0, pos - window + 1)
    return pos + 1 - low + min(sinks, low)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("chunk", "step"):
        return _exact_recurrence(st, case)
    if case["op"] == "attend":
        return _exact_attend(st, case)
    y, r = st["y"].double(), st["residual"].double()
    if st["z"] is not None:
        z = st["z"].double()
        y = y * z * torch.sigmoid(z)
    if st["post_weight"] is not None:
        parts = [p / torch.sqrt(p.pow(2).sum(1, keepdim=True) / p.shape[1] + EPS) for p in y.chunk(case["groups"], 1)]
        y = torch.cat(parts, 1) * st["post_weight"].double()
    r = r + y * (0.7 * st["channel_scale"].double())
    return r, r / torch.sqrt(r.pow(2).sum(1, keepdim=True) / case["C"] + EPS) * st["pre_weight"].double()


def _exact_recurrence(st, case):
    """Token by token: S <- exp(dt A) S + dt x B^T, y = S C + D x."""
    lens = _lengths(case["S"], case["L"], case["even"]) if case["op"] == "chunk" else [1] * case["S"]
    starts = _starts(lens)
    if sum(lens) * case["H"] > 9000000 or max(lens) > 20000:
        return None
    dt = torch.nn.functional.softplus(st["dt"].double() + st["dt_bias"].double(), threshold=1e9)
    slots = st["slots"].tolist()
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device=DEV)
    pool = st["state"].double()
    S = torch.stack([pool[s] if case["op"] == "step" or int(st["load_state"][i]) else torch.zeros_like(pool[s])
                     for i, s in enumerate(slots)])
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    S = S[order]
    t = 0
    while t < max(lens):
        rows = [i for i in order if lens[i] > t]
        n = torch.tensor([starts[i] for i in rows], device=DEV)
        live = len(rows)
        until = min(lens[i] for i in rows)
        Sl = S[:live].contiguous()
        while t < until:
            at = n + t
            d = dt[at]
            Bt = st["B"][at].double().repeat_interleave(case["hpg"], 1)
            Ct = st["C"][at].double().repeat_interleave(case["hpg"], 1)
            Sl.mul_(torch.exp(d * st["A"].double())[:, :, None, None])
            Sl.addcmul_((d[:, :, None] * st["x"][at].double())[..., None], Bt[:, :, None, :])
            y[at] = torch.matmul(Sl, Ct[..., None])[..., 0]
            t += 1
        S[:live] = Sl
    y += st["D"].double()[:, None] * st["x"].double()
    if st["z"] is not None:
        y *= st["z"].double() * torch.sigmoid(st["z"].double())
    for k, i in enumerate(order):
        pool[slots[i]] = S[k]
    return y, pool


def _exact_attend(st, case):
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    page, group, starts = case["page"], case["Hq"] // case["Hkv"], st["seq_start"].tolist()
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for s, n in enumerate(st["kv_len"].tolist()):
        a, b = starts[s], starts[s + 1]
        pages = st["page_table"][s, :(n + page - 1) // page].long()
        pos = torch.arange(n - (b - a), n, device=DEV)
        kc[pages[pos // page], pos % page] = st["k_new"][a:b].double()
        vc[pages[pos // page], pos % page] = st["v_new"][a:b].double()
        j = torch.arange(n, device=DEV)
        far = j[None] > pos[:, None]
        if case["window"]:
            far = far | ((pos[:, None] - j[None] >= case["window"]) & (j[None] >= case["sinks"]))
        for h in range(case["Hkv"]):
            K, V = kc[pages, :, h].reshape(-1, case["D"])[:n], vc[pages, :, h].reshape(-1, case["D"])[:n]
            for e in range(h * group, (h + 1) * group):
                s_ = (st["q"][a:b, e].double() @ K.T) / math.sqrt(case["D"])
                s_[far] = -math.inf
                out[a:b, e] = torch.softmax(s_, 1) @ V
    return out, kc, vc
