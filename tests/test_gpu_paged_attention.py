"""rssm_paged_append and rssm_paged_attention against the definition in 64 bits."""
import math

import pytest
import torch

import operators_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


def make(kv, ql, Hq, Hkv, D, page, it, *, seed=0, spare=3, extra_cols=2):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g).to(ref.DT[it])       # noqa: E731
    need = [(n + page - 1) // page for n in kv]
    P = sum(need) + spare
    table = torch.full((len(kv), max(need + [1]) + extra_cols), -1, dtype=torch.int32)
    order, at = torch.randperm(P, generator=g).int(), 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in ql:
        starts.append(starts[-1] + n)
    N = starts[-1]
    return dict(q=rn(N, Hq, D), kc=rn(P, page, Hkv, D), vc=rn(P, page, Hkv, D), kn=rn(N, Hkv, D), vn=rn(N, Hkv, D),
                table=table, seq_start=torch.tensor(starts, dtype=torch.int32), kv=torch.tensor(kv, dtype=torch.int32),
                seqs=[(starts[i], n) for i, n in enumerate(ql)])


def attend(rp, p, *, lse=True, out=None, **kw):
    c = {k: p[k].cuda() for k in ("q", "kc", "vc", "table", "seq_start", "kv")}
    out = torch.full(p["q"].shape, math.nan, dtype=p["q"].dtype, device="cuda") if out is None else out
    l = torch.full(p["q"].shape[:2], math.nan, device="cuda") if lse else None
    kw = dict(dict(max_seq_len=max([n for _, n in p["seqs"]], default=0), max_kv_len=int(p["kv"].max())), **kw)
    rp.rssm_paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["seq_start"], c["kv"], out, lse=l, **kw)
    torch.cuda.synchronize()
    return out, l


def check(rp, p, **kw):
    out, l = attend(rp, p, **kw)
    e, mag, lse, err = ref.paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seqs"], p["kv"],
                                           **{k: v for k, v in kw.items() if k in ("scale", "window", "sinks")})
    ref.check(out, e, ref.out_bound(e, mag, err, out.dtype), "out")
    empty = lse == -math.inf
    got = l.cpu().double()
    assert torch.equal(got == -math.inf, empty)
    assert (out.cpu()[empty] == 0).all()
    bound = err + 2.0 ** -20 * lse.abs().clamp(min=1)
    ref.check(got[~empty], lse[~empty], bound[~empty], "lse")
    return out, l


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 16, 24, 100])
def test_single_tokens(rp, it, D, page):
    check(rp, make([1, 31, 32, 33, 200], [1] * 5, 8, 2, D, page, it, seed=1))


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (6, 2), (8, 1)])
def test_chunks(rp, it, D, Hq, Hkv):
    check(rp, make([1, 70, 64, 130, 40], [1, 37, 64, 5, 0], Hq, Hkv, D, 16, it, seed=2))


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (50, 0), (50, 3), (64, 130), (1000, 2)])
@pytest.mark.parametrize("ql", [1, 90])
def test_window_and_sinks(rp, it, window, sinks, ql):
    check(rp, make([300, 129, 90], [ql, ql, min(ql, 90)], 4, 2, 64, 24, it, seed=3), window=window, sinks=sinks)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ql", [1, 40])
def test_long_cache_is_split(rp, it, ql):
    p = make([2500, 600], [ql, 1], 4, 2, 128, 48, it, seed=4)
    c = [p[k].cuda() for k in ("q", "kc", "vc", "table", "seq_start", "kv", "q")]
    assert rp.rssm_paged_attention_workspace(*c, max_seq_len=ql, max_kv_len=2500) > 0
    a = check(rp, p)
    b = attend(rp, p)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(rp, p, window=700, sinks=70)


def test_queries_that_see_nothing(rp):
    """More new tokens than cached ones: the first positions are negative."""
    check(rp, make([3, 0, 20], [10, 4, 20], 4, 2, 64, 16, "bf16", seed=5))
    check(rp, make([0, 2], [1, 1], 4, 2, 64, 16, "bf16", seed=5))


@pytest.mark.parametrize("ql", [1, 50])
def test_pages_outside_the_cache_are_not_visible(rp, ql):
    p = make([200, 120], [ql, ql], 4, 2, 64, 16, "bf16", seed=6)
    p["table"][0, 3] = -7
    p["table"][0, 5] = p["kc"].shape[0]
    p["table"][1, :] = -1
    check(rp, p)
    check(rp, p, window=30, sinks=60)


def test_tokens_past_the_table_are_not_visible(rp):
    p = make([200], [20], 4, 2, 64, 16, "bf16", seed=7, extra_cols=0)
    p["table"] = p["table"][:, :9].contiguous()
    check(rp, p)
    p = make([200], [1], 4, 2, 64, 16, "bf16", seed=7, extra_cols=0)
    p["table"] = p["table"][:, :9].contiguous()
    check(rp, p)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("ql", [3, 70])
def test_masked_nonfinite_values_stay_masked(rp, it, value, ql):
    """A non-finite key or value reaches only the queries that see it."""
    kw = dict(window=40, sinks=2)
    p = make([150, 90], [ql, ql], 4, 2, 64, 16, it, seed=8)
    clean, _ = attend(rp, p, **kw)
    late, early = 150 - ql + 1, 150 - ql - 39       # seen from the second query on; only by the first
    for pos in (late, early):
        page = int(p["table"][0, pos // 16])
        for t in ("kc", "vc"):
            p[t][page, pos % 16] = value
    # and everything beside the sequences' own tokens
    used = {(int(p["table"][s, j // 16]), j % 16) for s, n in enumerate((150, 90)) for j in range(n)}
    for a in range(p["kc"].shape[0]):
        for b in range(16):
            if (a, b) not in used:
                p["kc"][a, b], p["vc"][a, b] = value, value
    out, _ = attend(rp, p, **kw)
    pos = torch.arange(150 - ql, 150)
    sees = ((pos >= late) & (late > pos - 40)) | ((pos >= early) & (early > pos - 40))
    rows = torch.cat([~sees, torch.ones(ql, dtype=torch.bool)])
    assert bool(rows[:ql].any()) or ql == 3
    off = (out[rows].float() - clean[rows].float()).abs()
    e, mag, _, err = ref.paged_attention(p["q"], torch.nan_to_num(p["kc"], 0, 0, 0), torch.nan_to_num(p["vc"], 0, 0, 0),
                                         p["table"], p["seqs"], p["kv"], **kw)
    assert torch.isfinite(out[rows]).all()
    ref.check(out[rows], e[rows], ref.out_bound(e, mag, err, out.dtype)[rows], "out")
    assert off.numel() == 0 or torch.isfinite(off).all()


def test_scores_of_large_size(rp):
    """Scores in the hundreds: the running maximum carries the sums."""
    p = make([500, 70], [64, 70], 4, 2, 128, 16, "f32", seed=9)
    p["q"] *= 30
    check(rp, p)
    check(rp, p, scale=0.003)


def test_equal_keys(rp):
    p = make([100], [1], 4, 2, 64, 16, "bf16", seed=10)
    p["kc"][:] = 1.0
    check(rp, p)


def test_layouts(rp):
    """Head-major caches, rows of wider tensors, a table with longer rows."""
    p = make([90, 33], [20, 1], 4, 2, 64, 16, "bf16", seed=11)
    want, _ = attend(rp, p)
    kc, vc = (p[k].transpose(1, 2).contiguous().cuda().transpose(1, 2) for k in ("kc", "vc"))
    q = torch.full((21, 6, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    q[:, 1:5] = p["q"].cuda()
    out = torch.zeros(21, 8, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.full((2, 40), 10 ** 6, dtype=torch.int32, device="cuda")
    table[:, :p["table"].shape[1]] = p["table"].cuda()
    rp.rssm_paged_attention(q[:, 1:5], kc, vc, table[:, :p["table"].shape[1]], p["seq_start"].cuda(), p["kv"].cuda(),
                            out[:, 2:6], max_seq_len=20, max_kv_len=90)
    assert torch.equal(out[:, 2:6], want)
    assert (out[:, :2] == 0).all() and (out[:, 6:] == 0).all()


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("page,head_major", [(16, False), (7, True)])
def test_append(rp, it, page, head_major):
    p = make([40, 3, 0, 25], [13, 3, 2, 0], 4, 2, 64, page, it, seed=12)
    p["table"][0, 39 // page] = -1       # the last page of the first sequence is missing
    kc, vc = p["kc"].clone(), p["vc"].clone()
    for s, (a, n) in enumerate(p["seqs"]):
        for t in range(n):
            pos = int(p["kv"][s]) - n + t
            pg = int(p["table"][s, pos // page]) if pos >= 0 else -1
            if 0 <= pg < kc.shape[0]:
                kc[pg, pos % page], vc[pg, pos % page] = p["kn"][a + t], p["vn"][a + t]
    put = (lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2)) if head_major else (lambda t: t.cuda())
    k, v = put(p["kc"]), put(p["vc"])
    rp.rssm_paged_append(k, v, p["kn"].cuda(), p["vn"].cuda(), p["table"].cuda(), p["seq_start"].cuda(), p["kv"].cuda())
    assert torch.equal(k.cpu(), kc) and torch.equal(v.cpu(), vc)


def test_chunked_prompt_and_decode_equal_one_prompt(rp):
    """A prompt in chunks, then single tokens, each appended first: the outputs
    are those of attending all tokens at once."""
    p = make([150], [150], 4, 2, 64, 16, "f32", seed=13)
    c = {k: p[k].cuda() for k in ("q", "kc", "vc", "kn", "vn", "table")}
    got = torch.zeros_like(c["q"])
    at = 0
    for n in (70, 64, 1, 14, 1):
        ss = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        kv = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        rp.rssm_paged_append(c["kc"], c["vc"], c["kn"][at:at + n], c["vn"][at:at + n], c["table"], ss, kv)
        rp.rssm_paged_attention(c["q"][at:at + n], c["kc"], c["vc"], c["table"], ss, kv, got[at:at + n], max_seq_len=n,
                                max_kv_len=at + n)
        at += n
    p["kc"], p["vc"] = c["kc"].cpu(), c["vc"].cpu()
    e, mag, _, err = ref.paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seqs"], p["kv"])
    ref.check(got, e, ref.out_bound(e, mag, err, got.dtype), "out")


def test_streams_and_graph(rp):
    p = make([2500], [1], 4, 2, 64, 16, "bf16", seed=14)
    c = {k: p[k].cuda() for k in ("q", "kc", "vc", "kn", "vn", "table", "seq_start", "kv")}
    out = torch.zeros_like(c["q"])

    def go(**kw):
        rp.rssm_paged_append(c["kc"], c["vc"], c["kn"], c["vn"], c["table"], c["seq_start"], c["kv"],
                             **{k: v for k, v in kw.items() if k == "stream"})
        rp.rssm_paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["seq_start"], c["kv"], out, max_seq_len=1,
                                max_kv_len=2500, **kw)

    go()
    want = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    go(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        go()
    for k in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {k}"


def test_cache_offsets_past_32_bits(rp):
    p = make([100], [5], 4, 2, 128, 16, "bf16", seed=15)
    P = 1100000                                                   # 16 x 2 x 128 x 1.1e6 = 4.5e9 elements
    kc = torch.empty(P, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    far = torch.arange(P - 8, P - 1, dtype=torch.int32)
    old = p["table"][0, :7].long()
    kc[far.long()], vc[far.long()] = p["kc"][old].cuda(), p["vc"][old].cuda()
    want, _ = check(rp, p)
    table = p["table"].clone()
    table[0, :7] = far
    out = torch.zeros_like(want)
    rp.rssm_paged_attention(p["q"].cuda(), kc, vc, table.cuda(), p["seq_start"].cuda(), p["kv"].cuda(), out,
                            max_seq_len=5, max_kv_len=100)
    assert torch.equal(out, want)


def test_nothing_to_do(rp):
    p = make([10, 0], [0, 0], 4, 2, 64, 16, "bf16", seed=16)
    attend(rp, p)
