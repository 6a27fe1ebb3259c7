"""rssm_rotary_append against its formula in 64 bits."""
import math

import pytest
import torch

import more_operators_ref as ref
from operators_ref import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


def inputs(ql, kv, Hq, Hkv, D, rot, it="bf16", page=16, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)          # noqa: E731
    S, N = len(ql), sum(ql)
    starts = [0]
    for n in ql:
        starts.append(starts[-1] + n)
    per = max([-(-n // page) for n in kv] + [1])
    table = torch.full((S, per), -1, dtype=torch.int32)
    first = [max(0, n - q) // page for n, q in zip(kv, ql)]
    count = [-(-n // page) - f if n else 0 for n, f in zip(kv, first)]
    order, at = torch.randperm(sum(count) + 2, generator=g).int(), 0
    for i in range(S):
        table[i, first[i]:first[i] + count[i]] = order[at:at + count[i]]
        at += count[i]
    P = sum(count) + 2
    return dict(q=rn(N, Hq, D).to(DT[it]), k=rn(N, Hkv, D).to(DT[it]), v=rn(N, Hkv, D).to(DT[it]),
                kc=rn(P, page, Hkv, D).to(DT[it]), vc=rn(P, page, Hkv, D).to(DT[it]), table=table,
                starts=torch.tensor(starts, dtype=torch.int32), kv=torch.tensor(kv, dtype=torch.int32),
                freq=torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float32),
                pos=torch.tensor([n - m + t for n, m in zip(kv, ql) for t in range(m)], dtype=torch.int32),
                seq=[i for i, m in enumerate(ql) for _ in range(m)], page=page)


def check(rp, p, *, inter=False, factor=1.0, positions=None, out=None, d=None):
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)} if d is None else d
    out = torch.full(p["q"].shape, math.nan, dtype=p["q"].dtype, device="cuda") if out is None else out
    rp.rssm_rotary_append(d["q"], out, d["kc"], d["vc"], d["k"], d["v"], d["table"], d["starts"], d["kv"], d["freq"],
                          interleaved=inter, factor=factor, positions=None if positions is None else positions.cuda())
    angle = p["pos"] if positions is None else positions
    want, m = ref.turned(p["q"], angle, p["freq"], inter, factor)
    ref.check(out, want, ref.turned_bound(want, m, out.dtype), "q")
    kc, vc = p["kc"].double(), p["vc"].clone()
    bound = torch.zeros_like(kc)
    kt, km = ref.turned(p["k"], angle, p["freq"], inter, factor)
    kb = ref.turned_bound(kt, km, p["kc"].dtype)
    for t, s in enumerate(p["seq"]):
        j = int(p["pos"][t])
        if j < 0 or j // p["page"] >= p["table"].shape[1]:
            continue
        pg = int(p["table"][s, j // p["page"]])
        if 0 <= pg < kc.shape[0]:
            kc[pg, j % p["page"]], bound[pg, j % p["page"]], vc[pg, j % p["page"]] = kt[t], kb[t], p["v"][t]
    diff = (d["kc"].cpu().double() - kc).abs()
    assert (diff <= bound).all(), f"k: {float((diff - bound).max())} past the bound"
    assert torch.equal(d["vc"].cpu(), vc)
    return out


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 112)])
def test_layouts_and_parts_of_the_head(rp, it, inter, D, rot):
    check(rp, inputs([3, 1, 0, 40], [50, 1, 9, 40], 8, 2, D, rot, it, seed=rot), inter=inter, factor=1.25)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (32, 8), (64, 1), (3, 3)])
def test_heads(rp, Hq, Hkv):
    check(rp, inputs([1, 17], [33, 17], Hq, Hkv, 128, 128, seed=Hq))


@pytest.mark.parametrize("page", [1, 7, 16, 48, 256])
def test_pages(rp, page):
    check(rp, inputs([5, 60, 1], [30, 200, 257], 4, 2, 64, 64, page=page, seed=page), inter=True)


def test_one_share_a_token(rp):
    """Many tokens: a wavefront takes all heads of one."""
    check(rp, inputs([4097, 300], [5000, 300], 4, 1, 64, 32, page=64, seed=3))


def test_many_sequences(rp):
    check(rp, inputs([i % 3 for i in range(300)], [i % 3 + i for i in range(300)], 2, 1, 64, 64, seed=4))


@pytest.mark.parametrize("it", ["f32", "bf16"])
def test_far_positions(rp, it):
    """Angles of millions of turns keep their fraction."""
    far = [2 ** 31 - 1, 10 ** 9 + 7, 2 ** 24 + 1, 131071, -5, 0]
    p = inputs([6], [6], 4, 2, 128, 128, it, seed=5)
    check(rp, p, positions=torch.tensor(far, dtype=torch.int32))


def test_in_place_and_views(rp):
    p = inputs([9, 20], [9, 100], 8, 2, 128, 96, "f16", seed=6)
    N = 29
    wide = torch.full((N, (8 + 2 + 2) * 128 + 8), math.nan, dtype=torch.float16, device="cuda")
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
    for k, a, h in (("q", 0, 8), ("k", 1024, 2), ("v", 1280, 2)):
        wide[:, a:a + h * 128] = p[k].reshape(N, -1).cuda()
        d[k] = wide[:, a:a + h * 128].unflatten(1, (h, 128))
    check(rp, p, d=d, out=d["q"])
    assert torch.isnan(wide[:, -8:]).all()


def test_strided_caches(rp):
    """Pages of [heads, tokens, dim], keys and values of a page side by side."""
    p = inputs([9, 20], [9, 100], 4, 2, 64, 64, seed=7)
    P = p["kc"].shape[0]
    both = torch.zeros(P, 2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
    for i, k in enumerate(("kc", "vc")):
        view = both[:, i].transpose(1, 2)
        view.copy_(p[k])
        d[k] = view
    check(rp, p, d=d)


def test_bad_pages_and_positions_before_the_first(rp):
    """Their queries are turned, nothing is appended."""
    p = inputs([6, 8, 3], [40, 30, 3], 4, 2, 64, 64, seed=8)
    p["table"][0, 2] = 10 ** 6
    p["table"][1, 1] = -1
    p["kv"][2] = 1                        # two of the three new tokens lie before the first place
    p["pos"][-3:] = torch.tensor([-2, -1, 0], dtype=torch.int32)
    check(rp, p)


def test_rows_of_no_sequence_are_left_alone(rp):
    p = inputs([6, 4], [40, 30], 4, 2, 64, 64, seed=9)
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
    d["starts"] = torch.tensor([2, 6, 8], dtype=torch.int32, device="cuda")
    out = torch.full((10, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    rp.rssm_rotary_append(d["q"], out, d["kc"], d["vc"], d["k"], d["v"], d["table"], d["starts"], d["kv"], d["freq"])
    assert (out[:2] == 7).all() and (out[8:] == 7).all() and not (out[2:8] == 7).all(2).any()


def test_queries_alone_and_keys_alone(rp):
    p = inputs([6, 4], [40, 30], 4, 2, 64, 64, seed=10)
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
    both, alone, free = (torch.zeros_like(d["q"]) for _ in range(3))
    kc, vc = d["kc"].clone(), d["vc"].clone()
    rp.rssm_rotary_append(d["q"], both, d["kc"], d["vc"], d["k"], d["v"], d["table"], d["starts"], d["kv"], d["freq"])
    rp.rssm_rotary_append(d["q"], alone, None, None, None, None, None, d["starts"], d["kv"], d["freq"])
    rp.rssm_rotary_append(d["q"], free, None, None, None, None, None, None, None, d["freq"], positions=d["pos"])
    rp.rssm_rotary_append(None, None, kc, vc, d["k"], d["v"], d["table"], d["starts"], d["kv"], d["freq"])
    assert torch.equal(both, alone) and torch.equal(both, free)
    assert torch.equal(kc, d["kc"]) and torch.equal(vc, d["vc"])


def test_attention_sees_what_append_and_torch_would_give(rp):
    """Through the attention that reads the cache: relative positions alone matter."""
    p = inputs([12], [12], 4, 2, 64, 64, "f32", seed=11)
    outs = []
    for shift in (0, 1000):
        d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
        q, o = torch.empty_like(d["q"]), torch.empty_like(d["q"])
        rp.rssm_rotary_append(d["q"], q, d["kc"], d["vc"], d["k"], d["v"], d["table"], d["starts"], d["kv"], d["freq"], positions=d["pos"] + shift)
        rp.rssm_paged_attention(q, d["kc"], d["vc"], d["table"], d["starts"], d["kv"], o, max_seq_len=12, max_kv_len=12)
        outs.append(o)
    # scores of up to 64 terms of size about 64 / 8, each with 12 half steps twice; weights change by as much
    assert (outs[0] - outs[1]).abs().max() <= 2 * 24 * ref.STEP * 64 * 4


def test_no_tokens(rp):
    p = inputs([0], [5], 4, 2, 64, 64, seed=12)
    check(rp, p)


def test_captured_and_replayed(rp):
    p = inputs([1] * 5, [40, 3, 100, 17, 64], 8, 2, 128, 128, seed=13)
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
    a, b = torch.zeros_like(d["q"]), torch.zeros_like(d["q"])
    ka, va = d["kc"].clone(), d["vc"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rp.rssm_rotary_append(d["q"], b, d["kc"], d["vc"], d["k"], d["v"], d["table"], d["starts"], d["kv"], d["freq"])
    for i in range(4):
        d["q"].add_(1.0)
        d["kv"].sub_(1)
        rp.rssm_rotary_append(d["q"], a, ka, va, d["k"], d["v"], d["table"], d["starts"], d["kv"], d["freq"])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(ka, d["kc"]) and torch.equal(va, d["vc"])
