"""rssm_selective_scan and rssm_selective_scan_step against their formula in 64 bits."""
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


def inputs(lens, Ch, n=16, G=1, it="bf16", st="f32", seed=0, slots=None, extra=2):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)          # noqa: E731
    ru = lambda *s: torch.rand(s, generator=g)           # noqa: E731
    S, N = len(lens), sum(lens)
    starts = [0]
    for k in lens:
        starts.append(starts[-1] + k)
    return dict(state=rn(S + extra, Ch, n).to(DT[st]), A=-(1 + ru(Ch, n)) * torch.arange(1, n + 1) * 0.6, D=0.5 + ru(Ch),
                bias=torch.log(torch.expm1(0.001 + 0.099 * ru(Ch))), x=rn(N, Ch).to(DT[it]), dt=(0.3 * rn(N, Ch)).to(DT[it]),
                z=rn(N, Ch).to(DT[it]), B=rn(N, G, n).to(DT[it]), C=(rn(N, G, n) / n ** 0.5).to(DT[it]),
                slots=torch.randperm(S + extra, generator=g)[:S].int() if slots is None else torch.tensor(slots, dtype=torch.int32),
                starts=torch.tensor(starts, dtype=torch.int32), seqs=[(starts[i], lens[i]) for i in range(S)],
                load=torch.tensor([i % 3 != 2 for i in range(S)], dtype=torch.int32))


def call(rp, p, d, y, st, *, use=("D", "bias", "z", "load"), step=False, softplus=True, pad=-1, most=None, ws=None):
    kw = dict(D=d["D"] if "D" in use else None, dt_bias=d["bias"] if "bias" in use else None, z=d["z"] if "z" in use else None,
              dt_softplus=softplus, pad_slot_id=pad)
    args = (st, d["A"], d["x"], d["B"], d["C"], d["dt"], y, d["slots"])
    if step:
        rp.rssm_selective_scan_step(*args, **kw)
    else:
        longest = max([n for _, n in p["seqs"]], default=0) if most is None else most
        rp.rssm_selective_scan(*args, d["starts"], max_seq_len=longest, load_state=d["load"] if "load" in use else None,
                               workspace=ws, **kw)


def on_device(p):
    return {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}


def check(rp, p, *, use=("D", "bias", "z", "load"), step=False, softplus=True, pad=-1, most=None, d=None, y=None, st=None, ws=None):
    d = on_device(p) if d is None else d
    y = torch.full(p["x"].shape, math.nan, dtype=p["x"].dtype, device="cuda") if y is None else y
    st = p["state"].cuda() if st is None else st
    call(rp, p, d, y, st, use=use, step=step, softplus=softplus, pad=pad, most=most, ws=ws)
    h = lambda k: p[k] if k in use else None             # noqa: E731
    seqs = [(a, min(n, most) if most is not None else n) for a, n in p["seqs"]]
    want, m, pool, pm = ref.scan(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], seqs, D=h("D"),
                                 bias=h("bias"), z=h("z"), load=None if step else h("load"), softplus=softplus, pad=pad)
    chain = ref.scan_chain(max([n for _, n in seqs], default=0), p["state"].shape[2])
    ref.check(y, want, ref.scan_bound(want, m, y.dtype, chain), "y")
    assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want)), "rows of no sequence are left alone, all others written"
    ref.check(st, pool, ref.scan_bound(pool, pm, st.dtype, chain), "state")
    return y, st


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("st", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Ch,n,G", [(8, 16, 1), (104, 16, 1), (96, 32, 2), (128, 64, 8)])
def test_ragged_prompts(rp, it, st, Ch, n, G):
    """Short ones: no stretches."""
    check(rp, inputs([0, 1, 2, 15, 16, 17, 33, 0, 48], Ch, n, G, it, st, seed=Ch + n))


@pytest.mark.parametrize("lens", [[1], [0], [], [16], [100], [0, 0], [1] * 40])
def test_lengths(rp, lens):
    check(rp, inputs(lens, 64, seed=len(lens)))


@pytest.mark.parametrize("it,st,n", [("bf16", "f32", 16), ("f16", "f16", 32), ("f32", "bf16", 64)])
def test_stretches(rp, it, st, n):
    """Few channels and long sequences: the token axis is split, ends fall inside, at and before the borders."""
    lens = [400, 64, 65, 0, 1, 129, 63, 300]
    p = inputs(lens, 40, n, 1, it, st, seed=n)
    assert rp.rssm_selective_scan_workspace(p["state"].cuda(), *(p[k].cuda() for k in ("A", "x", "B", "C", "dt", "z", "slots", "starts")),
                                            max_seq_len=400) > 0
    check(rp, p)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("st,n,G", [("f32", 16, 1), ("bf16", 32, 4), ("f16", 64, 2)])
def test_wide_batches(rp, it, st, n, G):
    """Enough channels for the form with 16 of them a wavefront, no stretches; with and without all inputs."""
    p = inputs([17, 0, 1, 48, 15, 16, 33, 2, 31], 2048, n, G, it, st, seed=n)
    check(rp, p)
    check(rp, p, use=("bias",))


@pytest.mark.parametrize("n,lens,Ch", [(32, [700], 2056), (64, [600, 3], 1040), (32, [700, 40], 4200)])
def test_long_sequences_of_many_states(rp, n, lens, Ch):
    """At either side of the choice between the forms."""
    check(rp, inputs(lens, Ch, n, 1, "bf16", "f32", seed=n))


def test_more_sequences_than_are_sorted(rp):
    check(rp, inputs([(7 * i) % 23 for i in range(70)], 512, seed=3))


def test_channels_fill_the_device(rp):
    check(rp, inputs([70, 3, 40], 64 * 100, seed=4))


@pytest.mark.parametrize("use", [(), ("D",), ("z",), ("bias",), ("D", "z", "load")])
def test_optional_inputs(rp, use):
    p = inputs([5, 130, 1], 64, it="f16", seed=5)
    check(rp, p, use=use)
    check(rp, inputs([1] * 5, 64, it="f16", seed=6), use=use, step=True)


def test_step_sizes_as_they_are(rp):
    p = inputs([5, 130, 1], 64, it="f32", seed=7)
    p["dt"] = p["dt"].abs() * 0.1
    check(rp, p, softplus=False, use=("D",))


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("st", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("S,Ch,n,G", [(1, 8, 16, 1), (5, 104, 16, 1), (67, 96, 32, 2), (9, 128, 64, 2), (260, 64 * 20, 16, 1),
                                       (3, 96, 16, 6), (6, 240, 32, 5), (130, 16 * 66, 16, 66)])
def test_step(rp, it, st, S, Ch, n, G):
    check(rp, inputs([1] * S, Ch, n, G, it, st, seed=S + n), step=True)


@pytest.mark.parametrize("step", [False, True])
def test_pads_and_slots_outside_the_pool(rp, step):
    p = inputs([1] * 6 if step else [4, 9, 1, 0, 150, 3], 72, seed=8, slots=[-1, 3, 7, 900, -5, 0])
    check(rp, p, step=step)
    check(rp, p, step=step, pad=3)


def test_longer_than_said(rp):
    """Sequences past max_seq_len are cut to it."""
    check(rp, inputs([200, 30, 41], 64, seed=9), most=40)


def test_starts_past_the_rows_and_rows_of_no_sequence(rp):
    p = inputs([10, 20, 5], 64, seed=10)
    g = torch.Generator().manual_seed(1)
    for k, s in (("x", (60, 64)), ("dt", (60, 64)), ("z", (60, 64)), ("B", (60, 1, 16)), ("C", (60, 1, 16))):
        p[k] = torch.randn(s, generator=g).to(torch.bfloat16)
    p["starts"], p["seqs"] = torch.tensor([3, 13, 33, 38], dtype=torch.int32), [(3, 10), (13, 20), (33, 5)]
    check(rp, p)
    p["starts"], p["seqs"] = torch.tensor([-3, 13, 33, 70], dtype=torch.int32), [(0, 13), (13, 20), (33, 27)]
    check(rp, p, most=60)


@pytest.mark.parametrize("step", [False, True])
def test_views(rp, step):
    """B and C as views of one projection's rows, x, dt, z and y of wider rows, slots of a wider pool."""
    p = inputs([1] * 3 if step else [100, 7, 30], 72, seed=11)
    d = on_device(p)
    N = p["x"].shape[0]
    wide = torch.full((N, 8 + 16 + 16 + 72 * 3), math.nan, dtype=torch.bfloat16, device="cuda")
    at = 8
    for k in ("B", "C", "x", "dt", "z"):
        w = p[k][0].numel()
        wide[:, at:at + w] = p[k].reshape(N, w).cuda()
        d[k] = wide[:, at:at + w].view(N, 1, 16) if k in "BC" else wide[:, at:at + w]
        at += w
    out = torch.full((N, 96), math.nan, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(5, 72 * 16 + 12, device="cuda")
    st = pool[:, :72 * 16].unflatten(1, (72, 16))
    st.copy_(p["state"])
    check(rp, p, d=d, y=out[:, 8:80], st=st, step=step)
    assert torch.isnan(out[:, :8]).all() and torch.isnan(out[:, 80:]).all() and (pool[:, 72 * 16:] == 0).all()


def test_chunks_and_steps_equal_a_whole_prompt(rp):
    p = inputs([90], 64, it="f32", seed=12)
    whole, st_w = check(rp, p, use=("D", "bias", "z"))
    d = on_device(p)
    parts, st = torch.empty_like(whole), p["state"].cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")      # noqa: E731
    for a, b in ((0, 33), (33, 34), (34, 80)):
        rp.rssm_selective_scan(st, d["A"], *(d[k][a:b] for k in ("x", "B", "C", "dt")), parts[a:b], d["slots"], i32(0, b - a),
                               max_seq_len=b - a, D=d["D"], dt_bias=d["bias"], z=d["z"][a:b])
    for a in range(80, 90):
        rp.rssm_selective_scan_step(st, d["A"], *(d[k][a:a + 1] for k in ("x", "B", "C", "dt")), parts[a:a + 1], d["slots"],
                                    D=d["D"], dt_bias=d["bias"], z=d["z"][a:a + 1])
    want, m, pool, pm = ref.scan(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"], D=p["D"],
                                 bias=p["bias"], z=p["z"])
    ref.check(parts, want, ref.scan_bound(want, m, parts.dtype, ref.scan_chain(90, 16)), "y")
    ref.check(st, pool, ref.scan_bound(pool, pm, st.dtype, ref.scan_chain(90, 16)), "state")


def test_extreme_rates_and_steps(rp):
    """States that forget everything (A of -infinity), that keep everything (A = 0), steps of 0 and huge ones."""
    p = inputs([40, 17], 64, it="f32", seed=13)
    p["A"][:, 3], p["A"][:, 4], p["A"][:, 5] = -1e30, 0.0, -3e38
    p["dt"] = p["dt"].abs()
    p["dt"][5] = 0.0
    p["dt"][9] = 1e4
    check(rp, p, use=("D",), softplus=False)
    y, st = torch.empty(57, 64, device="cuda"), p["state"].cuda()
    p["A"][:, 3] = -math.inf
    p["dt"][5] = 1e-30
    d = on_device(p)
    call(rp, p, d, y, st, use=("D",), softplus=False)
    q = dict(p, A=p["A"].clone())
    q["A"][:, 3] = -3e38
    want, m, pool, pm = ref.scan(q["state"], q["A"], q["x"], q["B"], q["C"], q["dt"], q["slots"], q["seqs"], D=q["D"], softplus=False)
    ref.check(y, want, ref.scan_bound(want, m, y.dtype, ref.scan_chain(40, 16)), "y")


@pytest.mark.parametrize("it", ["bf16", "f32"])
@pytest.mark.parametrize("Ch", [64, 8448])
def test_a_bad_value_reaches_later_tokens_of_its_channel_only(rp, it, Ch):
    p = inputs([50, 9], Ch, it=it, seed=14)
    p["x"][21, 5] = math.inf
    p["z"][30, 6] = math.nan
    p["dt"][40, 7] = math.nan
    y = torch.empty(59, Ch, dtype=DT[it], device="cuda")
    call(rp, p, on_device(p), y, p["state"].cuda())
    odd = ~torch.isfinite(y.float().cpu())
    seen = torch.zeros(59, Ch, dtype=torch.bool)
    seen[21:50, 5] = seen[30, 6] = seen[40:50, 7] = True
    assert not (odd & ~seen).any() and odd[21:50, 5].all()


@pytest.mark.parametrize("lens,Ch", [([20, 9], 64), ([700], 64), ([20] * 9, 2048)])
def test_a_rate_that_is_not_a_number(rp, lens, Ch):
    """In each of the forms it reaches its channel, and that one alone."""
    p = inputs(lens, Ch, seed=18)
    p["A"][5, 7] = math.nan
    y = torch.empty(sum(lens), Ch, dtype=torch.bfloat16, device="cuda")
    call(rp, p, on_device(p), y, p["state"].cuda())
    odd = ~torch.isfinite(y.float())
    assert odd[:, 5].all() and int(odd.sum()) == sum(lens)


def test_bad_values_of_other_sequences_rows(rp):
    """The rows after a sequence's end belong to others: whatever they hold, no NaN comes over."""
    p = inputs([5, 20, 5], 64, seed=15)
    for k in ("x", "dt", "B", "C", "z"):
        p[k][5:25] = math.nan
    y = torch.empty(30, 64, dtype=torch.bfloat16, device="cuda")
    st = p["state"].cuda()
    call(rp, p, on_device(p), y, st)
    assert torch.isfinite(y[:5].float()).all() and torch.isfinite(y[25:].float()).all()
    assert torch.isfinite(st[p["slots"][[0, 2]].long().cuda()].float()).all()


@pytest.mark.parametrize("lens", [[4, 30, 0, 9], [700, 120], None])
def test_captured_and_replayed(rp, lens):
    step = lens is None
    p = inputs([1] * 4 if step else lens, 128, seed=16)
    d = on_device(p)
    ya, sa = torch.zeros_like(d["x"]), d["state"].clone()
    yb, sb = ya.clone(), sa.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(rp, p, d, yb, sb, step=step)
    for _ in range(4):
        call(rp, p, d, ya, sa, step=step)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya, yb) and torch.equal(sa, sb)


def test_workspace_given_and_other_stream(rp):
    p = inputs([500], 64, seed=17)
    d = on_device(p)
    need = rp.rssm_selective_scan_workspace(d["state"], d["A"], d["x"], d["B"], d["C"], d["dt"], d["z"], d["slots"], d["starts"], max_seq_len=500)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")     # NaN before use
    check(rp, p, ws=ws)
    ya, sa = torch.zeros_like(d["x"]), d["state"].clone()
    yb, sb = ya.clone(), sa.clone()
    call(rp, p, d, ya, sa)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rp.rssm_selective_scan(sb, d["A"], d["x"], d["B"], d["C"], d["dt"], yb, d["slots"], d["starts"], max_seq_len=500, load_state=d["load"],
                           D=d["D"], dt_bias=d["bias"], z=d["z"], stream=s)
    s.synchronize()
    assert torch.equal(ya, yb) and torch.equal(sa, sb)
