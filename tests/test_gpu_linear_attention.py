"""rssm_linear_attention and rssm_linear_attention_step against the recurrence in 64 bits."""
import math

import pytest
import torch

import operators_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


def make(lens, H, hpg, it, st, *, dim=64, dstate=128, seed=0, z=True, D=True, dt=True, scale=1.0, wide=0, extra_slots=2):
    """Inputs on the CPU, and `wide`: elements a token row is longer than its dense size."""
    g = torch.Generator().manual_seed(seed)
    N, G = sum(lens), H // hpg
    rn = lambda *s: torch.randn(s, generator=g)          # noqa: E731
    idt, sdt = ref.DT[it], ref.DT[st]
    p = dict(
        state=rn(len(lens) + extra_slots, H, dim, dstate).to(sdt),
        A=-torch.exp(torch.rand(H, generator=g) * math.log(16.0)),
        x=(rn(N, H, dim) * scale).to(idt), B=(rn(N, G, dstate) / math.sqrt(dstate)).to(idt),
        C=(rn(N, G, dstate) / math.sqrt(dstate)).to(idt), dt=rn(N, H) * 0.3 if dt else None,
        dt_bias=torch.log(torch.expm1(0.001 + 0.099 * torch.rand(H, generator=g))) if dt else None,
        D=0.5 + torch.rand(H, generator=g) if D else None, z=rn(N, H, dim).to(idt) if z else None,
        slots=torch.randperm(len(lens) + extra_slots, generator=g)[:len(lens)].int())
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    p["seq_start"] = torch.tensor(starts, dtype=torch.int32)
    p["seqs"] = [(starts[i], lens[i]) for i in range(len(lens))]
    p["wide"] = wide
    return p


def spread(t, wide):
    """`t` on the device as a view of rows `wide` elements longer, filled with NaN beside it."""
    if t is None:
        return None
    if not wide:
        return t.cuda()
    n = t[0].numel() if t.shape[0] else math.prod(t.shape[1:])
    big = torch.full((t.shape[0], n + wide), math.nan, dtype=t.dtype, device="cuda")
    view = big[:, :n].view(t.shape)
    view.copy_(t)
    return view


def run_prompt(rp, p, *, load=None, softplus=True, max_len=None, **kw):
    d = {k: spread(p[k], p["wide"]) for k in ("x", "B", "C", "z", "dt")}
    y = spread(torch.full(p["x"].shape, math.nan, dtype=p["x"].dtype), p["wide"])
    state = p["state"].cuda()
    c = lambda t: t.cuda() if t is not None else None    # noqa: E731
    rp.rssm_linear_attention(state, c(p["A"]), d["x"], d["B"], d["C"], d["dt"], y, c(p["slots"]), c(p["seq_start"]),
                             max_seq_len=max([n for _, n in p["seqs"]], default=0) if max_len is None else max_len,
                             load_state=c(load), D=c(p["D"]), dt_bias=c(p["dt_bias"]), z=d["z"], dt_softplus=softplus, **kw)
    torch.cuda.synchronize()
    return y, state


def check_prompt(rp, p, *, load=None, softplus=True, **kw):
    y, state = run_prompt(rp, p, load=load, softplus=softplus, **kw)
    ey, ym, pool, pm = ref.linear_attention(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"],
                                            load=load, D=p["D"], dt_bias=p["dt_bias"], z=p["z"], softplus=softplus)
    ref.check(y, ey, ref.y_bound(ey, ym, y.dtype), "y")
    chunks = 1 + max([n for _, n in p["seqs"]], default=0) // 64
    ref.check(state, pool, ref.state_bound(pool, pm, state.dtype, chunks), "state")
    untouched = [s for s in range(state.shape[0]) if s not in p["slots"].tolist()]
    assert torch.equal(state.cpu()[untouched], p["state"][untouched])
    return y, state


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("st", ["f32", "bf16", "f16"])
def test_ragged_prompts(rp, it, st):
    p = make([1, 63, 0, 64, 65, 130, 17], H=8, hpg=4, it=it, st=st, seed=1)
    check_prompt(rp, p, load=torch.tensor([1, 0, 0, 1, 1, 0, 1], dtype=torch.int32))


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,dstate", [(64, 64), (128, 64), (128, 128)])
def test_shapes(rp, it, dim, dstate):
    check_prompt(rp, make([70, 5], H=4, hpg=2, it=it, st="f32", dim=dim, dstate=dstate, seed=2))


@pytest.mark.parametrize("H,hpg", [(1, 1), (3, 1), (5, 5), (12, 3)])
def test_head_layouts(rp, H, hpg):
    check_prompt(rp, make([33, 80], H=H, hpg=hpg, it="bf16", st="f32", seed=3))


@pytest.mark.parametrize("it,st", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("lens", [[1500], [1100, 0, 513]])
def test_long_axis_is_split(rp, it, st, lens):
    """Few (sequence, head) tiles: the token axis runs in stretches."""
    p = make(lens, H=2, hpg=2, it=it, st=st, seed=4)
    args = [p[k].cuda() for k in ("state", "A", "x", "B", "C", "dt", "x", "slots", "seq_start")]
    assert rp.rssm_linear_attention_workspace(*args, max_seq_len=max(lens)) > 0
    check_prompt(rp, p, load=torch.tensor(([1, 1, 0])[:len(lens)], dtype=torch.int32))


def test_given_workspace_and_other_stream(rp):
    p = make([1500], H=2, hpg=1, it="bf16", st="f32", seed=5)
    a = run_prompt(rp, p)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run_prompt(rp, p, workspace=ws)
    c = run_prompt(rp, p, stream=s)
    d = run_prompt(rp, p, stream=s.cuda_stream)
    for o in (b, c, d):      # the same bits on every stream and in every run
        assert torch.equal(a[0], o[0]) and torch.equal(a[1], o[1])


def test_optional_inputs(rp):
    check_prompt(rp, make([90], H=4, hpg=2, it="bf16", st="f32", seed=6, z=False, D=False))
    p = make([90], H=4, hpg=2, it="bf16", st="f32", seed=7, dt=False)       # constant decay for each head
    p["A"] = -torch.tensor([0.001, 0.05, 0.5, 3.0])
    check_prompt(rp, p)
    p = make([90], H=4, hpg=2, it="f16", st="f32", seed=8)
    p["dt"], p["dt_bias"] = p["dt"].abs() * 0.2, None
    check_prompt(rp, p, softplus=False)


@pytest.mark.parametrize("it,wide", [("bf16", 8), ("f16", 24), ("f32", 4)])
def test_rows_of_a_wider_tensor(rp, it, wide):
    check_prompt(rp, make([65, 3], H=4, hpg=4, it=it, st="bf16", seed=9, wide=wide))


@pytest.mark.parametrize("scale", [1e-4, 3000.0])
def test_f16_range(rp, scale):
    """Small and large values: states beyond fp16's range, scores below it."""
    p = make([100], H=4, hpg=2, it="f16", st="f32", seed=10, scale=scale, z=False, D=False)
    p["state"] *= 1e5 if scale > 1 else 1e-6
    p["B"] = (p["B"].float() * (100.0 if scale > 1 else 0.01)).half()
    p["C"] = (p["C"].float() * (1e-5 if scale > 1 else 1.0)).half()
    check_prompt(rp, p)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
def test_strong_and_weak_decay(rp, it):
    p = make([200], H=4, hpg=2, it=it, st="f32", seed=11)
    p["A"] = -torch.tensor([1e-6, 1.0, 300.0, 5000.0])
    check_prompt(rp, p)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("where", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_nonfinite_token_stays_causal(rp, it, where, value):
    """A non-finite token changes no output before it, in its sequence or another."""
    p = make([80, 40], H=4, hpg=2, it=it, st="f32", seed=12)
    ey, ym, _, _ = ref.linear_attention(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"],
                                        D=p["D"], dt_bias=p["dt_bias"], z=p["z"])
    p[where][37] = value
    y, state = run_prompt(rp, p)
    rows = torch.ones(120, dtype=torch.bool)
    rows[37:80] = False
    if where == "C":
        rows[38:80] = True
    ref.check(y[rows], ey[rows], ref.y_bound(ey, ym, y.dtype)[rows], "y")


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
def test_dt_of_minus_infinity_skips_a_token(rp, it):
    """softplus(-inf) = 0: the state passes the token unchanged, in both forms."""
    p = make([70, 1], H=4, hpg=2, it=it, st="f32", seed=16)
    p["dt"][5], p["dt"][40], p["dt"][70] = -math.inf, -math.inf, -math.inf
    check_prompt(rp, p)
    q = make([1, 1], H=4, hpg=2, it=it, st="f32", seed=17)
    q["dt"][1] = -math.inf
    _, state = run_step(rp, q)
    s = int(q["slots"][1])
    assert torch.equal(state[s].cpu(), q["state"][s])


def test_pad_and_guarded_slots(rp):
    p = make([20, 30, 40], H=4, hpg=2, it="bf16", st="f32", seed=13)
    p["slots"] = torch.tensor([-1, 3, 1000], dtype=torch.int32)
    y, state = run_prompt(rp, p)
    ey, ym, pool, pm = ref.linear_attention(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"],
                                            D=p["D"], dt_bias=p["dt_bias"], z=p["z"])
    assert torch.isnan(y[:20]).all() and torch.isnan(y[50:]).all()
    ref.check(y[20:50], ey[20:50], ref.y_bound(ey, ym, y.dtype)[20:50], "y")
    ref.check(state, pool, ref.state_bound(pool, pm, state.dtype), "state")


def test_no_tokens(rp):
    p = make([0, 0], H=4, hpg=2, it="bf16", st="f32", seed=14)
    _, state = run_prompt(rp, p, load=torch.tensor([1, 0], dtype=torch.int32))
    want = p["state"].clone()
    want[int(p["slots"][1])] = 0
    assert torch.equal(state.cpu(), want)


def test_sequences_are_cut_to_max_seq_len(rp):
    p = make([50, 90], H=4, hpg=2, it="bf16", st="f32", seed=15)
    y, state = run_prompt(rp, p, max_len=70)
    p["seqs"] = [(0, 50), (50, 70)]
    ey, ym, pool, pm = ref.linear_attention(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"],
                                            D=p["D"], dt_bias=p["dt_bias"], z=p["z"])
    ref.check(y[:120], ey[:120], ref.y_bound(ey, ym, y.dtype)[:120], "y")
    ref.check(state, pool, ref.state_bound(pool, pm, state.dtype, 2), "state")
    assert torch.isnan(y[120:]).all()


def run_step(rp, p, **kw):
    d = {k: spread(p[k], p["wide"]) for k in ("x", "B", "C", "z", "dt")}
    y = spread(torch.full(p["x"].shape, math.nan, dtype=p["x"].dtype), p["wide"])
    state = p["state"].cuda()
    c = lambda t: t.cuda() if t is not None else None    # noqa: E731
    rp.rssm_linear_attention_step(state, c(p["A"]), d["x"], d["B"], d["C"], d["dt"], y, c(p["slots"]), D=c(p["D"]),
                                  dt_bias=c(p["dt_bias"]), z=d["z"], **kw)
    torch.cuda.synchronize()
    return y, state


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("st", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,dstate,wide", [(64, 128, 0), (128, 64, 8), (64, 64, 8), (128, 128, 0)])
def test_step(rp, it, st, dim, dstate, wide):
    p = make([1] * 5, H=6, hpg=3, it=it, st=st, dim=dim, dstate=dstate, seed=20, wide=wide, z=wide == 0, D=wide == 0)
    p["slots"][2] = -1
    y, state = run_step(rp, p)
    ey, ym, pool, pm = ref.linear_attention(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"],
                                            D=p["D"], dt_bias=p["dt_bias"], z=p["z"])
    assert torch.isnan(y[2]).all()
    live = [0, 1, 3, 4]
    bound = ref.half_step(y.dtype) * ey.abs() + ref.FP32_CHAIN * ym + torch.finfo(y.dtype).tiny
    ref.check(y[live], ey[live], bound[live], "y")
    ref.check(state, pool, ref.state_bound(pool, pm, state.dtype), "state")


def test_steps_continue_a_prompt(rp):
    """A prompt of n tokens and k steps are a prompt of n + k tokens."""
    p = make([100, 37], H=4, hpg=2, it="f32", st="f32", seed=21)
    whole_y, whole_state = run_prompt(rp, p)
    c = lambda t: t.cuda()                               # noqa: E731
    state = c(p["state"])
    tok = {k: c(p[k]) for k in ("x", "B", "C", "dt", "z")}
    y = torch.zeros_like(tok["x"])
    part = torch.tensor([0, 96, 96 + 33], dtype=torch.int32, device="cuda")
    rows = list(range(96)) + list(range(100, 133))
    yp = torch.zeros(129, 4, 64, device="cuda")
    rp.rssm_linear_attention(state, c(p["A"]), *(tok[k][rows] for k in ("x", "B", "C", "dt")), yp, c(p["slots"]), part,
                             max_seq_len=96, D=c(p["D"]), dt_bias=c(p["dt_bias"]), z=tok["z"][rows])
    for t in range(4):
        at = [96 + t, 133 + t]
        ys = torch.zeros(2, 4, 64, device="cuda")
        rp.rssm_linear_attention_step(state, c(p["A"]), *(tok[k][at] for k in ("x", "B", "C", "dt")), ys, c(p["slots"]),
                                      D=c(p["D"]), dt_bias=c(p["dt_bias"]), z=tok["z"][at])
        y[at] = ys
    y[rows] = yp
    _, ym, _, pm = ref.linear_attention(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"],
                                        D=p["D"], dt_bias=p["dt_bias"], z=p["z"])
    assert ((y - whole_y).abs().cpu().double() <= 2 * ref.FP32_CHAIN * ym).all()
    assert ((state - whole_state).abs().cpu().double() <= 2 * ref.FP32_CHAIN * pm).all()


def test_prompt_state_feeds_the_replay_decode_step(rp):
    """The pool a prompt fills is the checkpoint that rssm_ssu_decode reads."""
    p = make([50], H=8, hpg=4, it="bf16", st="f32", seed=22)
    _, state = run_prompt(rp, p)
    q = make([1], H=8, hpg=4, it="bf16", st="f32", seed=23)
    c = lambda t: t.cuda()                               # noqa: E731
    R, S = 4, state.shape[0]
    y = torch.zeros(1, 1, 8, 64, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    rp.rssm_ssu_decode(state, torch.zeros(S, R, 8, 64, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(S, R, 2, 128, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(S, R, 8, device="cuda"), c(p["A"]), c(q["x"])[:, None], c(q["B"])[:, None],
                       c(q["C"])[:, None], c(q["dt"])[:, None], y, c(p["slots"]), zero, zero, ring_buffer_len=R,
                       D=c(p["D"]), dt_bias=c(p["dt_bias"]), z=c(q["z"])[:, None])
    ys = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device="cuda")
    before = state.clone()
    rp.rssm_linear_attention_step(state, c(p["A"]), c(q["x"]), c(q["B"]), c(q["C"]), c(q["dt"]), ys, c(p["slots"]),
                                  D=c(p["D"]), dt_bias=c(p["dt_bias"]), z=c(q["z"]))
    ey, ym, _, _ = ref.linear_attention(before.cpu(), p["A"], q["x"], q["B"], q["C"], q["dt"], p["slots"], [(0, 1)],
                                        D=p["D"], dt_bias=p["dt_bias"], z=q["z"])
    ref.check(y[:, 0], ey, 2 * ref.FP32_CHAIN * ym, "decode step")
    ref.check(ys, ey, ref.y_bound(ey, ym, ys.dtype), "single-token form")


def test_graph_replay(rp):
    """Prompt and steps in one captured graph, replayed among eager work."""
    p = make([700, 30], H=2, hpg=1, it="bf16", st="f32", seed=24)
    c = lambda t: t.cuda() if t is not None else None    # noqa: E731
    d = {k: c(p[k]) for k in ("state", "A", "x", "B", "C", "dt", "z", "D", "dt_bias", "slots", "seq_start")}
    q = {k: c(v) for k, v in make([1, 1], H=2, hpg=1, it="bf16", st="f32", seed=25).items() if isinstance(v, torch.Tensor)}
    y, ys = torch.zeros_like(d["x"]), torch.zeros_like(q["x"])
    ws = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")

    def go():
        rp.rssm_linear_attention(d["state"], d["A"], d["x"], d["B"], d["C"], d["dt"], y, d["slots"], d["seq_start"],
                                 max_seq_len=700, D=d["D"], dt_bias=d["dt_bias"], z=d["z"], workspace=ws)
        rp.rssm_linear_attention_step(d["state"], d["A"], q["x"], q["B"], q["C"], q["dt"], ys, d["slots"], D=d["D"],
                                      dt_bias=d["dt_bias"], z=q["z"])

    start = d["state"].clone()
    go()
    want = [t.clone() for t in (y, ys, d["state"])]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        go()
    for k in range(3):
        d["state"].copy_(start)
        y.zero_()
        ys.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((y, ys, d["state"]), want):
            assert torch.equal(got, w), f"replay {k}"


def test_large_pool_offsets(rp):
    """A slot past 2^32 bytes of the state pool."""
    p = make([40], H=64, hpg=8, it="bf16", st="f32", seed=26, extra_slots=0)
    big = torch.empty(2100, 64, 64, 128, device="cuda")          # 4.4 GB
    big[2099].copy_(p["state"][0])
    y = torch.zeros(p["x"].shape, dtype=torch.bfloat16, device="cuda")
    c = lambda t: t.cuda()                               # noqa: E731
    rp.rssm_linear_attention(big, c(p["A"]), c(p["x"]), c(p["B"]), c(p["C"]), c(p["dt"]), y,
                             torch.tensor([2099], dtype=torch.int32, device="cuda"), c(p["seq_start"]), max_seq_len=40,
                             D=c(p["D"]), dt_bias=c(p["dt_bias"]), z=c(p["z"]))
    ey, ym, pool, pm = ref.linear_attention(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], [0], [(0, 40)],
                                            D=p["D"], dt_bias=p["dt_bias"], z=p["z"])
    ref.check(y, ey, ref.y_bound(ey, ym, y.dtype), "y")
    ref.check(big[2099], pool[0], ref.state_bound(pool, pm, torch.float32)[0], "state")
