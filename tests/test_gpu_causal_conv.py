"""rssm_causal_conv and rssm_causal_conv_step against their formula in 64 bits."""
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


def inputs(lens, C, W, it, seed=0, slots=None, extra=2):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)          # noqa: E731
    S, N = len(lens), sum(lens)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    p = dict(x=rn(N, C).to(DT[it]), weight=rn(W, C) / math.sqrt(W), bias=0.1 * rn(C), state=rn(S + extra, W - 1, C).to(DT[it]),
             slots=torch.randperm(S + extra, generator=g)[:S].int() if slots is None else torch.tensor(slots, dtype=torch.int32),
             starts=torch.tensor(starts, dtype=torch.int32), seqs=[(starts[i], lens[i]) for i in range(S)],
             load=torch.tensor([i % 3 != 2 for i in range(S)], dtype=torch.int32))
    return p


def check(rp, p, *, bias=True, load=True, on=True, step=False, pad=-1, y=None, x=None, state=None):
    x = p["x"].cuda() if x is None else x
    y = torch.full_like(x, math.nan) if y is None else y
    st = p["state"].cuda() if state is None else state
    b = p["bias"] if bias else None
    kw = dict(bias=b.cuda() if bias else None, silu=on, pad_slot_id=pad)
    if step:
        rp.rssm_causal_conv_step(x, p["weight"].cuda(), y, st, p["slots"].cuda(), **kw)
    else:
        rp.rssm_causal_conv(x, p["weight"].cuda(), y, st, p["slots"].cuda(), p["starts"].cuda(),
                            load_state=p["load"].cuda() if load else None, **kw)
    want, m, pool = ref.conv(p["x"], p["weight"], p["state"], p["slots"], p["seqs"], bias=b, on=on, pad=pad,
                             load=p["load"] if load and not step else None)
    ref.check(y, want, ref.conv_bound(want, m, y.dtype), "y")
    assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want)), "rows of no sequence are left alone, all others written"
    assert torch.equal(st.cpu(), pool), "the state is the inputs' bytes"
    return y


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [8, 520, 1024])
def test_ragged_prompts(rp, it, W, C):
    check(rp, inputs([0, 1, 2, 3, 33, 64, 7, 95, 0, 31, 32, 5], C, W, it, seed=C + W))


@pytest.mark.parametrize("lens", [[1], [0], [], [3], [8], [9], [200], [0, 0, 0], [1] * 70, [40, 0, 0, 1, 39]])
def test_lengths(rp, lens):
    check(rp, inputs(lens, 64, 4, "bf16", seed=len(lens)))


def test_many_channels(rp):
    """More than a launch of the small cases: sequence ends inside tiles and at their borders."""
    check(rp, inputs([31, 1, 32, 33, 0, 64, 2, 95, 100], 512 * 300, 4, "bf16", seed=3))


@pytest.mark.parametrize("it,W", [("bf16", 2), ("f16", 3), ("f32", 4), ("bf16", 4)])
def test_longer_tiles(rp, it, W):
    """Over 8,192 wavefronts' work: tiles of 8 tokens, ends inside and at their borders."""
    check(rp, inputs([7, 8, 9, 0, 1, 2, 16, 41, 3, 0], 512 * 420, W, it, seed=W))


def test_more_sequences_than_a_wavefront(rp):
    check(rp, inputs([i % 5 for i in range(333)], 16, 3, "f16", seed=4))


@pytest.mark.parametrize("kw", [dict(bias=False), dict(on=False), dict(load=False), dict(bias=False, on=False, load=False)])
def test_optional_inputs(rp, kw):
    check(rp, inputs([5, 40, 1], 128, 4, "f32", seed=5), **kw)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("S,C", [(1, 8), (5, 520), (67, 1032), (8, 512 * 520)])
def test_step(rp, it, W, S, C):
    check(rp, inputs([1] * S, C, W, it, seed=S), step=True)


@pytest.mark.parametrize("step", [False, True])
def test_pads_and_slots_outside_the_pool(rp, step):
    p = inputs([1] * 6 if step else [4, 9, 1, 0, 50, 3], 72, 4, "bf16", seed=6, slots=[-1, 3, 7, 900, -5, 0])
    check(rp, p, step=step)
    check(rp, p, step=step, pad=3)


def test_rows_of_no_sequence(rp):
    p = inputs([10, 20, 5], 64, 4, "bf16", seed=7)
    g = torch.Generator().manual_seed(1)
    p["x"] = torch.randn(60, 64, generator=g).to(torch.bfloat16)
    p["starts"] = torch.tensor([3, 13, 33, 38], dtype=torch.int32)
    p["seqs"] = [(3, 10), (13, 20), (33, 5)]
    check(rp, p)


def test_starts_past_the_rows_are_clamped(rp):
    p = inputs([10, 20], 64, 4, "bf16", seed=8)
    p["starts"] = torch.tensor([-4, 10, 1000], dtype=torch.int32)
    check(rp, p)


@pytest.mark.parametrize("step", [False, True])
def test_views(rp, step):
    """Rows of a wider projection in and out, slots of a wider pool."""
    p = inputs([1, 1, 1] if step else [30, 2, 41], 136, 4, "f16", seed=9)
    N = p["x"].shape[0]
    wide = torch.full((N, 304), math.nan, dtype=torch.float16, device="cuda")
    wide[:, 16:152] = p["x"].cuda()
    out = torch.full((N, 160), math.nan, dtype=torch.float16, device="cuda")
    pool = torch.zeros(5, 504, dtype=torch.float16, device="cuda")
    st = pool[:, :408].unflatten(1, (3, 136))
    st.copy_(p["state"])
    check(rp, p, x=wide[:, 16:152], y=out[:, 8:144], state=st, step=step)
    assert torch.isnan(out[:, :8]).all() and torch.isnan(out[:, 144:]).all() and (pool[:, 408:] == 0).all()


def test_rows_off_their_alignment_are_refused(rp):
    """Rows 600 and slots 1,000 bytes apart: not multiples of 16."""
    p = inputs([1, 1, 1], 136, 4, "f16", seed=9)
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
    wide = torch.zeros(3, 300, dtype=torch.float16, device="cuda")
    pool = torch.zeros(5, 500, dtype=torch.float16, device="cuda")
    for x, st in ((wide[:, 16:152], d["state"]), (d["x"], pool[:, :408].unflatten(1, (3, 136)))):
        with pytest.raises(rp.RssmError, match="16 bytes"):
            rp.rssm_causal_conv_step(x, d["weight"], torch.empty_like(d["x"]), st, d["slots"])


def test_step_in_place(rp):
    p = inputs([1] * 9, 264, 4, "bf16", seed=10)
    x = p["x"].cuda()
    check(rp, p, x=x, y=x, step=True)


def test_chunks_equal_a_whole_prompt_and_steps(rp):
    """Bit for bit: the same sums in the same order."""
    g = torch.Generator().manual_seed(11)
    x, w = torch.randn(77, 96, generator=g).bfloat16().cuda(), torch.randn(4, 96, generator=g).cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")      # noqa: E731
    whole, parts = torch.empty_like(x), torch.empty_like(x)
    a = torch.zeros(1, 3, 96, dtype=torch.bfloat16, device="cuda")
    b = torch.full_like(a, 7.0)
    rp.rssm_causal_conv(x, w, whole, a, i32(0), i32(0, 77), load_state=i32(0))
    at = 0
    for n in (1, 2, 40, 1, 30):
        rp.rssm_causal_conv(x[at:at + n], w, parts[at:at + n], b, i32(0), i32(0, n), load_state=i32(int(at > 0)))
        at += n
    while at < 77:
        rp.rssm_causal_conv_step(x[at:at + 1], w, parts[at:at + 1], b, i32(0))
        at += 1
    assert torch.equal(whole, parts) and torch.equal(a, b)


def test_a_bad_value_stays_in_its_taps_and_channel(rp):
    p = inputs([50], 64, 4, "f32", seed=12)
    p["x"][20, 5] = math.inf
    p["x"][30, 6] = math.nan
    y = torch.empty(50, 64, device="cuda")
    rp.rssm_causal_conv(p["x"].cuda(), p["weight"].cuda(), y, p["state"].cuda(), p["slots"].cuda(), p["starts"].cuda())
    odd = ~torch.isfinite(y.cpu())
    seen = torch.zeros(50, 64, dtype=torch.bool)
    seen[20:24, 5] = seen[30:34, 6] = True
    assert not (odd & ~seen).any()


@pytest.mark.parametrize("step", [False, True])
def test_captured_and_replayed(rp, step):
    p = inputs([1] * 4 if step else [4, 30, 0, 9], 256, 4, "bf16", seed=13)
    c = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}

    def call(y, st):
        if step:
            rp.rssm_causal_conv_step(c["x"], c["weight"], y, st, c["slots"], bias=c["bias"])
        else:
            rp.rssm_causal_conv(c["x"], c["weight"], y, st, c["slots"], c["starts"], bias=c["bias"])
    ya, yb, sa, sb = torch.zeros_like(c["x"]), torch.zeros_like(c["x"]), c["state"].clone(), c["state"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(yb, sb)
    for _ in range(4):
        call(ya, sa)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya, yb) and torch.equal(sa, sb)
