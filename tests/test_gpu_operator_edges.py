"""Edges of the prompt-side operators: inputs that are not finite or of very different size, lengths and
counts past the usual ones.  Against the definitions in 64 bits."""
import math

import pytest
import torch

import operators_ref as ref
from test_gpu_linear_attention import check_prompt, run_prompt, run_step
from test_gpu_linear_attention import make as linear
from test_gpu_paged_attention import attend
from test_gpu_paged_attention import make as paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


SPLITS = [(1, 1500), (1, 6000), (40, 1500), (40, 6000)]      # both kernels, few and many splits


def check_nonfinite(rp, p, **kw):
    """Against the definition, NaN included: NaN where the formula has it and nowhere else."""
    c = [p[k].cuda() for k in ("q", "kc", "vc", "table", "seq_start", "kv", "q")]
    longest = max(n for _, n in p["seqs"])
    assert rp.rssm_paged_attention_workspace(*c, max_seq_len=longest, max_kv_len=int(p["kv"].max()), **kw) > 0
    out, lse = attend(rp, p, **kw)
    e, mag, el, err = ref.paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seqs"], p["kv"], **kw)
    ref.check(out, e, ref.out_bound(e, mag, err, out.dtype), "out")
    ref.check(lse, el, err + 2.0 ** -20 * el.abs().clamp(min=1), "lse")
    assert torch.isnan(el).any() and torch.equal(torch.isnan(lse.cpu()), torch.isnan(el))
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(e))


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ql,kv", SPLITS)
def test_nan_query_of_a_split_axis(rp, it, ql, kv):
    p = paged([kv, 600], [ql, ql], 4, 2, 64, 48, it, seed=30)
    p["q"][0, 1, 5] = math.nan
    check_nonfinite(rp, p)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ql,kv", SPLITS)
def test_split_of_nan_keys(rp, it, ql, kv):
    """Positions 256 .. 767 hold whole splits."""
    p = paged([kv, 200], [ql, ql], 4, 2, 64, 48, it, seed=31)
    for j in range(256, 768):
        p["kc"][int(p["table"][0, j // 48]), j % 48, 0] = math.nan
    check_nonfinite(rp, p)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ql,kv", SPLITS)
def test_nan_key_in_a_split_of_low_scores(rp, it, ql, kv):
    """The other splits' scores are so much larger that this one's weight is zero."""
    p = paged([kv], [ql], 2, 1, 64, 48, it, seed=32)
    p["q"][:] = p["q"][0, 0]
    for j in range(256):
        p["kc"][int(p["table"][0, j // 48]), j % 48] = 0
    p["kc"][int(p["table"][0, 0]), 5, 0] = math.nan
    p["kc"][int(p["table"][0, 1000 // 48]), 1000 % 48, 0] = 50 * p["q"][0, 0]
    check_nonfinite(rp, p)


def decays(it, st, A, seed, **kw):
    """dt as given (no softplus), and nothing but the recurrence in y."""
    p = linear(it=it, st=st, H=len(A), hpg=len(A), seed=seed, z=False, D=False, **kw)
    p["A"], p["dt_bias"] = -torch.tensor(A), None
    return p


@pytest.mark.parametrize("it,far", [("f16", 100.0)] + [(it, far) for it in ("bf16", "f32") for far in (100.0, 1e4, 1e8, 1e30)])
def test_small_decays_after_a_far_one(rp, it, far):
    """One token whose decay forgets everything leaves the decays between later tokens as they are."""
    p = decays(it, "f32", [16.0, 5000.0, 0.5], 40, lens=[100, 33])
    p["dt"] = torch.tensor([0.01, 1e-4, 0.02]).expand(133, 3) * (0.5 + torch.rand(133, 1, generator=torch.Generator().manual_seed(1)))
    for t in (0, 3, 31, 40, 41, 70, 102):
        p["dt"][t], p["x"][t] = far, 0
    check_prompt(rp, p, softplus=False)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", [[1, 70, 130], [1500]])
@pytest.mark.parametrize("constant", [False, True])
def test_heads_without_memory(rp, it, lens, constant):
    """A of -infinity: the state is the last token's term alone, in prompts and in single tokens."""
    p = decays(it, "f32", [math.inf, 1.0], 41, lens=lens, dt=not constant)
    if not constant:
        p["dt"] = 0.01 + 0.1 * torch.rand(p["dt"].shape, generator=torch.Generator().manual_seed(2))
    check_prompt(rp, p, softplus=False)
    q = decays(it, "f32", [math.inf, 1.0], 42, lens=[1, 1], dt=not constant)
    if not constant:
        q["dt"] = q["dt"].abs() + 0.01
    y, state = run_step(rp, q, dt_softplus=False)
    ey, ym, pool, pm = ref.linear_attention(q["state"], q["A"], q["x"], q["B"], q["C"], q["dt"], q["slots"], q["seqs"],
                                            softplus=False)
    ref.check(y, ey, ref.half_step(y.dtype) * ey.abs() + ref.FP32_CHAIN * ym + torch.finfo(y.dtype).tiny, "y")
    ref.check(state, pool, ref.state_bound(pool, pm, state.dtype), "state")


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("ql", [1, 40])
def test_masked_values_change_no_bit(rp, it, value, window, ql):
    """Finite or not, a value that no query sees leaves every output as it is."""
    lens = [150, 90, 3000]
    p = paged(lens, [ql] * 3, 4, 2, 64, 16, it, seed=60)
    spare = next(a for a in range(p["kc"].shape[0]) if a not in p["table"])
    p["table"][p["table"] == 0] = spare                     # no sequence holds page 0,
    p["table"][1, 2] = -1                                   # whose first row is read in place of what is off the cache
    seen = {(int(p["table"][s, j // 16]), j % 16) for s, n in enumerate(lens) for j in range(n)
            if int(p["table"][s, j // 16]) >= 0 and (window == 0 or j > n - ql - window)}
    out, lse = attend(rp, p, window=window)
    for a in range(p["kc"].shape[0]):
        for b in range(16):
            if (a, b) not in seen:
                p["vc"][a, b] = value
    again, lse2 = attend(rp, p, window=window)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_f16_weights_far_below_the_largest(rp):
    """60,000 keys of weight just below 2^-25 of the largest are 1/600 of the sum: row tiles that walk the
    whole cache (enough sequences that it is not split) may not lose them."""
    n, S, ql = 60000, 257, 17
    p = paged([n], [ql], 1, 1, 64, 1000, "f16", seed=61, spare=0, extra_cols=0)
    p["kc"][:], p["vc"][:], p["q"][:] = 0, 1, 0
    p["q"][:, :, 0] = 12
    p["kc"][int(p["table"][0, 0]), 0, 0, 0] = 11.6          # 12 x 11.6 / 8 = 17.4 = 25.1 log(2)
    e, mag, el, err = ref.paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seqs"], p["kv"])
    p["q"], p["table"], p["kv"] = p["q"].repeat(S, 1, 1), p["table"].repeat(S, 1), p["kv"].repeat(S)
    p["seqs"] = [(s * ql, ql) for s in range(S)]
    p["seq_start"] = torch.arange(S + 1).int() * ql
    c = [p[k].cuda() for k in ("q", "kc", "vc", "table", "seq_start", "kv", "q")]
    assert rp.rssm_paged_attention_workspace(*c, max_seq_len=ql, max_kv_len=n) == 0
    out, lse = attend(rp, p)
    rep = lambda t: t.repeat(S, *[1] * (t.dim() - 1))       # noqa: E731
    ref.check(out, rep(e), rep(ref.out_bound(e, mag, err, out.dtype)), "out")
    ref.check(lse, rep(el), rep(err + 2.0 ** -20 * el.abs().clamp(min=1)), "lse")


@pytest.mark.parametrize("st", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("A", [4.0, 16.0, 60.0])
def test_f16_state_terms_of_any_size(rp, st, A):
    """Each token writes a column of its own, so its term is all that the column holds: at least 22
    bits of it down to 2^-29 of the row's largest term, and 2^-51 of that largest below."""
    p = linear([64], H=1, hpg=1, it="f16", st=st, dim=64, dstate=64, seed=50, z=False, D=False)
    p["A"], p["dt_bias"], p["dt"][:] = -torch.tensor([A]), None, 0.1
    p["B"] = torch.eye(64).half()[:, None]
    load = torch.zeros(1, dtype=torch.int32)
    _, state = run_prompt(rp, p, load=load, softplus=False)
    _, _, pool, pm = ref.linear_attention(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"],
                                          load=load, softplus=False)
    s = int(p["slots"][0])
    bound = ref.state_bound(pool, pm, state.dtype)[s] + 2.0 ** -51 * pool[s].abs().amax(-1, keepdim=True)
    ref.check(state[s], pool[s], bound, "state")


@pytest.mark.parametrize("it", ["bf16", "f32"])
@pytest.mark.parametrize("ql", [1, 40])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 0), (60, 3), (120, 0)])
def test_kv_len_past_max_kv_len(rp, it, ql, window, sinks):
    """Positions stay those of kv_len (where the append put the tokens); keys from max_kv_len on are hidden."""
    p = paged([200, 130, 90], [ql] * 3, 4, 2, 64, 16, it, seed=62)
    out, lse = attend(rp, p, window=window, sinks=sinks, max_kv_len=96)
    p["table"] = p["table"][:, :6]
    e, mag, el, err = ref.paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seqs"], p["kv"], window=window,
                                          sinks=sinks)
    ref.check(out, e, ref.out_bound(e, mag, err, out.dtype), "out")
    empty = el == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty) and (out.cpu()[empty] == 0).all()


@pytest.mark.parametrize("longest", [6, 15])
@pytest.mark.parametrize("kv", [100, 2500])
def test_new_tokens_past_max_seq_len(rp, longest, kv):
    """The first rows of a longer sequence are computed, at their own positions; the others stay as they are."""
    p = paged([kv, 90], [20, 3], 4, 2, 64, 16, "bf16", seed=63)
    out, lse = attend(rp, p, max_seq_len=longest)
    e, mag, el, err = ref.paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seqs"], p["kv"])
    rows = [*range(longest), 20, 21, 22]
    ref.check(out[rows], e[rows], ref.out_bound(e, mag, err, out.dtype)[rows], "out")
    ref.check(lse[rows], el[rows], (err + 2.0 ** -20 * el.abs().clamp(min=1))[rows], "lse")
    assert torch.isnan(out[longest:20]).all() and torch.isnan(lse[longest:20]).all()


def test_norm_of_more_rows_than_one_launch_takes(rp):
    R, C = 2 ** 24 + 3, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn(R, C, generator=g, device="cuda", dtype=torch.bfloat16)
    z = torch.randn(R, C, generator=g, device="cuda", dtype=torch.bfloat16)
    res = torch.randn(R, C, generator=g, device="cuda")
    out, n = torch.full_like(res, math.nan), torch.full_like(y, math.nan)
    rp.rssm_block_norm(y, res, out, n)
    assert torch.equal(out, res + y.float())                # one fp32 addition
    rows = [0, 1, 2 ** 23, 2 ** 24 - 3, 2 ** 24 - 2, 2 ** 24 - 1, 2 ** 24, 2 ** 24 + 1, 2 ** 24 + 2]
    _, _, nn, nm = ref.block_norm(y[rows].cpu(), res[rows].cpu())
    ref.check(n[rows], nn, ref.norm_bound(nn, nm, n.dtype), "normed")
    assert not torch.isnan(n).any()
    rp.rssm_block_norm(y, res, out, None, z=z)              # no normed; with a gate
    r, rm, _, _ = ref.block_norm(y[rows].cpu(), res[rows].cpu(), z=z[rows].cpu())
    ref.check(out[rows], r, ref.norm_bound(r, rm, out.dtype), "residual")


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(16, 1), (24, 1), (64, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
def test_single_tokens_of_many_heads_a_page(rp, it, Hq, Hkv, window, sinks):
    """Up to 16 rows a key/value head stream the cache, more take row tiles."""
    p = paged([1, 31, 200, 2500], [1] * 4, Hq, Hkv, 64, 16, it, seed=64)
    out, lse = attend(rp, p, window=window, sinks=sinks)
    e, mag, el, err = ref.paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seqs"], p["kv"], window=window,
                                          sinks=sinks)
    ref.check(out, e, ref.out_bound(e, mag, err, out.dtype), "out")
    ref.check(lse, el, err + 2.0 ** -20 * el.abs().clamp(min=1), "lse")
