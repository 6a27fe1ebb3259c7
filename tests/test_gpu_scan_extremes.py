"""The selective scan at the ends of its numbers, in each of its forms: few channels (short), stretches, one pass (wide)
and single tokens."""
import math

import pytest
import torch

import more_operators_ref as ref
import test_gpu_selective_scan as scan

pytestmark = pytest.mark.gpu

FORMS = {"short": ([40, 17], 64), "stretches": ([700, 17], 64), "wide": ([40, 17] + [3] * 7, 2048), "step": ([1] * 60, 64)}


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


@pytest.mark.parametrize("n", [16, 32, 64])
@pytest.mark.parametrize("form", FORMS)
def test_rates_of_zero_and_minus_infinity(rp, form, n):
    """A of -infinity keeps nothing of earlier tokens (in 64 bits: a rate that makes nothing of steps from 1e-30 on), A of 0
    everything; steps that are tiny and huge.  Outputs and states."""
    lens, Ch = FORMS[form]
    p = scan.inputs(lens, Ch, n, it="f32", seed=13 + n)
    p["dt"] = p["dt"].abs() + 1e-3
    p["dt"][5], p["dt"][9] = 1e-30, 1e4
    p["A"][:, 3], p["A"][:, 4], p["A"][:, n - 1] = -math.inf, 0.0, -1e30
    d = scan.on_device(p)
    y, st = torch.full_like(d["x"], math.nan), d["state"].clone()
    scan.call(rp, p, d, y, st, use=("D",), softplus=False, step=form == "step")
    A = p["A"].clone()
    A[:, 3] = -3e38
    want, m, pool, pm = ref.scan(p["state"], A, p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"], D=p["D"], softplus=False)
    chain = ref.scan_chain(max(lens), n)
    ref.check(y, want, ref.scan_bound(want, m, y.dtype, chain), "y")
    assert not torch.isnan(y).any()
    ref.check(st, pool, ref.scan_bound(pool, pm, st.dtype, chain), "state")


@pytest.mark.parametrize("form", FORMS)
def test_a_step_of_zero_leaves_the_state(rp, form):
    """Whatever the rate."""
    lens, Ch = FORMS[form]
    p = scan.inputs(lens, Ch, it="f32", seed=14)
    p["A"][:, 3], p["A"][:, 4], p["A"][:, 5] = -math.inf, 0.0, -3e38
    p["dt"][:] = 0.0
    d = scan.on_device(p)
    y, st = torch.empty_like(d["x"]), d["state"].clone()
    scan.call(rp, p, d, y, st, use=(), softplus=False, step=form == "step")
    assert torch.equal(st, d["state"]) and torch.isfinite(y).all()


@pytest.mark.parametrize("it,n", [("bf16", 16), ("f16", 32), ("f32", 64)])
def test_infinities_across_borders(rp, it, n):
    """Stretches of 48 tokens: an infinity in x or dt reaches all later tokens of its channel, one in the pool all tokens;
    no other channel and no earlier token."""
    p = scan.inputs([700], 72, n, it=it, seed=15 + n)
    p["x"][100, 5] = math.inf
    p["dt"][300, 9] = math.inf
    p["dt"][310, 12] = -math.inf                 # a step of size 0
    p["state"][int(p["slots"][0]), 17, n - 1] = -math.inf
    p["x"][699, 30] = -math.inf                  # the last token
    d = scan.on_device(p)
    y, st = torch.empty_like(d["x"]), d["state"].clone()
    scan.call(rp, p, d, y, st)
    seen = torch.zeros(700, 72, dtype=torch.bool)
    seen[100:, 5] = seen[300:, 9] = seen[:, 17] = seen[699, 30] = True
    assert torch.equal(~torch.isfinite(y.float().cpu()), seen)
    odd = ~torch.isfinite(st.cpu())
    assert odd.any(2).nonzero().tolist() == [[int(p["slots"][0]), c] for c in (5, 9, 17, 30)]
    assert odd.sum(2)[int(p["slots"][0]), 17] == 1


def test_an_infinity_that_a_stretch_decays_to_nothing(rp):
    """NaN from the next stretch on, as the header says; not a number that hides it."""
    p = scan.inputs([700], 64, it="f32", seed=16)
    p["A"][5, 2] = -1e4
    p["state"][int(p["slots"][0]), 5, 2] = math.inf
    d = scan.on_device(p)
    y, st = torch.empty_like(d["x"]), d["state"].clone()
    scan.call(rp, p, d, y, st, use=("D", "bias"))
    assert not torch.isfinite(y[:, 5]).any() and torch.isnan(y[48:, 5]).all()
    y[:, 5] = 0
    assert torch.isfinite(y).all()
