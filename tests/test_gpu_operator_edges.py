"""Edges of the prompt-side operators: inputs that are not finite or of very different size, lengths and
counts past the usual ones.  Against the definitions in 64 bits."""
import math

import pytest
import torch

import operators_ref as ref
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
