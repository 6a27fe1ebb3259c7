"""The example decoder: prompts in chunks, prompts at once and tokens fed as a
prompt all have to see the same model."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

# fp32 all through.  Per block at most 512 half steps of rounding on terms of the size of the
# values (2^-15), through two norms and a gate each; two evaluations; four blocks and the head.
TOL = 2 * 5 * 3 * 2.0 ** -15


@pytest.fixture(scope="module")
def ex():
    import hybrid_decoder
    return hybrid_decoder


def prompts(ex):
    g = torch.Generator().manual_seed(1)
    return [torch.randint(0, ex.HybridDecoder.VOCAB, (n,), generator=g).tolist() for n in (300, 17, 129, 1)]


def test_chunked_prompts_equal_whole_ones(ex):
    m = ex.HybridDecoder(dtype="f32")
    ps = prompts(ex)
    a = ex.prefill(m, m.new_cache(4, 300), ps, 1000)
    b = ex.prefill(m, m.new_cache(4, 300), ps, 70)
    assert (a - b).abs().max() <= TOL * a.abs().max()


def test_decoded_tokens_equal_a_longer_prompt(ex):
    m = ex.HybridDecoder(dtype="f32")
    ps = prompts(ex)
    tokens, logits = ex.generate(m, ps, 6, 128)
    whole = ex.prefill(m, m.new_cache(4, 310), [p + t for p, t in zip(ps, tokens)], 1000)
    assert (whole - logits[-1]).abs().max() <= TOL * whole.abs().max()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sixteen_bits_run(ex, dtype):
    tokens, logits = ex.generate(ex.HybridDecoder(dtype=dtype), prompts(ex), 4, 64)
    assert torch.isfinite(logits.float()).all() and all(len(t) == 4 for t in tokens)


def test_binding_refusals():
    """Device tensors of the wrong kind: named by the binding, nothing enqueued."""
    import replayssm_persistent_rssm_amd as rp
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")      # noqa: E731
    i = lambda *s: z(*s, dtype=torch.int32)                                              # noqa: E731
    good = dict(state=z(2, 4, 64, 128), A=z(4), x=z(3, 4, 64), B=z(3, 2, 128), C=z(3, 2, 128), dt=z(3, 4), y=z(3, 4, 64),
                slots=i(1), seq_start=i(2))
    for name, bad in (("A", z(5)), ("x", z(3, 4, 128)), ("B", z(3, 2, 128, dtype=torch.bfloat16)), ("C", z(3, 128, 2).transpose(1, 2)),
                      ("dt", z(3, 4, dtype=torch.float16)), ("y", z(2, 4, 64)), ("slots", z(1)), ("seq_start", i(3)), ("A", z(4).cpu())):
        with pytest.raises(ValueError, match=name):
            rp.rssm_linear_attention(**{**good, name: bad}, max_seq_len=3)
    with pytest.raises(rp.RssmError, match="dim=32"):
        rp.rssm_linear_attention_step(z(2, 4, 32, 128), z(4), z(1, 4, 32), z(1, 2, 128), z(1, 2, 128), z(1, 4), z(1, 4, 32), i(1))
    kc, t, s, k, q = z(4, 16, 2, 64), i(1, 4), i(2), i(1), z(1, 4, 64)
    with pytest.raises(ValueError, match="v_cache"):
        rp.rssm_paged_append(kc, z(4, 16, 2, 128), z(1, 2, 64), z(1, 2, 64), t, s, k)
    with pytest.raises(ValueError, match="out"):
        rp.rssm_paged_attention(q, kc, kc, t, s, k, z(1, 4, 64, dtype=torch.float16), max_seq_len=1, max_kv_len=1)
    with pytest.raises(rp.RssmError, match="window"):
        rp.rssm_paged_attention(q, kc, kc, t, s, k, z(1, 4, 64), max_seq_len=1, max_kv_len=1, window=-1)
    with pytest.raises(rp.RssmError, match="workspace"):
        rp.rssm_paged_attention(q, kc, kc, t, s, k, z(1, 4, 64), max_seq_len=1, max_kv_len=10 ** 6,
                                workspace=z(16, dtype=torch.uint8))
    with pytest.raises(rp.RssmError, match="groups"):
        rp.rssm_block_norm(z(2, 64), z(2, 64), z(2, 64), groups=3)
    with pytest.raises(ValueError, match="residual_out"):
        rp.rssm_block_norm(z(2, 64), z(2, 64), z(2, 72))
