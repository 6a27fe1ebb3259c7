"""The example decoder's sequences forked, released and packed: every one has to go on as if it had been alone."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

# fp32 all through.  Per block at most 512 half steps of rounding on terms of the size of the
# values (2^-15), through a convolution, two norms and a gate each; two evaluations; four blocks and the head.
TOL = 2 * 5 * 4 * 2.0 ** -15


@pytest.fixture(scope="module")
def ex():
    import hybrid_decoder
    return hybrid_decoder


def tokens(ex, n, seed):
    return torch.randint(0, ex.HybridDecoder.VOCAB, (n,), generator=torch.Generator().manual_seed(seed)).tolist()


def close(a, b):
    assert (a - b).abs().max() <= TOL * b.abs().max()


@pytest.mark.parametrize("page", [16, 7])
def test_forks_go_their_own_ways(ex, page):
    m = ex.HybridDecoder(dtype="f32")
    base, one, two = tokens(ex, 45, 1), tokens(ex, 20, 2), tokens(ex, 9, 3)
    c = m.new_cache(5, 120, page)
    ex.prefill(m, c, [base, tokens(ex, 70, 4), [], [], []], 64)
    m.fork(c, [0, 0], [2, 3])
    out = m.forward(c, [[5], [], one, two, []])
    for got, text in zip(out, (base + [5], base + one, base + two)):
        close(got, ex.prefill(m, m.new_cache(1, 120), [text], 1000)[0])
    # the second sequence ends, the pool is packed, a fork of a fork takes its place
    live = m.release(c, [1], pack=True)
    assert live == int((c["ref"] > 0).sum()) and (c["ref"][:live] > 0).all()
    m.fork(c, [2], [1])
    out = m.forward(c, [[7], [8], [9], [], [11]])
    for got, text in zip(out, (base + [5, 7], base + one + [8], base + one + [9], [11])):
        close(got, ex.prefill(m, m.new_cache(1, 120), [text], 1000)[0])
    m.release(c, [0, 1, 2, 3, 4])
    assert not c["ref"].any() and (c["table"] == -1).all() and not c["kv_len"].any()


def test_single_tokens_after_a_fork(ex):
    m = ex.HybridDecoder(dtype="f32")
    base = tokens(ex, 33, 5)
    c = m.new_cache(2, 64)
    ex.prefill(m, c, [base, []], 1000)
    m.fork(c, [0], [1])
    for i in range(5):
        out = m.forward(c, [[i], [100 + i]])
    for got, text in zip(out, (base + [0, 1, 2, 3, 4], base + [100, 101, 102, 103, 104])):
        close(got, ex.prefill(m, m.new_cache(1, 64), [text], 1000)[0])


def test_a_taken_row_is_not_forked_onto(ex):
    m = ex.HybridDecoder(dtype="f32")
    c = m.new_cache(2, 64)
    ex.prefill(m, c, [tokens(ex, 20, 6), tokens(ex, 3, 7)], 1000)
    with pytest.raises(RuntimeError, match="not forked"):
        m.fork(c, [0], [1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sixteen_bits_run(ex, dtype):
    m = ex.HybridDecoder(dtype=dtype)
    c = m.new_cache(3, 100)
    ex.prefill(m, c, [tokens(ex, 50, 8), tokens(ex, 2, 9), []], 32)
    m.fork(c, [0], [2])
    out = m.forward(c, [[1], [2], [1]])
    assert torch.isfinite(out.float()).all() and torch.equal(out[0], out[2])
