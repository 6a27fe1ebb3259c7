"""The example decoder where the page pool refuses: an error, and every sequence goes on as if it had not been asked."""
import pytest
import torch

from test_gpu_hybrid_fork import close, ex, tokens  # noqa: F401

pytestmark = pytest.mark.gpu


def snapshot(m, c):
    return [c[k].clone() for k in ("table", "kv_len", "ref")] + [t.clone() for kept in c["layer"] for t in kept] + [list(c["length"])]


def same(a, b):
    return all(torch.equal(x, y) if torch.is_tensor(x) else x == y for x, y in zip(a, b))


def test_a_refused_extend_beside_a_fork(ex):  # noqa: F811
    m = ex.HybridDecoder(dtype="f32")
    base, more = tokens(ex, 20, 1), tokens(ex, 13, 2)
    c = m.new_cache(3, 32)
    ex.prefill(m, c, [base, [], []], 1000)
    m.fork(c, [0], [1])                      # the first page is shared
    before = snapshot(m, c)
    with pytest.raises(RuntimeError, match=r"not extended: \[2, 0, 0\]"):
        m.forward(c, [more, [5], [6]])       # 33 tokens do not fit the first row; the others did
    assert same(before, snapshot(m, c))
    out = m.forward(c, [more[:12], [5], [6]])
    for got, text in zip(out, (base + more[:12], base + [5], [6])):
        close(got, ex.prefill(m, m.new_cache(1, 32), [text], 1000)[0])


def test_a_refused_fork_beside_others(ex):  # noqa: F811
    m = ex.HybridDecoder(dtype="f32")
    base, other = tokens(ex, 21, 3), tokens(ex, 3, 4)
    c = m.new_cache(4, 32)
    ex.prefill(m, c, [base, other, [], []], 1000)
    before = snapshot(m, c)
    with pytest.raises(RuntimeError, match=r"not forked: \[0, 2, 0\]"):
        m.fork(c, [0, 0, 1], [2, 1, 3])
    after = snapshot(m, c)
    # the copies went to pages that are free again
    assert same(before[:3], after[:3]) and before[-1] == after[-1]
    m.fork(c, [0], [2])
    out = m.forward(c, [[7], [8], [9], []])
    for got, text in zip(out, (base + [7], other + [8], base + [9])):
        close(got, ex.prefill(m, m.new_cache(1, 32), [text], 1000)[0])


def test_nothing_to_do(ex):  # noqa: F811
    """No tokens at all: no logits, nothing changed.  A prompt of none cannot be continued."""
    m = ex.HybridDecoder(dtype="f32")
    c = m.new_cache(2, 32)
    assert ex.prefill(m, c, [[], []], 10).shape == (0, m.VOCAB)
    ex.prefill(m, c, [tokens(ex, 5, 5), []], 10)
    before = snapshot(m, c)
    assert m.forward(c, [[], []]).shape == (0, m.VOCAB) and same(before, snapshot(m, c))
    with pytest.raises(ValueError, match="without tokens"):
        ex.generate(m, [[1, 2], []], 3, 10)
