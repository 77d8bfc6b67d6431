"""The oracles of beam selection, page operations and masked attention, pinned by hand."""
import numpy as np

from oracle import beam, kv_cache, kv_pages


def test_selection_by_hand():
    x = np.log(np.array([[[1.0, 2.0, 1.0], [4.0, 2.0, 2.0]]]))     # p = 1/4 1/2 1/4 and 1/2 1/4 1/4
    s, p, t, f, _ = beam.select(x, np.log([[0.5, 0.25]]), 4, np.zeros((1, 2), bool), 1)
    assert np.allclose(np.exp(s), [[0.25, 0.125, 0.125, 0.125]])
    # three at 1/8: beam 0's tokens 0 and 2, then beam 1's token 0
    assert p.tolist() == [[0, 0, 0, 1]] and t.tolist() == [[1, 0, 2, 0]] and f.tolist() == [[True, False, False, False]]
    # beam 1 has ended: one candidate, its score as it is
    s, p, t, f, _ = beam.select(x, np.log([[0.5, 0.3]]), 3, np.array([[False, True]]), 2)
    assert np.allclose(np.exp(s), [[0.3, 0.25, 0.125]]) and t.tolist() == [[2, 1, 0]] and f.tolist() == [[True, False, False]]
    # nothing left
    s, p, t, f, _ = beam.select(x, np.array([[-np.inf, np.nan]]), 2)
    assert np.all(np.isneginf(s)) and np.all(p == -1) and np.all(t == -1)


def test_masks_count_as_nothing():
    x = np.array([0.0, -np.inf, -3e38, 0.0])
    assert np.isclose(beam.log_sum(x), np.log(2.0))
    assert np.isnan(beam.log_sum([0.0, np.nan])) and np.isnan(beam.log_sum([0.0, np.inf])) and np.isnan(beam.log_sum([-np.inf]))


def pages(n, heads=1, page=16, D=64):
    c = [np.zeros((n, heads, page, D // 2), np.uint8), np.zeros((n, heads, page, D // 16), np.uint8),
         np.zeros((n, heads, page, D // 2), np.uint8), np.zeros((n, heads, D // 16, page), np.uint8)]
    for i in range(n):
        for b in c:
            b[i] = i + 1
    return c


def test_fork_by_hand():
    # one sequence of 20 tokens in pages 4 and 1; two children and a page held elsewhere
    refs, tables = np.array([0, 1, 1, 0, 1]), np.array([[4, 1, -1]])
    t, n, r, s, c, short = kv_pages.fork(pages(5), refs, tables, [20], [0, 0, -1], 1)
    assert t.tolist() == [[4, 1, -1], [4, 0, -1], [-1, -1, -1]] and n.tolist() == [21, 21, 0]
    assert r.tolist() == [1, 1, 1, 0, 2] and s.tolist() == [[20 - 16 + 16], [4], [-1]] and not short
    assert np.all(c[0][0] == 2) and np.all(c[3][0] == 2) and np.all(c[1][3] == 4)
    # a full last page is shared, the new token begins a page of its own; pages run out
    t, n, r, s, _, short = kv_pages.fork(pages(5), refs, tables, [32], [0, 0, 0], 1)
    assert t.tolist() == [[4, 1, 0], [4, 1, 3], [4, 1, -1]] and s.tolist() == [[0], [48], [-1]] and short


def test_trim_and_compact_by_hand():
    refs, tables = np.array([0, 1, 2, 0, 1, 1]), np.array([[5, 2, 4], [2, 1, -1]])
    t, n, r = kv_pages.trim(16, refs, tables, [40, 20], [17, 0], [40, 0])
    assert t.tolist() == [[-1, 2, 4], [-1, -1, -1]] and n.tolist() == [40, 0] and r.tolist() == [0, 0, 1, 0, 1, 0]
    t, r, m, live, c = kv_pages.compact(pages(6), r, t, n)
    assert live == 2 and m.tolist() == [-1, -1, 0, -1, 1, -1] and t.tolist() == [[-1, 0, 1], [-1, -1, -1]] and r.tolist() == [1, 1, 0, 0, 0, 0]
    assert np.all(c[2][0] == 3) and np.all(c[2][1] == 5)


def test_masked_attention_by_hand():
    """Four keys of equal products: windows, prefixes and biases decide alone."""
    D, cache = 64, [np.zeros(s, np.uint8) for s in ((1, 1, 16, 32), (1, 1, 16, 4), (1, 1, 16, 32), (1, 1, 4, 16))]
    v = np.repeat(np.array([1.5, 3.0, 6.0, 12.0])[:, None, None], D, 2)
    kv_cache.append(cache, np.zeros((4, 1, D)), v, np.arange(4))
    q = np.ones((2, 1, D))
    run = lambda **kw: kv_cache.attention(q, cache, np.array([[0]]), [4], [0, 2], **kw).out[:, 0, 0]   # noqa: E731
    assert np.allclose(run(), [10.5 / 3, 22.5 / 4])
    assert np.allclose(run(window=2), [4.5, 9])
    assert np.allclose(run(prefix=[4]), [22.5 / 4] * 2)
    assert np.allclose(run(prefix=[1], window=1), [6, 12])
    w = np.array([0.25, 0.5, 1.0])
    assert np.allclose(run(slopes=np.log([2.0]))[0], (w * [1.5, 3, 6]).sum() / w.sum())
    # a prefix's keys behind the row count by their distance, too
    w = np.array([0.25, 0.5, 1.0, 0.5])
    assert np.allclose(run(slopes=np.log([2.0]), prefix=[4])[0], (w * [1.5, 3, 6, 12]).sum() / w.sum())
    # products of 3 and 0, capped at 1
    kv_cache.append(cache, np.full((1, 1, D), 3.0 / D), np.full((1, 1, D), 1.5), np.array([0]))
    k = kv_cache.gather(cache, [0])[0][0, 0].sum()
    e = np.exp(np.tanh(k))
    assert np.allclose(run(softcap=1.0)[1], (e * 1.5 + 3 + 6 + 12) / (e + 3))
