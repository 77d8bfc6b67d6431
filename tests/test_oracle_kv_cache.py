"""Pins of the key/value cache oracle (no GPU): closed forms, layouts, masks."""
import numpy as np
import pytest

import oracle
from oracle import kv_cache as okv


def empty(pages=4, heads=2, page=16, D=64):
    z = lambda *s: np.zeros((pages, heads, *s), np.uint8)  # noqa: E731
    return [z(page, D // 2), z(page, D // 16), z(page, D // 2), z(D // 16, page)]


def table(n, rot):
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n)[:, None] * freq
    return np.concatenate([np.cos(a), np.sin(a)], -1).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_angles(interleaved):
    rng = np.random.default_rng(0)
    cs = table(64, 64)
    x, y = rng.standard_normal((2, 1, 1, 64)).astype(np.float32)
    dots = []
    for p in (0, 5, 40):       # q at p + 7, k at p: the product depends on the distance only
        a = okv.rotate(x, np.array([p + 7]), cs, interleaved)
        b = okv.rotate(y, np.array([p]), cs, interleaved)
        assert np.isclose(np.linalg.norm(a), np.linalg.norm(x), rtol=1e-6)
        dots.append(float((a * b).sum()))
    assert np.allclose(dots, dots[0], rtol=1e-5)
    assert np.array_equal(okv.rotate(x, np.array([0]), cs, interleaved), x)


def test_partial_rotation_leaves_the_rest():
    x = np.arange(64, dtype=np.float32).reshape(1, 1, 64)
    y = okv.rotate(x, np.array([3]), table(8, 32), False)
    assert np.array_equal(y[..., 32:], x[..., 32:]) and not np.array_equal(y[..., :32], x[..., :32])


def test_append_places_tokens_and_gather_returns_grid_values():
    rng = np.random.default_rng(1)
    c = empty()
    # values of the E2M1 grid with a 6 in every block: the scale is 1 and nothing is lost
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -.5, -1, -1.5, -2, -3, -4, -6, 6], np.float32)
    k = np.tile(rng.permutation(grid), (3, 2, 4)).astype(np.float32)
    v = -k
    slots = np.array([17, -1, 63])
    okv.append(c, k, v, slots)
    gk, gv = okv.gather(c, [17, 63])
    assert np.array_equal(gk, k[[0, 2]]) and np.array_equal(gv, v[[0, 2]])
    untouched = np.setdiff1d(np.arange(64), [17, 63])
    assert not c[0].transpose(0, 2, 1, 3).reshape(64, -1)[untouched].any()
    assert not c[3].transpose(0, 3, 1, 2).reshape(64, -1)[untouched].any()


def test_append_is_the_producers_quantization():
    rng = np.random.default_rng(2)
    c = empty(D=128)
    k, v = rng.standard_normal((2, 20, 2, 128)).astype(np.float32)
    okv.append(c, k, v, np.arange(20), k_gs=2.0, v_gs=0.5)
    o = oracle.quantize(v[:, 1], "nvfp4", "rowmajor", global_scale=0.5)
    flat = c[2].transpose(0, 2, 1, 3).reshape(64, 2, 64)
    assert np.array_equal(flat[:20, 1], o.packed)


def test_attention_closed_forms():
    c = empty()
    k = np.zeros((32, 2, 64), np.float32)
    v = np.ones((32, 2, 64), np.float32) * 6
    v[:16] = -6
    okv.append(c, k, v, np.arange(32))
    tables = np.array([[0, 1]])
    q = np.ones((1, 4, 64))
    r = okv.attention(q, c, tables, [32])
    assert np.allclose(r.out, 0) and np.allclose(r.lse, np.log(32)) and np.allclose(r.weight, 6)
    r = okv.attention(q, c, tables, [16])
    assert np.allclose(r.out, -6) and np.allclose(r.lse, np.log(16))
    r = okv.attention(q, c, tables, [0])
    assert np.all(r.out == 0) and np.all(np.isneginf(r.lse))
    r = okv.attention(q, c, np.array([[-1, 1]]), [32])      # a masked page
    assert np.allclose(r.out, 6) and np.allclose(r.lse, np.log(16))
    # 4 query rows, 2 keys: the first two rows see nothing, then one key, then two
    r = okv.attention(np.ones((4, 4, 64)), c, tables, [2], cu=[0, 4])
    assert list(r.keys) == [0, 0, 1, 2] and np.all(r.out[:2] == 0)
    r = okv.attention(np.ones((4, 4, 64)), c, tables, [2], cu=[0, 4], causal=False)
    assert list(r.keys) == [2, 2, 2, 2]


def test_attention_picks_the_matching_key():
    c = empty()
    k = np.zeros((8, 2, 64), np.float32)
    for j in range(8):
        k[j, :, j] = 6
    v = np.zeros((8, 2, 64), np.float32)
    v[:, 0, 0], v[:, 1, 0] = [.5, 1, 1.5, 2, 3, 4, 6, 6], 6
    okv.append(c, k, v, np.arange(8))
    q = np.zeros((1, 4, 64))
    q[0, 1, 3] = 100       # head 1 reads key/value head 0
    r = okv.attention(q, c, np.array([[0]]), [8])
    assert np.isclose(r.out[0, 1, 0], 6 / 6 * 2 * (6 / 6), rtol=0.2)
    assert np.isclose(r.lse[0, 1], 600, atol=1)


def test_attention_weights_by_hand():
    """Two keys whose logits differ by log 3: weights 1/4 and 3/4, in each head of a group."""
    c = empty()
    k = np.zeros((2, 2, 64), np.float32)
    k[1, :, 0] = 6
    v = np.zeros((2, 2, 64), np.float32)
    v[0, :, 0], v[1, :, 0], v[1, 1, 17] = 6, -6, 3            # 3 alone in its block: code 6, scale 1/2
    okv.append(c, k, v, np.arange(2))
    q = np.zeros((1, 4, 64))
    q[0, :, 0] = [np.log(3) / 6, -np.log(3) / 6, np.log(3) / 6, 0]
    r = okv.attention(q, c, np.array([[0]]), [2])
    p1 = np.array([0.75, 0.25, 0.75, 0.5])
    assert np.allclose(r.out[0, :, 0], 6 * (1 - p1) - 6 * p1, rtol=1e-12)
    assert np.allclose(r.out[0, :, 17], [0, 0, 3 * 0.75, 3 * 0.5], rtol=1e-12)
    assert np.allclose(r.lse[0], np.log([4, 4 / 3, 4, 2]), rtol=1e-12)
    assert np.allclose(r.weight[0, :, 0], 6) and np.allclose(r.logit[0], np.log(3) * np.array([1, 1, 1, 0]))
    half = okv.attention(2 * q, c, np.array([[0]]), [2], sm_scale=0.5)
    assert np.allclose(half.out, r.out, rtol=1e-12) and np.allclose(half.lse, r.lse, rtol=1e-12)
    scaled = okv.attention(2 * q, c, np.array([[0]]), [2], k_gs=2.0, v_gs=4.0)
    assert np.allclose(4 * scaled.out, r.out, rtol=1e-12) and np.allclose(scaled.lse, r.lse, rtol=1e-12)
