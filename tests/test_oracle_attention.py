"""Pins of the attention step's oracle (closed forms, exact cases, hand-worked tables) and of the host function
svq_rope_frequencies, which needs no GPU."""
import math

import numpy as np
import pytest

from oracle import attention as oa

import bit_spherical_vector_b200 as svq


def test_kv_assign_hand_worked():
    """Pages of 4: request 0 (5 tokens on pages 7, 2) gets 4 -> one page; request 1 is done (pages 5, 9 back, 9 on
    top); request 2 (4 tokens, page 1 full) gets 1 -> one page; request 3 idles.  The stack 0 3 | 5 9 gives 9 to
    request 0 and 5 to request 2."""
    table = np.full((4, 4), -1)
    table[0, :2], table[1, :2], table[2, 0], table[3, 0] = (7, 2), (5, 9), 1, 4
    free = np.array([0, 3, -1, -1, -1, -1, -1, -1, -1, -1])
    r = oa.kv_assign([5, 6, 4, 1], [4, -1, 1, 0], 4, table, free, 2, 7)
    assert r["cu_rows"].tolist() == [0, 4, 4, 5, 5]
    assert r["positions"].tolist() == [5, 6, 7, 8, 4, -1, -1]
    assert r["slots"].tolist() == [9, 10, 11, 36, 20, -1, -1]
    assert r["block_table"][0].tolist() == [7, 2, 9, -1] and r["block_table"][2].tolist() == [1, 5, -1, -1]
    assert r["lens_out"].tolist() == [9, 0, 5, 1] and r["n_free_out"] == 2
    assert r["free_pages"].tolist() == free.tolist()


def test_kv_assign_released_pages_that_stay_free():
    table = np.array([[3, 4, 5], [0, -1, -1]])
    free = np.array([1, 2, -1, -1, -1, -1])
    r = oa.kv_assign([12, 4], [-1, 1], 4, table, free, 2, 4)
    assert r["block_table"][1].tolist() == [0, 5, -1]
    assert r["n_free_out"] == 4 and r["free_pages"].tolist() == [1, 2, 3, 4, -1, -1]


@pytest.mark.parametrize("lens,new,n_free,rows", [([-1], [1], 2, 4), ([5], [8], 2, 9), ([1], [5], 2, 4),
                                                  ([4], [5], 1, 8), ([1], [1], 4, 4)])
def test_kv_assign_refusals(lens, new, n_free, rows):
    assert oa.kv_assign(lens, new, 4, np.zeros((1, 3)), np.zeros(3), n_free, rows) is None


def test_rotate_closed_forms():
    x = np.arange(1.0, 9.0)
    assert np.array_equal(oa.rotate(x, 0, [1.0, 0.5]), x)
    y = oa.rotate(x, 1, [math.pi / 2])                        # a quarter turn of the pair (0, 1)
    assert np.allclose(y, [-2, 1, 3, 4, 5, 6, 7, 8], atol=1e-15)
    y = oa.rotate(x, 3, [math.pi / 2, math.pi / 3], interleaved=True)
    assert np.allclose(y, [2, -1, -3, -4, 5, 6, 7, 8], atol=1e-14)
    y = oa.rotate(x, 2, [math.pi / 4, math.pi / 2], factor=2.0)   # pairs (0, 2) and (1, 3)
    assert np.allclose(y, [-6, -4, 2, -8, 5, 6, 7, 8], atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_keeps_lengths_and_relative_positions(interleaved):
    rng = np.random.default_rng(1)
    f = svq.svq_rope_frequencies(64, 10000.0)[0]
    a, b = rng.standard_normal((2, 64))
    ra, rb = oa.rotate(a, 1234, f, 1.0, interleaved), oa.rotate(b, 1200, f, 1.0, interleaved)
    assert np.allclose(oa.pair_size(ra, 64, interleaved), oa.pair_size(a, 64, interleaved), rtol=1e-13)
    shifted = oa.rotate(a, 34, f, 1.0, interleaved) @ b
    assert abs(ra @ rb - shifted) < 1e-10


def test_head_norm_constant_head_gives_gamma():
    g = np.linspace(-2, 3, 64)
    assert np.allclose(oa.head_norm(np.full((2, 64), -4.0), g, 0.0), -np.tile(g, (2, 1)), rtol=1e-15)


def test_attention_closed_forms():
    # equal scores: the mean; one key: its value; a score far ahead: its value
    v = np.arange(12.0).reshape(3, 4)
    o, lse, size, _ = oa.attend(np.zeros(4), np.ones((3, 4)), v, 0.5)
    assert np.allclose(o, v.mean(0)) and lse == pytest.approx(math.log(3.0)) and np.allclose(size, v.mean(0))
    o, lse, _, _ = oa.attend(np.ones(4), np.full((1, 4), 2.0), v[1:2], 0.25)
    assert np.array_equal(o, v[1]) and lse == pytest.approx(2.0)
    o, lse, _, _ = oa.attend(np.ones(4), np.array([[0.0] * 4, [500.0] * 4]), v[:2], 1.0)
    assert np.array_equal(o, v[1]) and lse == 2000.0
    o, lse, _, _ = oa.attend(np.ones(4), np.zeros((0, 4)), np.zeros((0, 4)), 1.0)
    assert np.array_equal(o, np.zeros(4)) and lse == -math.inf
    # two keys with odds 3 : 1
    o, _, _, _ = oa.attend(np.array([math.log(3.0)]), np.array([[1.0], [0.0]]), np.array([[8.0], [4.0]]), 1.0)
    assert o[0] == pytest.approx(7.0)


def test_paged_attention_follows_the_table():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 6, 4, 2, 8))
    q = rng.standard_normal((2, 4, 8))
    table = np.array([[5, 1, -1], [3, 0, 2]])
    r = oa.paged_attention(q, k, v, [6, 0], table, 0.3)
    keys = np.concatenate([k[5], k[1][:2]])
    vals = np.concatenate([v[5], v[1][:2]])
    for h in range(4):
        want = oa.attend(q[0, h], keys[:, h // 2], vals[:, h // 2], 0.3)[0]
        assert np.allclose(r[0][0][h], want)
    assert np.array_equal(r[1][0], np.zeros((4, 8))) and np.all(r[1][1] == -math.inf)
    r = oa.paged_attention(q, k, v, [6, 2], table, 0.3, cu_rows=[0, 0, 2])
    assert list(r) == [1]


def test_rope_frequencies_plain_linear_ntk():
    f, c = svq.svq_rope_frequencies(128, 1e6)
    want = 1e6 ** (-np.arange(64) / 64.0)
    assert c == 1.0 and np.allclose(f, want, rtol=1e-14)
    g, c = svq.svq_rope_frequencies(128, 1e6, svq.SVQ_ROPE_LINEAR, 4.0)
    assert c == 1.0 and np.allclose(g, want / 4, rtol=1e-14)
    g, c = svq.svq_rope_frequencies(128, 1e6, svq.SVQ_ROPE_NTK, 4.0)
    # the fastest pair is untouched and the slowest is slowed by exactly the scale
    assert c == 1.0 and g[0] == 1.0 and g[-1] == pytest.approx(want[-1] / 4, rel=1e-12)


def test_rope_frequencies_yarn():
    """Pairs that turn more than 32 times over the trained length keep their frequency, pairs that turn less than
    once are divided by the scale, between them the ramp is monotone; factor 0.1 ln s + 1."""
    s, n = 4.0, 32768
    f, c = svq.svq_rope_frequencies(128, 1e6, svq.SVQ_ROPE_YARN, s, n)
    plain = svq.svq_rope_frequencies(128, 1e6)[0]
    turns = plain * n / (2 * math.pi)
    ratio = f / plain
    assert c == pytest.approx(0.1 * math.log(4.0) + 1.0, rel=1e-6)
    at = lambda t: 128 * math.log(n / (t * 2 * math.pi)) / (2 * math.log(1e6))
    i = np.arange(64)
    assert np.all(ratio[i <= math.floor(at(32.0))] == 1.0) and np.all(turns[i <= math.floor(at(32.0))] >= 32.0)
    slow = i >= math.ceil(at(1.0))
    assert slow.any() and np.allclose(ratio[slow], 1 / s, rtol=1e-14) and np.all(turns[slow] <= 1.0)
    assert np.all(np.diff(ratio) <= 1e-15)
    # scale 1 changes nothing
    f1, c1 = svq.svq_rope_frequencies(128, 1e6, svq.SVQ_ROPE_YARN, 1.0, n)
    assert c1 == 1.0 and np.allclose(f1, plain, rtol=1e-15)


@pytest.mark.parametrize("args,status", [((24, 1e4), svq.SVQ_ERR_UNSUPPORTED_SHAPE),
                                         ((0, 1e4), svq.SVQ_ERR_UNSUPPORTED_SHAPE),
                                         ((512, 1e4), svq.SVQ_ERR_UNSUPPORTED_SHAPE),
                                         ((64, 1.0), svq.SVQ_ERR_INVALID_ARG),
                                         ((64, float("nan")), svq.SVQ_ERR_INVALID_ARG),
                                         ((64, 1e4, 4), svq.SVQ_ERR_INVALID_ARG),
                                         ((64, 1e4, svq.SVQ_ROPE_LINEAR, 0.5), svq.SVQ_ERR_INVALID_ARG),
                                         ((64, 1e4, svq.SVQ_ROPE_YARN, 2.0, 0), svq.SVQ_ERR_INVALID_ARG)])
def test_rope_frequencies_refusals(args, status):
    with pytest.raises(svq.SvqError) as e:
        svq.svq_rope_frequencies(*args)
    assert e.value.status == status
