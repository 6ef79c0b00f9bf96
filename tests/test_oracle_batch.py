"""The oracle of the batch operators against worked values and counts."""

import numpy as np

from oracle import batch


def test_extend_worked():
    # pages of 4; request 0 fills its page and takes one, 1 has room, 2 starts, 3 wants more than is left
    table = np.array([[7, 0, 0], [8, 0, 0], [0, 0, 0], [9, 0, 0]], np.int32)
    got = batch.extend([3, 1, 0, 4], [2, 1, 1, 8], table, np.array([1, 2, 3, 0]), 3, 4, 14)
    assert got["table"].tolist() == [[7, 3, 0], [8, 0, 0], [2, 0, 0], [9, 0, 0]]
    assert got["served"].tolist() == [True, True, True, False] and got["free_count"] == 1
    assert got["lengths"].tolist() == [5, 2, 1, 4]
    assert got["starts"].tolist() == [0, 2, 3, 4, 12]
    assert got["positions"].tolist() == [3, 4, 1, 0, 4, 5, 6, 7, 8, 9, 10, 11, 0, 0]
    assert got["slots"].tolist() == [31, 12, 33, 8] + [-1] * 10
    assert got["request"].tolist() == [0, 0, 1, 2] + [3] * 8 + [-1, -1]
    assert got["row_lengths"].tolist() == [4, 5, 2, 1] + [0] * 10
    assert got["row_tables"][1].tolist() == [7, 3, 0] and got["row_tables"][0].tolist() == [7, 0, 0]


def test_trim_takes_back_what_extend_took():
    r = np.random.default_rng(1)
    lengths, new = r.integers(0, 40, 9), r.integers(0, 30, 9)
    stack = np.arange(100, dtype=np.int32)
    grown = batch.extend(np.zeros(9, int), lengths, np.zeros((9, 12), np.int32), stack, 100, 7, 400)
    more = batch.extend(grown["lengths"], new, grown["table"], stack, grown["free_count"], 7, 400)
    after, count, back = batch.trim(more["lengths"], lengths, more["table"], stack, more["free_count"], 7)
    assert after.tolist() == lengths.tolist() and count == grown["free_count"]
    held = [int(p) for b in range(9) for p in grown["table"][b, :-(-int(lengths[b]) // 7)]]
    assert sorted(held + back[:count].tolist()) == list(range(100))


def test_lora_is_the_dense_matrix():
    r = np.random.default_rng(2)
    x, y = r.standard_normal((3, 5)), r.standard_normal((3, 4))
    a, b, s = r.standard_normal((2, 2, 5)), r.standard_normal((2, 4, 2)), np.array([0.5, -2.0])
    out, mag = batch.lora(y, x, a, b, [1, -1, 0], s)
    for t, i in ((0, 1), (2, 0)):
        assert np.allclose(out[t], y[t] + x[t] @ (s[i] * b[i] @ a[i]).T)
    assert np.array_equal(out[1], y[1]) and np.all(mag[1] == 0)
    assert np.all(mag + 1e-12 >= np.abs(out - y))


def test_kept_worked():
    l = np.log([0.1, 0.4, 0.1, 0.3, 0.1])
    assert batch.kept(l, 1.0)[0].tolist() == [0, 1, 2, 3, 4]
    assert batch.kept(l, 1.0, top_k=3)[0].tolist() == [0, 1, 3]          # equal ones: the lower index
    assert batch.kept(l, 1.0, top_p=0.6)[0].tolist() == [1, 3]
    assert batch.kept(l, 1.0, top_p=0.75)[0].tolist() == [0, 1, 3]
    assert batch.kept(l, 1.0, top_k=2, top_p=0.5)[0].tolist() == [1]      # 4/7 of the two
    assert batch.kept(l, 1.0, min_p=0.5)[0].tolist() == [1, 3]
    assert batch.kept(l, 0.0)[0].tolist() == [1]
    assert batch.kept([np.nan, -np.inf, 2.0], 1.0)[0].tolist() == [2]
    assert batch.kept([np.inf, 0.0, np.inf], 1.0)[1].tolist()[::2] == [1.0, 1.0]
    assert batch.draw([np.nan, -np.inf], 0.3, 1.0) == (-1, -np.inf)


def test_draw_follows_the_weights():
    l = np.log([0.1, 0.4, 0.2, 0.3])
    u = (np.arange(1000) + 0.5) / 1000
    tokens = [batch.draw(l, v, 1.0)[0] for v in u]
    assert np.bincount(tokens).tolist() == [100, 400, 200, 300]
    assert np.isclose(batch.draw(l, 0.2, 1.0)[1], np.log(0.4))
    half = [batch.draw(l, v, 1.0, top_k=2)[0] for v in u]
    assert set(half) == {1, 3} and abs(np.mean(np.array(half) == 1) - 4 / 7) < 2e-3
