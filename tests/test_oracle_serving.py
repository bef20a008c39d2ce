"""Pins of oracle/serving.py that do not restate its formulas."""
import itertools
import math

import numpy as np

from oracle import attention, serving
from oracle.kv_cache import FP8
from tests.serving_testlib import P, Pool


def test_shared_prefix_equals_decode_over_the_joined_table():
    pool = Pool(40, 2, 64, FP8, 1)
    pre, own = pool.table([64, 32]), [5, 16, 33]
    mine = pool.table(own)
    _, q = pool.query(3, 3)
    out, _ = serving.shared_prefix_decode(q, pool.k, pool.v, pool.k_scale, pool.v_scale, pre, [64, 32], [0, 2, 3], mine, own,
                                          0.2, FP8)
    for b, i, n in ((0, 0, 64), (1, 0, 64), (2, 1, 32)):
        joined = np.concatenate([pre[i][:n // P], mine[b]])[None]
        ref, _ = attention.paged_decode(q[b:b + 1], pool.k, pool.v, pool.k_scale, pool.v_scale, joined, [n + own[b]], 0.2,
                                        mode="pure")
        # the oracle's own scale is rounded to float32 there
        assert np.allclose(out[b], ref[0], rtol=1e-6, atol=1e-7)


def test_weights_sum_to_the_heads_and_reproduce_the_output():
    pool = Pool(20, 2, 64, FP8, 2)
    lens = [100, 40]
    table = pool.table(lens)
    _, q = pool.query(2, 1)
    w0 = np.zeros((2, 2, table.shape[1] * P))
    out, _, acc, _ = serving.decode_weights(q, pool.k, pool.v, pool.k_scale, pool.v_scale, table, lens, w0, 1.0, 0.125, -1, FP8)
    assert np.allclose(acc.sum(-1), 1.0)
    for b, L in enumerate(lens):  # one query head per KV head: the weights are its probabilities
        for h in range(2):
            _, v, _ = serving.tokens(pool.k, pool.v, pool.k_scale, pool.v_scale, table[b], np.arange(L), h, FP8)
            assert np.allclose(acc[b, h, :L] @ v, out[b, h])
    _, _, win, _ = serving.decode_weights(q, pool.k, pool.v, pool.k_scale, pool.v_scale, table, lens, w0 + 1, 0.5, 0.125, 16, FP8)
    assert np.allclose(win[0, :, :84], 0.5) and np.allclose(win[0, :, 100:], 1.0)


def test_kept_positions_by_exhaustion():
    """Over every subset: the kept set has the largest total weight, and among
    equal totals the lowest positions."""
    rng = np.random.default_rng(3)
    for trial in range(60):
        L, sink, recent = 9, int(rng.integers(0, 3)), int(rng.integers(0, 4))
        keep = int(rng.integers(0, L + 2))
        w = rng.integers(0, 4, L).astype(np.float64)
        got = serving.kept_positions(w, L, keep, sink, recent)
        n = min(keep, L)
        s = min(sink, n)
        r = min(recent, n - s)
        must = set(range(s)) | set(range(L - r, L))
        best = max((c for c in itertools.combinations(range(L), n) if must <= set(c)),
                   key=lambda c: (sum(w[j] for j in c), [-j for j in c]))
        assert sum(w[j] for j in got) == sum(w[j] for j in best) and must <= set(got) and len(got) == n
        assert got == sorted(got)
        out = [j for j in range(s, L - r) if j not in got]
        assert all(w[a] > w[b] or (w[a] == w[b] and a < b) for a in got if a not in must for b in out)


def test_nan_ranks_lowest():
    w = np.array([math.nan, -math.inf, 0.0, -0.0, math.nan, 1.0])
    assert serving.kept_positions(w, 6, 4, 0, 0) == [1, 2, 3, 5]
    assert serving.kept_positions(w, 6, 5, 0, 0) == [0, 1, 2, 3, 5]
    assert serving.kept_positions(w, 6, 2, 0, 0) == [2, 5]
