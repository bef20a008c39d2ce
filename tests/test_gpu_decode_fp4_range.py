"""The 4-bit decode where scores are large."""
import numpy as np
import pytest
import torch

from oracle import e2m1
from tests.fp4_testlib import P, Pool4, assert_within, i32
from tests.test_gpu_decode_fp4 import _k, _run

pytestmark = pytest.mark.gpu


def _write(pool, row, k, v):
    """Tokens k, v [n, heads, dim] into the pages of a table row."""
    n = len(k)
    at, off = row[np.arange(n) // P], np.arange(n) % P
    pool.k[at, :, off], pool.ks[at, :, off] = e2m1.quantize(k, pool.k_scale[None])
    pool.v[at, :, off], pool.vs[at, :, off] = e2m1.quantize(v, pool.v_scale[None])


def _pool(n, heads, dim, k_scale, v_scale, seed=0):
    pool = Pool4(-(-n // P) + 2, heads, dim, seed)
    pool.k_scale[:], pool.v_scale[:] = k_scale, v_scale
    return pool, np.array([[pool.order.pop() for _ in range(-(-n // P))]], np.int32)


def _expected(pool, row, n, q, sm):
    """(out, bound on the error) of one sequence's queries [heads * group, dim].

    Half a step of the bf16 output, 2^-8 |out|; of the float16 weight and of its product with the block scale,
    2^-11 sum p |v| each; 2^-12 sum p |v| for the float32 scores and sums and the approximate exponential.  Below
    2^-14 the steps of float16 are 2^-24: 2^-25 of error per token, of the weight and of its product with the block
    scale, where the weights' sum is at least 2^base, base 12 for block scales of an exponent field up to 7 (below
    2) and one less for each beyond."""
    g = len(q) // pool.H
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    j = np.arange(n)
    for h in range(pool.H):
        k, v = pool.tokens(row, 0, n, h)
        rows = slice(h * g, (h + 1) * g)
        out[rows], mag = e2m1.attend(q[rows], k, v, sm)
        field = max(7, int(pool.vs[row[j // P], h, j % P].max()) >> 3)
        tol[rows] = 2.0 ** -8 * np.abs(out[rows]) + (2 * 2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -133
        tol[rows] += 2.0 ** (-25 - 12 + field - 7) * (np.abs(v).sum(0) + n * 6 * float(pool.v_scale[h]))
    return out, tol


@pytest.mark.parametrize("score", [1e7, -1e7, 1e9, -1e9, 1e20, -1e31])
@pytest.mark.parametrize("n", [1, 30])
def test_large_scores_that_are_equal(score, n):
    """Of one key, so that each token weighs the same, however coarse float32 is there."""
    heads, dim = 2, 64
    pool, table = _pool(n, heads, dim, 1.0, 0.003, seed=5)
    rng = np.random.default_rng(6)
    k = np.zeros((n, heads, dim), np.float32)
    k[..., 0] = 1000.0
    _write(pool, table[0], k, rng.standard_normal((n, heads, dim)).astype(np.float32))
    q = torch.zeros(1, 2 * heads, dim, dtype=torch.bfloat16)
    q[0, :, 0] = score / 1000
    ref, tol = _expected(pool, table[0], n, q[0].double().numpy(), 1.0)
    out, st = _run((q.cuda(), *pool.device(), *pool.scales(), i32(table), i32([n])), dict(sm_scale=1.0))
    assert st == 0
    assert_within(out[0], ref, tol)
