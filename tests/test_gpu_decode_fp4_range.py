"""The 4-bit decode where the scales of V are far below or far apart from one
another, where scores are large, and where rows have many pieces."""
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


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [0.01, 0.05, 1.0, 300.0])
def test_a_first_token_that_draws_most_and_a_long_flat_tail(size, dim):
    """Head scales of 1, so that block scales are those of the data: subnormal ones at 0.01.  The first token has
    no part in every other dim, whose output is the tail's.  The sequences share their pages, as many as it takes for
    pieces of thousands of tokens."""
    n, heads, batch = 16_003, 2, 512
    pool, table = _pool(n, heads, dim, 1.0, 1.0)
    rng = np.random.default_rng(1)
    k, v = np.zeros((n, heads, dim), np.float32), np.empty((n, heads, dim), np.float32)
    k[0, :, 0] = 10.0  # 14.4 in base 2 above the others
    v[:] = size * np.where(np.arange(dim) % 4 < 2, 1, -1) * rng.uniform(0.7, 1.0, (n, heads, dim))
    v[0, :, ::2] = 0
    _write(pool, table[0], k, v)
    q = torch.zeros(1, 4 * heads, dim, dtype=torch.bfloat16)
    q[0, :, 0] = torch.tensor([1.0, 0.95, 0.9, 0.8] * heads)
    ref, tol = _expected(pool, table[0], n, q[0].double().numpy(), 1.0)
    args = (q.expand(batch, -1, -1).contiguous().cuda(), *pool.device(), *pool.scales(), i32(np.repeat(table, batch, 0)), i32([n] * batch))
    out, st = _run(args, dict(sm_scale=1.0))
    assert st == 0
    assert_within(out, ref[None], tol[None])


@pytest.mark.parametrize("dim,heads,batch,n", [(64, 2, 64, 4001), (128, 1, 60, 4099), (128, 1, 1, 62_005), (64, 1, 1, 1500), (64, 8, 300, 45)])
@pytest.mark.parametrize("first,last", [(1e-3, 2000.0), (2000.0, 1e-3), (5e-3, 5e-3)])
def test_block_scales_that_grow_and_shrink(dim, heads, batch, n, first, last):
    """Parts of several stages, pieces of one, CTAs that join theirs: the sequences share their pages."""
    pool, table = _pool(n, heads, dim, 0.7, 1.0, seed=3)
    rng = np.random.default_rng(4)
    size = np.exp(np.linspace(np.log(first), np.log(last), n))[:, None, None]
    _write(pool, table[0], rng.standard_normal((n, heads, dim)).astype(np.float32),
           (size * rng.standard_normal((n, heads, dim))).astype(np.float32))
    q = torch.from_numpy(rng.standard_normal((1, heads * 3, dim))).bfloat16()
    ref, tol = _expected(pool, table[0], n, q[0].double().numpy(), dim ** -0.5)
    args = (q.expand(batch, -1, -1).contiguous().cuda(), *pool.device(), *pool.scales(), i32(np.repeat(table, batch, 0)), i32([n] * batch))
    out, st = _run(args, {})
    assert st == 0
    assert_within(out, ref[None], tol[None])


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


@pytest.mark.parametrize("scale", [1e-37, 1e-33, 1e-20, 1e20, 1e34, 1.2e35])
@pytest.mark.parametrize("n,dim", [(20, 64), (40_000, 128)])
def test_head_scales_of_any_size(scale, n, dim):
    """One piece, and many that are joined: values of 500 head scales, up to 2,688."""
    pool, table = _pool(n, 1, dim, 0.01, scale, seed=9)
    rng = np.random.default_rng(10)
    v = 500 * (1 + 0.2 * rng.standard_normal((n, 1, dim))) * float(np.float32(scale))
    _write(pool, table[0], rng.standard_normal((n, 1, dim)).astype(np.float32), v.astype(np.float32))
    q = torch.from_numpy(rng.standard_normal((1, 4, dim))).bfloat16()
    ref, tol = _expected(pool, table[0], n, q[0].double().numpy(), dim ** -0.5)
    out, st = _run((q.cuda(), *pool.device(), *pool.scales(), i32(table), i32([n])), {})
    assert st == 0
    assert_within(out[0], ref, tol)


@pytest.mark.parametrize("dim,heads,lengths", [
    (64, 1, [61_000]), (128, 1, [61_000]),        # 32 warps join a row: more pieces than a round's 256
    (64, 4, [15_500]), (128, 2, [12, 16_000]),    # 8 warps: more than 64
    (64, 1, [21_000] + [9] * 239), (128, 2, [5] * 119 + [21_000])])  # 2 warps: more than 16
def test_rows_of_more_pieces_than_a_round_joins(dim, heads, lengths):
    pool = Pool4(sum(-(-n // P) for n in lengths) + 3, heads, dim, 7)
    table = pool.table(lengths)
    qd, q = pool.query(len(lengths), 2)
    ref, tol = pool.attend(q, table, lengths, dim ** -0.5)
    args = (qd, *pool.device(), *pool.scales(), i32(table), i32(lengths))
    out, st = _run(args, {})
    assert st == 0
    assert_within(out, ref, tol)
    again, _ = _run(args, {})
    assert torch.equal(out, again)


def test_the_same_lengths_under_tables_of_several_widths():
    """The joining's form goes by the table's width: each of them within the bound, and each the same every time."""
    lengths = [190, 33]
    pool = Pool4(20, 1, 64, 8)
    table = pool.table(lengths)
    qd, q = pool.query(2, 4)
    ref, tol = pool.attend(q, table, lengths, 0.125)
    for width in (12, 40, 1100):
        wide = np.zeros((2, width), np.int32)
        wide[:, :12] = table
        args = (qd, *pool.device(), *pool.scales(), i32(wide), i32(lengths))
        out, st = _run(args, {})
        assert st == 0
        assert_within(out, ref, tol)
        assert torch.equal(out, _run(args, {})[0])
