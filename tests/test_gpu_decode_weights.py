"""kvq_paged_decode_attention_weights against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import serving
from oracle.kv_cache import BF16, FP8, FP8_E5M2
from tests.serving_testlib import P, Pool, assert_output, i32

pytestmark = pytest.mark.gpu


def _k():
    import fp8_kv_cache_reshape_gb300 as k
    return k


def _run(pool, table, lens, q, weights, decay=1.0, window=-1, paired=False, **kw):
    k = _k()
    kd, vd = pool.device(paired)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    w = torch.from_numpy(weights).cuda()
    k.kvq_paged_decode_attention_weights(q, kd, vd, *pool.device_scales(), i32(table), i32(lens), out, w, decay=decay,
                                         window=window, cache_dtype=pool.dtype, per_token=pool.per_token, dev_status=st,
                                         **kw)
    torch.cuda.synchronize()
    return out, w.double().cpu().numpy(), int(st.item())


def _check(pool, table, lens, qv, weights, decay, window, out, got):
    D = pool.D
    ref, mag, acc, size = serving.decode_weights(qv, pool.k, pool.v, pool.k_scale, pool.v_scale, table, lens, weights,
                                                 decay, 1.0 / np.sqrt(D), window, pool.dtype, pool.scales)
    assert_output(out, ref, mag)
    # a score is a sum of D products in float32 (at most a step, 2^-23, per addition, of sums no larger than
    # sum |q k|), the maximum's score likewise: a probability is off by twice that share; 2^-20 for the
    # exponential and the row sum; then 2^-23 for the update of the stored weight
    B, H = weights.shape[:2]
    rel = 2 * D * 2.0 ** -23 * size.reshape(B, H, -1).max(-1) + 2.0 ** -20
    drawn = acc - decay * weights
    bound = np.abs(drawn) * rel[..., None] + 2.0 ** -23 * np.abs(acc) + 1e-12
    for b, L in enumerate(lens):
        assert np.all(np.abs(got[b, :, :L] - acc[b, :, :L]) <= bound[b, :, :L])
        assert np.array_equal(got[b, :, L:], weights[b, :, L:].astype(np.float64)), "entries behind the sequence changed"


CASES = {
    # lengths, KV heads, group, head dim, dtype, per token, window, decay
    "one_token": ([1], 1, 1, 64, FP8, False, -1, 1.0),
    "lengths": ([0, 1, 15, 16, 17, 500], 2, 4, 128, FP8, False, -1, 1.0),
    "odd_group": ([33, 200], 2, 3, 128, FP8, False, -1, 0.5),
    "group_8": ([700, 5, 64], 1, 8, 64, FP8, False, -1, 0.9),
    "group_1": ([300], 4, 1, 128, FP8, False, -1, 0.0),
    "window": ([40, 500, 100], 2, 4, 128, FP8, False, 100, 0.75),
    "window_plain_sum": ([40, 500, 100], 2, 4, 64, FP8, False, 33, 1.0),
    "e5m2": ([100, 777], 2, 4, 128, FP8_E5M2, False, -1, 1.0),
    "e5m2_d64": ([100, 777], 2, 5, 64, FP8_E5M2, False, -1, 1.0),
    "bf16": ([100, 777, 0], 2, 4, 128, BF16, False, -1, 0.99),
    "bf16_window_d64": ([100, 777], 2, 8, 64, BF16, False, 128, 1.0),
    "per_token": ([100, 777], 2, 4, 128, FP8, True, -1, 1.0),
    "per_token_e5m2_d64": ([1, 300], 2, 7, 64, FP8_E5M2, True, -1, 0.5),
    "single_long": ([6000], 1, 4, 128, FP8, False, -1, 1.0),
    "ragged": ([3000, 1, 900, 16], 1, 4, 128, FP8, False, -1, 1.0),
}


@pytest.mark.parametrize("paired", [False, True], ids=["separate", "paired"])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(name, paired):
    lens, heads, group, dim, dtype, per_token, window, decay = CASES[name]
    pool = Pool(sum(-(-n // P) for n in lens) + 2, heads, dim, dtype, 3, per_token)
    table = pool.table(lens)
    q, qv = pool.query(len(lens), group)
    weights = pool.rng.exponential(size=(len(lens), heads, table.shape[1] * P + 5)).astype(np.float32)
    weights[..., ::7] = 0
    out, got, st = _run(pool, table, lens, q, weights, decay, window, paired)
    assert st == 0
    _check(pool, table, lens, qv, weights, decay, window, out, got)


@pytest.mark.parametrize("splits", [1, 2, 7])
def test_split_counts(splits):
    lens = [400, 90]
    pool = Pool(40, 2, 128, FP8, 5)
    table = pool.table(lens)
    q, qv = pool.query(2, 4)
    weights = np.zeros((2, 2, table.shape[1] * P), np.float32)
    out, got, st = _run(pool, table, lens, q, weights, num_splits=splits)
    assert st == 0
    _check(pool, table, lens, qv, weights, 1.0, -1, out, got)
    # the weights of one step sum to the query heads of the group
    assert np.allclose(got.sum(-1), 4.0, rtol=1e-5)


@pytest.mark.parametrize("splits", [3, 9, 20, 60])
@pytest.mark.parametrize("blocks", [150, 5000])  # table columns: four and eight tokens per thread of the last kernel
def test_every_merge_width(splits, blocks):
    lens = [2300, 900]
    pool = Pool(220, 8, 64, FP8, 6)
    table = np.full((2, blocks), -1, np.int32)
    short = pool.table(lens)
    table[:, :short.shape[1]] = short
    q, qv = pool.query(2, 3)
    weights = pool.rng.exponential(size=(2, 8, blocks * P)).astype(np.float32)
    out, got, st = _run(pool, table, lens, q, weights, 0.5, num_splits=splits)
    assert st == 0
    _check(pool, table, lens, qv, weights, 0.5, -1, out, got)


@pytest.mark.parametrize("dtype,per_token", [(FP8, False), (FP8_E5M2, False), (BF16, False), (FP8, True)])
def test_output_is_the_plain_decodes(dtype, per_token):
    """The same plan and kernels as kvq_paged_decode_attention: equal bits
    (several ranges per sequence, so that both merge in the combine)."""
    k = _k()
    lens = [1500, 1333]
    pool = Pool(200, 2, 128, dtype, 7, per_token)
    table = pool.table(lens)
    q, _ = pool.query(2, 4)
    out, _, _ = _run(pool, table, lens, q, np.zeros((2, 2, table.shape[1] * P), np.float32))
    kd, vd = pool.device()
    ref = torch.empty_like(out)
    if per_token:
        k.kvq_paged_decode_attention_per_token(q, kd, vd, i32(table), i32(lens), ref, cache_dtype=dtype)
    else:
        k.kvq_paged_decode_attention(q, kd, vd, *pool.device_scales(), i32(table), i32(lens), ref, cache_dtype=dtype)
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))


def test_bad_pages_draw_no_weight():
    lens = [200, 60]
    pool = Pool(40, 2, 128, FP8, 9)
    table = pool.table(lens)
    q, qv = pool.query(2, 4)
    table[0, 4], table[1, :] = -3, pool.blocks
    weights = np.ones((2, 2, table.shape[1] * P), np.float32)
    out, got, st = _run(pool, table, lens, q, weights, 0.5)
    assert st == 0x2
    _check(pool, table, lens, qv, weights, 0.5, -1, out, got)
    assert np.all(got[1, :, :60] == 0.5) and not out[1].any()


def test_bad_length_is_clamped():
    pool = Pool(40, 1, 64, FP8, 9)
    table = pool.table([100, 32])
    q, qv = pool.query(2, 2)
    weights = np.zeros((2, 1, table.shape[1] * P), np.float32)
    table[1, 2:] = table[0, 2:]  # pages for a length beyond the table
    _, got, st = _run(pool, table, [-7, 10 ** 6], q, weights)
    assert st & 0x4
    assert not got[0].any()


def test_steps_in_a_graph_accumulate():
    k = _k()
    lens = [300, 77]
    pool = Pool(40, 2, 128, FP8, 11)
    table = pool.table(lens)
    q, qv = pool.query(2, 4)
    kd, vd = pool.device()
    w = torch.zeros(2, 2, table.shape[1] * P, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(k.kvq_decode_weights_workspace_size(2, 8, 2, 128, table.shape[1]), dtype=torch.uint8, device="cuda")
    args = (q, kd, vd, *pool.device_scales(), i32(table), i32(lens), out, w)
    k.kvq_paged_decode_attention_weights(*args, workspace=ws)
    torch.cuda.synchronize()
    one = w.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k.kvq_paged_decode_attention_weights(*args, workspace=ws)
    w.zero_()
    for _ in range(4):
        g.replay()
    torch.cuda.synchronize()
    # four additions of the same value to a float32 sum: at most half a step each
    assert ((w - 4 * one).abs() <= 4 * 2.0 ** -24 * (4 * one)).all()
