"""kvq_paged_decode_attention_shared_prefix against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import serving
from oracle.kv_cache import FP8, FP8_E5M2
from tests.serving_testlib import P, Pool, assert_output, i32

pytestmark = pytest.mark.gpu


def _k():
    import fp8_kv_cache_reshape_gb300 as k
    return k


def _case(prefixes, starts, own, heads, group, dim, dtype, seed=1, width=None):
    pages = sum(-(-n // P) for n in prefixes + own)
    pool = Pool(pages + 3, heads, dim, dtype, seed)
    pre = pool.table(prefixes)
    mine = pool.table(own, width)
    return pool, pre, mine, pool.query(len(own), group), starts


def _run(pool, pre, plens, starts, mine, lens, q, paired=False, workspace=None, **kw):
    k = _k()
    kd, vd = pool.device(paired)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    k.kvq_paged_decode_attention_shared_prefix(q, kd, vd, *pool.device_scales(), i32(pre), i32(plens), i32(starts),
                                               i32(mine), i32(lens), out, cache_dtype=pool.dtype, workspace=workspace,
                                               dev_status=st, **kw)
    torch.cuda.synchronize()
    return out, int(st.item())


CASES = {
    # prefixes, group starts, own lengths, KV heads, group, head dim, dtype
    "one_group": ([300], [0, 4], [1, 17, 64, 5], 2, 4, 128, FP8),
    "tile_exact": ([256], [0, 3], [16, 32, 128], 1, 8, 64, FP8),
    "no_own_tokens": ([129], [0, 2], [0, 0], 2, 2, 128, FP8),
    "empty_rows": ([0, 40], [0, 2, 3], [0, 33, 0], 2, 4, 64, FP8),
    "outside_groups": ([77], [1, 3], [12, 0, 50, 21], 2, 1, 128, FP8),
    "groups_ragged": ([513, 1, 128, 0, 2000], [0, 3, 4, 4, 6, 9], [3, 0, 200, 1, 16, 15, 7, 90, 2], 2, 4, 128, FP8),
    "one_token": ([1], [0, 1], [1], 1, 1, 64, FP8),
    "single_head_long": ([5000], [0, 2], [100, 3], 1, 1, 128, FP8),
    "two_tiles": ([700], [0, 40], [(7 * i) % 50 for i in range(40)], 2, 4, 128, FP8),
    "three_tiles": ([1500], [0, 45], [(5 * i) % 33 for i in range(45)], 1, 8, 64, FP8),
    "five_tiles_e5m2": ([1000, 333], [0, 75, 90], [(3 * i) % 20 for i in range(90)], 2, 8, 128, FP8_E5M2),
    "e5m2_d64": ([2049], [0, 5], [16, 0, 1, 300, 31], 4, 3, 64, FP8_E5M2),
    "many_groups": ([(37 * i) % 300 for i in range(40)], list(range(0, 82, 2)), [(11 * i) % 60 for i in range(80)], 1, 2,
                    64, FP8),
    "batch_256": ([40, 300], [0, 100, 250], [(13 * i) % 70 for i in range(256)], 1, 1, 64, FP8),
    "batch_300": ([100], [5, 300], [(13 * i) % 40 for i in range(300)], 2, 2, 64, FP8),
    "more_heads_than_sms": ([200], [0, 2], [3, 40], 160, 1, 64, FP8),
}


@pytest.mark.parametrize("paired", [False, True], ids=["separate", "paired"])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(name, paired):
    prefixes, starts, own, heads, group, dim, dtype = CASES[name]
    pool, pre, mine, (q, qv), starts = _case(prefixes, starts, own, heads, group, dim, dtype)
    out, st = _run(pool, pre, prefixes, starts, mine, own, q, paired)
    assert st == 0
    ref, mag = serving.shared_prefix_decode(qv, pool.k, pool.v, pool.k_scale, pool.v_scale, pre, prefixes, starts, mine,
                                            own, 1.0 / np.sqrt(dim), dtype)
    assert_output(out, ref, mag)


# prefixes long enough, for their KV heads, that the prefix's grid goes first (eight tiles per CTA or more)
PREFIX_FIRST = {
    "one_slot_per_head": ([1000], [0, 2], [3, 40], 160, 1, 64, FP8),
    "two_tiles": ([1500], [0, 32], [(29 * i) % 100 for i in range(32)], 40, 8, 64, FP8_E5M2),
    "groups": ([1100, 0, 700], [0, 20, 22, 39], [(17 * i) % 50 for i in range(40)], 40, 8, 128, FP8),
    "nothing_of_their_own": ([1500], [0, 32], [0] * 32, 40, 8, 128, FP8),
}


@pytest.mark.parametrize("name", list(PREFIX_FIRST))
def test_long_prefix_first(name):
    prefixes, starts, own, heads, group, dim, dtype = PREFIX_FIRST[name]
    pool, pre, mine, (q, qv), starts = _case(prefixes, starts, own, heads, group, dim, dtype)
    out, st = _run(pool, pre, prefixes, starts, mine, own, q)
    assert st == 0
    ref, mag = serving.shared_prefix_decode(qv, pool.k, pool.v, pool.k_scale, pool.v_scale, pre, prefixes, starts, mine,
                                            own, 1.0 / np.sqrt(dim), dtype)
    assert_output(out, ref, mag)
    # in stream order over one workspace, eager and captured: the same bits
    k = _k()
    kd, vd = pool.device()
    args = [q, kd, vd, *pool.device_scales(), i32(pre), i32(prefixes), i32(starts), i32(mine), i32(own)]
    ws = torch.empty(k.kvq_shared_prefix_workspace_size(len(own), len(prefixes), heads * group, heads, dim, pre.shape[1],
                                                        mine.shape[1]), dtype=torch.uint8, device="cuda")
    outs, g = [torch.zeros_like(q) for _ in range(4)], torch.cuda.CUDAGraph()
    for o in outs[:2]:
        k.kvq_paged_decode_attention_shared_prefix(*args, o, cache_dtype=dtype, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for o in outs[2:]:
            k.kvq_paged_decode_attention_shared_prefix(*args, o, cache_dtype=dtype, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o.view(torch.int16), out.view(torch.int16)) for o in outs)


def test_equals_plain_decode_over_the_joined_table():
    """A prefix of whole pages: the same attention as plain decode over the
    prefix's and the sequence's pages in one table."""
    k = _k()
    prefixes, starts, own = [512], [0, 6], [1, 16, 40, 7, 100, 64]
    pool, pre, mine, (q, _), _ = _case(prefixes, starts, own, 2, 4, 128, FP8)
    out, st = _run(pool, pre, prefixes, starts, mine, own, q)
    joined = np.concatenate([np.repeat(pre, len(own), 0), mine], 1)
    kd, vd = pool.device()
    ref = torch.empty_like(out)
    k.kvq_paged_decode_attention(q, kd, vd, *pool.device_scales(), i32(joined), i32([512 + n for n in own]), ref)
    assert st == 0
    # both round to bf16 (half a step each) and their probabilities to float16 (|v| < 8 here)
    assert ((out.float() - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs() + 8 * 2.0 ** -10).all()


def test_large_scores_keep_their_order():
    """Scores far apart: the largest key's value row comes out alone."""
    pool, pre, mine, (q, qv), starts = _case([400], [0, 3], [20, 0, 5], 1, 4, 128, FP8)
    out, st = _run(pool, pre, [400], starts, mine, [20, 0, 5], q, sm_scale=40.0)
    ref, mag = serving.shared_prefix_decode(qv, pool.k, pool.v, pool.k_scale, pool.v_scale, pre, [400], starts, mine,
                                            [20, 0, 5], 40.0, FP8)
    assert st == 0
    # a score's error is 2^-18 max|q| sum|k| sm_scale and 2^-24 per product: p moves by that share
    err = 40.0 * 128 * 4 * 2 * (2.0 ** -18 + 2.0 ** -22)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + min(1.0, err)) * mag)


def test_bad_pages_are_masked_and_reported():
    prefixes, starts, own = [300], [0, 3], [40, 3, 20]
    pool, pre, mine, (q, qv), _ = _case(prefixes, starts, own, 2, 4, 128, FP8)
    pre, mine = pre.copy(), mine.copy()
    pre[0, 3], pre[0, 18], mine[0, 1], mine[2, 0] = -1, pool.blocks, pool.blocks + 7, -5
    out, st = _run(pool, pre, prefixes, starts, mine, own, q)
    assert st == 0x2
    ref, mag = serving.shared_prefix_decode(qv, pool.k, pool.v, pool.k_scale, pool.v_scale, pre, prefixes, starts, mine,
                                            own, 1.0 / np.sqrt(128), FP8)
    assert_output(out, ref, mag)


def test_every_prefix_page_bad():
    prefixes, starts, own = [40], [0, 2], [5, 0]
    pool, pre, mine, (q, qv), _ = _case(prefixes, starts, own, 1, 2, 64, FP8)
    pre = np.full_like(pre, -1)
    out, st = _run(pool, pre, prefixes, starts, mine, own, q)
    assert st == 0x2
    ref, mag = serving.shared_prefix_decode(qv, pool.k, pool.v, pool.k_scale, pool.v_scale, pre, prefixes, starts, mine,
                                            own, 0.125, FP8)
    assert_output(out, ref, mag)
    assert not out[1].any()


@pytest.mark.parametrize("plens,starts,bits", [
    ([-4, 20], [0, 1, 3], 0x4), ([20, 9999], [0, 1, 3], 0x4), ([20, 20], [0, 5, 3], 0x20), ([20, 20], [2, 0, 3], 0x20),
    ([20, 20], [-1, 1, 3], 0x20), ([20, 20], [0, 1, 7], 0x20)])
def test_bad_groups_are_clamped_and_reported(plens, starts, bits):
    pool, pre, mine, (q, _), _ = _case([20, 20], [0, 1, 3], [4, 4, 4], 1, 2, 64, FP8)
    _, st = _run(pool, pre, plens, starts, mine, [4, 4, 4], q)
    assert st & bits


def test_repeatable_and_in_a_graph():
    """Two replays of a captured step and an eager one: the same bits; a
    second call on another stream with its own workspace too."""
    k = _k()
    prefixes, starts, own = [1000], [0, 33], [(7 * i) % 40 for i in range(33)]
    pool, pre, mine, (q, _), _ = _case(prefixes, starts, own, 2, 4, 128, FP8)
    kd, vd = pool.device()
    args = [q, kd, vd, *pool.device_scales(), i32(pre), i32(prefixes), i32(starts), i32(mine), i32(own)]
    ws = torch.empty(k.kvq_shared_prefix_workspace_size(33, 1, 8, 2, 128, pre.shape[1], mine.shape[1]), dtype=torch.uint8,
                     device="cuda")
    eager = torch.empty_like(q)
    k.kvq_paged_decode_attention_shared_prefix(*args, eager, workspace=ws)
    torch.cuda.synchronize()
    out, g = torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k.kvq_paged_decode_attention_shared_prefix(*args, out, workspace=ws)
    for _ in range(2):
        out.zero_()
        ws.fill_(0xFF)  # NaN in every partial
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
    other, side = torch.zeros_like(q), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    k.kvq_paged_decode_attention_shared_prefix(*args, other, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(other.view(torch.int16), eager.view(torch.int16))


def test_back_to_back_calls_share_a_workspace():
    """Calls in stream order reuse one workspace without waiting in between."""
    k = _k()
    prefixes, starts, own = [700], [0, 8], [5, 0, 100, 7, 64, 16, 3, 31]
    pool, pre, mine, (q, _), _ = _case(prefixes, starts, own, 2, 4, 64, FP8)
    kd, vd = pool.device()
    ws = torch.empty(k.kvq_shared_prefix_workspace_size(8, 1, 8, 2, 64, pre.shape[1], mine.shape[1]), dtype=torch.uint8,
                     device="cuda")
    tables = [i32(pre), i32(prefixes), i32(starts), i32(mine), i32(own)]
    qs = [q * (i + 1) for i in range(6)]
    alone = []
    for x in qs:
        alone.append(k.kvq_paged_decode_attention_shared_prefix(x, kd, vd, *pool.device_scales(), *tables,
                                                                torch.empty_like(x), workspace=ws))
        torch.cuda.synchronize()
    outs = [torch.empty_like(x) for x in qs]
    for x, o in zip(qs, outs):
        k.kvq_paged_decode_attention_shared_prefix(x, kd, vd, *pool.device_scales(), *tables, o, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(alone, outs))
