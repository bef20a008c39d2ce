"""Shared-prefix decode where a CTA goes through several units of work:
against the float64 oracle, and again to the same bits."""
import numpy as np
import pytest
import torch

from oracle import serving
from oracle.kv_cache import FP8
from tests.serving_testlib import P, Pool, assert_output, i32
from tests.test_serving_segments import SEGMENTS, most_segments, starts_of

pytestmark = pytest.mark.gpu


def _k():
    import fp8_kv_cache_reshape_gb300 as k
    return k


@pytest.mark.parametrize("name", list(SEGMENTS))
def test_matches_oracle_and_repeats(name):
    k = _k()
    prefixes, sizes, heads, group, dim, dtype, least = SEGMENTS[name]
    slots = torch.cuda.get_device_properties(0).multi_processor_count // heads
    assert most_segments(prefixes, sizes, group, max(1, slots)) >= least
    starts = starts_of(sizes)
    own = [(17 * i) % 50 for i in range(starts[-1])]
    pool = Pool(sum(-(-n // P) for n in prefixes + own) + 3, heads, dim, dtype, 7)
    pre, mine = pool.table(prefixes), pool.table(own)
    q, qv = pool.query(len(own), group)
    kd, vd = pool.device()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q, kd, vd, *pool.device_scales(), i32(pre), i32(prefixes), i32(starts), i32(mine), i32(own))
    ws = torch.empty(k.kvq_shared_prefix_workspace_size(len(own), len(sizes), heads * group, heads, dim, pre.shape[1],
                                                        mine.shape[1]), dtype=torch.uint8, device="cuda")
    outs = [torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    for o in outs:
        k.kvq_paged_decode_attention_shared_prefix(*args, o, cache_dtype=dtype, workspace=ws, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, mag = serving.shared_prefix_decode(qv, pool.k, pool.v, pool.k_scale, pool.v_scale, pre, prefixes, starts, mine, own,
                                            1 / np.sqrt(dim), dtype)
    assert_output(outs[0], ref, mag)
    assert all(torch.equal(o.view(torch.int16), outs[0].view(torch.int16)) for o in outs[1:])


@pytest.mark.parametrize("prefixes", [[1100, 700], [200, 100]], ids=["prefix_first", "own_first"])
def test_inputs_written_by_the_preceding_kernels(prefixes):
    """The call's inputs change in place between calls, in stream order: each
    call sees its own, whichever of its grids goes first, eager and captured."""
    k = _k()
    heads, group, dim, B = 40, 8, 128, 40
    pool = Pool(sum(-(-n // P) for n in prefixes) + 4 * B + 3, heads, dim, FP8, 11)
    pre, mine = pool.table(prefixes), pool.table([64] * B)
    kd, vd = pool.device()
    ks, vs = pool.device_scales()
    sets = []
    for i in range(4):
        q, qv = pool.query(B, group)
        own = [(29 * j + 13 * i) % 65 for j in range(B)]
        sets.append(((q, ks * (1 + 0.25 * i), vs * (1 + 0.5 * i), i32(pre[::-1].copy() if i % 2 else pre),
                      i32([(min(prefixes) - 37 * i), min(prefixes) - i]), i32([0, 20 + i, 39 - i]), i32(np.roll(mine, i, 0)), i32(own)),
                     qv, own))

    def call(a, out, ws):
        q, s, t, *tables = a
        k.kvq_paged_decode_attention_shared_prefix(q, kd, vd, s, t, *tables, out, workspace=ws)

    ws = torch.empty(k.kvq_shared_prefix_workspace_size(B, 2, heads * group, heads, dim, pre.shape[1], mine.shape[1]),
                     dtype=torch.uint8, device="cuda")
    alone = [torch.zeros_like(sets[0][0][0]) for _ in sets]
    for (a, _, _), o in zip(sets, alone):
        call(a, o, ws)
        torch.cuda.synchronize()
    for i in (0, 3):
        a, qv, own = sets[i]
        table, plens, starts, rows = (t.cpu().numpy() for t in a[3:7])
        ref, mag = serving.shared_prefix_decode(qv, pool.k, pool.v, a[1].cpu().numpy(), a[2].cpu().numpy(), table, plens, starts,
                                                rows, own, 1 / np.sqrt(dim), FP8)
        assert_output(alone[i], ref, mag)
    now = [torch.zeros_like(t) for t in sets[0][0]]
    outs = [torch.zeros_like(o) for o in alone]

    def steps():
        for (a, _, _), o in zip(sets, outs):
            for dst, src in zip(now, a):
                dst.copy_(src)
            call(now, o, ws)

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(alone, outs))
        for o in outs:
            o.zero_()

    for _ in range(3):
        steps()
        check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        steps()
    for _ in range(3):
        g.replay()
        check()


@pytest.mark.parametrize("dim", [64, 128])
def test_scores_below_the_smallest_float(dim):
    """Queries and a K scale so small that no score differs from 0: every key
    counts alike, and those behind the prefix's end still count nothing."""
    k = _k()
    prefixes, own = [300], [20, 0, 5]
    pool = Pool(30, 1, dim, FP8, 13)
    pre, mine = pool.table(prefixes), pool.table(own)
    pool.k_scale[:] = 2.0 ** -45
    q, _ = pool.query(3, 4)
    q = q * 2.0 ** -110
    kd, vd = pool.device()
    out, st = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    k.kvq_paged_decode_attention_shared_prefix(q, kd, vd, *pool.device_scales(), i32(pre), i32(prefixes), i32([0, 3]), i32(mine),
                                               i32(own), out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, mag = serving.shared_prefix_decode(q.double().cpu().numpy(), pool.k, pool.v, pool.k_scale, pool.v_scale, pre, prefixes,
                                            [0, 3], mine, own, 1 / np.sqrt(dim), FP8)
    assert_output(out, ref, mag)


def test_calls_on_two_streams_at_once():
    """Calls with several segments per CTA on two streams, each with its own
    workspace, beside each other: the bits of each alone."""
    k = _k()
    calls = []
    for seed, (prefixes, sizes, heads, group, dim) in enumerate([([700, 900], [10, 32], 80, 4, 128), ([1500], [40], 8, 4, 128)]):
        own = [(31 * i) % 90 for i in range(sum(sizes))]
        pool = Pool(sum(-(-n // P) for n in prefixes + own) + 3, heads, dim, FP8, 17 + seed)
        pre, mine = pool.table(prefixes), pool.table(own)
        q, _ = pool.query(len(own), group)
        args = (q, *pool.device(), *pool.device_scales(), i32(pre), i32(prefixes), i32(starts_of(sizes)), i32(mine), i32(own))
        alone = k.kvq_paged_decode_attention_shared_prefix(*args, torch.zeros_like(q))
        calls.append((args, alone, [torch.zeros_like(q) for _ in range(20)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(20):
        for args, _, outs, side in calls:
            k.kvq_paged_decode_attention_shared_prefix(*args, outs[i], stream=side)
    torch.cuda.synchronize()
    for _, alone, outs, _ in calls:
        assert all(torch.equal(alone.view(torch.int16), o.view(torch.int16)) for o in outs)
