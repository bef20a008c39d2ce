"""Calls without a workspace on a side stream, while the current stream still
writes memory that it has given back: the same bits as alone."""
import pytest
import torch

from oracle.kv_cache import FP8
from tests.serving_testlib import P, Pool, i32

pytestmark = pytest.mark.gpu


def _k():
    import fp8_kv_cache_reshape_gb300 as k
    return k


def _shared(k):
    prefixes, starts, own = [1000], [0, 33], [(7 * i) % 40 for i in range(33)]
    pool = Pool(sum(-(-n // P) for n in prefixes + own) + 3, 2, 128, FP8, 5)
    pre, mine = pool.table(prefixes), pool.table(own)
    q, _ = pool.query(33, 4)
    args = (q, *pool.device(), *pool.device_scales(), i32(pre), i32(prefixes), i32(starts), i32(mine), i32(own))
    return (k.kvq_shared_prefix_workspace_size(33, 1, 8, 2, 128, pre.shape[1], mine.shape[1]), [torch.zeros_like(q)],
            lambda outs, **kw: k.kvq_paged_decode_attention_shared_prefix(*args, *outs, **kw))


LENS = [2000, 31, 700]


def _decode_inputs(per_token=False):
    pool = Pool(sum(-(-n // P) for n in LENS) + 3, 2, 128, FP8, 6, per_token)
    table = pool.table(LENS)
    q, _ = pool.query(3, 4)
    return pool, q, (i32(table), i32(LENS)), table.shape[1]


def _weights(k):
    pool, q, tables, width = _decode_inputs()
    args = (q, *pool.device(), *pool.device_scales(), *tables)
    return (k.kvq_decode_weights_workspace_size(3, 8, 2, 128, width), [torch.zeros_like(q), torch.zeros(3, 2, width * P, device="cuda")],
            lambda outs, **kw: k.kvq_paged_decode_attention_weights(*args, *outs, **kw))


def _plain(k):
    pool, q, tables, width = _decode_inputs()
    args = (q, *pool.device(), *pool.device_scales(), *tables)
    return (k.kvq_decode_workspace_size(3, 8, 2, 128, width), [torch.zeros_like(q)],
            lambda outs, **kw: k.kvq_paged_decode_attention(*args, *outs, **kw))


def _append(k):
    pool, q, tables, width = _decode_inputs()
    new, slots = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.full((3,), -1, device="cuda")  # no slot: nothing written
    args = (q, new, new, slots, *pool.device(), *pool.device_scales(), *tables)
    return (k.kvq_decode_workspace_size(3, 8, 2, 128, width), [torch.zeros_like(q)],
            lambda outs, **kw: k.kvq_paged_decode_attention_append(*args, *outs, **kw))


def _per_token(k):
    pool, q, tables, width = _decode_inputs(per_token=True)
    args = (q, *pool.device(), *tables)
    return (k.kvq_decode_workspace_size(3, 8, 2, 128, width), [torch.zeros_like(q)],
            lambda outs, **kw: k.kvq_paged_decode_attention_per_token(*args, *outs, **kw))


@pytest.mark.parametrize("make", [_shared, _weights, _plain, _append, _per_token])
def test_memory_given_back_by_another_stream_is_left_alone(make):
    k = _k()
    size, outs, call = make(k)
    call(outs)
    torch.cuda.synchronize()
    alone = [o.clone() for o in outs]
    side, big = torch.cuda.Stream(), torch.ones(4096, 4096, device="cuda")
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    given_back = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        big @ big
    for _ in range(300):
        given_back.fill_(0xFF)
    del given_back
    call(outs, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(alone, outs))
