"""Shared-prefix decode where a CTA goes through several units of work:
against the float64 oracle, and again to the same bits."""
import numpy as np
import pytest
import torch

from oracle import serving
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
