"""The serving calls as they are used together: a prompt is cached and
observed for some decode steps (attention weights), cut to its heaviest
tokens, and the cut prompt becomes the shared prefix of a batch that decodes
on.  Every step is checked against the float64 oracle on the cache's own
bytes; the whole run again from a captured graph gives the same bits."""
import numpy as np
import pytest
import torch

from oracle import layout, serving
from oracle.kv_cache import FP8, FP8_E5M2
from tests.serving_testlib import P, Pool, assert_output, i32

pytestmark = pytest.mark.gpu


def _k():
    import fp8_kv_cache_reshape_gb300 as k
    return k


@pytest.mark.parametrize("dtype,dim,group,paired", [(FP8, 128, 4, True), (FP8_E5M2, 64, 8, False)])
def test_observe_evict_share(dtype, dim, group, paired):
    k = _k()
    H, B, L, keep, steps = 2, 5, 700, 301, 3
    Hq = H * group
    gen = torch.Generator(device="cuda").manual_seed(31)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    top = 448.0 if dtype == FP8 else 57344.0
    ks = torch.tensor([5.5 / top, 6.0 / top], device="cuda")
    vs = torch.tensor([5.0 / top, 6.5 / top], device="cuda")
    prompt_pages, cut_pages, own_pages = -(-L // P), -(-keep // P), 2
    blocks = prompt_pages + cut_pages + B * own_pages + 3
    order = torch.randperm(blocks, generator=torch.Generator().manual_seed(2)).int()
    prompt, cut = order[:prompt_pages][None], order[prompt_pages:prompt_pages + cut_pages][None]
    own = order[prompt_pages + cut_pages:prompt_pages + cut_pages + B * own_pages].view(B, own_pages)
    kd, vd = k.alloc_kv_cache(blocks, H, dim, dtype, fill=0x7F, paired=paired)  # 0x7F: NaN in both formats
    kp, vp = randn(L, H, dim), randn(L, H, dim)
    pos = torch.arange(L)
    slots = (prompt[0][pos // P].long() * P + pos % P).cuda()
    q_seen = [2 * randn(1, Hq, dim) for _ in range(steps)]
    q_own = [2 * randn(B, Hq, dim) for _ in range(steps)]
    k_own, v_own = ([randn(B, H, dim) for _ in range(steps)] for _ in range(2))
    own_slot = [(own[:, (14 + s) // P].long() * P + (14 + s) % P).cuda() for s in range(steps)]
    starting = torch.cat([(own[b, 0].long() * P + torch.arange(14)) for b in range(B)]).cuda()
    k0, v0 = randn(14 * B, H, dim), randn(14 * B, H, dim)
    weights = torch.zeros(1, H, prompt_pages * P, device="cuda")
    cut_weights = torch.empty(1, H, cut_pages * P, device="cuda")
    kept = torch.zeros(1, H, cut_pages * P, dtype=torch.int32, device="cuda")
    cut_len = torch.zeros(1, dtype=torch.int32, device="cuda")
    tables = dict(prompt=prompt.cuda(), cut=cut.cuda(), own=own.cuda())
    lens = {n: i32([n]) for n in (L, keep)}
    own_lens = [i32([15 + s] * B) for s in range(steps)]
    starts = i32([0, B])
    seen = [torch.empty(1, Hq, dim, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
    outs = [torch.empty(B, Hq, dim, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(k.kvq_decode_weights_workspace_size(1, Hq, H, dim, prompt_pages),
                         k.kvq_shared_prefix_workspace_size(B, 1, Hq, H, dim, cut_pages, own_pages)), dtype=torch.uint8,
                     device="cuda")

    def run():
        weights.zero_()
        k.kvq_reshape_and_cache(kp, vp, slots, kd, vd, ks, vs, dtype, dev_status=st)
        k.kvq_reshape_and_cache(k0, v0, starting, kd, vd, ks, vs, dtype, dev_status=st)
        for s in range(steps):
            k.kvq_paged_decode_attention_weights(q_seen[s], kd, vd, ks, vs, tables["prompt"], lens[L], seen[s], weights,
                                                 num_blocks=blocks, cache_dtype=dtype, workspace=ws, dev_status=st)
        k.kvq_evict_tokens(weights, kd, vd, tables["prompt"], lens[L], lens[keep], tables["cut"], cut_weights, cut_len, kept,
                           head_dim=dim, sink=4, recent=32, num_blocks=blocks, cache_dtype=dtype, dev_status=st)
        for s in range(steps):
            k.kvq_reshape_and_cache(k_own[s], v_own[s], own_slot[s], kd, vd, ks, vs, dtype, dev_status=st)
            k.kvq_paged_decode_attention_shared_prefix(q_own[s], kd, vd, ks, vs, tables["cut"], cut_len, starts, tables["own"],
                                                       own_lens[s], outs[s], num_blocks=blocks, cache_dtype=dtype,
                                                       workspace=ws, dev_status=st)

    run()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # the oracle on the cache as it stands (tokens are only ever added)
    raw = kd.cpu().numpy()
    kpage = P * dim
    kb, vb = (raw[..., :kpage], raw[..., kpage:]) if paired else (raw, vd.cpu().numpy())
    kl, vl = layout.from_device_format(np.ascontiguousarray(kb), np.ascontiguousarray(vb), dim, 1)
    kss, vss, scale = ks.cpu().numpy(), vs.cpu().numpy(), 1 / np.sqrt(dim)
    acc = np.zeros((1, H, prompt_pages * P))
    for s in range(steps):
        ref, mag, acc, _ = serving.decode_weights(q_seen[s].double().cpu().numpy(), kl, vl, kss, vss, prompt.numpy(), [L], acc, 1.0,
                                                  scale, -1, dtype)
        assert_output(seen[s], ref, mag)
    got_w = weights.cpu().numpy()
    assert np.allclose(got_w, acc, rtol=1e-4, atol=1e-9)
    for h in range(H):  # the kept positions by the weights as accumulated
        at = serving.kept_positions(got_w[0, h], L, keep, 4, 32)
        assert kept[0, h, :keep].tolist() == at
        src, _, _ = serving.tokens(kl, vl, kss, vss, prompt[0].numpy(), np.array(at), h, dtype)
        dst, _, _ = serving.tokens(kl, vl, kss, vss, cut[0].numpy(), np.arange(keep), h, dtype)
        assert np.array_equal(src, dst)
    for s in range(steps):
        ref, mag = serving.shared_prefix_decode(q_own[s].double().cpu().numpy(), kl, vl, kss, vss, cut.numpy(), [keep], [0, B],
                                                own.numpy(), [15 + s] * B, scale, dtype)
        assert_output(outs[s], ref, mag)
    first = [t.clone() for t in (kd, weights, cut_weights, kept, *seen, *outs)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for t in (cut_weights, kept, *seen, *outs):
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for a, b in zip(first, (kd, weights, cut_weights, kept, *seen, *outs)))


def test_stuck_wait_ends_the_shared_prefix_call():
    """The test hook of the bounded waits: the call returns, says so in the
    status word, and the next call is right."""
    k = _k()
    pool = Pool(80, 2, 128, FP8, 41)
    pre, mine = pool.table([700]), pool.table([20, 5, 0, 33])
    q, qv = pool.query(4, 4)
    kd, vd = pool.device()
    args = (q, kd, vd, *pool.device_scales(), i32(pre), i32([700]), i32([0, 4]), i32(mine), i32([20, 5, 0, 33]))
    out = torch.empty_like(q)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    k.kvq_debug_set_stall_ns(1_000_000)
    try:
        k.kvq_paged_decode_attention_shared_prefix(*args, out, dev_status=st)
        torch.cuda.synchronize()
    finally:
        k.kvq_debug_set_stall_ns(0)
    assert int(st.item()) & k.KVQ_DEV_TIMEOUT
    st.zero_()
    k.kvq_paged_decode_attention_shared_prefix(*args, out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, mag = serving.shared_prefix_decode(qv, pool.k, pool.v, pool.k_scale, pool.v_scale, pre, [700], [0, 4], mine,
                                            [20, 5, 0, 33], 1 / np.sqrt(128), FP8)
    assert_output(out, ref, mag)


def test_pages_beyond_32_bit_offsets():
    """Pages at the end of caches of 5 GB each: byte offsets beyond 2^32."""
    k = _k()
    dim, L, own, keep = 128, 300, [20, 33], 90
    pool = Pool(60, 1, dim, FP8, 43)
    table, mine, dst = pool.table([L]), pool.table(own), pool.table([keep], fill=False)
    q, qv = pool.query(2, 4)
    weights = pool.rng.exponential(size=(1, 1, table.shape[1] * P)).astype(np.float32)
    blocks = 5 * (1 << 30) // (P * dim)
    small_k, small_v = pool.device()
    kd, vd = (torch.empty(blocks, 1, P * dim, dtype=torch.uint8, device="cuda") for _ in range(2))
    kd[-60:], vd[-60:] = small_k, small_v
    up = blocks - 60
    scales, st = pool.device_scales(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    k.kvq_paged_decode_attention_shared_prefix(q, kd, vd, *scales, i32(table + up), i32([L]), i32([0, 2]), i32(mine + up), i32(own),
                                               out, dev_status=st)
    one = torch.empty_like(q[:1])
    w = torch.zeros(1, 1, table.shape[1] * P, device="cuda")
    k.kvq_paged_decode_attention_weights(q[:1].contiguous(), kd, vd, *scales, i32(table + up), i32([L]), one, w, dev_status=st)
    dw, dl = torch.zeros(1, 1, dst.shape[1] * P, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.zeros(1, 1, dst.shape[1] * P, dtype=torch.int32, device="cuda")
    k.kvq_evict_tokens(torch.from_numpy(weights).cuda(), kd, vd, i32(table + up), i32([L]), i32([keep]), i32(dst + up), dw, dl,
                       kept, head_dim=dim, sink=2, recent=8, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, mag = serving.shared_prefix_decode(qv, pool.k, pool.v, pool.k_scale, pool.v_scale, table, [L], [0, 2], mine, own,
                                            1 / np.sqrt(dim), FP8)
    assert_output(out, ref, mag)
    ref, mag, acc, _ = serving.decode_weights(qv[:1], pool.k, pool.v, pool.k_scale, pool.v_scale, table, [L],
                                              np.zeros(weights.shape), 1.0, 1 / np.sqrt(dim), -1, FP8)
    assert_output(one, ref, mag)
    assert np.allclose(w.cpu().numpy(), acc, rtol=1e-4, atol=1e-9)
    ek, ev, _, rw, _, rk = serving.evict(weights, pool.k, pool.v, table, [L], [keep], dst, np.zeros(dw.shape, np.float32),
                                         np.zeros(kept.shape, np.int32), 2, 8)
    pk, pv = layout.to_device_format(ek, ev)
    assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(dw.cpu().numpy(), rw)
    assert np.array_equal(kd[-60:].cpu().numpy(), pk) and np.array_equal(vd[-60:].cpu().numpy(), pv)
