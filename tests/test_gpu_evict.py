"""kvq_evict_tokens: bytes, positions, weights and lengths equal to the
oracle's, everything else left as it was."""
import numpy as np
import pytest
import torch

from oracle import layout, serving
from oracle.kv_cache import BF16, FP8, FP8_E5M2
from tests.serving_testlib import P, Pool, i32

pytestmark = pytest.mark.gpu


def _k():
    import fp8_kv_cache_reshape_gb300 as k
    return k


def _run(pool, weights, table, lens, keep, dst, sink, recent, paired=False, extra=0):
    k = _k()
    B, H = weights.shape[:2]
    cap = dst.shape[1] * P
    kd, vd = pool.device(paired)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = torch.full((B, H, cap + extra), 7.0, device="cuda")
    kept = torch.full((B, H, cap), -9, dtype=torch.int32, device="cuda")
    dl = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    k.kvq_evict_tokens(torch.from_numpy(weights).cuda(), kd, vd, i32(table), i32(lens), i32(keep), i32(dst), dw, dl, kept,
                       head_dim=pool.D, sink=sink, recent=recent, cache_dtype=pool.dtype, per_token=pool.per_token,
                       dev_status=st)
    torch.cuda.synchronize()
    return kd.cpu().numpy(), vd.cpu().numpy(), dw.cpu().numpy(), dl.cpu().numpy(), kept.cpu().numpy(), int(st.item())


def _check(pool, weights, table, lens, keep, dst, sink, recent, paired=False, extra=0):
    kd, vd, dw, dl, kept, st = _run(pool, weights, table, lens, keep, dst, sink, recent, paired, extra)
    assert st == 0
    B, H = weights.shape[:2]
    cap = dst.shape[1] * P
    k, v, sc, rw, rl, rk = serving.evict(weights, pool.k, pool.v, table, lens, keep, dst,
                                         np.zeros((B, H, cap + extra), np.float32), np.full((B, H, cap), -9, np.int32),
                                         sink, recent, pool.scales)
    assert np.array_equal(dl, rl) and np.array_equal(kept, rk)
    assert np.array_equal(dw, rw, equal_nan=True)
    if paired:
        assert np.array_equal(kd, layout.to_device_format_paired(k, v, sc))
        return
    ek, ev = layout.to_device_format(k, v) if sc is None else layout.to_device_format_per_token(k, v, sc)
    assert np.array_equal(kd, ek) and np.array_equal(vd, ev)


def _weights(rng, B, H, W, kind):
    w = rng.exponential(size=(B, H, W)).astype(np.float32)
    if kind == "ties":
        w = np.floor(w * 2).astype(np.float32)
        w[..., ::5] = -0.0
    elif kind == "equal":
        w[:] = 1.25
    elif kind == "odd":
        w[..., ::3], w[..., 1::7], w[..., 2::11], w[..., 4::13] = np.nan, np.inf, -np.inf, -w[..., 4::13]
        w[..., 5::17] = 1e-40  # subnormal
    return w


CASES = {
    # lengths, keep, KV heads, head dim, dtype, per token, sink, recent, weights
    "one": ([1], [1], 1, 64, FP8, False, 0, 0, "plain"),
    "none_kept": ([40, 0], [0, 5], 2, 64, FP8, False, 4, 4, "plain"),
    "all_kept": ([40, 17], [40, 99], 2, 128, FP8, False, 4, 4, "plain"),
    "half": ([500, 333, 16], [250, 100, 15], 2, 128, FP8, False, 4, 32, "plain"),
    "ties": ([500, 333], [250, 101], 2, 128, FP8, False, 3, 10, "ties"),
    "equal": ([300, 333], [20, 101], 1, 64, FP8, False, 0, 0, "equal"),
    "odd_values": ([400, 399], [200, 390], 2, 64, FP8, False, 0, 0, "odd"),
    "sink_takes_all": ([300], [5], 2, 128, FP8, False, 9, 9, "plain"),
    "recent_takes_the_rest": ([300], [50], 2, 128, FP8, False, 9, 100, "plain"),
    "d256": ([200, 70], [77, 33], 2, 256, FP8, False, 2, 8, "plain"),
    "e5m2": ([200, 70], [77, 33], 2, 128, FP8_E5M2, False, 2, 8, "plain"),
    "bf16_d128": ([200, 70], [77, 33], 2, 128, BF16, False, 2, 8, "plain"),
    "bf16_d64": ([200, 70], [78, 32], 2, 64, BF16, False, 2, 8, "ties"),
    "per_token": ([200, 70], [77, 33], 2, 128, FP8, True, 2, 8, "plain"),
    "per_token_e5m2_d64": ([200, 70], [77, 33], 2, 64, FP8_E5M2, True, 2, 8, "plain"),
    "cluster_2": ([8000, 5], [3001, 5], 1, 64, FP8, False, 4, 64, "plain"),
    "sparse": ([9000], [300], 1, 64, FP8, False, 4, 64, "ties"),
}


@pytest.mark.parametrize("paired", [False, True], ids=["separate", "paired"])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(name, paired):
    lens, keep, heads, dim, dtype, per_token, sink, recent, kind = CASES[name]
    need = [min(a, b) for a, b in zip(lens, keep)]
    pool = Pool(sum(-(-n // P) for n in lens + need) + 3, heads, dim, dtype, 13, per_token)
    table = pool.table(lens)
    dst = pool.table(need, max(1, -(-max(need) // P)) + 1, fill=False)
    weights = _weights(pool.rng, len(lens), heads, table.shape[1] * P + 3, kind)
    _check(pool, weights, table, lens, keep, dst, sink, recent, paired, extra=5)


def test_source_pages_may_be_shared():
    """Two sequences over the same pages (a shared prompt), cut differently."""
    pool = Pool(80, 2, 64, FP8, 17)
    one = pool.table([600])
    table = np.repeat(one, 2, 0)
    dst = pool.table([200, 111], fill=False)
    weights = _weights(pool.rng, 2, 2, table.shape[1] * P, "plain")
    _check(pool, weights, table, [600, 590], [200, 111], dst, 4, 16)


def test_selection_of_a_long_sequence():
    """Positions and weights at 300,000 tokens, beyond what a CTA holds in
    shared memory in some plans; many equal weights around the threshold."""
    k = _k()
    L, keep = 300_000, 77_777
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = torch.floor(torch.rand(1, 2, L, generator=gen, device="cuda") * 300)
    blocks = -(-L // P)
    table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    nd = -(-keep // P)
    dst = torch.arange(blocks, blocks + nd, dtype=torch.int32, device="cuda")[None]
    kd, vd = k.alloc_kv_cache(blocks + nd, 2, 64, fill=0)
    dw, kept = torch.empty(1, 2, nd * P, device="cuda"), torch.zeros(1, 2, nd * P, dtype=torch.int32, device="cuda")
    dl = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = torch.zeros(1, 2, blocks * P, device="cuda")
    wide[..., :L] = w
    k.kvq_evict_tokens(wide, kd, vd, table, i32([L]), i32([keep]), dst, dw, dl, kept, head_dim=64, sink=5, recent=1000)
    score = wide.clone()
    score[..., :5] = float("inf")
    score[..., L - 1000:L] = float("inf")
    score[..., L:] = float("-inf")
    best = torch.sort(score, descending=True, stable=True).indices[..., :keep].sort().values
    assert torch.equal(kept[..., :keep].long(), best)
    assert torch.equal(dw[..., :keep], wide.gather(-1, best))
    assert int(dl) == keep


@pytest.mark.parametrize("L,heads,keep", [(20_000, 50, 3000), (20_001, 20, 9999), (70_000, 9, 501),  # clusters of 2, 4, 8
                                          (420_000, 2, 30_000), (60_000, 80, 2000)])  # keys read from memory each pass
def test_selection_over_clusters_and_lengths(L, heads, keep):
    k = _k()
    gen = torch.Generator(device="cuda").manual_seed(L)
    blocks, nd = -(-L // P), -(-keep // P)
    table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    dst = torch.arange(blocks, blocks + nd, dtype=torch.int32, device="cuda")[None]
    kd, vd = k.alloc_kv_cache(blocks + nd, heads, 64, fill=0)
    w = torch.zeros(1, heads, blocks * P, device="cuda")
    # ties around every threshold; in the odd heads a value for most tokens
    w[..., :L] = torch.floor(torch.rand(1, heads, L, generator=gen, device="cuda") * 300)
    w[:, 1::2] = torch.maximum(w[:, 1::2], torch.tensor(250.0, device="cuda"))
    dw, kept = torch.empty(1, heads, nd * P, device="cuda"), torch.zeros(1, heads, nd * P, dtype=torch.int32, device="cuda")
    dl = torch.zeros(1, dtype=torch.int32, device="cuda")
    k.kvq_evict_tokens(w, kd, vd, table, i32([L]), i32([keep]), dst, dw, dl, kept, head_dim=64, sink=4, recent=100)
    score = w.clone()
    score[..., :4] = float("inf")
    score[..., L - 100:L] = float("inf")
    score[..., L:] = float("-inf")
    best = torch.sort(score, descending=True, stable=True).indices[..., :keep].sort().values
    assert torch.equal(kept[..., :keep].long(), best)
    assert torch.equal(dw[..., :keep], w.gather(-1, best))
    assert int(dl) == keep


def test_bad_pages_and_lengths_are_reported():
    pool = Pool(60, 1, 64, FP8, 19)
    table = pool.table([200, 60])
    dst = pool.table([64, 32], fill=False)
    weights = _weights(pool.rng, 2, 1, table.shape[1] * P, "plain")
    t2, d2 = table.copy(), dst.copy()
    t2[0, 2], d2[1, 1] = -1, pool.blocks
    kd, vd, dw, dl, kept, st = _run(pool, weights, t2, [200, 60], [64, 32], d2, 0, 0)
    assert st == 0x2 and list(dl) == [64, 32]
    k, v, _, rw, _, rk = serving.evict(weights, pool.k, pool.v, table, [200, 60], [64, 32], dst,
                                       np.zeros((2, 1, dst.shape[1] * P), np.float32),
                                       np.full((2, 1, dst.shape[1] * P), -9, np.int32), 0, 0)
    assert np.array_equal(kept, rk) and np.array_equal(dw, rw)
    # the tokens of the bad source page and the bad destination page stay unwritten
    for i, j in enumerate(rk[0, 0, :64]):
        if j // P == 2:
            k[dst[0, i // P], 0, i % P] = pool.k[dst[0, i // P], 0, i % P]
            v[dst[0, i // P], 0, :, i % P] = pool.v[dst[0, i // P], 0, :, i % P]
    k[dst[1, 1]], v[dst[1, 1]] = pool.k[dst[1, 1]], pool.v[dst[1, 1]]
    ek, ev = layout.to_device_format(k, v)
    assert np.array_equal(kd, ek) and np.array_equal(vd, ev)
    for lens, keep, n in (([-3, 60], [64, 32], [0, 32]), ([10 ** 6, 60], [64, 32], [64, 32]), ([200, 60], [-1, 32], [0, 32]),
                          ([200, 60], [100, 32], [64, 32])):
        _, _, _, dl, _, st = _run(pool, weights, table, lens, keep, dst, 0, 0)
        assert st & 0x4 and list(dl) == n


def test_in_a_graph():
    k = _k()
    pool = Pool(80, 2, 128, FP8, 23)
    table, dst = pool.table([500]), pool.table([100], fill=False)
    kd, vd = pool.device()
    w = torch.from_numpy(_weights(pool.rng, 1, 2, table.shape[1] * P, "plain")).cuda()
    dw, kept = torch.zeros(1, 2, dst.shape[1] * P, device="cuda"), torch.zeros(1, 2, dst.shape[1] * P, dtype=torch.int32,
                                                                                device="cuda")
    dl = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (w, kd, vd, i32(table), i32([500]), i32([100]), i32(dst), dw, dl, kept)
    k.kvq_evict_tokens(*args, head_dim=128, sink=4, recent=16)
    torch.cuda.synchronize()
    first = [t.clone() for t in (kd, vd, dw, dl, kept)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k.kvq_evict_tokens(*args, head_dim=128, sink=4, recent=16)
    for t in (dw, dl, kept):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (kd, vd, dw, dl, kept)))
