"""kvq_gather_cache: bits against the oracle's codecs for every format, and
the step from projection to attention as it is used: rotation into a 4-bit
cache, decode over it, and the context read back."""
import numpy as np
import pytest
import torch

from oracle import e2m1, rotary
from oracle.kv_cache import BF16, FP8, FP8_E5M2
from tests.fp4_testlib import Pool4, assert_within, i32
from tests.serving_testlib import P, Pool

pytestmark = pytest.mark.gpu


def _k():
    import fp8_kv_cache_reshape_gb300 as k
    return k


def _bf16(x):
    """float32 -> bf16 as torch rounds it."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16()


def _orders(slots, seed=0):
    """The tokens as they lie, and in any order with repeats and gaps."""
    rng = np.random.default_rng(seed)
    some = rng.choice(slots, len(slots) + 7)
    some[rng.random(len(some)) < 0.2] = -3
    return [slots, slots[5:], some]


def _check(k, slots, caches, scales, want, **kw):
    """want(slots) -> k, v bf16 rows of valid slots."""
    for s in _orders(slots):
        T, (H, D) = len(s), want(slots[:1])[0].shape[1:]
        ko, vo = (torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        k.kvq_gather_cache(torch.from_numpy(s).cuda(), *caches, ko, vo, *scales, dev_status=st, **kw)
        assert int(st) == 0
        live = s >= 0
        for got, ref in zip((ko.cpu(), vo.cpu()), want(s[live])):
            assert torch.equal(got[torch.from_numpy(live)].view(torch.int16), ref.view(torch.int16))
            assert torch.all(got[torch.from_numpy(~live)] == 9.0)


@pytest.mark.parametrize("dtype,per_token", [(FP8, False), (FP8_E5M2, False), (FP8, True), (FP8_E5M2, True), (BF16, False)])
@pytest.mark.parametrize("dim,heads,paired,n", [(64, 3, False, 1), (64, 3, False, 16), (128, 2, True, 100), (128, 2, True, 555), (64, 5, True, 10000),
                                                (128, 6, False, 10000)])
def test_formats(dtype, per_token, dim, heads, paired, n):
    from oracle import e4m3, e5m2
    pool = Pool(-(-n // P) + 4, heads, dim, dtype, 3, per_token)
    table = pool.table([n])
    j = np.arange(n)
    slots = table[0, j // P].astype(np.int64) * P + j % P

    def want(s):
        at, off = s // P, s % P
        kc, vc = pool.k[at, :, off], pool.v.transpose(0, 1, 3, 2)[at, :, off]
        if dtype == BF16:
            return [torch.from_numpy(x.astype(np.int16)).view(torch.bfloat16) for x in (kc, vc)]
        codec = e4m3 if dtype == FP8 else e5m2
        out = []
        for i, (c, s1) in enumerate(((kc, pool.k_scale), (vc, pool.v_scale))):
            sc = pool.scales[at, :, i, off][..., None] if per_token else s1[:, None]
            out.append(_bf16(codec.decode(c).astype(np.float32) * sc))
        return out

    _check(_k(), slots, pool.device(paired), pool.device_scales(), want, cache_dtype=dtype, per_token=per_token)


@pytest.mark.parametrize("dim,heads,paired,n", [(64, 3, True, 1), (64, 3, True, 16), (128, 2, False, 100), (128, 2, False, 555), (64, 5, False, 10000)])
def test_fp4(dim, heads, paired, n):
    pool = Pool4(-(-n // P) + 4, heads, dim, 3)
    table = pool.table([n])
    j = np.arange(n)
    slots = table[0, j // P].astype(np.int64) * P + j % P

    def want(s):
        at, off = s // P, s % P
        return [_bf16(e2m1.dequantize(c[at, :, off], sb[at, :, off]).astype(np.float32) * sc[:, None])
                for c, sb, sc in ((pool.k, pool.ks, pool.k_scale), (pool.v, pool.vs, pool.v_scale))]

    _check(_k(), slots, pool.device(paired), pool.scales(), want, cache_dtype="fp4")


@pytest.mark.parametrize("name", ["fp8_e4m3", "fp8_e5m2"])
def test_head_dim_256(name):
    """Back from kvq_reshape_and_cache with powers of two as scales: half a step of the codes, and exact where they are."""
    k = _k()
    gen = torch.Generator(device="cuda").manual_seed(1)
    kk, v = (torch.randn(75, 2, 256, generator=gen, device="cuda").bfloat16() for _ in range(2))
    slots = torch.randperm(8 * P, generator=torch.Generator().manual_seed(2))[:75].cuda()
    one = torch.full((2,), 2.0 ** -5, device="cuda")
    caches = k.alloc_kv_cache(8, 2, 256, name, fill=0x7F)
    k.kvq_reshape_and_cache(kk, v, slots, *caches, one, one, cache_dtype=name)
    ko, vo = torch.zeros_like(kk), torch.zeros_like(v)
    k.kvq_gather_cache(slots, *caches, ko, vo, one, one, cache_dtype=name)
    t = torch.float8_e4m3fn if name == "fp8_e4m3" else torch.float8_e5m2
    for got, x in ((ko, kk), (vo, v)):
        assert torch.equal(got, ((x.float() * 32).to(t).float() / 32).bfloat16())


def test_bad_slots_leave_their_rows():
    k = _k()
    pool = Pool(5, 2, 64, FP8, 3)
    pool.table([64])
    ko, vo = (torch.full((4, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    k.kvq_gather_cache(torch.tensor([80, -1, 2**50, -(2**60)]).cuda(), *pool.device(), ko, vo, *pool.device_scales(), dev_status=st)
    assert int(st) == k.KVQ_DEV_BAD_SLOT and torch.all(ko == 9) and torch.all(vo == 9)


@pytest.mark.parametrize("dim,group,axes,captured", [(128, 4, 1, False), (64, 8, 3, True)])
def test_a_layer_step_over_a_4_bit_cache(dim, group, axes, captured):
    """Prompts of three sequences, then decode steps: rotate and append, attend, and at the end the context read back."""
    k = _k()
    H, lens, steps = 2, [37, 160, 5], 4
    Hq, B = H * group, len(lens)
    gen = torch.Generator(device="cuda").manual_seed(7)
    width = -(-(max(lens) + steps) // P)
    order = torch.randperm(B * width + 2, generator=torch.Generator().manual_seed(1))
    table = order[:B * width].view(B, width).int()
    kd, vd = k.alloc_kv_cache(B * width + 2, H, dim, "fp4", fill=0x7F, paired=True)
    ks, vs = torch.tensor([0.0021, 0.0024], device="cuda"), torch.tensor([0.0019, 0.002], device="cuda")
    inv = (10000.0 ** (-torch.arange(dim // 2) / (dim // 2))).cuda()
    axis = (torch.arange(dim // 2) % axes).int().cuda() if axes > 1 else None
    w = [(1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).bfloat16() for _ in range(2)]

    def qkv(T):
        x = torch.randn(T, (Hq + 2 * H) * dim, generator=gen, device="cuda").bfloat16()
        return [y.unflatten(1, (-1, dim)) for y in x.split([Hq * dim, H * dim, H * dim], 1)]

    def where(b, t):
        return table[b, t // P].long() * P + t % P

    seen = [[] for _ in lens]  # (k, v, position) of each sequence's tokens
    turn = dict(pair_axis=axis, q_weight=w[0], k_weight=w[1], cache_dtype="fp4")
    q, kk, v = qkv(sum(lens))
    at = torch.cat([torch.arange(n) for n in lens])
    slots = torch.cat([where(b, torch.arange(n)) for b, n in enumerate(lens)])
    pos = at if axes == 1 else torch.stack([at, at // 7, at % 7])
    k.kvq_rope_and_cache(q, kk, v, pos.cuda(), inv, slots.cuda(), kd, vd, ks, vs, q_out=torch.empty(sum(lens), Hq, dim, dtype=torch.bfloat16, device="cuda"), **turn)
    start = 0
    for b, n in enumerate(lens):
        seen[b] += [(kk[start + i], v[start + i], pos[..., start + i]) for i in range(n)]
        start += n

    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    state = dict(x=torch.zeros(B, (Hq + 2 * H) * dim, dtype=torch.bfloat16, device="cuda"),
                 pos=torch.zeros((B,) if axes == 1 else (axes, B), dtype=torch.int64, device="cuda"),
                 slots=torch.zeros(B, dtype=torch.int64, device="cuda"), lens=i32(lens), q=torch.zeros(B, Hq, dim, dtype=torch.bfloat16, device="cuda"),
                 out=torch.zeros(B, Hq, dim, dtype=torch.bfloat16, device="cuda"), ws=torch.empty(k.kvq_decode_fp4_workspace_size(B, Hq, H, dim, width), dtype=torch.uint8, device="cuda"))
    dev_table = table.cuda()

    def step():
        q, kk, v = (y.unflatten(1, (-1, dim)) for y in state["x"].split([Hq * dim, H * dim, H * dim], 1))
        k.kvq_rope_and_cache(q, kk, v, state["pos"], inv, state["slots"], kd, vd, ks, vs, q_out=state["q"], dev_status=st, **turn)
        k.kvq_paged_decode_attention_fp4(state["q"], kd, vd, ks, vs, dev_table, state["lens"], state["out"], workspace=state["ws"], dev_status=st)

    graph = None
    if captured:
        state["slots"].fill_(-1)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    host_w = [x.double().cpu().numpy() for x in w]
    host_axis = None if axis is None else axis.cpu().numpy()
    for s in range(steps):
        q, kk, v = qkv(B)
        now = torch.tensor([n + s for n in lens])
        p = now if axes == 1 else torch.stack([now, now // 7, now % 7])
        state["x"].copy_(torch.cat([y.flatten(1) for y in (q, kk, v)], 1))
        state["pos"].copy_(p)
        state["slots"].copy_(torch.stack([where(b, now[b]) for b in range(B)]))
        state["lens"].copy_(now + 1)
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        assert int(st) == 0
        for b in range(B):
            seen[b].append((kk[b], v[b], p[..., b]))
        # the queries by the formula, attention by the oracle on the cache's own codes
        want = rotary.turn(q.double().cpu().numpy(), p.numpy(), inv.cpu().numpy(), host_axis, host_w[0], 1e-6)
        slop = rotary.slop(q.double().cpu().numpy(), host_w[0], 1e-6)
        assert np.all(np.abs(state["q"].double().cpu().numpy() - want) <= 2.0 ** -8 * (np.abs(want) + slop) + slop)
        pool = Pool4(B * width + 2, H, dim, 0)
        kpage = 16 * (dim // 2 + dim // 16)
        pool.k, pool.ks, pool.v, pool.vs = e2m1.from_pages(kd[..., :kpage].cpu().numpy(), kd[..., kpage:].cpu().numpy(), dim)
        pool.k_scale, pool.v_scale = ks.cpu().numpy(), vs.cpu().numpy()
        ref, tol = pool.attend(state["q"].double().cpu().numpy(), table.numpy(), (now + 1).tolist(), dim ** -0.5)
        assert_within(state["out"], ref, tol)
    # the context back, against the keys turned by the formula: half a step of E2M1 at its widest, 1 of 6, of the block's largest
    # value, and half a step of its E4M3 scale, 2^-4, on top; bf16's and float32's own far below the last term
    for b, n in enumerate(lens):
        t = torch.arange(n + steps)
        ko, vo = (torch.zeros(n + steps, H, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k.kvq_gather_cache(where(b, t).cuda(), kd, vd, ko, vo, ks, vs, cache_dtype="fp4")
        kh, vh = (torch.stack([x[i] for x in seen[b]]).double().cpu().numpy() for i in range(2))
        ph = torch.stack([x[2] for x in seen[b]], -1).numpy()
        kh = rotary.turn(kh, ph, inv.cpu().numpy(), host_axis, host_w[1], 1e-6)
        for got, ref in ((ko, kh), (vo, vh)):
            top = np.abs(ref.reshape(n + steps, H, -1, 16)).max(-1).repeat(16, -1)
            assert np.all(np.abs(got.double().cpu().numpy() - ref) <= (1 / 6 + 2.0 ** -4) * (1 + 2.0 ** -4) * top + 2.0 ** -7 * top)


@pytest.mark.parametrize("fmt", ["fp8_e4m3", "fp8_e5m2", "bf16", "fp4"])
def test_nan_comes_back_as_nan(fmt):
    """Of 4 bits the whole block of 16 dims, of the others the value."""
    k = _k()
    x = torch.ones(20, 2, 128, dtype=torch.bfloat16)
    x[3, 1, 37] = x[19, 0, 127] = float("nan")
    x = x.cuda()
    slots = torch.arange(7, 27).cuda()
    s = None if fmt == "bf16" else torch.ones(2, device="cuda")
    kc, vc = k.alloc_kv_cache(2, 2, 128, fmt, fill=0)
    k.kvq_reshape_and_cache(x, x, slots, kc, vc, s, s, cache_dtype=fmt)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    k.kvq_gather_cache(slots, kc, vc, ko, vo, s, s, cache_dtype=fmt)
    want, one = x.isnan(), 1.0
    if fmt == "fp4":
        one = 33 / 32  # the block scale is 1/6 in E4M3: 11/64; 64/11 is 6 in E2M1
        want = want.unflatten(-1, (-1, 16)).any(-1, keepdim=True).expand(-1, -1, -1, 16).flatten(-2)
    for y in (ko, vo):
        assert torch.equal(y.isnan(), want) and bool((y[~want] == one).all())
