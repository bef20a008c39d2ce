"""kvq_qk_norm_rope and kvq_rope_and_cache against the float64 oracle: rows to
half a step of bf16, codes between those of the exact value's error bounds."""
import numpy as np
import pytest
import torch

from oracle import e2m1, e4m3, e5m2, layout, rotary

pytestmark = pytest.mark.gpu
P = 16


def _k():
    import fp8_kv_cache_reshape_gb300 as k
    return k


def _inputs(T, Hq, H, D, seed=0):
    """q, k, v as slices of one projection output."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, (Hq + 2 * H) * D, generator=gen).bfloat16()
    cut = [x.cuda()[:, a:b].unflatten(1, (-1, D)) for a, b in ((0, Hq * D), (Hq * D, (Hq + H) * D), ((Hq + H) * D, (Hq + 2 * H) * D))]
    host = [c.double().cpu().numpy() for c in cut]
    return cut, host


def _turn(T, rot, axes, norm, D, far, seed=0):
    """Keyword arguments of the calls and of the oracle."""
    rng = np.random.default_rng(seed)
    inv = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    pos = rng.integers(-far // 8, far, (axes, T))
    axis = rng.integers(0, axes, rot // 2).astype(np.int32) if axes > 1 else None
    w = [torch.from_numpy(1 + 0.4 * rng.standard_normal(D)).bfloat16() if norm else None for _ in range(2)]
    dev = dict(positions=torch.from_numpy(pos if axes > 1 else pos[0]).cuda(), inv_freq=torch.from_numpy(inv).cuda())
    more = dict(pair_axis=None if axis is None else torch.from_numpy(axis).cuda(),
                **{n: None if x is None else x.cuda() for n, x in zip(("q_weight", "k_weight"), w)})
    host = dict(positions=pos, inv_freq=inv, pair_axis=axis)
    weights = [None if x is None else x.double().numpy() for x in w]
    return dev, more, host, weights


def _expected(x, host, weight, interleaved, scale):
    eps = 0.0 if weight is None else 1e-6
    return (rotary.turn(x, **host, weight=weight, eps=eps, interleaved=interleaved, scale=scale),
            rotary.slop(x, weight, eps, scale) + 1e-30)


def _rows_ok(got, ref, slop):
    got = got.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + slop) + slop)


CASES = [(1, 4, 1, 64, 64, 1, False, False), (1, 32, 8, 128, 128, 1, True, False), (17, 3, 3, 64, 32, 2, True, True), (5, 8, 2, 128, 16, 3, False, True),
         (100, 2, 1, 128, 112, 4, True, False), (33, 5, 5, 256, 256, 1, True, False), (16, 1, 1, 256, 48, 3, False, False), (300, 16, 4, 64, 48, 1, False, True),
         (47, 8, 8, 256, 256, 2, True, True)]


@pytest.mark.parametrize("T,Hq,H,D,rot,axes,norm,interleaved", CASES)
def test_norm_rope(T, Hq, H, D, rot, axes, norm, interleaved):
    (q, kk, _), (qh, kh, _) = _inputs(T, Hq, H, D)
    dev, more, host, w = _turn(T, rot, axes, norm, D, 100000)
    qo, ko = (torch.full(x.shape, 9.0, dtype=torch.bfloat16, device="cuda") for x in (q, kk))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _k().kvq_qk_norm_rope(q, kk, **dev, q_out=qo, k_out=ko, interleaved=interleaved, rope_scale=1.25, dev_status=st, **more)
    assert int(st) == 0
    _rows_ok(qo, *_expected(qh, host, w[0], interleaved, 1.25))
    _rows_ok(ko, *_expected(kh, host, w[1], interleaved, 1.25))
    # in place, in the projection's own memory, beside v
    before = (q.clone(), kk.clone())
    _k().kvq_qk_norm_rope(q, kk, **dev, q_out=q, k_out=kk, interleaved=interleaved, rope_scale=1.25, **more)
    assert torch.equal(q, qo) and torch.equal(kk, ko) and not (T > 4 and torch.equal(before[0], q))


def test_norm_alone_rotation_alone_and_one_tensor():
    (q, kk, v), (qh, kh, _) = _inputs(21, 4, 2, 128)
    dev, more, host, w = _turn(21, 128, 1, True, 128, 5000)
    keep = v.clone()
    out = torch.zeros(21, 4, 128, dtype=torch.bfloat16, device="cuda")
    _k().kvq_qk_norm_rope(q, None, None, None, out, None, q_weight=more["q_weight"])
    _rows_ok(out, *_expected(qh, dict(positions=None, inv_freq=None), w[0], False, 1.0))
    out = torch.zeros(21, 2, 128, dtype=torch.bfloat16, device="cuda")
    _k().kvq_qk_norm_rope(None, kk, **dev, q_out=None, k_out=out)
    _rows_ok(out, *_expected(kh, host, None, False, 1.0))
    # a norm of the keys alone, both tensors turned
    qo, ko = torch.zeros_like(q), torch.zeros_like(kk)
    _k().kvq_qk_norm_rope(q, kk, **dev, q_out=qo, k_out=ko, k_weight=more["k_weight"])
    _rows_ok(qo, *_expected(qh, host, None, False, 1.0))
    _rows_ok(ko, *_expected(kh, host, w[1], False, 1.0))
    # neither: the rows themselves
    _k().kvq_qk_norm_rope(q, kk, None, None, qo, ko)
    assert torch.equal(qo, q) and torch.equal(ko, kk) and torch.equal(v, keep)


@pytest.mark.parametrize("pos", [[2**31 - 1, -(2**31), 10**6 + 1, 0]])
def test_far_positions(pos):
    (q, _, _), (qh, _, _) = _inputs(4, 2, 1, 64)
    inv = (500000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    out = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    _k().kvq_qk_norm_rope(q, None, torch.tensor(pos).cuda(), torch.from_numpy(inv).cuda(), out, None)
    _rows_ok(out, *_expected(qh, dict(positions=np.array(pos), inv_freq=inv), None, False, 1.0))


@pytest.mark.parametrize("T,Hq,H,D", [(5000, 35, 9, 64), (2600, 33, 10, 128)])
def test_norm_rope_many_heads_to_a_cta(T, Hq, H, D):
    (q, kk, _), (qh, kh, _) = _inputs(T, Hq, H, D)
    dev, more, host, w = _turn(T, D // 2, 2, True, D, 100000)
    qo, ko = (torch.full(x.shape, 9.0, dtype=torch.bfloat16, device="cuda") for x in (q, kk))
    _k().kvq_qk_norm_rope(q, kk, **dev, q_out=qo, k_out=ko, **more)
    _rows_ok(qo, *_expected(qh, host, w[0], False, 1.0))
    _rows_ok(ko, *_expected(kh, host, w[1], False, 1.0))


def test_one_row_of_positions_for_all_axes():
    (q, kk, _), _ = _inputs(40, 2, 1, 64)
    pos, inv = torch.randint(0, 9999, (40,)).cuda(), torch.rand(32).cuda()
    outs = [torch.zeros_like(q) for _ in range(2)]
    _k().kvq_qk_norm_rope(q, None, pos, inv, outs[0], None)
    _k().kvq_qk_norm_rope(q, None, pos.expand(3, 40), inv, outs[1], None, pair_axis=(torch.arange(32) % 3).int().cuda())
    assert torch.equal(*outs)


def test_zero_rows_and_values_beyond_float32_squares():
    q = torch.zeros(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[1, 0, 5] = 1e18
    q[2] = 1e-20
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 9.0)
    _k().kvq_qk_norm_rope(q, None, None, None, out, None, q_weight=w, eps=1e-6)
    assert not out[0].any() and float(out[1, 0, 5]) == 8.0 and float(out[2].abs().max()) <= 1e-16


def test_an_axis_out_of_range_counts_as_the_first():
    k = _k()
    (q, _, _), _ = _inputs(20, 2, 1, 64)
    pos = torch.arange(40).view(2, 20).cuda()
    inv = torch.rand(32, generator=torch.Generator().manual_seed(1)).cuda()
    outs = []
    for bad, want in ((0, 0), (2, k.KVQ_DEV_BAD_AXIS), (-1, k.KVQ_DEV_BAD_AXIS), (2**31 - 1, k.KVQ_DEV_BAD_AXIS)):
        axis = (torch.arange(32) % 2).int()
        axis[7] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs.append(torch.zeros(20, 2, 64, dtype=torch.bfloat16, device="cuda"))
        k.kvq_qk_norm_rope(q, None, pos, inv, outs[-1], None, pair_axis=axis.cuda(), dev_status=st)
        assert int(st) == want
    axis = (torch.arange(32) % 2).int()
    axis[7] = 0
    k.kvq_qk_norm_rope(q, None, pos, inv, outs[0], None, pair_axis=axis.cuda())
    assert all(torch.equal(o, outs[0]) for o in outs)


# ------------------------------------------------------------ into the cache ---
CODECS = {"e4m3": (e4m3, 448.0), "e5m2": (e5m2, 57344.0)}


def _between(got, lo, hi, codec):
    """Each code is that of a value in [lo, hi]: rounding is monotone."""
    got = codec.decode(got)
    assert np.all((codec.decode(codec.encode(lo)) <= got) & (got <= codec.decode(codec.encode(hi))))


def _slots(T, kind, seed=0):
    """Slots of a chunk: in order from a page's start or its middle, several
    sequences' ends, one token of each of many sequences, or any order; some skipped."""
    rng = np.random.default_rng(seed)
    blocks = T + 5
    order = rng.permutation(blocks)
    at = np.arange(T)
    if kind == "aligned":
        s = order[at // P] * P + at % P
    elif kind == "middle":
        s = order[(at + 11) // P] * P + (at + 11) % P
    elif kind == "sequences":  # pieces of 1 to 40 tokens, each from a random place of a page of its own
        s, page, left = [], 0, 0
        for _ in range(T):
            if left == 0:
                left, page, off = int(rng.integers(1, 41)), page + 1, int(rng.integers(0, P))
            s.append(order[page % blocks] * P + off)
            off += 1
            left -= 1
            if off == P:
                page, off = page + 1, 0
        s = np.array(s)
        s[len(set(s.tolist())):] = -1 if len(set(s.tolist())) < T else s[len(set(s.tolist())):]
    elif kind == "steps":
        s = order[at] * P + rng.integers(0, P, T)
    else:
        s = rng.permutation(blocks * P)[:T]
        s[rng.random(T) < 0.2] = -1
    return s.astype(np.int64), blocks


def _logical(kd, vd, fmt, per_token, D):
    """The device caches as logical codes (k, v [nb, H, 16, D]; v transposed back) and scales."""
    kd, vd = kd.cpu().numpy(), vd.cpu().numpy()
    if fmt == "fp4":
        return e2m1.from_pages(kd, vd, D)
    if fmt == "bf16":
        kd, vd = kd.view(np.uint16), vd.view(np.uint16)
    scales = None
    if per_token:
        scales = vd[..., P * D:].copy().view(np.float32).reshape(*vd.shape[:2], 2, P)
        vd = np.ascontiguousarray(vd[..., :P * D])
    k, v = _from_device(kd, vd, D)
    return k, v, scales


def _from_device(kd, vd, D):
    """layout.to_device_format() inverted by pushing positions through it."""
    nb, H = kd.shape[:2]
    wide = kd.dtype == np.uint16
    n = P * D
    index = np.arange(n)
    parts = []
    for shift in range(0, 16, 8):
        x = ((index >> shift) & 0xFF).astype(np.uint8).astype(np.uint16 if wide else np.uint8)
        kk = x.reshape(1, 1, P, D)
        vv = x.reshape(1, 1, D, P)
        a, b = layout.to_device_format(kk, vv)
        parts.append([y.view(np.uint16 if wide else np.uint8).reshape(-1).astype(np.int64) << shift for y in (a, b)])
    kat, vat = (parts[0][i] | parts[1][i] for i in range(2))
    k, v = np.empty((nb, H, n), kd.dtype), np.empty((nb, H, n), kd.dtype)
    k[..., kat], v[..., vat] = kd.reshape(nb, H, n), vd.reshape(nb, H, n)
    return k.reshape(nb, H, P, D), v.reshape(nb, H, D, P).transpose(0, 1, 3, 2)


FORMATS = [("e4m3", False), ("e5m2", False), ("e4m3", True), ("e5m2", True), ("bf16", False), ("fp4", False)]
APPEND = [(1, 4, 1, 64, 64, 1, False, False, "steps"), (40, 8, 2, 128, 128, 1, False, False, "steps"), (64, 2, 2, 128, 64, 3, True, True, "aligned"),
          (150, 4, 3, 64, 64, 1, True, False, "middle"), (333, 0, 2, 128, 128, 2, False, False, "sequences"), (90, 6, 6, 64, 16, 1, False, True, "any"),
          (700, 2, 1, 128, 128, 1, False, False, "middle")]


@pytest.mark.parametrize("fmt,per_token", FORMATS)
@pytest.mark.parametrize("T,Hq,H,D,rot,axes,norm,interleaved,kind", APPEND)
@pytest.mark.parametrize("paired", [False, True])
def test_rope_and_cache(T, Hq, H, D, rot, axes, norm, interleaved, kind, fmt, per_token, paired):
    _check_append(T, Hq, H, D, rot, axes, norm, interleaved, kind, fmt, per_token, paired)


@pytest.mark.parametrize("fmt,per_token", FORMATS)
@pytest.mark.parametrize("T,H,D,kind", [(5000, 5, 64, "sequences"), (2600, 10, 128, "middle"), (2600, 3, 128, "any")])
def test_rope_and_cache_many_heads_to_a_cta(T, H, D, kind, fmt, per_token):
    _check_append(T, 2 * H, H, D, D, 1, True, False, kind, fmt, per_token, False)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["middle", "steps"])
def test_rope_and_cache_head_dim_256(fmt, kind):
    _check_append(70, 3, 2, 256, 256, 1, True, False, kind, fmt, False, False)


def _check_append(T, Hq, H, D, rot, axes, norm, interleaved, kind, fmt, per_token, paired):
    k = _k()
    (q, kk, v), (qh, kh, vh) = _inputs(T, Hq or 1, H, D, seed=T)
    dev, more, host, w = _turn(T, rot, axes, norm, D, 30000, seed=T)
    slots, blocks = _slots(T, kind)
    name = {"e4m3": "fp8_e4m3", "e5m2": "fp8_e5m2", "bf16": "bf16", "fp4": "fp4"}[fmt]
    top = {"e4m3": 448.0, "e5m2": 57344.0, "fp4": 6 * 448.0, "bf16": 1.0}[fmt]
    kd, vd = k.alloc_kv_cache(blocks, H, D, name, fill=0x5A, per_token=per_token, paired=paired)
    ks = ((5.3 + 0.37 * np.arange(H)) / top).astype(np.float32)
    vs = ((3.9 + 0.41 * np.arange(H)) / top).astype(np.float32)  # some values saturate
    given = () if per_token or fmt == "bf16" else (torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda())
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    qs = torch.full((1,), 4.1 / 448, device="cuda")
    outs = {}
    if Hq:
        outs = dict(q_out=torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
                    q8=torch.zeros(T, Hq, D, dtype=torch.uint8, device="cuda"), q_scale=qs)
    k.kvq_rope_and_cache(q if Hq else None, kk, v, **dev, slot_mapping=torch.from_numpy(slots).cuda(), k_cache=kd, v_cache=vd,
                         **dict(zip(("k_scale", "v_scale"), given)), interleaved=interleaved, cache_dtype=name,
                         per_token=per_token, dev_status=st, **outs, **more)
    torch.cuda.synchronize()
    assert int(st) == 0
    if Hq:
        ref, slop = _expected(qh, host, w[0], interleaved, 1.0)
        _rows_ok(outs["q_out"], ref, slop)
        s = float(qs[0])
        _between(outs["q8"].cpu().numpy(), (ref - slop) / s, (ref + slop) / s, e4m3)
    kpage = kd.shape[-1] if not paired else k._page_bytes(D, k._dtype_code(name))
    pages = (kd, vd) if not paired else (kd[..., :kpage], kd[..., kpage:])
    kx, kslop = _expected(kh, host, w[1], interleaved, 1.0)
    live = slots >= 0
    at, off = slots[live] // P, slots[live] % P
    if fmt == "fp4":
        kc, ksb, vc, vsb = _logical(*pages, fmt, per_token, D)
        for codes, sb, x, slop, s in ((kc, ksb, kx, kslop, ks), (vc, vsb, vh, np.zeros((T, 1, 1)), vs)):
            codes, sb, x, slop = codes[at, :, off], sb[at, :, off], x[live], np.broadcast_to(slop, x.shape)[live]
            amax = np.abs(x.reshape(*x.shape[:2], -1, 16)).max(-1)
            room = slop[..., :1] + 2.0 ** -23 * amax
            _between(sb, (amax - room) / (6 * s[:, None]), (amax + room) / (6 * s[:, None]), e4m3)
            step = np.repeat(e4m3.decode(sb) * s[:, None], 16, -1)
            ok = step > 0
            room = slop + 2.0 ** -23 * np.abs(x)
            with np.errstate(divide="ignore", invalid="ignore"):
                _between(codes[ok], ((x - room) / step)[ok], ((x + room) / step)[ok], e2m1)
            assert not codes[~ok].any()
        want_k, want_v = e2m1.quantize(kh[live].astype(np.float32), ks), e2m1.quantize(vh[live].astype(np.float32), vs)
        assert np.array_equal(vc[at, :, off], want_v[0]) and np.array_equal(vsb[at, :, off], want_v[1])  # v is neither turned nor normed
        untouched = np.ones((blocks, P), bool)
        untouched[at, off] = False
        assert np.all(kc.transpose(0, 2, 1, 3)[untouched] == np.tile([0xA, 0x5], D // 2)) and np.all(ksb.transpose(0, 2, 1, 3)[untouched] == 0x5A)
        assert np.all(vc.transpose(0, 2, 1, 3)[untouched] == np.tile([0xA, 0x5], D // 2)) and np.all(vsb.transpose(0, 2, 1, 3)[untouched] == 0x5A)
        return
    kc, vc, scales = _logical(*(x.contiguous() for x in pages), fmt, per_token, D)
    untouched = np.ones((blocks, P), bool)
    untouched[at, off] = False
    fill = 0x5A5A if fmt == "bf16" else 0x5A
    assert np.all(kc.transpose(0, 2, 1, 3)[untouched] == fill) and np.all(vc.transpose(0, 2, 1, 3)[untouched] == fill)
    got_k, got_v, x, slop = kc[at, :, off], vc[at, :, off], kx[live], kslop[live]
    if fmt == "bf16":
        value = (got_k.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        assert np.all(np.abs(value - x) <= 2.0 ** -8 * (np.abs(x) + slop) + slop)
        assert np.array_equal(got_v, v.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)[live])
        return
    codec, top = CODECS[fmt]
    if per_token:
        assert np.all(scales.view(np.uint32).transpose(0, 3, 1, 2)[untouched] == 0x5A5A5A5A)
        sk, sv = scales[at, :, 0, off][..., None], scales[at, :, 1, off][..., None]
        amax = np.abs(x).max(-1, keepdims=True)
        assert np.all(np.abs(sk.astype(np.float64) - amax / top) <= (slop + 2.0 ** -22 * amax) / top)
        assert np.array_equal(sv[..., 0], (np.abs(vh[live]).max(-1) / top).astype(np.float32))
    else:
        sk, sv = ks[:, None], vs[:, None]
    room = slop + 2.0 ** -23 * np.abs(x)
    _between(got_k, (x - room) / sk.astype(np.float64), (x + room) / sk.astype(np.float64), codec)
    assert np.array_equal(got_v, codec.encode(vh[live].astype(np.float32) / sv.astype(np.float32)))


def test_without_norm_or_rotation_the_bytes_are_those_of_the_plain_write():
    k = _k()
    for fmt, per_token in FORMATS:
        name = {"e4m3": "fp8_e4m3", "e5m2": "fp8_e5m2"}.get(fmt, fmt)
        (_, kk, v), _ = _inputs(77, 1, 3, 128, seed=4)
        kk[5], v[6, 1], kk[30, 2], v[30] = 0, 0, 0, 0  # tokens of zeros
        slots, blocks = _slots(77, "middle")
        sd = torch.from_numpy(slots).cuda()
        scales = () if per_token or fmt == "bf16" else (torch.full((3,), 0.011, device="cuda"), torch.full((3,), 0.017, device="cuda"))
        a, b = (k.alloc_kv_cache(blocks, 3, 128, name, fill=0x11, per_token=per_token) for _ in range(2))
        k.kvq_rope_and_cache(None, kk, v, None, None, sd, *a, *scales, cache_dtype=name, per_token=per_token)
        if per_token:
            k.kvq_reshape_and_cache_per_token(kk.contiguous(), v.contiguous(), sd, *b, cache_dtype=name)
        else:
            k.kvq_reshape_and_cache(kk.contiguous(), v.contiguous(), sd, *b, *scales, cache_dtype=name)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), fmt


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -7, 3.0, 0.011, 1e-38, 2.0 ** -126, 1e-44, 2.0 ** 120, 3e38])
def test_quotients_are_those_of_a_division(scale):
    """Scales that give many ties, that are powers of two, and beyond those that the enclosure covers: the bytes of the plain write."""
    k = _k()
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(64, 2, 64, generator=gen).bfloat16()
    x[:20] = (x[:20].float() * min(scale, 1e36)).bfloat16()
    x[20:24] = torch.arange(4 * 2 * 64).view(4, 2, 64).bfloat16()
    x[24] = 0
    x = x.cuda()
    slots = torch.arange(5, 69).cuda()
    s = torch.full((2,), scale, device="cuda")
    for name in ("fp8_e4m3", "fp8_e5m2"):
        a, b = (k.alloc_kv_cache(6, 2, 64, name, fill=0) for _ in range(2))
        k.kvq_rope_and_cache(None, x, x, None, None, slots, *a, s, s, cache_dtype=name)
        k.kvq_reshape_and_cache(x, x, slots, *b, s, s, cache_dtype=name)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q8, want = (torch.zeros(64, 2, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    k.kvq_rope_and_cache(x, x, x, None, None, slots, *a, s, s, q8=q8, q_scale=s[:1], cache_dtype=name)
    k.kvq_quantize_query(x, want, s[:1])
    assert torch.equal(q8, want)
    kd, vd = k.alloc_kv_cache(6, 2, 64, "fp4", fill=0)
    k.kvq_reshape_and_cache(x, x, slots, kd, vd, s, s, cache_dtype="fp4")
    codes, sb, vc, vsb = e2m1.from_pages(kd.cpu().numpy(), vd.cpu().numpy(), 64)
    at, off = np.arange(5, 69) // P, np.arange(5, 69) % P
    want = e2m1.quantize(x.float().cpu().numpy(), np.float32(scale))
    for got, ref in ((codes, want[0]), (sb, want[1]), (vc, want[0]), (vsb, want[1])):
        assert np.array_equal(got[at, :, off], ref)


@pytest.mark.parametrize("scale", [1.0, 0.011, 2.0 ** -126, 1e-44, 3e38])
def test_quotients_of_infinities_nan_and_zeros(scale):
    """The bytes of the plain write, whose values are divided; 4 bits: the oracle's."""
    k = _k()
    x = torch.zeros(16, 1, 64, dtype=torch.bfloat16)
    odd = torch.tensor([float("inf"), float("-inf"), 0.0, -0.0, 1.0, -2.5, 3e38, 1e-38])
    for t in range(16):
        x[t, 0] = odd.repeat(8).roll(t).bfloat16()
    x[12, 0, :8] = float("inf")
    x[13, 0, :8] = -0.0
    slots = torch.arange(16).cuda()
    s = torch.full((1,), scale, device="cuda")
    x[14, 0, ::3] = float("nan")
    x[15, 0, :8] = float("nan")
    kd, vd = k.alloc_kv_cache(1, 1, 64, "fp4", fill=0)
    k.kvq_reshape_and_cache(x.cuda(), x.cuda(), slots, kd, vd, s, s, cache_dtype="fp4")
    with np.errstate(all="ignore"):
        want = e2m1.quantize(x.float().numpy(), np.float32(scale))
    codes, sb, vc, vsb = e2m1.from_pages(kd.cpu().numpy(), vd.cpu().numpy(), 64)
    for got, ref in ((codes, want[0]), (sb, want[1]), (vc, want[0]), (vsb, want[1])):
        assert np.array_equal(got[0].transpose(1, 0, 2), ref)
    x = x.cuda()
    for name in ("fp8_e4m3", "fp8_e5m2"):
        a, b = (k.alloc_kv_cache(1, 1, 64, name, fill=0) for _ in range(2))
        k.kvq_rope_and_cache(None, x, x, None, None, slots, *a, s, s, cache_dtype=name)
        k.kvq_reshape_and_cache(x, x, slots, *b, s, s, cache_dtype=name)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_fp4_write_against_the_oracle():
    """kvq_reshape_and_cache: every byte, zero blocks and saturation among them."""
    k = _k()
    for D, T, kind in ((64, 41, "any"), (128, 200, "middle"), (128, 3, "steps")):
        H = 3
        gen = torch.Generator().manual_seed(D + T)
        kk, v = (torch.randn(T, H, D, generator=gen).bfloat16() for _ in range(2))
        kk[T // 2, 1, :16] = 0
        kk[T // 2, 2, 16:32] = 1e-6
        v[0, 0, :5] = torch.tensor([1e4, -1e4, 0.0, -0.0, 3e38])
        slots, blocks = _slots(T, kind)
        ks, vs = np.float32([0.002, 1.0, 0.0007]), np.float32([0.25, 0.0013, 0.004])
        kd, vd = k.alloc_kv_cache(blocks, H, D, "fp4", fill=0x33)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        k.kvq_reshape_and_cache(kk.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), kd, vd, torch.from_numpy(ks).cuda(),
                                torch.from_numpy(vs).cuda(), cache_dtype="fp4", dev_status=st)
        assert int(st) == 0
        logical = [np.full((blocks, H, P, D), 3, np.uint8), np.full((blocks, H, P, D // 16), 0x33, np.uint8),
                   np.full((blocks, H, P, D), 3, np.uint8), np.full((blocks, H, P, D // 16), 0x33, np.uint8)]
        live = slots >= 0
        at, off = slots[live] // P, slots[live] % P
        for i, (x, s) in enumerate(((kk, ks), (v, vs))):
            logical[2 * i][at, :, off], logical[2 * i + 1][at, :, off] = e2m1.quantize(x.float().numpy()[live], s)
        want = e2m1.pages(*logical)
        assert np.array_equal(kd.cpu().numpy(), want[0]) and np.array_equal(vd.cpu().numpy(), want[1])


@pytest.mark.parametrize("fmt,per_token", FORMATS)
def test_bad_slots(fmt, per_token):
    """One past the end is reported and written nowhere; negative ones are skipped."""
    k = _k()
    name = {"e4m3": "fp8_e4m3", "e5m2": "fp8_e5m2"}.get(fmt, fmt)
    (_, kk, v), _ = _inputs(20, 1, 2, 64)
    kd, vd = k.alloc_kv_cache(4, 2, 64, name, fill=1, per_token=per_token)
    slots = torch.full((20,), -1, device="cuda")
    slots[3], slots[17], slots[5] = 64, 2**62, -(2**40)
    one = torch.ones(2, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    scales = {} if per_token or fmt == "bf16" else dict(k_scale=one, v_scale=one)
    k.kvq_rope_and_cache(None, kk, v, None, None, slots, kd, vd, **scales, cache_dtype=name, per_token=per_token, dev_status=st)
    assert int(st) == k.KVQ_DEV_BAD_SLOT and torch.all(kd == 1) and torch.all(vd == 1)


@pytest.mark.parametrize("T", [3, 700])
def test_queries_in_place_beside_their_keys(T):
    """In the projection's own memory, whose k and v go to the cache: the bits of a call with an output of its own."""
    k = _k()
    dev, more, _, _ = _turn(T, 128, 1, True, 128, 9999)
    slots, blocks = _slots(T, "middle")
    sd, s = torch.from_numpy(slots).cuda(), torch.full((2,), 0.01, device="cuda")
    found = []
    for own in (True, False):
        (q, kk, v), _ = _inputs(T, 6, 2, 128, seed=2)
        before = (kk.clone(), v.clone())
        cache = k.alloc_kv_cache(blocks, 2, 128, fill=0)
        out = torch.empty(T, 6, 128, dtype=torch.bfloat16, device="cuda") if own else q
        k.kvq_rope_and_cache(q, kk, v, **dev, slot_mapping=sd, k_cache=cache[0], v_cache=cache[1], k_scale=s, v_scale=s, q_out=out, **more)
        assert torch.equal(kk, before[0]) and torch.equal(v, before[1])
        found.append((out.contiguous(), *cache))
    assert all(torch.equal(a, b) for a, b in zip(*found))


def test_no_tokens():
    k = _k()
    kd, vd = k.alloc_kv_cache(4, 2, 64, fill=1)
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos, inv, slots = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.ones(32, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    k.kvq_qk_norm_rope(none, none, pos, inv, none, none)
    k.kvq_rope_and_cache(none, none, none, pos, inv, slots, kd, vd, torch.ones(2, device="cuda"), torch.ones(2, device="cuda"), q_out=none)
    k.kvq_gather_cache(slots, kd, vd, none, none, torch.ones(2, device="cuda"), torch.ones(2, device="cuda"))
    torch.cuda.synchronize()
    assert torch.all(kd == 1)


def test_offsets_beyond_32_bits():
    """Rows more than 2^31 elements from the first, slots beyond 4 GiB."""
    k = _k()
    T, wide = 70000, 32768
    x = torch.zeros(T, wide, dtype=torch.bfloat16, device="cuda")
    rows = x[:, :128].unflatten(1, (2, 64))
    rows[-1] = torch.randn(2, 64, device="cuda").bfloat16()
    pos, inv = torch.arange(T, device="cuda"), torch.rand(32, device="cuda")
    out = x[:, 128:256].unflatten(1, (2, 64))
    k.kvq_qk_norm_rope(rows, None, pos, inv, out, None)
    alone = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    k.kvq_qk_norm_rope(rows[-1:], None, pos[-1:], inv, alone, None)
    assert torch.equal(alone[0], out[-1]) and alone.any()
    blocks = 2_200_000
    kd, vd = k.alloc_kv_cache(blocks, 2, 64, fill=0)
    assert kd.nbytes > 2**32
    slots = torch.arange(blocks * 16 - 33, blocks * 16, device="cuda")
    kk, v = (torch.randn(33, 2, 64, device="cuda").bfloat16() for _ in range(2))
    one = torch.full((2,), 0.02, device="cuda")
    k.kvq_rope_and_cache(None, kk, v, None, None, slots, kd, vd, one, one)
    small = k.alloc_kv_cache(3, 2, 64, fill=0)
    k.kvq_reshape_and_cache(kk, v, slots - (blocks - 3) * 16, *small, one, one)
    assert torch.equal(kd[-3:], small[0]) and torch.equal(vd[-3:], small[1])
    ko, vo = torch.zeros_like(kk), torch.zeros_like(v)
    k.kvq_gather_cache(slots, kd, vd, ko, vo, one, one)
    k1, v1 = torch.zeros_like(kk), torch.zeros_like(v)
    k.kvq_gather_cache(slots - (blocks - 3) * 16, *small, k1, v1, one, one)
    assert torch.equal(ko, k1) and torch.equal(vo, v1) and ko.any()
