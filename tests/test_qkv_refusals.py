"""Refusals of the rotation, gather and 4-bit calls, in the C ABI and in the
binding: each comes before any CUDA call (this runs without a GPU)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "fp8_kv_cache_reshape_gb300", "libkvq.so")
p, i, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
OK, INVALID, UNSUPPORTED = 0, 1, 2
FAR = 1 << 40  # a fake address that is never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    return ctypes.CDLL(LIB)


@pytest.fixture(scope="module")
def k(lib):
    import fp8_kv_cache_reshape_gb300 as kvq
    return kvq


class Rotary(ctypes.Structure):
    _fields_ = [("positions", p), ("stride", i64), ("inv_freq", p), ("pair_axis", p), ("axes", i), ("rot", i), ("inter", i),
                ("scale", f32)]


class Norm(ctypes.Structure):
    _fields_ = [("q", p), ("k", p), ("eps", f32)]


ROTARY = dict(positions=FAR, stride=4, inv_freq=FAR, pair_axis=None, axes=1, rot=64, inter=0, scale=1.0)
NORM = dict(q=FAR, k=FAR, eps=1e-6)


def _turn(change):
    norm = None if change.pop("norm", 1) is None else ctypes.pointer(Norm(**{**NORM, **{n: change.pop(n) for n in ("eps", "qw") if n in change}}))
    rotary = ctypes.pointer(Rotary(**{**ROTARY, **{n: change.pop(n) for n in list(change) if n in ROTARY}}))
    return ctypes.cast(norm, p), ctypes.cast(rotary, p)


ROPE = dict(q=FAR, qs=1024, k=FAR, ks=256, norm_p=0, rotary_p=0, qo=FAR, qos=1024, ko=FAR, kos=256, T=4, Hq=8, Hkv=2, D=128,
            st=None, stream=None)
ROPE_SIG = [p, i64, p, i64, p, p, p, i64, p, i64, i, i, i, i, p, p]

TURNS = [({"rot": 8}, UNSUPPORTED), ({"rot": 144}, UNSUPPORTED), ({"rot": 40}, UNSUPPORTED), ({"axes": 0}, UNSUPPORTED),
         ({"axes": 5}, UNSUPPORTED), ({"axes": 2, "stride": 3}, INVALID), ({"positions": None}, INVALID), ({"inv_freq": None}, INVALID),
         ({"positions": FAR + 4}, INVALID), ({"inv_freq": FAR + 2}, INVALID), ({"pair_axis": FAR + 2}, INVALID), ({"scale": NAN}, INVALID),
         ({"scale": INF}, INVALID), ({"eps": -1.0}, INVALID), ({"eps": NAN}, INVALID), ({"eps": INF}, INVALID)]


@pytest.mark.parametrize("change,status", TURNS + [
    ({"T": -1}, INVALID), ({"Hq": 0, "Hkv": 0}, INVALID), ({"Hq": -1}, INVALID), ({"D": 96}, UNSUPPORTED), ({"D": 32}, UNSUPPORTED),
    ({"q": None}, INVALID), ({"ko": None}, INVALID), ({"q": FAR + 8}, INVALID), ({"qs": 1020}, INVALID), ({"qs": 1016}, INVALID),
    ({"kos": 248}, INVALID), ({"T": 0, "q": None}, OK), ({"T": (1 << 31) - 1, "Hq": 512, "qs": 1 << 16, "qos": 1 << 16}, UNSUPPORTED)])
def test_qk_norm_rope(lib, change, status):
    change = dict(change)
    norm, rotary = _turn(change)
    a = {**ROPE, "norm_p": norm, "rotary_p": rotary, **change}
    lib.kvq_qk_norm_rope.argtypes = ROPE_SIG
    assert lib.kvq_qk_norm_rope(*a.values()) == status


CACHE = dict(q=FAR, qs=1024, k=FAR, ks=256, v=FAR, vs=256, norm_p=0, rotary_p=0, slots=FAR, kc=FAR * 2, vc=FAR * 3, ksc=FAR, vsc=FAR,
             qo=FAR, qos=1024, q8=FAR, qsc=FAR, T=4, Hq=8, Hkv=2, D=128, P=16, nb=9, dtype=0, per_token=0, st=None, stream=None)
CACHE_SIG = [p, i64, p, i64, p, i64, p, p, p, p, p, p, p, p, i64, p, p, i, i, i, i, i, i64, i, i, p, p]


@pytest.mark.parametrize("change,status", TURNS + [
    ({"T": -1}, INVALID), ({"Hkv": 0}, INVALID), ({"nb": 0}, INVALID), ({"P": 32}, UNSUPPORTED), ({"dtype": 4}, INVALID),
    ({"dtype": 1, "per_token": 1}, INVALID), ({"dtype": 3, "per_token": 1}, INVALID), ({"D": 96}, UNSUPPORTED),
    ({"D": 256, "dtype": 1}, UNSUPPORTED), ({"D": 256, "dtype": 3}, UNSUPPORTED), ({"D": 256, "per_token": 1}, UNSUPPORTED),
    ({"k": None}, INVALID), ({"v": None}, INVALID), ({"q": None}, INVALID), ({"qo": None, "q8": None}, INVALID), ({"qsc": None}, INVALID),
    ({"q8": FAR + 8}, INVALID), ({"ks": 255}, INVALID), ({"vs": 248}, INVALID), ({"v": FAR + 2}, INVALID), ({"slots": None}, INVALID),
    ({"slots": FAR + 4}, INVALID), ({"kc": None}, INVALID), ({"vc": FAR * 3 + 8}, INVALID), ({"ksc": None}, INVALID),
    ({"vsc": FAR + 2}, INVALID), ({"dtype": 3, "vsc": None}, INVALID), ({"T": 0, "k": None}, OK)])
def test_rope_and_cache(lib, change, status):
    change = dict(change)
    norm, rotary = _turn(change)
    a = {**CACHE, "norm_p": norm, "rotary_p": rotary, **change}
    lib.kvq_rope_and_cache.argtypes = CACHE_SIG
    assert lib.kvq_rope_and_cache(*a.values()) == status


GATHER = dict(slots=FAR, kc=FAR * 2, vc=FAR * 3, ksc=FAR, vsc=FAR, ko=FAR * 4, vo=FAR * 5, T=4, Hkv=2, D=128, P=16, nb=9, dtype=0,
              per_token=0, st=None, stream=None)


@pytest.mark.parametrize("change,status", [
    ({"T": -1}, INVALID), ({"Hkv": 0}, INVALID), ({"nb": 0}, INVALID), ({"P": 8}, UNSUPPORTED), ({"dtype": 9}, INVALID),
    ({"dtype": 1, "per_token": 1}, INVALID), ({"dtype": 3, "per_token": 1}, INVALID), ({"D": 96}, UNSUPPORTED),
    ({"D": 256, "dtype": 3}, UNSUPPORTED), ({"D": 256, "dtype": 1}, UNSUPPORTED), ({"slots": None}, INVALID), ({"ko": None}, INVALID),
    ({"ksc": None}, INVALID), ({"dtype": 3, "vsc": None}, INVALID), ({"vo": FAR + 8}, INVALID), ({"kc": FAR * 2 + 4}, INVALID),
    ({"slots": FAR + 4}, INVALID), ({"vsc": FAR + 1}, INVALID), ({"T": 0, "slots": None}, OK)])
def test_gather(lib, change, status):
    a = {**GATHER, **change}
    lib.kvq_gather_cache.argtypes = [p] * 7 + [i, i, i, i, i64, i, i, p, p]
    assert lib.kvq_gather_cache(*a.values()) == status


DECODE = dict(q=FAR, kc=FAR * 2, vc=FAR * 3, ks=FAR, vs=FAR, bt=FAR, sl=FAR, out=FAR, B=4, Hq=8, Hkv=2, D=128, P=16, max_blocks=4,
              nb=9, scale=0.1, window=-1, ws=FAR * 4, wb=1 << 40, st=None, stream=None)


@pytest.mark.parametrize("change,status", [
    ({"B": 0}, INVALID), ({"Hkv": 3}, INVALID), ({"max_blocks": 0}, INVALID), ({"nb": 0}, INVALID), ({"window": 0}, INVALID),
    ({"window": -2}, INVALID), ({"scale": 0.0}, INVALID), ({"scale": NAN}, INVALID), ({"scale": INF}, INVALID), ({"P": 32}, UNSUPPORTED),
    ({"D": 256}, UNSUPPORTED), ({"Hq": 18}, UNSUPPORTED), ({"max_blocks": 1 << 27}, UNSUPPORTED),
    ({"B": 1 << 10, "max_blocks": 1 << 20}, UNSUPPORTED), ({"q": None}, INVALID), ({"ks": None}, INVALID), ({"ws": None}, INVALID),
    ({"sl": None}, INVALID), ({"q": FAR + 8}, INVALID), ({"ws": FAR + 4}, INVALID), ({"bt": FAR + 2}, INVALID), ({"out": FAR + 2}, INVALID),
    ({"wb": 16}, INVALID)])
def test_decode_fp4(lib, change, status):
    a = {**DECODE, **change}
    lib.kvq_paged_decode_attention_fp4.argtypes = [p] * 8 + [i] * 6 + [i64, f32, i, p, sz, p, p]
    assert lib.kvq_paged_decode_attention_fp4(*a.values()) == status


def test_fp4_workspace_size(lib):
    f = lib.kvq_decode_fp4_workspace_size
    f.restype, f.argtypes = sz, [i] * 6
    assert f(0, 8, 2, 128, 16, 4) == f(4, 8, 3, 128, 16, 4) == f(4, 8, 2, 96, 16, 4) == f(4, 8, 2, 128, 8, 4) == 0
    # 4 sequences of 2 KV heads and 4 pages: 16 parts of 2 pages; rows of D + 1 floats, and the pages before each sequence
    assert f(4, 8, 2, 128, 16, 4) == ((16 + 8) * 4 * 129 + 5) * 4 + 12


def test_other_calls_refuse_the_4_bit_cache(k):
    """Every call that reads caches and has no 4-bit form."""
    lib, ptr = k.lib, FAR
    assert lib.kvq_reshape_and_cache(ptr, ptr, ptr, ptr, ptr, ptr, ptr, 4, 2, 256, 16, 9, 3, None, None) == UNSUPPORTED
    assert lib.kvq_reshape_and_cache(ptr, ptr, ptr, ptr, ptr, None, ptr, 4, 2, 128, 16, 9, 3, None, None) == INVALID
    assert lib.kvq_reshape_and_cache(None, None, None, None, None, None, None, 0, 2, 128, 16, 9, 3, None, None) == OK
    assert lib.kvq_reshape_and_cache_per_token(ptr, ptr, ptr, ptr, ptr, 4, 2, 128, 16, 9, 3, None, None) == INVALID
    head, tail = [ptr] * 8 + [1, 8, 2, 128, 16, 4, 64, 0.1], [0, ptr, 1 << 40, None, None]
    assert lib.kvq_paged_decode_attention(*head, -1, 3, *tail) == INVALID
    assert lib.kvq_paged_decode_attention_acc(*head, -1, 3, *tail, 0) == INVALID
    assert lib.kvq_paged_decode_attention_append(*[ptr] * 3, *head, -1, 3, *tail) == INVALID
    assert lib.kvq_paged_decode_attention_per_token(*[ptr] * 6, *head[8:], -1, 3, *tail) == INVALID
    assert lib.kvq_paged_decode_attention_weights(*[ptr] * 9, 64, 1.0, 1, 8, 2, 128, 16, 4, 64, 0.1, -1, 3, 0, 0, ptr, 1 << 40, None, None) == INVALID
    assert lib.kvq_paged_decode_attention_shared_prefix(*[ptr] * 11, 1, 1, 8, 2, 128, 16, 4, 4, 64, 0.1, 3, ptr, 1 << 40, None, None) == UNSUPPORTED
    assert lib.kvq_evict_tokens(FAR, 64, FAR * 2, FAR * 3, FAR * 4, FAR * 5, FAR * 6, FAR * 7, FAR * 8, 32, FAR * 10, FAR * 11, 4, 2, 128, 16, 4, 2, 64,
                                4, 8, 3, 0, None, None) == INVALID
    sizes = [1, 8, 2, 128, 16, 4, 64, 16, 0.1, 1]
    assert lib.kvq_prefill_attention_dtype(*[ptr] * 10, *sizes, None, None, 3) in (INVALID, UNSUPPORTED)
    assert lib.kvq_prefill_attention_per_token(*[ptr] * 8, *sizes, 3, None, None) in (INVALID, UNSUPPORTED)


# ------------------------------------------------------------- the binding ---
T, Hq, H, D, NB = 3, 4, 2, 64, 5
bf16 = torch.bfloat16


def _base(k):
    kd, vd = k.alloc_kv_cache(NB, H, D, device="cpu", fill=0)
    f4 = k.alloc_kv_cache(NB, H, D, "fp4", device="cpu", fill=0)
    s = torch.ones(H)
    return dict(q=torch.zeros(T, Hq, D, dtype=bf16), k=torch.zeros(T, H, D, dtype=bf16), v=torch.zeros(T, H, D, dtype=bf16),
                pos=torch.zeros(T, dtype=torch.int64), inv=torch.zeros(D // 2), slots=torch.zeros(T, dtype=torch.int64), kd=kd, vd=vd,
                k4=f4[0], v4=f4[1], ks=s, vs=s.clone(), qo=torch.zeros(T, Hq, D, dtype=bf16), ko=torch.zeros(T, H, D, dtype=bf16),
                vo=torch.zeros(T, H, D, dtype=bf16), bt=torch.zeros(T, 2, dtype=torch.int32), sl=torch.zeros(T, dtype=torch.int32))


def _rope(kvq, **change):
    a = {**_base(kvq), **change}
    kw = {n: a[n] for n in ("q_weight", "k_weight", "pair_axis") if n in a}
    return kvq.kvq_qk_norm_rope(a["q"], a["k"], a["pos"], a["inv"], a["qo"], a["ko"], **kw)


def _append(kvq, **change):
    a = {**_base(kvq), **change}
    kw = {n: a[n] for n in ("q_weight", "k_weight", "pair_axis", "q8", "q_scale", "num_blocks", "cache_dtype", "per_token") if n in a}
    return kvq.kvq_rope_and_cache(a["q"], a["k"], a["v"], a["pos"], a["inv"], a["slots"], a["kd"], a["vd"], a["ks"], a["vs"], q_out=a["qo"], **kw)


def _gather(kvq, **change):
    a = {**_base(kvq), **change}
    kw = {n: a[n] for n in ("num_blocks", "cache_dtype", "per_token") if n in a}
    return kvq.kvq_gather_cache(a["slots"], a["kd"], a["vd"], a["ko"], a["vo"], a["ks"], a["vs"], **kw)


def _decode(kvq, **change):
    a = {**_base(kvq), **change}
    kw = {n: a[n] for n in ("num_blocks",) if n in a}
    return kvq.kvq_paged_decode_attention_fp4(a["q"], a["k4"], a["v4"], a["ks"], a["vs"], a["bt"], a["sl"], a["qo"], **kw)


def _write(kvq, **change):
    a = {**_base(kvq), **change}
    return kvq.kvq_reshape_and_cache(a["k"], a["v"], a["slots"], a["k4"], a["v4"], a["ks"], a["vs"], cache_dtype="fp4")


wide = torch.zeros(T, Hq, 2 * D, dtype=bf16)


@pytest.mark.parametrize("call,change,words", [
    (_rope, {"q": None, "k": None}, "q or k"), (_rope, {"q": torch.zeros(T, Hq, D)}, "q must be"), (_rope, {"k": torch.zeros(T, H, 128, dtype=bf16)}, "k must be"),
    (_rope, {"q": wide[..., :D]}, "contiguous"), (_rope, {"q": wide[..., ::2]}, "contiguous"), (_rope, {"qo": None}, "needs q_out"),
    (_rope, {"k": torch.zeros(T + 1, H, D, dtype=bf16)}, "tokens like"), (_rope, {"qo": torch.zeros(T, Hq + 1, D, dtype=bf16)}, "shaped like q"),
    (_rope, {"pos": torch.zeros(T, dtype=torch.int32)}, "positions"), (_rope, {"pos": torch.zeros(T + 1, dtype=torch.int64)}, "positions"),
    (_rope, {"pos": torch.zeros(2, T, dtype=torch.int64)}, "pair_axis"), (_rope, {"pos": torch.zeros(T, 2, dtype=torch.int64)[:, 0]}, "contiguous"),
    (_rope, {"inv": None}, "inv_freq"), (_rope, {"inv": torch.zeros(D // 2, dtype=torch.float64)}, "inv_freq"), (_rope, {"pos": None}, "need positions"),
    (_rope, {"pair_axis": torch.zeros(3, dtype=torch.int32)}, "pair_axis"), (_rope, {"q_weight": torch.zeros(D)}, "q_weight"),
    (_rope, {"k_weight": torch.zeros(D + 8, dtype=bf16)}, "k_weight"),
    (_append, {"v": torch.zeros(T + 1, H, D, dtype=bf16)}, "v must have"), (_append, {"v": torch.zeros(T, H + 1, D, dtype=bf16)}, "v must be"), (_append, {"q": torch.zeros(T + 1, Hq, D, dtype=bf16)}, "q must"),
    (_append, {"qo": None}, "q needs"), (_append, {"q": None}, "need q"), (_append, {"q8": torch.zeros(T, Hq, D)}, "q8 must"),
    (_append, {"q8": torch.zeros(T, Hq, D, dtype=torch.uint8)}, "q_scale"), (_append, {"slots": torch.zeros(T + 1, dtype=torch.int64)}, "slot_mapping"),
    (_append, {"ks": torch.ones(1)}, "k_scale"), (_append, {"cache_dtype": "bf16"}, "alloc_kv_cache"), (_append, {"per_token": True}, "alloc_kv_cache"),
    (_append, {"cache_dtype": "fp4"}, "alloc_kv_cache"), (_append, {"num_blocks": NB + 1}, "num_blocks"), (_append, {"inv": torch.zeros(D // 2).half()}, "inv_freq"),
    (_gather, {"vo": torch.zeros(T, H, D)}, "v_out"), (_gather, {"slots": torch.zeros(T, dtype=torch.int32)}, "slot_mapping"),
    (_gather, {"cache_dtype": "fp4"}, "alloc_kv_cache"), (_gather, {"num_blocks": NB + 1}, "num_blocks"), (_gather, {"per_token": True}, "alloc_kv_cache"),
    (_decode, {"q": torch.zeros(T, Hq, D)}, "q must"), (_decode, {"bt": torch.zeros(T, 2, dtype=torch.int64)}, "block_table"),
    (_decode, {"sl": torch.zeros(T + 1, dtype=torch.int32)}, "seq_lens"), (_decode, {"vs": torch.ones(H + 1)}, "v_scale"),
    (_decode, {"k4": torch.zeros(NB, H, 16 * D, dtype=torch.uint8)}, "alloc_kv_cache"), (_decode, {"num_blocks": NB + 1}, "num_blocks"),
    (_decode, {"qo": torch.zeros(T, Hq, D)}, "out must"), (_write, {"k4": torch.zeros(NB, H, 16 * D, dtype=torch.uint8)}, "alloc_kv_cache"),
    (_write, {"v": torch.zeros(T - 1, H, D, dtype=bf16)}, "v must"), (_write, {"slots": torch.zeros(T - 1, dtype=torch.int64)}, "slot_mapping"),
    (_write, {"ks": torch.ones(H + 1)}, "k_scale"), (_gather, {"ko": torch.zeros(H, T, D, dtype=bf16).transpose(0, 1)}, "contiguous"),
    (_decode, {"q": torch.zeros(T, D, Hq, dtype=bf16).transpose(1, 2)}, "contiguous")])
def test_binding_refuses(k, call, change, words):
    with pytest.raises(ValueError, match=words):
        call(k, **change)


@pytest.mark.parametrize("call", [_rope, _append, _gather, _decode, _write])
def test_cpu_tensors_are_refused(k, call):
    with pytest.raises(ValueError, match="CUDA tensors only"):
        call(k)


def test_fp4_allocation(k):
    kd, vd = k.alloc_kv_cache(7, 2, 128, "fp4_e2m1", device="cpu", fill=3)
    assert kd.shape == vd.shape == (7, 2, 1152)
    kd, vd = k.alloc_kv_cache(7, 2, 64, "fp4", device="cpu", paired=True)
    assert kd.shape == (7, 2, 1152) and vd.data_ptr() == kd.data_ptr() + 576
    for bad in ({"per_token": True}, {"head_dim": 256}):
        with pytest.raises(ValueError):
            k.alloc_kv_cache(**{**dict(num_blocks=7, kv_heads=2, head_dim=128, cache_dtype="fp4", device="cpu"), **bad})


class _OnGpu:
    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 16 * self.index


def test_tensors_of_another_device_are_refused(k, monkeypatch):
    """Any of them, whatever its place in the call."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert k._addresses(None, _OnGpu(1), _OnGpu(1)) == [None, 16, 16]
    for bad in ((_OnGpu(0),), (_OnGpu(1), None, _OnGpu(0))):
        with pytest.raises(ValueError, match=r"cuda:0\) must be the current one \(cuda:1\)"):
            k._addresses(*bad)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        k._addresses(_OnGpu(1), torch.zeros(1))


@pytest.mark.parametrize("dt,D,per_token", [(0, 64, False), (0, 64, True), (1, 128, False), (3, 128, False)])
def test_separate_tensors_of_one_page_may_lie_side_by_side(k, dt, D, per_token):
    """As an allocator may place them; with more pages the same addresses would be read as pairs."""
    kpage = k._page_bytes(D, dt)
    vpage = kpage + (k.SCALE_TAIL_BYTES if per_token else 0)
    buf = torch.zeros(2 * (kpage + vpage), dtype=torch.uint8)
    kc, vc = buf[:kpage].view(1, 1, -1), buf[kpage:kpage + vpage].view(1, 1, -1)
    assert k._check_cache(kc, vc, 1, D, dt, per_token, None) == 1
    if per_token:
        assert k._check_per_token_cache(kc, vc, 1, D) == 1
    two = (buf[:2 * kpage].view(2, 1, -1), buf[kpage:kpage + 2 * vpage].view(2, 1, -1))
    with pytest.raises(ValueError):
        k._check_cache(*two, 1, D, dt, per_token, None)
