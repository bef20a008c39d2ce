"""Host-side refusals of the shared-prefix, weights and eviction calls: every
one returns its status before any CUDA call (this runs without a GPU)."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "fp8_kv_cache_reshape_gb300", "libkvq.so")
p, i, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
INVALID, UNSUPPORTED = 1, 2
FAR = 1 << 40  # a fake address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    return ctypes.CDLL(LIB)


def _call(lib, name, sig, base, change):
    args = dict(base)
    assert set(change) <= set(args)
    args.update(change)
    f = getattr(lib, name)
    f.restype, f.argtypes = i, sig
    return f(*args.values())


def _pointers(*names):
    return {n: FAR * (k + 1) for k, n in enumerate(names)}


SHARED = {**_pointers("q", "k", "v", "ks", "vs", "pt", "pl", "gs", "bt", "sl", "out"), "B": 4, "G": 2, "Hq": 8, "Hkv": 2,
          "D": 128, "P": 16, "max_prefix": 8, "max_blocks": 4, "num_blocks": 64, "scale": 0.1, "dtype": 0, "ws": FAR * 20,
          "wb": BIG, "st": None, "stream": None}
SHARED_SIG = [p] * 11 + [i] * 8 + [i64, f32, i, p, sz, p, p]


@pytest.mark.parametrize("change,status", [
    ({"B": 0}, INVALID), ({"G": 0}, INVALID), ({"Hkv": 3}, INVALID), ({"max_prefix": 0}, INVALID), ({"max_blocks": 0}, INVALID),
    ({"num_blocks": 0}, INVALID), ({"scale": 0.0}, INVALID), ({"scale": float("nan")}, INVALID), ({"P": 32}, UNSUPPORTED),
    ({"D": 96}, UNSUPPORTED), ({"D": 256}, UNSUPPORTED), ({"Hq": 18}, UNSUPPORTED), ({"dtype": 1}, UNSUPPORTED),
    ({"q": None}, INVALID), ({"pt": None}, INVALID), ({"pl": None}, INVALID), ({"gs": None}, INVALID), ({"ks": None}, INVALID),
    ({"ws": None}, INVALID), ({"q": FAR + 8}, INVALID), ({"k": FAR + 4}, INVALID), ({"ws": FAR + 8}, INVALID),
    ({"gs": FAR + 2}, INVALID), ({"out": FAR + 2}, INVALID), ({"wb": 1024}, INVALID), ({"max_prefix": 1 << 28}, UNSUPPORTED),
    ({"B": 1 << 28, "Hq": 16}, UNSUPPORTED)])
def test_shared_prefix(lib, change, status):
    assert _call(lib, "kvq_paged_decode_attention_shared_prefix", SHARED_SIG, SHARED, change) == status


WEIGHTS = {**_pointers("q", "k", "v", "ks", "vs", "bt", "sl", "out", "w"), "stride": 64, "decay": 1.0, "B": 4, "Hq": 8,
           "Hkv": 2, "D": 128, "P": 16, "max_blocks": 4, "num_blocks": 64, "scale": 0.1, "window": -1, "dtype": 0,
           "per_token": 0, "splits": 0, "ws": FAR * 20, "wb": BIG, "st": None, "stream": None}
WEIGHTS_SIG = [p] * 9 + [i64, f32] + [i] * 6 + [i64, f32] + [i] * 4 + [p, sz, p, p]


@pytest.mark.parametrize("change,status", [
    ({"w": None}, INVALID), ({"w": FAR + 2}, INVALID), ({"stride": 63}, INVALID), ({"decay": -0.1}, INVALID),
    ({"decay": 1.5}, INVALID), ({"decay": float("nan")}, INVALID), ({"B": 0}, INVALID), ({"window": 0}, INVALID),
    ({"D": 256}, UNSUPPORTED), ({"Hq": 18}, UNSUPPORTED), ({"ks": None}, INVALID), ({"per_token": 1, "dtype": 1}, INVALID),
    ({"wb": 4096}, INVALID), ({"out": None}, INVALID), ({"B": 1 << 29}, UNSUPPORTED),
    ({"max_blocks": 134217727, "stride": 1 << 40}, UNSUPPORTED)])
def test_weights(lib, change, status):
    assert _call(lib, "kvq_paged_decode_attention_weights", WEIGHTS_SIG, WEIGHTS, change) == status


EVICT = {"w": FAR, "stride": 64, **{n: FAR * (k + 2) for k, n in enumerate(["k", "v", "bt", "sl", "kl", "dt", "dw"])},
         "dstride": 32, "dl": FAR * 10, "kept": FAR * 11, "B": 4, "Hkv": 2, "D": 128, "P": 16, "max_blocks": 4, "max_dst": 2,
         "num_blocks": 64, "sink": 4, "recent": 8, "dtype": 0, "per_token": 0, "st": None, "stream": None}
EVICT_SIG = [p, i64] + [p] * 7 + [i64, p, p] + [i] * 6 + [i64] + [i] * 4 + [p, p]


@pytest.mark.parametrize("change,status", [
    ({"B": 0}, INVALID), ({"Hkv": 0}, INVALID), ({"max_blocks": 0}, INVALID), ({"max_dst": 0}, INVALID), ({"sink": -1}, INVALID),
    ({"recent": -1}, INVALID), ({"P": 8}, UNSUPPORTED), ({"D": 96}, UNSUPPORTED), ({"D": 256, "dtype": 1}, UNSUPPORTED),
    ({"D": 256, "per_token": 1}, UNSUPPORTED), ({"dtype": 9}, INVALID), ({"dtype": 1, "per_token": 1}, INVALID),
    ({"stride": 63}, INVALID), ({"dstride": 31}, INVALID), ({"kept": None}, INVALID), ({"w": None}, INVALID),
    ({"kl": None}, INVALID), ({"k": FAR * 2 + 8}, INVALID), ({"dw": FAR * 8 + 2}, INVALID), ({"dw": FAR + 64}, INVALID),
    ({"dl": FAR * 5}, INVALID), ({"dl": FAR * 6 + 4}, INVALID), ({"B": 70000}, UNSUPPORTED),
    ({"max_blocks": 1 << 28, "stride": 1 << 40}, UNSUPPORTED)])
def test_evict(lib, change, status):
    assert _call(lib, "kvq_evict_tokens", EVICT_SIG, EVICT, change) == status


def test_workspace_sizes(lib):
    for name in ("kvq_shared_prefix_workspace_size", "kvq_decode_weights_workspace_size"):
        f = getattr(lib, name)
        f.restype, f.argtypes = sz, [i] * 8
        assert f(0, 1, 8, 2, 128, 16, 4, 4) == 0
    assert lib.kvq_shared_prefix_workspace_size(4, 1, 8, 3, 128, 16, 4, 4) == 0
    assert lib.kvq_shared_prefix_workspace_size(4, 1, 8, 2, 128, 16, 4, 4) > 0
    base = lib.kvq_decode_workspace_size
    base.restype, base.argtypes = sz, [i] * 8
    a, b = base(4, 6, 2, 128, 16, 4, -1, 0), lib.kvq_decode_weights_workspace_size(4, 6, 2, 128, 16, 4, -1, 0)
    assert b - a == 4 * 2 * 4 * 16 * 4 * 4 + 128  # float32 scores of four heads (three rounded up), and room to align them
