"""The Python wrappers' refusals of the shared-prefix, weights and eviction
calls: shapes, types and cache sizes are checked before anything is launched
(CPU tensors: this runs without a GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def k():
    try:
        import fp8_kv_cache_reshape_gb300 as kvq
    except ImportError:
        import __graft_entry__
        __graft_entry__.build()
        import fp8_kv_cache_reshape_gb300 as kvq
    return kvq


B, Hq, H, D, NB = 2, 4, 2, 64, 9


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _base(k):
    kd, vd = k.alloc_kv_cache(NB, H, D, device="cpu", fill=0)
    q = torch.zeros(B, Hq, D, dtype=torch.bfloat16)
    s = torch.ones(H)
    return dict(q=q, kd=kd, vd=vd, ks=s, vs=s.clone(), out=torch.zeros_like(q), bt=_i(B, 3), sl=_i(B))


def _shared(k, **change):
    a = {**_base(k), "pt": _i(1, 4), "pl": _i(1), "gs": _i(2), **change}
    kw = {n: a[n] for n in ("num_blocks", "cache_dtype") if n in a}
    return k.kvq_paged_decode_attention_shared_prefix(a["q"], a["kd"], a["vd"], a["ks"], a["vs"], a["pt"], a["pl"], a["gs"],
                                                      a["bt"], a["sl"], a["out"], **kw)


def _weights(k, **change):
    a = {**_base(k), "w": torch.zeros(B, H, 48), **change}
    kw = {n: a[n] for n in ("num_blocks", "cache_dtype", "per_token") if n in a}
    return k.kvq_paged_decode_attention_weights(a["q"], a["kd"], a["vd"], a["ks"], a["vs"], a["bt"], a["sl"], a["out"], a["w"],
                                                **kw)


def _evict(k, **change):
    a = {**_base(k), "w": torch.zeros(B, H, 48), "keep": _i(B), "dt": _i(B, 2), "dw": torch.zeros(B, H, 32), "dl": _i(B),
         "kept": _i(B, H, 32), "head_dim": D, **change}
    kw = {n: a[n] for n in ("num_blocks", "cache_dtype", "per_token") if n in a}
    return k.kvq_evict_tokens(a["w"], a["kd"], a["vd"], a["bt"], a["sl"], a["keep"], a["dt"], a["dw"], a["dl"], a["kept"],
                              head_dim=a["head_dim"], **kw)


LONG = dict(dtype=torch.int64)


@pytest.mark.parametrize("call,change,words", [
    (_shared, {"q": torch.zeros(B, Hq, D)}, "q must be"), (_shared, {"out": torch.zeros(B, Hq, D)}, "out must be"),
    (_shared, {"pt": torch.zeros(1, 4, **LONG)}, "prefix_table"), (_shared, {"pl": _i(2)}, "prefix_lens"),
    (_shared, {"gs": _i(3)}, "group_starts"), (_shared, {"sl": _i(3)}, "seq_lens"), (_shared, {"bt": _i(3, 3)}, "block_table"),
    (_shared, {"ks": torch.ones(1)}, "k_scale"), (_shared, {"vs": torch.ones(H, dtype=torch.float64)}, "v_scale"),
    (_shared, {"cache_dtype": "bf16"}, "alloc_kv_cache"), (_shared, {"num_blocks": NB + 1}, "num_blocks"),
    (_weights, {"w": torch.zeros(B, 1, 48)}, "weights"), (_weights, {"w": torch.zeros(B, H, 48, dtype=torch.float64)}, "weights"),
    (_weights, {"per_token": True}, "alloc_kv_cache"), (_weights, {"cache_dtype": "bf16"}, "alloc_kv_cache"),
    (_weights, {"bt": torch.zeros(B, 3, **LONG)}, "block_table"),
    (_evict, {"head_dim": 128}, "alloc_kv_cache"), (_evict, {"per_token": True}, "alloc_kv_cache"), (_evict, {"keep": _i(1)}, "keep_lens"),
    (_evict, {"kept": _i(B, H, 16)}, "kept"), (_evict, {"dl": torch.zeros(B, **LONG)}, "dst_seq_lens"),
    (_evict, {"dw": torch.zeros(B, 1, 32)}, "dst_weights"), (_evict, {"dt": _i(1, 2)}, "dst_block_table"),
    (_evict, {"num_blocks": NB + 1}, "num_blocks")])
def test_refused(k, call, change, words):
    with pytest.raises(ValueError, match=words):
        call(k, **change)


@pytest.mark.parametrize("call", [_shared, _weights, _evict])
def test_cpu_tensors_are_refused(k, call):
    """Everything else in order: the tensors are not on a GPU."""
    with pytest.raises(ValueError, match="CUDA tensors only"):
        call(k)


class _OnGpu:
    is_cuda = True

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 16 * self.index


def test_tensors_of_another_device_are_refused(k, monkeypatch):
    """Any of them, whatever its place in the call."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert k._device_ptrs(_OnGpu(1), None, _OnGpu(1)) == [16, None, 16]
    for bad in ((_OnGpu(0),), (_OnGpu(1), None, _OnGpu(0))):
        with pytest.raises(ValueError, match=r"cuda:0\) must be the current one \(cuda:1\)"):
            k._device_ptrs(*bad)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        k._device_ptrs(_OnGpu(1), torch.zeros(1))


def test_a_protected_end_beyond_32_bits_means_every_token(k, monkeypatch):
    seen = {}
    monkeypatch.setattr(k, "_device_ptrs", lambda *t: [None] * len(t))
    monkeypatch.setattr(k, "_stream", lambda s: None)
    monkeypatch.setattr(k.lib, "kvq_evict_tokens", lambda *a: seen.update(sink=a[19], recent=a[20]) or 0)
    a = _base(k)
    k.kvq_evict_tokens(torch.zeros(B, H, 48), a["kd"], a["vd"], a["bt"], a["sl"], _i(B), _i(B, 2), torch.zeros(B, H, 32),
                       _i(B), _i(B, H, 32), D, sink=2**32, recent=10**12)
    assert seen == {"sink": 2**31 - 1, "recent": 2**31 - 1}
