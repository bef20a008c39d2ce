"""The workspace that a call allocates for itself comes from the memory of the
stream the call runs on (the allocator's blocks are ordered by their stream
alone).  A stand-in for CUDA streams: this runs without a GPU."""
import contextlib

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


@pytest.fixture
def allocated(k, monkeypatch):
    """(bytes, stream) of every allocation made while the test runs."""
    seen, current = [], [None]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    empty = torch.empty

    def recorded(n, **kw):
        seen.append((n, current[-1]))
        return empty(n, **{**kw, "device": "cpu"})

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: ("raw", raw))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    monkeypatch.setattr(k.torch, "empty", recorded)
    return seen


@pytest.mark.parametrize("stream,on", [(None, None), ("side", "side"), (0x1234, ("raw", 0x1234)), (0, ("raw", 0))])
def test_workspace_of_the_calls_stream(k, allocated, stream, on):
    like = torch.zeros(1)
    assert k._workspace(100, like, stream).numel() == 100
    assert k._workspace(0, like, stream).numel() == 16
    assert allocated == [(100, on), (16, on)]


def test_every_decode_call_allocates_there(k, allocated, monkeypatch):
    """Whatever becomes of the call afterwards (these tensors are not on a GPU)."""
    q, bt, lens = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    new, slots = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    s = torch.ones(2)
    kd, vd = torch.zeros(9, 2, 1024, dtype=torch.uint8), torch.zeros(9, 2, 1024, dtype=torch.uint8)
    vt = torch.zeros(9, 2, 1024 + k.SCALE_TAIL_BYTES, dtype=torch.uint8)
    calls = [lambda: k.kvq_paged_decode_attention(q, kd, vd, s, s, bt, lens, q, stream="side"),
             lambda: k.kvq_paged_decode_attention_append(q, new, new, slots, kd, vd, s, s, bt, lens, q, stream="side"),
             lambda: k.kvq_paged_decode_attention_per_token(q, kd, vt, bt, lens, q, stream="side"),
             lambda: k.kvq_paged_decode_attention_weights(q, kd, vd, s, s, bt, lens, q, torch.zeros(2, 2, 48), stream="side"),
             lambda: k.kvq_paged_decode_attention_shared_prefix(q, kd, vd, s, s, bt[:1], lens[:1], lens, bt, lens, q, stream="side")]
    for call in calls:
        before = len(allocated)
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
        assert [on for _, on in allocated[before:]] == ["side"]
