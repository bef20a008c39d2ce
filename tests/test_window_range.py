"""Windows at the end of 32 bits and beyond reach the library as what they mean,
in every decode call: wider than any sequence, or an error (CPU tensors: the
library's calls are replaced by ones that keep their arguments)."""
import ctypes

import pytest
import torch

from tests.test_serving_binding import k  # noqa: F401  (the fixture)

B, Hq, H, D, NB = 2, 4, 2, 64, 9
CALLS = ("kvq_paged_decode_attention", "kvq_paged_decode_attention_append", "kvq_paged_decode_attention_per_token",
         "kvq_paged_decode_attention_weights", "kvq_paged_decode_attention_fp4")


class Taken(Exception):
    pass


def _windows(k, monkeypatch, name, window):  # noqa: F811
    """The call's window argument, and that of its workspace's size where it has one."""
    lib, real = k.lib, getattr(k.lib, name)
    size = {"kvq_paged_decode_attention_weights": "kvq_decode_weights_workspace_size",
            "kvq_paged_decode_attention_fp4": None}.get(name, "kvq_decode_workspace_size")
    found = []

    types = list(real.argtypes)  # the window comes behind sm_scale, the last float; in a size, last but one
    position = len(types) - types[::-1].index(ctypes.c_float)

    def keep(window):
        assert ctypes.c_int(window).value == window, "ctypes cuts it"
        found.append(window)

    class Lib:
        def __getattr__(self, attr):
            def call(*args):
                keep(args[position])
                raise Taken

            def need(*args):
                keep(args[-2])
                return 64

            return {name: call, size: need}.get(attr) or getattr(lib, attr)

    monkeypatch.setattr(k, "lib", Lib())
    monkeypatch.setattr(k, "_ptr", lambda t: None)
    monkeypatch.setattr(k, "_stream", lambda s: 0)
    monkeypatch.setattr(k, "_device_ptrs", lambda *t: [None] * len(t))
    monkeypatch.setattr(k, "_addresses", lambda *t: [None] * len(t))
    fp4, per_token = name.endswith("fp4"), name.endswith("per_token")
    kd, vd = k.alloc_kv_cache(NB, H, D, "fp4" if fp4 else "fp8", device="cpu", fill=0, per_token=per_token)
    q, s = torch.zeros(B, Hq, D, dtype=torch.bfloat16), torch.ones(H)
    table, lens = torch.zeros(B, 3, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    new, scales = torch.zeros(B, H, D, dtype=torch.bfloat16), () if per_token else (s, s)
    more = (new, new, torch.zeros(B, dtype=torch.int64)) if name.endswith("append") else ()
    last = (torch.zeros(B, H, 48),) if name.endswith("weights") else ()
    with pytest.raises(Taken):
        getattr(k, name)(q, *more, kd, vd, *scales, table, lens, q.clone(), *last, window=window)
    assert found
    return found


@pytest.mark.parametrize("name", CALLS)
def test_windows_wider_than_32_bits(k, monkeypatch, name):  # noqa: F811
    for window in (2**31, 2**32, 2**32 + 5, 2**62):
        assert set(_windows(k, monkeypatch, name, window)) == {2**31 - 1}
        monkeypatch.undo()
    for window in (-1, 1, 500, 2**31 - 1):
        assert set(_windows(k, monkeypatch, name, window)) == {window}
        monkeypatch.undo()


@pytest.mark.parametrize("name", CALLS)
def test_negative_windows_stay_wrong(k, monkeypatch, name):  # noqa: F811
    for window in (-2, -2**31 - 1, -2**32 - 1, -2**32 + 7):
        assert max(_windows(k, monkeypatch, name, window)) < -1
        monkeypatch.undo()


def test_the_widest_window_is_planned_like_none(k):  # noqa: F811
    for window in (2**31 - 16, 2**31 - 15, 2**31 - 1, 2**40):
        assert k.kvq_decode_num_splits(1, 8, 8192, window) == k.kvq_decode_num_splits(1, 8, 8192)
        assert k.kvq_decode_workspace_size(1, 32, 8, 128, 8192, window) == k.kvq_decode_workspace_size(1, 32, 8, 128, 8192)
