"""Rows in place with another stride are refused: a token's output would take the
place of one that is still to be read (no GPU)."""
import pytest

from tests.test_qkv_refusals import CACHE, CACHE_SIG, FAR, INVALID, ROPE, ROPE_SIG, _turn, lib  # noqa: F401


@pytest.mark.parametrize("change", [{"qos": 2048}, {"qs": 2048}, {"kos": 512}, {"ks": 264, "qo": FAR * 2}])
def test_norm_rope(lib, change):  # noqa: F811
    norm, rotary = _turn({})
    lib.kvq_qk_norm_rope.argtypes = ROPE_SIG
    assert lib.kvq_qk_norm_rope(*{**ROPE, "norm_p": norm, "rotary_p": rotary, **change}.values()) == INVALID


@pytest.mark.parametrize("change", [{"qos": 2048}, {"qs": 1032}, {"qos": 1032, "q8": None}])
def test_rope_and_cache(lib, change):  # noqa: F811
    norm, rotary = _turn({})
    lib.kvq_rope_and_cache.argtypes = CACHE_SIG
    assert lib.kvq_rope_and_cache(*{**CACHE, "norm_p": norm, "rotary_p": rotary, **change}.values()) == INVALID
