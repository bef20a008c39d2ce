"""Windows at the end of 32 bits: wider than any sequence."""
from tests.test_serving_binding import k  # noqa: F401  (the fixture)


def test_the_widest_window_is_planned_like_none(k):  # noqa: F811
    for window in (2**31 - 16, 2**31 - 15, 2**31 - 1):
        assert k.kvq_decode_num_splits(1, 8, 8192, window) == k.kvq_decode_num_splits(1, 8, 8192)
        assert k.kvq_decode_workspace_size(1, 32, 8, 128, 8192, window) == k.kvq_decode_workspace_size(1, 32, 8, 128, 8192)
