"""Calls of arc_kv_attend whose query rows would not fit the kernel's 32-bit counts are refused."""
import ctypes

from test_kv_cache import FAKE, fake_cache, fake_query, fake_step, lib  # noqa: F401


def test_too_many_rows_of_a_sequence(lib):  # noqa: F811
    ref = ctypes.addressof

    def call(T, heads, q_heads):
        cache = fake_cache(heads=heads, page_stride=heads * 64 * 128)
        step, query = fake_step(T=T, row_offsets=FAKE), fake_query(q_heads=q_heads)
        return lib.arc_kv_attend(ref(cache), ref(step), ref(query), None, FAKE, 0, None)  # (no workspace: the next check)

    assert call(1 << 24, 1, 64) == -8 and call(1 << 24, 1, 65) == -2
    assert call(1 << 20, 1, 1 << 10) == -8 and call((1 << 20) + 1, 1, 1 << 10) == -2
    assert call(1 << 24, 8, 512) == -8 and call(1 << 24, 4, 512) == -2
