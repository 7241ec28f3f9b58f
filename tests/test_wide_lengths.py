"""Lengths past 32 bits in the dense decodes' workspace sizes: cut as the calls cut them.  CPU only."""
import pytest


@pytest.fixture(scope="module")
def m():
    from sparse_mla_decode_kv_gb300 import build
    build.build()
    import sparse_mla_decode_kv_gb300 as m
    m.load()
    return m


def test_lengths_are_cut(m):
    top = 2 ** 31 - 1
    w, p = m.mla_window_decode_workspace_size, m.mla_prefix_decode_workspace_size
    for wide in (2 ** 32 + 1, 2 ** 40):
        assert w(1, 1, 16, 1000, 0, wide) == w(1, 1, 16, 1000, 0, top) > 0
        assert w(1, 1, 16, 1000, wide, 5) == w(1, 1, 16, 1000, top, 5) > 0
        assert p(1, 1, 16, 100, 1000, wide) == p(1, 1, 16, 100, 1000, top) > 0


def test_what_a_c_int_would_wrap_is_refused(m):
    with pytest.raises(ValueError):
        m.mla_window_decode_workspace_size(1, 1, 16, 10, 0, 5 - 2 ** 32)
    for prefix, ctx in ((2 ** 32 + 5, 100), (5 - 2 ** 32, 100), (5, 100 - 2 ** 32)):
        with pytest.raises(ValueError):
            m.mla_prefix_decode_workspace_size(1, 1, 16, prefix, 10, ctx)
