"""How the shared-prefix decode divides its rows, seen through its workspace: a
float output row and LSE per column and part.  CPU only."""
import pytest

COLUMN = (512 + 1) * 4


@pytest.fixture(scope="module")
def m():
    from sparse_mla_decode_kv_gb300 import build
    build.build()
    import sparse_mla_decode_kv_gb300 as m
    m.load()
    return m


def parts(m, batch, q_len, heads, prefix, own):
    """Parts a column is joined from; 1 where nothing is joined."""
    size = m.mla_prefix_decode_workspace_size(batch, q_len, heads, prefix, -(-own // 64), own)
    return max(1, size // (batch * q_len * heads * COLUMN))


@pytest.mark.parametrize("batch,q_len,heads,own", [(64, 1, 64, 140000), (32, 1, 16, 140000), (64, 3, 64, 2000),
                                                   (1, 1, 16, 140000), (7, 2, 48, 9000), (200, 1, 16, 1000)])
@pytest.mark.parametrize("prefix", [1, 32, 500])
def test_a_short_prefix_does_not_shred_long_own_rows(m, batch, q_len, heads, own, prefix):
    alone = parts(m, batch, q_len, heads, 0, own)
    # the prefix has 16 tiles at most, so 16 slices; the own rows at most those they have without it
    assert 2 <= parts(m, batch, q_len, heads, prefix, own) <= alone + min(16, -(-prefix // 32))


@pytest.mark.parametrize("prefix", [1, 5000, 2 ** 31 - 257])
@pytest.mark.parametrize("batch", [1, 9, 300, 4096])
def test_parts_are_bounded(m, prefix, batch):
    """However long the contexts may be, at most one slice an SM of the prefix and one of the own rows."""
    size = m.mla_prefix_decode_workspace_size(batch, 1, 16, prefix, 1 << 25, 2 ** 31 - 1)
    assert 2 <= size // (batch * 16 * COLUMN) <= 2 * 160


def test_long_prefixes_fill_the_machine_once(m):
    """Eight groups of columns over a long prefix: one wave of slices, and own rows in one slice each."""
    assert 160 // 8 - 4 <= parts(m, 32, 1, 16, 140000, 200) <= 160 // 8 + 1
    assert parts(m, 1, 1, 16, 0, 32) == 1
