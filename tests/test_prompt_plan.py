"""How the attention over packed prompts divides its work: the plan query against the
workspace, and what it refuses.  CPU only (without a GPU for 148 SMs)."""
import pytest

SIZES = [(1, 1, 1, 1, 1, 64), (51, 51, 3, 8, 8, 64), (6000, 6000, 1, 16, 16, 128), (2048, 32768, 1, 16, 16, 128),
         (15000, 15000, 16, 32, 4, 128), (32, 150000, 32, 64, 8, 128), (1, 8192, 1, 32, 8, 128), (600, 18000, 3, 4, 2, 80),
         (231, 2205, 7, 28, 4, 128), (5, 0, 2, 4, 4, 64), (700, 5200, 1, 16, 16, 128), (2, 2 ** 31 - 256, 1, 1, 1, 8)]


@pytest.fixture(scope="module")
def m():
    from sparse_mla_decode_kv_gb300 import build
    build.build()
    import sparse_mla_decode_kv_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("sizes", SIZES)
def test_plan_and_workspace(m, sizes):
    q_tokens, kv_tokens, batch, heads, kv_heads, dv = sizes
    p = m.mla_prompt_attention_plan(*sizes)
    assert p["row_tiles"] in (1, 2) and p["slices"] >= 1 and p["variant"] in ("plain", "turns", "pairs")
    # a sequence has a place for each started span of tokens, and one more at most
    span = p["row_tiles"] * (128 // (heads // kv_heads))
    assert p["units"] == (q_tokens // span + batch) * kv_heads * p["slices"]
    # a float row, a reference and a sum for each slice
    rows = q_tokens * heads * p["slices"] * (dv + 2) * 4
    assert m.mla_prompt_attention_workspace_size(*sizes) == (-(-rows // 256) * 256 if p["slices"] > 1 else 0)
    # no slice is longer than what a role without rows may wait for
    assert -(-kv_tokens // 128) <= 65536 * p["slices"]


def test_variants(m):
    plan = m.mla_prompt_attention_plan
    assert plan(4096, 5200, 1, 16, 16, 128)["variant"] == "turns"     # both tiles, many keys
    sliced = plan(700, 5200, 1, 16, 16, 128)                          # as many keys, but few a slice
    assert sliced["slices"] > 1 and sliced["variant"] == "plain"
    assert plan(9600, 9600, 24, 16, 16, 128)["variant"] == "plain"    # both tiles, few keys
    assert plan(32, 150000, 32, 64, 8, 128)["variant"] == "pairs"     # a token each
    assert plan(600, 18000, 3, 4, 2, 128)["row_tiles"] == 1           # rows that leave SMs idle


def test_refusals(m):
    lib = m.load()
    args = [10, 10, 1, 4, 4, 64]
    assert lib.mla_prompt_attention_plan(*args, None, None, None, None) == 0
    for at, value, status in ((0, 0, 1), (1, -1, 1), (2, 0, 1), (3, 0, 1), (3, 5, 1), (4, 0, 1), (4, 3, 1), (5, 4, 1),
                              (5, 20, 1), (5, 136, 2), (3, 129 * 4, 2), (0, 2 ** 31, 2), (1, 2 ** 31, 2),
                              (2, 2 ** 31 - 1, 2)):
        bad = list(args)
        bad[at] = value
        assert lib.mla_prompt_attention_plan(*bad, None, None, None, None) == status, (at, value)
    with pytest.raises(ValueError, match="32 bits"):
        m.mla_prompt_attention_plan(10, 10, 2 ** 32 + 1, 4, 4, 64)
    with pytest.raises(m.MlaError):
        m.mla_prompt_attention_plan(10, 10, 1, 4, 3, 64)
