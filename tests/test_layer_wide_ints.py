"""Sizes that a C int would keep the low 32 bits of, in the layer's operators.  CPU only:
the binding refuses them before the library is reached."""
import pytest
import torch


class Wide:
    """Looks like a CUDA tensor of any shape, of which nothing is stored."""

    is_cuda = True

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 0

    def stride(self):
        out, n = [], 1
        for x in reversed(self.shape):
            out.append(n)
            n *= x
        return tuple(reversed(out))

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True


@pytest.fixture
def m(monkeypatch):
    import sparse_mla_decode_kv_gb300 as m
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return m


BF16, U8, E4M3, I32 = torch.bfloat16, torch.uint8, torch.float8_e4m3fn, torch.int32


def test_rows_and_k_of_products(m):
    for groups, n, k in ((1, 2 ** 32 + 5, 32), (1, 5, 2 ** 32 + 32), (2 ** 32 + 3, 5, 32)):
        with pytest.raises(ValueError, match="32 bits"):
            m.mla_fp4_matvec(Wide((1, groups, k), BF16), Wide((groups, n, k // 2), U8), Wide((groups, n, k // 16), E4M3))


def test_dims_of_the_norm(m):
    d = 2 ** 32 + 128
    with pytest.raises(ValueError, match="32 bits"):
        m.mla_add_norm_quant(Wide((1, d), BF16), Wide((d,), BF16))


def test_heads_and_sequences(m):
    for heads, dk, batch in ((2 ** 32 + 1, 64, 1), (1, 2 ** 32 + 64, 1), (1, 64, 2 ** 32 + 1)):
        q, at = Wide((1, heads, dk), BF16), Wide((batch + 1,), I32)
        with pytest.raises(ValueError, match="32 bits"):
            m.mla_prompt_attention(q, q, q, at, at, 1.0)


@pytest.mark.parametrize("query", ["mla_prompt_attention_workspace_size", "mla_prompt_attention_plan"])
def test_sizes_of_a_prompt_batch(m, query):
    for at in (2, 3, 4, 5):
        sizes = [32, 10 ** 6, 32, 8, 1, 128]
        sizes[at] += 2 ** 32
        with pytest.raises(ValueError, match="32 bits"):
            getattr(m, query)(*sizes)
