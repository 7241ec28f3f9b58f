"""Arguments past 32 bits: a C int keeps their low 32 bits, so they are refused
before the call, negative ones too."""
import pytest
import torch

from dense_ref import SCALE, random_pool
from gpu_helpers import lib
from test_gpu_dense_decode import DEV, gen, lens_tensor, queries, tables

pytestmark = pytest.mark.gpu
WRAP = 2 ** 32


@pytest.fixture(scope="module")
def m():
    return lib()


@pytest.mark.parametrize("over", [dict(sinks=-WRAP), dict(window=5 - WRAP), dict(block_size=64 - WRAP),
                                  dict(block_size=64 + WRAP), dict(fmt=-WRAP)])
def test_window_decode(m, over):
    g = gen(1)
    bt, _, nb = tables(g, [100])
    pool, stride = random_pool(g, nb, 0)
    args = dict(sinks=0, window=5)
    args.update(over)
    with pytest.raises(ValueError):
        m.mla_window_decode(*queries(g, 1, 1, 16), pool, stride, nb, bt, lens_tensor([100]), SCALE, **args)


@pytest.mark.parametrize("prefix_len,max_ctx", [(64 - WRAP, 100), (64 + WRAP, 100), (64, 100 - WRAP)])
def test_prefix_decode(m, prefix_len, max_ctx):
    g = gen(2)
    bt, spare, nb = tables(g, [100])
    pool, stride = random_pool(g, nb, 0)
    with pytest.raises(ValueError):
        m.mla_prefix_decode(*queries(g, 1, 1, 16), pool, stride, nb, spare, prefix_len, bt, lens_tensor([100]), SCALE,
                            max_ctx)


def test_norms_and_tables(m):
    x = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device=DEV)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    inv = torch.ones(32, dtype=torch.float64, device=DEV)
    pool = torch.zeros((1, 64, 352), dtype=torch.uint8, device=DEV)
    for offset in (WRAP, -WRAP):
        with pytest.raises(ValueError):
            m.mla_qk_norm_rope(x, None, one, inv, rope_offset=offset)
    kv, w, slot = (torch.zeros((1, 576), dtype=torch.bfloat16, device=DEV),
                   torch.ones(512, dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV))
    for bad in (dict(block_size=64 - WRAP), dict(fmt=WRAP)):
        args = dict(block_size=64, fmt=0)
        args.update(bad)
        with pytest.raises(ValueError):
            m.mla_kv_norm_rope_append(kv, w, one, inv, slot, pool, 1, kv_block_stride=64 * 352, **args)
    with pytest.raises(ValueError):
        m.mla_block_table_extend(one, one, torch.zeros((1, 4), dtype=torch.int32, device=DEV), one,
                                 torch.zeros(3, dtype=torch.int64, device=DEV), 1, 4, block_size=64 + WRAP)
    assert not pool.any()
