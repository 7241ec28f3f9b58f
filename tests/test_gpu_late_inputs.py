"""Dense decodes behind a kernel that signals its dependents first and writes
their lengths, tables and queries late: the decode's grid is resident by then and
has to see what was written."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from dense_ref import SCALE, random_pool
from gpu_helpers import lib
from test_gpu_dense_decode import DEV, gen, lens_tensor, queries, tables

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def m():
    return lib()


@pytest.fixture(scope="module")
def late_write(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("late_writer") / "liblate.so")
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-shared",
                    "-Xcompiler", "-fPIC", os.path.join(HERE, "late_writer_kernel.cu"), "-o", out], check=True)
    so = C.CDLL(out)
    so.late_write.restype = C.c_int
    so.late_write.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p, C.c_longlong, C.c_void_p]

    def write(src, dst):
        assert all(s.numel() * s.element_size() == d.numel() * d.element_size() for s, d in zip(src, dst))
        at = (C.c_void_p * 4)
        words = (C.c_int * 4)(*[s.numel() * s.element_size() // 4 for s in src])
        err = so.late_write(at(*[s.data_ptr() for s in src]), at(*[d.data_ptr() for d in dst]), words, 40000,
                            torch.cuda.current_stream().cuda_stream)
        assert err == 0

    return write


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("batch,heads,prefix", [(3, 16, 0), (200, 64, 0), (3, 32, 700)])
def test_inputs_written_while_the_grid_waits(m, late_write, fmt, batch, heads, prefix):
    g = gen(90 + batch)
    lens = [[1 + (131 * b + 700 * k) % 1400 for b in range(batch)] for k in range(2)]
    bt, spare, nb = tables(g, [1400] * batch, extra_blocks=24)
    pool, stride = random_pool(g, nb, fmt)
    ctx = [lens_tensor(x) for x in lens]
    table = [bt, bt.flip(1).contiguous()]
    shared = [spare[:12].contiguous(), spare[12:24].contiguous()]
    query = [queries(g, batch, 1, heads) for _ in range(2)]

    def decode(ctx, table, shared, qn, qr):
        if prefix:
            return m.mla_prefix_decode(qn, qr, pool, stride, nb, shared, prefix, table, ctx, SCALE, 1400, fmt=fmt)[0]
        return m.mla_window_decode(qn, qr, pool, stride, nb, table, ctx, SCALE, 4, 600, fmt=fmt)[0]

    want = [decode(ctx[k], table[k], shared[k], *query[k]) for k in range(2)]
    assert not torch.equal(want[0], want[1])
    live = [ctx[0].clone(), table[0].clone(), shared[0].clone(), query[0][0].clone()]
    rope = query[0][1]
    want = [decode(ctx[k], table[k], shared[k], query[k][0], rope) for k in range(2)]
    torch.cuda.synchronize()
    for step in range(12):
        k = (step + 1) % 2
        late_write([ctx[k], table[k], shared[k], query[k][0]], live)
        got = decode(*live, rope)
        torch.cuda.synchronize()
        assert torch.equal(got, want[k]), f"step {step}"
    assert m.mla_device_fault() == 0
