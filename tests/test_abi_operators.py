"""Host-side validation of the operators around the paged cache: block tables
from lengths, norm and rotation, window and shared-prefix decode.

CPU only: every call here fails validation, is a no-op, or is a pure host
query; the pointers are never dereferenced."""
import ctypes as C

import pytest

INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 3
FAKE = C.c_void_p(0x10000)
ODD = C.c_void_p(0x10002)  # 2-byte aligned only
BIG = 1 << 40


@pytest.fixture(scope="module")
def m():
    from sparse_mla_decode_kv_gb300 import build
    build.build()
    import sparse_mla_decode_kv_gb300 as m
    m.load()
    return m


def call(m, name, defaults, over):
    assert set(over) <= set(defaults), over
    return getattr(m.load(), name)(*{**defaults, **over}.values(), None)


EXTEND = dict(ctx=FAKE, new=FAKE, batch=2, bt=FAKE, width=4, free=FAKE, cap=8, state=FAKE, nb=10, bs=64, slots=FAKE,
              pos=FAKE, n=16, start=FAKE, ctx_out=FAKE, state_out=FAKE)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, INVALID) for k in ("ctx", "new", "bt", "free", "state", "slots", "pos", "start", "ctx_out",
                                     "state_out")],
    *[({k: ODD}, INVALID) for k in ("ctx", "new", "bt", "free", "state", "slots", "pos", "start", "ctx_out",
                                    "state_out")],
    *[({k: -1}, INVALID) for k in ("batch", "cap", "nb", "n")],
    (dict(state=C.c_void_p(0x10004)), INVALID),  # int64
    (dict(width=0), INVALID), (dict(bs=48), INVALID), (dict(bs=32), UNSUPPORTED), (dict(n=1 << 31), INVALID),
])
def test_block_table_extend(m, over, status):
    assert call(m, "mla_block_table_extend", EXTEND, over) == status


def heads(m, **over):
    h = dict(in_=0x10000, out=0x20000, heads=4, in_token_stride=4 * 192, in_head_stride=192, out_token_stride=4 * 192,
             out_head_stride=192, weight=0x30000)
    h.update(over)
    return C.byref(m._Heads(*h.values()))


QK = dict(q=None, k=None, n=3, dim=192, offset=128, interleaved=1, eps=1e-6, pos=FAKE, inv=FAKE)
BAD_HEADS = [dict(heads=-1), dict(in_=None), dict(out=None), dict(in_=0x10008), dict(out=0x20008),
             dict(weight=0x30008), dict(in_token_stride=4 * 192 + 4), dict(in_head_stride=196),
             dict(out_token_stride=4 * 192 + 4), dict(out_head_stride=196),
             dict(out_token_stride=0), dict(out_head_stride=184),  # rows of the output that overlap
             dict(out=0x10000, out_token_stride=4 * 200, out_head_stride=200)]  # in place, other strides


@pytest.mark.parametrize("over", BAD_HEADS)
@pytest.mark.parametrize("which", ["q", "k"])
def test_head_sets(m, over, which):
    assert call(m, "mla_qk_norm_rope", QK, {which: heads(m, **over)}) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), INVALID), (dict(dim=56), INVALID), (dict(dim=100), INVALID), (dict(dim=264), UNSUPPORTED),
    (dict(offset=-8), INVALID), (dict(offset=132), INVALID), (dict(offset=136), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(pos=None), INVALID), (dict(inv=None), INVALID), (dict(pos=ODD), INVALID),
    (dict(inv=C.c_void_p(0x10004)), INVALID), (dict(n=0), 0), (dict(n=0, pos=None, inv=None), 0),
])
def test_qk_norm_rope(m, over, status):
    assert call(m, "mla_qk_norm_rope", QK, dict(q=heads(m), **over)) == status


def test_qk_norm_rope_needs_a_head_set(m):
    assert call(m, "mla_qk_norm_rope", QK, {}) == INVALID


APPEND = dict(kv=FAKE, kv_stride=576, w=FAKE, q=None, dim=192, offset=128, interleaved=1, eps=1e-6, pos=FAKE, inv=FAKE,
              slots=FAKE, n=3, pool=FAKE, nb=4, bs=64, stride=64 * 576, fmt=1)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, INVALID) for k in ("kv", "w", "pos", "inv", "slots", "pool")],
    *[({k: ODD}, INVALID) for k in ("kv", "w", "pos", "inv", "slots", "pool")],
    (dict(kv_stride=580), INVALID), (dict(n=-1), INVALID), (dict(nb=-1), INVALID), (dict(fmt=2), INVALID),
    (dict(bs=128), UNSUPPORTED), (dict(bs=40), INVALID), (dict(stride=64 * 576 - 16), INVALID),
    (dict(stride=64 * 576 + 8), INVALID), (dict(fmt=0, stride=64 * 352 - 16), INVALID), (dict(eps=0.0), INVALID),
    (dict(n=0, kv=None, w=None, pos=None, inv=None, slots=None, pool=None), 0),
])
def test_kv_norm_rope_append(m, over, status):
    assert call(m, "mla_kv_norm_rope_append", APPEND, over) == status


@pytest.mark.parametrize("over", BAD_HEADS)
def test_kv_norm_rope_append_head_set(m, over):
    assert call(m, "mla_kv_norm_rope_append", APPEND, dict(q=heads(m, **over))) == INVALID


WINDOW = dict(qn=FAKE, qr=FAKE, pool=FAKE, stride=64 * 352, nb=10, bt=FAKE, width=4096, ctx=FAKE, batch=2, q_len=1,
              heads=16, bs=64, sinks=4, window=100000, scale=0.07, fmt=0, out=FAKE, lse=None, ws=None, ws_bytes=0)
PREFIX = dict(qn=FAKE, qr=FAKE, pool=FAKE, stride=64 * 352, nb=10, pt=FAKE, prefix=5000, bt=FAKE, width=4, ctx=FAKE,
              batch=2, q_len=1, heads=16, bs=64, max_ctx=256, scale=0.07, fmt=0, out=FAKE, lse=None, ws=None,
              ws_bytes=0)
DENSE = [
    *[({k: None}, INVALID) for k in ("qn", "qr", "pool", "bt", "ctx", "out")],
    *[({k: ODD}, INVALID) for k in ("qn", "qr", "pool", "bt", "ctx", "out", "lse")],
    (dict(stride=64 * 352 - 16), INVALID), (dict(stride=64 * 352 + 8), INVALID), (dict(fmt=1), INVALID),
    (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID), (dict(nb=-1), INVALID), (dict(width=0), INVALID),
    (dict(batch=-1), INVALID), (dict(q_len=0), INVALID), (dict(q_len=65), INVALID), (dict(heads=8), INVALID),
    (dict(heads=24), INVALID), (dict(heads=144), INVALID), (dict(bs=32), UNSUPPORTED), (dict(bs=63), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(batch=1 << 24, q_len=64, heads=128), INVALID),  # more than 2^31 (token, head) pairs
    (dict(ws=None, ws_bytes=0), TOO_SMALL), (dict(ws=FAKE, ws_bytes=256), TOO_SMALL),
    (dict(ws=None, ws_bytes=BIG), INVALID), (dict(ws=C.c_void_p(0x10080), ws_bytes=BIG), INVALID),
    (dict(batch=0), 0), (dict(batch=0, qn=None, qr=None, pool=None, bt=None, ctx=None, out=None), 0),
]


@pytest.mark.parametrize("over,status", DENSE + [(dict(sinks=-1), INVALID), (dict(window=0), INVALID),
                                                 (dict(window=-5), INVALID)])
def test_window_decode(m, over, status):
    assert call(m, "mla_window_decode", WINDOW, over) == status


@pytest.mark.parametrize("over,status", DENSE + [(dict(pt=None), INVALID), (dict(pt=ODD), INVALID),
                                                 (dict(prefix=-1), INVALID), (dict(prefix=0x7FFFFFFF), INVALID),
                                                 (dict(max_ctx=-1), INVALID)])
def test_prefix_decode(m, over, status):
    assert call(m, "mla_prefix_decode", PREFIX, over) == status


def test_dense_workspace_sizes(m):
    w, p = m.mla_window_decode_workspace_size, m.mla_prefix_decode_workspace_size
    for bad in [(0, 1, 16, 4, 0, 5), (1, 0, 16, 4, 0, 5), (1, 1, 8, 4, 0, 5), (1, 1, 24, 4, 0, 5), (1, 1, 16, 0, 0, 5),
                (1, 1, 16, 4, -1, 5), (1, 1, 16, 4, 0, 0)]:
        assert w(*bad) == 0
    assert p(1, 1, 16, -1, 4, 5) == 0 and p(1, 1, 16, 5, 0, 5) == 0 and p(1, 1, 16, 5, 4, -1) == 0
    assert w(1, 1, 16, 4, 0, 32) == 0           # one tile: nothing to join
    assert w(4096, 4, 128, 4096, 64, 4096) == 0  # a batch that fills the machine is not split
    # an f16 output row and a float LSE per column and part: prefix and own rows are two parts at least
    assert p(3, 2, 32, 100, 4, 256) >= 3 * 2 * 32 * 2 * (512 * 2 + 4)
    assert p(3, 2, 32, 0, 4, 32) == 0
    # a table that holds less than the window bounds the rows
    assert w(1, 1, 16, 2, 0, 10 ** 9) == w(1, 1, 16, 2, 0, 128)
    assert w(2, 3, 16, 1 << 25, 2 ** 31 - 1, 2 ** 31 - 1) > 0
