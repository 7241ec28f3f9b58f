"""Host-side validation of prompt attention, residual + norm in 8 bits and
products with 4-bit weights.

CPU only: every call here fails validation, is a no-op, or is a pure host
query; the pointers are never dereferenced."""
import ctypes as C

import pytest

from test_abi_operators import BIG, FAKE, INVALID, ODD, TOO_SMALL, UNSUPPORTED, call, m  # noqa: F401

NAN, INF = float("nan"), float("inf")
MORE = C.c_void_p(0x20000)

ATTENTION = dict(q=FAKE, qt=20 * 192, qh=192, k=FAKE, kt=16 * 320, kh=320, v=FAKE, vt=16 * 320, vh=320, qs=FAKE, ks=FAKE,
                 batch=2, nq=100, nk=100, heads=16, kv_heads=16, dk=192, dv=128, causal=1, scale=0.07, out=MORE,
                 ot=16 * 128, oh=128, lse=None, ws=None, ws_bytes=0)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, INVALID) for k in ("q", "k", "v", "qs", "ks", "out")],
    *[({k: ODD}, INVALID) for k in ("q", "k", "v", "qs", "ks", "out", "lse")],
    *[({k: 4}, INVALID) for k in ("qt", "qh", "kt", "kh", "vt", "vh", "ot", "oh")],
    *[({k: -1}, INVALID) for k in ("batch", "nq", "nk", "heads", "kv_heads", "dk", "dv")],
    (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(kv_heads=32), INVALID),
    (dict(dk=4), INVALID), (dict(dk=100), INVALID), (dict(dv=12), INVALID), (dict(dk=200), UNSUPPORTED),
    (dict(dv=136), UNSUPPORTED), (dict(heads=129, kv_heads=1), UNSUPPORTED), (dict(nq=2 ** 31), UNSUPPORTED),
    (dict(nk=2 ** 31), UNSUPPORTED), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(ot=0), INVALID), (dict(oh=120), INVALID), (dict(ot=128, oh=128), INVALID),  # rows of out that overlap
    (dict(nq=2 ** 27, heads=64, kv_heads=64, ot=64 * 128), UNSUPPORTED),  # 2^33 rows
    # few rows over many keys are split: the partials need a workspace
    (dict(nq=2, nk=10 ** 6), TOO_SMALL), (dict(nq=2, nk=10 ** 6, ws=FAKE, ws_bytes=64), TOO_SMALL),
    (dict(nq=2, nk=10 ** 6, ws=None, ws_bytes=BIG), INVALID),
    (dict(nq=2, nk=10 ** 6, ws=C.c_void_p(0x10080), ws_bytes=BIG), INVALID),
    (dict(batch=0), 0), (dict(nq=0), 0), (dict(nq=0, q=None, k=None, v=None, qs=None, ks=None, out=None), 0),
])
def test_prompt_attention(m, over, status):  # noqa: F811
    assert call(m, "mla_prompt_attention", ATTENTION, over) == status


def test_prompt_attention_workspace(m):  # noqa: F811
    size = m.mla_prompt_attention_workspace_size
    for bad in [(0, 5, 1, 4, 4, 64), (5, -1, 1, 4, 4, 64), (5, 5, 0, 4, 4, 64), (5, 5, 1, 4, 3, 64), (5, 5, 1, 4, 0, 64),
                (5, 5, 1, 0, 1, 64), (5, 5, 1, 129, 1, 64), (5, 5, 1, 4, 4, 0), (2 ** 31, 5, 1, 4, 4, 64)]:
        assert size(*bad) == 0
    assert size(10, 100, 1, 4, 4, 64) == 0            # one tile of keys
    assert size(100000, 100000, 1, 64, 64, 128) == 0  # rows that fill the machine
    assert size(3, 0, 3, 4, 4, 64) == 0
    # two slices at least, each a float row and an LSE
    assert size(32, 10 ** 6, 32, 8, 1, 128) >= 32 * 8 * 2 * 129 * 4


NORM = dict(x=FAKE, xs=6144, kind=1, res=MORE, rs=6144, out=MORE, os=6144, w=FAKE, n=3, dim=6144, group=128, eps=1e-6,
            codes=FAKE, scales=FAKE)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, INVALID) for k in ("x", "res", "out", "w", "codes", "scales")],
    *[({k: ODD}, INVALID) for k in ("x", "res", "out", "w", "codes", "scales")],
    (dict(n=-1), INVALID), (dict(dim=0), INVALID), (dict(dim=12), INVALID), (dict(dim=16392), UNSUPPORTED),
    (dict(kind=3), INVALID), (dict(kind=-1), INVALID), (dict(group=-128), INVALID), (dict(group=100), INVALID),
    (dict(group=64), UNSUPPORTED), (dict(group=256), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(xs=6148), INVALID), (dict(rs=6148), INVALID),
    (dict(os=6148), INVALID), (dict(os=6136), INVALID), (dict(rs=6152), INVALID),  # in place with another stride
    (dict(kind=2, rs=6146, res=FAKE), INVALID), (dict(kind=2, os=6146, res=FAKE), INVALID),
    (dict(n=0), 0), (dict(n=0, x=None, res=None, out=None, w=None, codes=None, scales=None), 0),
])
def test_add_norm_quant(m, over, status):  # noqa: F811
    assert call(m, "mla_add_norm_quant", NORM, over) == status


MATVEC = dict(x=FAKE, kind=0, xt=16 * 192, xg=192, xs=None, xsg=0, codes=FAKE, scales=FAKE, ws=FAKE, n=4, groups=16, rows=512,
              k=128, out=FAKE, out_kind=0, ot=16 * 512, og=512)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, INVALID) for k in ("x", "codes", "scales", "out")],
    *[({k: C.c_void_p(0x10001)}, INVALID) for k in ("x", "codes", "scales", "ws", "out")],
    *[({k: -1}, INVALID) for k in ("n", "groups", "rows", "k")],
    (dict(x=ODD), INVALID), (dict(codes=C.c_void_p(0x10008)), INVALID), (dict(ws=ODD), INVALID),
    (dict(k=0), INVALID), (dict(k=40), INVALID), (dict(k=48), UNSUPPORTED), (dict(kind=2), INVALID), (dict(kind=-1), INVALID),
    (dict(out_kind=2), INVALID), (dict(out_kind=1, out=ODD), INVALID), (dict(xt=4), INVALID), (dict(xg=4), INVALID),
    (dict(kind=1, xs=FAKE, xsg=1, xt=16 * 192 + 8), INVALID), (dict(kind=1, xs=FAKE, xsg=1, xg=200), INVALID),
    (dict(kind=1, xs=None, xsg=1), INVALID), (dict(kind=1, xs=ODD, xsg=1), INVALID), (dict(kind=1, xs=FAKE, xsg=2), INVALID),
    (dict(kind=1, xs=FAKE, xsg=0), INVALID), (dict(kind=1, xs=FAKE, xsg=2, k=384, xg=384, xt=16 * 384), INVALID),
    (dict(groups=65536), UNSUPPORTED), (dict(n=2 ** 22), UNSUPPORTED),
    (dict(ot=0), INVALID), (dict(og=500), INVALID), (dict(ot=512, og=512), INVALID),  # rows of out that overlap
    (dict(n=0), 0), (dict(groups=0), 0), (dict(rows=0), 0),
    (dict(n=0, x=None, codes=None, scales=None, ws=None, out=None), 0),
])
def test_fp4_matvec(m, over, status):  # noqa: F811
    assert call(m, "mla_fp4_matvec", MATVEC, over) == status


@pytest.mark.parametrize("over,status", [
    *[({k: 0}, UNSUPPORTED) for k in ("qt", "qh", "kt", "kh", "vt", "vh")],  # an axis that is repeated
    *[({k: 184}, UNSUPPORTED) for k in ("qt", "qh", "kt", "kh")], *[({k: 120}, UNSUPPORTED) for k in ("vt", "vh")],
    *[({k: -1024}, UNSUPPORTED) for k in ("qt", "qh", "kt", "kh", "vt", "vh")],
    # what is not used is not looked at
    (dict(kv_heads=1, kh=0, vh=0, nq=2, nk=10 ** 6), TOO_SMALL), (dict(nk=1, kt=0, vt=0, kh=4), INVALID),
    (dict(nk=1, kt=0, vt=0, kh=0), UNSUPPORTED),
])
def test_prompt_attention_strides(m, over, status):  # noqa: F811
    assert call(m, "mla_prompt_attention", ATTENTION, over) == status


LARGE = 2 ** 31 - 256  # tokens, sequences


@pytest.mark.parametrize("over,status", [
    # sequences whose search would leave 32 bits
    *[(dict(batch=2 ** 31 - n, nq=1, nk=1, heads=1, kv_heads=1), UNSUPPORTED) for n in (1, 20, 32, 255)],
    # units of work: sequences x key heads x slices that are 0 or a few modulo 2^64
    (dict(batch=2 ** 30, nq=1, nk=LARGE, heads=2 ** 30, kv_heads=2 ** 30, qt=2 ** 39, kt=2 ** 39, vt=2 ** 39), UNSUPPORTED),
    (dict(batch=2 ** 30 + 1, nq=1, nk=LARGE, heads=2 ** 30, kv_heads=2 ** 30, qt=2 ** 39, kt=2 ** 39, vt=2 ** 39), UNSUPPORTED),
    (dict(batch=2 ** 16, nq=1, nk=1, heads=2 ** 15, kv_heads=2 ** 15), UNSUPPORTED),
    (dict(batch=LARGE + 1, nq=0), 0),
])
def test_prompt_attention_largest_sizes(m, over, status):  # noqa: F811
    assert call(m, "mla_prompt_attention", ATTENTION, over) == status


def test_prompt_attention_workspace_of_refused_sizes(m):  # noqa: F811
    size = m.mla_prompt_attention_workspace_size
    assert size(1, LARGE, LARGE + 1, 1, 1, 64) == 0
    assert size(1, LARGE, 2 ** 30, 2 ** 30, 2 ** 30, 64) == 0
    assert size(2 ** 27, LARGE, 1, 64, 64, 64) == 0
