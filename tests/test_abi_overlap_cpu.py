"""Outputs that share memory with themselves or with other arguments are refused before anything touches the
device (the pointers are made up): the operators' blocks would race."""

import ctypes

import numpy as np
import pytest

from bit_quantized_linear_hadamard_b200 import binding
from bit_quantized_linear_hadamard_b200 import build as qs_build

PTR, OVERLAP = 8, 10  # PTR: all checks but that of device memory passed
KB, MB = 1 << 10, 1 << 20


@pytest.fixture(scope="module")
def lib():
    qs_build.build()
    return binding.load()


def at(n):
    return ctypes.c_void_p(n * MB)


def st(batch, row, head):
    return ctypes.byref(binding._Strides(batch, row, head))


def rope(lib, x=at(1), y=at(64), xs=(1024, 128), ys=(1024, 128), rows=50, heads=8, pos=at(128), inv=at(129), axis=None, dtype=0):
    return lib.qs_rope(x, *xs, rows, heads, 128, 64, pos, 1, axis, inv, 1.0, 1, dtype, y, *ys, None)


def test_status_has_a_string(lib):
    assert b"unknown" not in lib.qs_status_str(OVERLAP) and binding.STATUS[OVERLAP] == "QS_ERR_OVERLAP"


@pytest.mark.parametrize("want,kw", [
    (PTR, {}), (PTR, dict(y=at(1))),                                     # apart; in place
    (OVERLAP, dict(y=at(1), ys=(2048, 128))),                            # in place with other strides
    (OVERLAP, dict(y=ctypes.c_void_p(MB + 2))), (OVERLAP, dict(y=ctypes.c_void_p(MB + 256))),
    (OVERLAP, dict(y=ctypes.c_void_p(MB - 2 * 127))), (PTR, dict(y=ctypes.c_void_p(MB + 50 * 2048))),
    (OVERLAP, dict(ys=(1000, 128))), (OVERLAP, dict(ys=(1024, 120))), (OVERLAP, dict(ys=(1024, 64))),
    (PTR, dict(ys=(128, 50 * 128))), (OVERLAP, dict(ys=(128, 50 * 128 - 1))), (OVERLAP, dict(ys=(128, 128))),
    # query and key heads of one row into the value heads' place, and one head too far
    (PTR, dict(y=ctypes.c_void_p(MB + 2048), xs=(3072 + 64, 128), ys=(3072 + 64, 128))),
    (OVERLAP, dict(y=ctypes.c_void_p(MB + 2048 - 256), xs=(3072 + 64, 128), ys=(3072 + 64, 128))),
    # every second head
    (PTR, dict(y=ctypes.c_void_p(MB + 256), xs=(2048, 256), ys=(2048, 256))),
    (OVERLAP, dict(y=ctypes.c_void_p(MB + 254), xs=(2048, 256), ys=(2048, 256))),
    (OVERLAP, dict(pos=at(64))), (OVERLAP, dict(inv=ctypes.c_void_p(64 * MB + 512))), (OVERLAP, dict(axis=at(64))),
    (PTR, dict(rows=1, heads=1, ys=(7, 7))),                             # strides of one row and head do not matter
    (OVERLAP, dict(dtype=2, ys=(1024, 64))), (PTR, dict(dtype=2, ys=(2000, 200)))])
def test_rope(lib, want, kw):
    assert rope(lib, **kw) == want


def test_rope_reach(lib):
    assert rope(lib, ys=(1 << 46, 128)) == 5 and rope(lib, xs=(1024, 1 << 44)) == 5


def lora(lib, **kw):
    a = dict(x=at(1), y=at(2), M=64, K=256, N=64, a=at(3), b=at(4), scale=None, adapters=2, R=16, start=at(5), ids=at(6),
             requests=2, ws=at(7), ws_bytes=MB, out=at(2), stream=None)
    a.update(kw)
    return lib.qs_lora_add(*a.values())


@pytest.mark.parametrize("want,kw", [
    (PTR, {}), (PTR, dict(out=at(8))), (OVERLAP, dict(out=at(1))), (OVERLAP, dict(out=ctypes.c_void_p(2 * MB + 128))),
    (PTR, dict(out=ctypes.c_void_p(2 * MB + 64 * 64 * 2))), (OVERLAP, dict(out=ctypes.c_void_p(2 * MB - 16))),
    (OVERLAP, dict(out=at(3))), (OVERLAP, dict(out=ctypes.c_void_p(4 * MB + 16))), (OVERLAP, dict(out=at(5))),
    (OVERLAP, dict(out=at(6))), (OVERLAP, dict(scale=at(2))), (OVERLAP, dict(ws=at(2))), (OVERLAP, dict(ws=at(1))),
    (OVERLAP, dict(ws=at(5))), (OVERLAP, dict(ws=at(8), out=at(8))), (OVERLAP, dict(ws=at(4)))])
def test_lora(lib, want, kw):
    assert lora(lib, **kw) == want


def test_block_means(lib):
    def f(x, strides, means, lens=None):
        return lib.qs_block_means(x, st(*strides), 2, 100, 3, 128, 0, lens, 0, means, None)
    assert f(at(1), (38400, 384, 128), at(2)) == PTR
    assert f(at(1), (38400, 384, 128), ctypes.c_void_p(MB + 64)) == OVERLAP
    assert f(at(1), (0, 384, 128), ctypes.c_void_p(MB + 76800)) == PTR     # one sequence for both
    assert f(at(1), (38400, 384, 128), at(2), at(2)) == OVERLAP


def select(lib, **kw):
    a = dict(q=at(1), st=st(38400, 384, 128), B=2, Lq=100, Hq=3, D=128, dtype=0, means=at(2), Lk=640, Hkv=1, ql=None, kl=None,
             T=4, first=0, last=0, flags=0, ws=None, ws_bytes=0, blocks=at(3), stream=None)
    a.update(kw)
    return lib.qs_block_select(*a.values())


@pytest.mark.parametrize("want,kw", [
    (PTR, {}), (OVERLAP, dict(blocks=at(1))), (OVERLAP, dict(blocks=at(2))), (OVERLAP, dict(ql=at(3))), (OVERLAP, dict(kl=at(3))),
    (PTR, dict(ws=at(3)))])  # no workspace is needed: it is not touched
def test_block_select(lib, want, kw):
    assert select(lib, **kw) == want


def test_block_select_workspace(lib):
    big = dict(q=at(1), st=st(1 << 30, 40 * 128, 128), B=1, Lq=32760, Hq=40, means=at(2000), Lk=640, Hkv=40, blocks=at(2100),
               ws=at(2200), ws_bytes=64 * MB)
    assert select(lib, **big) == PTR
    for p in (at(100), at(2000), at(2100)):
        assert select(lib, **{**big, "ws": p}) == OVERLAP


def attention(lib, **kw):
    a = dict(q=at(1), qs=st(38400, 384, 128), k=at(2), ks=st(0, 128, 0), v=at(3), vs=st(0, 128, 0), B=2, Lq=100, Lk=640, Hq=3,
             Hkv=3, D=128, dtype=0, blocks=at(4), T=10, ql=None, kl=None, scale=0.1, flags=0, ws=at(5), ws_bytes=1 << 30,
             out=at(4096), os=st(38400, 384, 128), lse=at(8192), stream=None)
    a.update(kw)
    return lib.qs_block_attention(*a.values())


@pytest.mark.parametrize("want,kw", [
    (PTR, {}), (PTR, dict(lse=None)), *[(OVERLAP, dict(out=at(i))) for i in (1, 2, 3, 4, 5)], (OVERLAP, dict(out=at(8192))),
    *[(OVERLAP, dict(lse=at(i))) for i in (1, 2, 3, 4, 5)], *[(OVERLAP, dict(ws=at(i))) for i in (1, 2, 3, 4)],
    (OVERLAP, dict(ql=at(4096))), (OVERLAP, dict(kl=at(8192))), (OVERLAP, dict(ql=at(5))),
    (OVERLAP, dict(os=st(38400, 376, 128))), (OVERLAP, dict(os=st(38392, 384, 128))), (OVERLAP, dict(os=st(38400, 384, 120))),
    (PTR, dict(os=st(38400, 128, 12800))), (OVERLAP, dict(os=st(38400, 128, 12792))),
    # into the wider row that q lies in, beside it, and one head into it
    (PTR, dict(qs=st(76800, 768, 128), out=ctypes.c_void_p(MB + 768), os=st(76800, 768, 128))),
    (OVERLAP, dict(qs=st(76800, 768, 128), out=ctypes.c_void_p(MB + 512), os=st(76800, 768, 128)))])
def test_attention(lib, want, kw):
    assert attention(lib, **kw) == want


def test_views_against_every_element(lib):
    """Random small rows and heads: refused exactly where an element is shared."""
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(3000):
        rows, heads = (int(rng.integers(1, 5)) for _ in range(2))
        xs, ys = ([int(rng.integers(1, 700)), int(rng.integers(1, 300))] for _ in range(2))
        if rng.random() < 0.5:
            ys = xs
        gap = int(rng.integers(0, 1500))
        el = lambda base, s: [base + r * s[0] + h * s[1] + e for r in range(rows) for h in range(heads) for e in range(128)]  # noqa: E731
        ex, ey = el(0, xs), el(gap, ys)
        same = gap == 0 and all(n == 1 or a == b for n, a, b in zip((rows, heads), xs, ys))
        bad = len(set(ey)) < len(ey) or (not same and bool(set(ex) & set(ey)))
        assert rope(lib, y=ctypes.c_void_p(MB + 2 * gap), xs=xs, ys=ys, rows=rows, heads=heads) == (OVERLAP if bad else PTR)
        seen.add(bad)
    assert seen == {True, False}
