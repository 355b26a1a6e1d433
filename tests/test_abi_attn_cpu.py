"""Refusals of the operators around the projections, without a GPU: every bad argument gives its
documented status before anything touches the device (the pointers are made up)."""

import ctypes
import math

import pytest
import torch

import bit_quantized_linear_hadamard_b200 as qs
from bit_quantized_linear_hadamard_b200 import binding
from bit_quantized_linear_hadamard_b200 import build as qs_build

OK, NULL, SHAPE, BITS, ALIGN, RANGE, CUDA, TIMEOUT, PTR, DTYPE = range(10)
A, B, C, D, E = (ctypes.c_void_p(0x10000 * i) for i in range(1, 6))
MIS, ODD = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def lib():
    qs_build.build()
    return binding.load()


def st(batch=1 << 20, row=128, head=1 << 14):
    return ctypes.byref(binding._Strides(batch, row, head))


def test_dtype_has_a_status_string(lib):
    assert lib.qs_status_str(DTYPE) and b"unknown" not in lib.qs_status_str(DTYPE)


def rope_args(**kw):
    a = dict(x=A, xr=256, xh=128, rows=4, heads=2, dim=128, rot=128, pos=B, axes=1, axis=None, inv=C, scale=1.0, flags=1,
             dtype=0, y=D, yr=256, yh=128, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(pos=None)), (NULL, dict(inv=None)), (NULL, dict(y=None)),
    (DTYPE, dict(dtype=3)), (DTYPE, dict(dtype=-1)),
    (SHAPE, dict(rows=0)), (SHAPE, dict(heads=0)), (SHAPE, dict(dim=0)), (SHAPE, dict(rot=0)), (SHAPE, dict(rot=3)),
    (SHAPE, dict(rot=130)), (SHAPE, dict(yr=0)), (SHAPE, dict(yh=0)), (SHAPE, dict(xr=-1)),
    (RANGE, dict(axes=0)), (RANGE, dict(axes=9)), (RANGE, dict(dim=1026)), (RANGE, dict(heads=65536)),
    (RANGE, dict(flags=4)), (RANGE, dict(scale=math.inf)), (RANGE, dict(scale=math.nan)),
    (ALIGN, dict(x=ODD)), (ALIGN, dict(pos=ctypes.c_void_p(0x10004))), (ALIGN, dict(inv=ctypes.c_void_p(0x10004))),
    (ALIGN, dict(axis=ctypes.c_void_p(0x10002))), (ALIGN, dict(dtype=2, x=ctypes.c_void_p(0x10002))),
])
def test_rope_refusals(lib, want, kw):
    assert lib.qs_rope(*rope_args(**kw)) == want


def lora_args(**kw):
    a = dict(x=A, y=B, M=64, K=256, N=64, a=C, b=D, scale=None, adapters=2, R=16, start=E, ids=E, requests=2, ws=A,
             ws_bytes=1 << 30, out=B, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("want,kw", [
    *[(NULL, {k: None}) for k in ("x", "y", "a", "b", "start", "ids", "ws", "out")],
    (SHAPE, dict(M=0)), (SHAPE, dict(K=200)), (SHAPE, dict(N=24)), (SHAPE, dict(N=0)), (SHAPE, dict(R=4)), (SHAPE, dict(R=20)),
    (SHAPE, dict(adapters=0)), (SHAPE, dict(requests=0)), (RANGE, dict(R=136)), (RANGE, dict(K=65536 + 128)),
    (RANGE, dict(adapters=1 << 28)), (RANGE, dict(ws_bytes=16)),
    (ALIGN, dict(x=MIS)), (ALIGN, dict(out=MIS)), (ALIGN, dict(ws=MIS)),
])
def test_lora_refusals(lib, want, kw):
    assert lib.qs_lora_add(*lora_args(**kw)) == want


def test_lora_workspace(lib):
    f = lib.qs_lora_workspace_bytes
    assert f(0, 256, 16, 1) == f(8, 200, 16, 1) == f(8, 256, 12, 1) == f(8, 256, 136, 1) == f(8, 256, 16, 0) == -1
    for M, K, R, n in ((1, 128, 8, 1), (64, 5120, 16, 64), (4099, 13824, 32, 9), (32760, 5120, 128, 2)):
        need = f(M, K, R, n)
        assert need >= 4 * M * R and need % (4 * M * R) == 0


def means_args(**kw):
    a = dict(x=A, st=st(), B=2, L=100, H=2, D=128, dtype=0, len=None, first=0, means=B, stream=None)
    a.update(kw)
    return list(a.values())


VIEWS = [(DTYPE, dict(dtype=2)), (SHAPE, dict(D=96)), (SHAPE, dict(B=0)), (RANGE, dict(B=65536)),
         (ALIGN, dict(st=st(row=132))), (SHAPE, dict(st=st(row=0))), (SHAPE, dict(st=st(head=-8))), (RANGE, dict(st=st(batch=1 << 39)))]


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(st=None)), (NULL, dict(means=None)), (ALIGN, dict(x=MIS)), (SHAPE, dict(L=0)),
    (RANGE, dict(L=(1 << 24) + 1)), *VIEWS])
def test_means_refusals(lib, want, kw):
    assert lib.qs_block_means(*means_args(**kw)) == want


def select_args(**kw):
    a = dict(q=A, st=st(), B=2, Lq=100, Hq=4, D=128, dtype=0, means=B, Lk=640, Hkv=2, ql=None, kl=None, T=4, first=0, last=0,
             flags=0, ws=None, ws_bytes=0, blocks=C, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(q=None)), (NULL, dict(st=None)), (NULL, dict(means=None)), (NULL, dict(blocks=None)), *VIEWS])
def test_select_refusals_of_views(lib, want, kw):
    assert lib.qs_block_select(*select_args(**kw)) == want


def attention_args(**kw):
    a = dict(q=A, qs=st(), k=B, ks=st(), v=C, vs=st(), B=2, Lq=100, Lk=640, Hq=4, Hkv=2, D=128, dtype=0, blocks=D, T=4, ql=None,
             kl=None, scale=0.1, flags=0, ws=E, ws_bytes=1 << 30, out=A, os=st(), lse=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("want,kw", [
    *[(NULL, {k: None}) for k in ("q", "qs", "k", "ks", "v", "vs", "blocks", "out", "os")],
    (DTYPE, dict(dtype=2)), (SHAPE, dict(D=32)), (SHAPE, dict(Lq=0)), (ALIGN, dict(q=MIS)), (ALIGN, dict(qs=st(head=12)))])
def test_attention_refusals_of_views(lib, want, kw):
    assert lib.qs_block_attention(*attention_args(**kw)) == want


def test_attention_workspace(lib):
    f = lib.qs_block_attention_workspace_bytes
    assert f(0, 1, 1, 64, 1) == f(1, 0, 1, 64, 1) == f(1, 1, 0, 64, 1) == f(1, 1, 1, 96, 1) == f(1, 1, 1, 64, 0) == -1
    assert f(1, 32760, 40, 128, 77) == 0           # enough query blocks: the lists stay whole
    assert f(1, 1, 40, 128, 77) > 0                # a single token: they are cut
    assert f(1, 1, 40, 128, 77) % (40 * 129 * 4) == 0
    g = lib.qs_block_select_workspace_bytes
    assert g(1, 0, 1, 64) == g(1, 1, 1, 32) == -1 and g(1, 1, 40, 128) == 0 and g(1, 32760, 40, 128) == 40 * 256 * 128 * 4


def test_python_refusals():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(TypeError):
        qs.rope(x, torch.zeros(2, dtype=torch.int64), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(TypeError):
        qs.block_means(torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        qs.lora_add(torch.zeros(2, 16), torch.zeros(2, 128), torch.zeros(1, 8, 256), torch.zeros(1, 16, 8),
                    torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_rope_frequencies():
    inv, axis, scale = qs.rope_frequencies(8, theta=10000.0, device="cpu")
    assert axis is None and scale == 1.0 and inv.dtype == torch.float64
    assert torch.allclose(inv, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    inv, axis, _ = qs.rope_frequencies(128, axes=(44, 42, 42), device="cpu")
    assert inv.shape == (64,) and axis.tolist() == [0] * 22 + [1] * 21 + [2] * 21 and inv[0] == inv[22] == inv[43] == 1.0
    base, _, _ = qs.rope_frequencies(64, device="cpu")
    lin, _, _ = qs.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, base / 4, rtol=1e-15)
    ntk, _, _ = qs.rope_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and abs(ntk[-1] / base[-1] * 4 - 1) < 1e-12
    yarn, _, scale = qs.rope_frequencies(64, scaling="yarn", factor=8.0, device="cpu")
    assert yarn[0] == base[0] and torch.allclose(yarn[-1], base[-1] / 8, rtol=1e-14)
    assert abs(scale - (0.1 * math.log(8) + 1)) < 1e-15
    ratio = yarn / base
    assert (ratio[1:] <= ratio[:-1] + 1e-15).all()
    for bad in (dict(rot_dim=7), dict(rot_dim=8, axes=(4, 2)), dict(rot_dim=8, axes=(5, 3)), dict(rot_dim=8, scaling="x"),
                dict(rot_dim=8, scaling="linear", factor=0.5), dict(rot_dim=8, axes=(4, 4), scaling="ntk")):
        with pytest.raises(ValueError):
            qs.rope_frequencies(device="cpu", **bad)
