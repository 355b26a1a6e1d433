"""The operators around the quantised projections against their binary64 forms.

Tolerances (u = 2^-24, half a step of binary32; e = half a step of the output's type):
  rope       sine and cosine: 2 ulp of CUDA's sincosf, the first-order correction, the scale's
             rounding and product: 4 u * scale; the two products and their sum: 2 u.  So
             e |y| + 6 u scale (|u| + |v|), and half of the type's smallest step near 0.
  lora       every summation of n binary32 terms is off by at most n 2 u of the sum of their
             magnitudes (the tensor cores may truncate: 2 u per addition): K + R + 8 terms, and 2^-17
             for the inner sum as two bf16 numbers.  So e |out| + (2 u (K + R + 8) + 2^-17) size.
  attention  scores: D additions, 2 u each, of sum |q||k| scale; the exponent's product and sum:
             u of the running maximum and of itself, each at most c = max |score|; exp2: 2^-22.
             w = 2 u (D c1 + 4 c) + 2^-22 is the relative error of a p, with c1 = scale max
             sum |q||k|.  P's rounding: e.  So e |out| + (e + 2 w + 2 u (n + 8)) size over n keys,
             and n 2^-25 max |v| for fp16's subnormal p.
  lse        w + 2 u (n + 4) + 4 u |lse| (the sum's additions; the logarithm and its product).
"""

import math

import numpy as np
import pytest
import torch

import bit_quantized_linear_hadamard_b200 as qs
from bit_quantized_linear_hadamard_b200 import build as qs_build
from oracle import attn_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qs_build.build()
    qs.load()
    yield
    assert qs.qs_device_error() == 0


def half(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(seed, *shape, dtype=BF16, by=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * by).to(dtype).cuda()


def close(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, what
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= tol)
    bad &= ~(got == want)  # infinities
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {want[bad][0]}"


# ------------------------------------------------------------------------------------- rope

def check_rope(x, pos, inv, axis, inter, scale, inverse=False, out=None):
    want = O.rope(f64(x), pos.cpu().numpy(), inv.cpu().numpy(), None if axis is None else axis.cpu().numpy(),
                  inter, scale, inverse)
    before = f64(x)
    got = qs.rope(x, pos, inv, axis, inter, scale, inverse, out=out)
    n = inv.numel()
    tol = half(x.dtype) * np.abs(want) + torch.finfo(x.dtype).smallest_normal * half(x.dtype)
    for p in range(n):
        i, j = (2 * p, 2 * p + 1) if inter else (p, p + n)
        size = 6 * U * scale * (np.abs(before[:, :, i]) + np.abs(before[:, :, j]))
        tol[:, :, i] += size
        tol[:, :, j] += size
    tol[:, :, 2 * n:] = 0.0
    close(got, want, tol, "rope")
    return got


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("rows,heads,dim,rot", [(1, 1, 2, 2), (1, 80, 128, 128), (3, 5, 128, 64), (300, 3, 64, 48),
                                                (7, 4, 80, 80), (5, 2, 34, 30), (2, 2, 700, 700), (40, 17, 96, 6)])
def test_rope(dtype, inter, rows, heads, dim, rot):
    x = randn(rows + dim, rows, heads, dim, dtype=dtype, by=3.0)
    inv, _, _ = qs.rope_frequencies(rot)
    pos = torch.arange(rows, device="cuda") * 977 + 12345
    got = check_rope(x, pos, inv, None, inter, 1.0)
    # the inverse brings x back within two roundings; in place is the same as into a new tensor
    back = qs.rope(got, pos, inv, None, inter, 1.0, inverse=True)
    # each output was off by e |y|; turning it back adds e of the result and the factors' 12 u
    size = f64(x).copy()
    n = rot // 2
    for p in range(n):
        i, j = (2 * p, 2 * p + 1) if inter else (p, p + n)
        size[:, :, i] = size[:, :, j] = np.abs(f64(x)[:, :, i]) + np.abs(f64(x)[:, :, j])
    e = half(dtype)
    close(back, f64(x), (2.1 * e + 16 * U) * 1.5 * np.abs(size) + 2 * torch.finfo(dtype).smallest_normal * e, "inverse")
    same = x.clone()
    qs.rope(same, pos, inv, None, inter, 1.0, out=same)
    assert torch.equal(same, got)


@pytest.mark.parametrize("inter", [True, False])
def test_rope_views_axes_and_far_positions(inter):
    """Query and key heads of a qkv row, three axes, positions to 10^9, scaled frequencies."""
    rows, heads, dim = 77, 6, 128
    qkv = randn(5, rows, (heads + 3) * dim)
    x = qkv[:, : heads * dim].view(rows, heads, dim)
    inv, axis, _ = qs.rope_frequencies(dim, axes=(44, 42, 42))
    pos = torch.randint(0, 10 ** 9, (rows, 3), generator=torch.Generator().manual_seed(1)).cuda()
    pos[3] = -pos[3]
    got = check_rope(x, pos, inv, axis, inter, 1.0)
    keep = qkv.clone()
    check_rope(x, pos, inv, axis, inter, 1.0, out=x)
    assert torch.equal(x, got) and torch.equal(qkv[:, heads * dim :], keep[:, heads * dim :])
    inv, _, scale = qs.rope_frequencies(64, scaling="yarn", factor=32.0)
    check_rope(randn(6, 9, 2, dim), torch.arange(9, device="cuda") + 10 ** 6, inv, None, inter, scale)


@pytest.mark.parametrize("dtype,offset,row", [(BF16, 1, 513), (F16, 8, 520), (F32, 2, 514)])
def test_rope_any_alignment_and_order(dtype, offset, row):
    """Element alignment, odd strides, heads-first order; what lies between the views stays."""
    base = randn(9, offset + 20 * row, dtype=dtype)
    x = base[offset:].as_strided((20, 4, 128), (row, 128, 1), offset)
    inv, _, _ = qs.rope_frequencies(128)
    pos = torch.arange(20, device="cuda") + 3
    out = torch.full((4, 20, 128), -7.0, dtype=dtype, device="cuda")
    check_rope(x, pos, inv, None, True, 1.0, out=out.transpose(0, 1))
    guard = torch.full((20, 4, 130), -7.0, dtype=dtype, device="cuda")
    check_rope(x, pos, inv, None, False, 1.0, out=guard[:, :, 1:129])
    assert (guard[:, :, 0] == -7).all() and (guard[:, :, 129] == -7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("rows,heads,dim,rot", [(1301, 5, 128, 128), (1301, 3, 64, 48), (2400, 2, 128, 48), (1211, 7, 44, 30),
                                                (1200, 1, 6, 6)])
def test_rope_more_rows_than_processors(dtype, inter, rows, heads, dim, rot):
    """Blocks of several rows, the last one not full; all heads of a row in one block."""
    x = randn(rows, rows, heads + 2, dim, dtype=dtype, by=3.0)[:, 1:-1]
    inv, axis, _ = qs.rope_frequencies(rot, axes=(rot - 4, 2, 2))
    pos = torch.randint(0, 10 ** 6, (rows, 3), generator=torch.Generator().manual_seed(rot)).cuda()
    got = check_rope(x, pos, inv, axis, inter, 1.25)
    same = x.clone()
    qs.rope(same, pos, inv, axis, inter, 1.25, out=same)
    assert torch.equal(same, got)


def test_rope_bad_axis_is_reported():
    x = randn(1, 2, 1, 8)
    inv, _, _ = qs.rope_frequencies(8)
    axis = torch.tensor([0, 5, 0, -1], dtype=torch.int32, device="cuda")
    pos = torch.arange(2, device="cuda")
    got = qs.rope(x, pos, inv, axis)
    assert qs.qs_device_error() == 5
    assert torch.equal(got, qs.rope(x, pos, inv))


# ------------------------------------------------------------------------------------- lora

def check_lora(seed, M, K, N, R, starts, ids, adapters, scaled=True, in_place=False, by=1.0):
    x, y = randn(seed, M, K), randn(seed + 1, M, N)
    a, b = randn(seed + 2, adapters, R, K, by=by / math.sqrt(K)), randn(seed + 3, adapters, N, R)
    scale = (torch.rand(adapters, generator=torch.Generator().manual_seed(seed)) + 0.5).cuda() if scaled else None
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    id_ = torch.tensor(ids, dtype=torch.int32, device="cuda")
    out = y.clone() if in_place else torch.full_like(y, -3.0)
    want, size = O.lora_add(f64(y), f64(x), f64(a), f64(b), starts, ids, None if scale is None else f64(scale), f64(out))
    got = qs.lora_add(out if in_place else y, x, a, b, st, id_, scale, out=None if in_place else out)
    assert got is out
    tol = half(BF16) * np.abs(want) + (2 * U * (K + R + 8) + 2.0 ** -17) * size
    inside = np.zeros(M, dtype=bool)
    for lo, hi in zip(starts, starts[1:]):
        inside[lo:hi] = True
    tol[~inside] = 0.0
    close(got, want, tol, "lora")


@pytest.mark.parametrize("R", [8, 16, 24, 40, 64, 72, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_lora_ragged_requests(R, in_place):
    # one row, an empty request, none, a tile and one more, rows in front and behind
    starts = [2, 3, 3, 20, 37, 166, 190]
    check_lora(R, 200, 256, 176, R, starts, [0, 1, 2, -1, 1, 0], 3, in_place=in_place)


@pytest.mark.parametrize("M,K,N,R,requests", [(1, 128, 16, 8, 1), (64, 1280, 528, 16, 64), (300, 640, 1040, 32, 1),
                                              (1000, 2560, 304, 64, 3), (333, 128, 48, 128, 333), (129, 384, 32, 96, 2)])
def test_lora_sizes(M, K, N, R, requests):
    starts = [M * i // requests for i in range(requests + 1)]
    check_lora(M, M, K, N, R, starts, [(3 * i) % 5 - 1 for i in range(requests)], 4, scaled=M % 2 == 0)


@pytest.mark.parametrize("R,M,K", [(8, 33000, 128), (16, 9300, 512), (24, 3300, 1280), (32, 2500, 1792),
                                   (40, 2000, 2176), (64, 1100, 4096), (128, 1100, 4096)])
def test_lora_long_requests(R, M, K):
    """Tiles of 128 rows at every rank: uneven lengths, rows in front, behind and without an adapter."""
    starts = [1, 2, M // 3 + 5, M // 3 + 5, M - 130, M - 2] if R > 32 else [1, M // 3 + 5, M - 130, M - 2]
    ids = [1, 0, 1, 2, -1] if R > 32 else [2, 0, -1]
    check_lora(50 + R, M, K, 80, R, starts, ids, 3, in_place=R % 16 == 0)


@pytest.mark.parametrize("R", [16, 64, 72, 128])
@pytest.mark.parametrize("M,K,N,starts", [
    (4200, 1024, 4112, [3, 700, 701, 1900, 4150]),                       # many column chunks for each tile
    (2200, 2048, 1040, [0, *range(1, 64), 2100]),                        # single tokens and one long prompt
    (300, 512, 15376, [0, 5, 100, 300])])                                # few rows, many columns
def test_lora_many_columns(R, M, K, N, starts):
    """The stages, both accumulators and the column ranges serve one chunk after another."""
    ids = [(3 * i) % 4 - 1 for i in range(len(starts) - 2)] + [1]
    check_lora(R, M, K, N, R, starts, ids, 3, in_place=R == 64)


def test_lora_update_far_larger_than_the_projection():
    check_lora(3, 40, 512, 64, 16, [0, 40], [0], 1, by=1000.0)


@pytest.mark.parametrize("M,K,N,R", [(40, 256, 80, 16), (70, 128, 48, 128), (33000, 128, 80, 16), (1100, 4096, 176, 72)])
def test_lora_infinite_weights(M, K, N, R):
    """An infinite element of B makes its column infinite, with the sign of its product with t, whether t
    is one bf16 number (then the rest of it is 0) or not, and an infinite sum of both signs is NaN; a
    NaN in x is its row's alone.  In tiles of 16 rows and of 128."""
    x, y = randn(0, M, K), randn(1, M, N)
    a, b = randn(2, 1, R, K, by=1 / math.sqrt(K)), randn(3, 1, N, R)
    x[: M // 2] = 0.0
    x[: M // 2, 5] = 2.0      # t = 2 A[:, 5]: bf16 numbers
    a[0, :3, 5] = torch.tensor([0.5, -0.25, 0.75])
    b[0, 3, 0], b[0, 7, 1], b[0, N - 1, 2] = float("inf"), float("inf"), -float("inf")
    b[0, 20, 0], b[0, 20, 1] = float("inf"), float("inf")
    b[0, 30, 4] = float("nan")
    x[M - 2, 9] = float("nan")
    st = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    with np.errstate(invalid="ignore"):
        want, size = O.lora_add(f64(y), f64(x), f64(a), f64(b), [0, M], [0])
    got = qs.lora_add(y, x, a, b, st, torch.zeros(1, dtype=torch.int32, device="cuda"), out=torch.empty_like(y))
    nan = np.isnan(want)
    assert nan[M - 2].all() and nan[:, 30].all() and nan[: M // 2, 20].all() and nan.sum() < M * N // 4
    assert np.array_equal(np.isnan(f64(got)), nan)
    inf = np.isinf(want)
    assert inf[: M // 2, [3, 7, N - 1]].all() and (want[: M // 2, 7] < 0).all()
    assert np.array_equal(f64(got)[inf], want[inf])
    fin = ~(nan | inf)
    tol = half(BF16) * np.abs(want) + (2 * U * (K + R + 8) + 2.0 ** -17) * size
    assert (np.abs(f64(got)[fin] - want[fin]) <= tol[fin]).all()


def test_lora_many_requests():
    """More requests than a block has threads; most rows in small tiles, empty ones between."""
    rng = np.random.default_rng(0)
    starts = np.sort(rng.integers(0, 2000, 701))
    starts[0], starts[-1] = 1, 1990
    check_lora(5, 2000, 128, 48, 8, starts.tolist(), rng.integers(-1, 3, 700).tolist(), 3)
    # 200 requests of 70 rows and more on average: large tiles, more of them than the threads that look
    starts = np.sort(rng.integers(0, 15000, 201))
    starts[0], starts[-1] = 0, 15000
    check_lora(6, 15000, 384, 48, 40, starts.tolist(), rng.integers(-1, 3, 200).tolist(), 3)


def test_lora_again_and_in_a_row():
    """The second kernel of a call runs into the first's time: calls that follow each other at once,
    each on the last one's output, with adapters in some rows only."""
    x, y = randn(0, 700, 1280), randn(1, 700, 528)
    a, b = randn(2, 3, 24, 1280, by=0.03), randn(3, 3, 528, 24)
    st = torch.tensor([0, 300, 301, 640], dtype=torch.int32, device="cuda")
    ids = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    want = y.clone()
    for _ in range(8):
        want = qs.lora_add(want, x, a, b, st, ids, out=want.clone())
        torch.cuda.synchronize()
    got = y.clone()
    for _ in range(8):
        qs.lora_add(got, x, a, b, st, ids)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_lora_bad_requests_are_left_out():
    x, y = randn(0, 32, 128), randn(1, 32, 32)
    a, b = randn(2, 2, 8, 128), randn(3, 2, 32, 8)
    st = torch.tensor([0, 8, 16, 40], dtype=torch.int32, device="cuda")
    id_ = torch.tensor([0, 2, 1], dtype=torch.int32, device="cuda")  # adapter 2: none such; rows to 40
    out = torch.full_like(y, -3.0)
    qs.lora_add(y, x, a, b, st, id_, out=out)
    assert qs.qs_device_error() == 5
    assert (out[8:] == -3).all()
    want, size = O.lora_add(f64(y), f64(x), f64(a), f64(b), [0, 8], [0], None, np.full((32, 32), -3.0))
    close(out, want, half(BF16) * np.abs(want) + (2 * U * 144 + 2.0 ** -17) * size, "lora")


@pytest.mark.parametrize("starts,ids", [([1000, 1010, 1011], [0, 1]), ([0, 8, 4000, 4001], [0, 1, 1]), ([32, 32, 30], [0, 1]),
                                        ([-400, -300], [0]), ([0, 0, 0], [0, 9]), ([0] * 400 + [2 ** 31 - 1], [0] * 400)])
def test_lora_every_bad_request_is_reported(starts, ids):
    """Requests whose rows no tile comes to, empty ones without an adapter, the last of many."""
    x, y = randn(0, 32, 128), randn(1, 32, 32)
    a, b = randn(2, 2, 8, 128), randn(3, 2, 32, 8)
    ints = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full_like(y, -3.0)
    qs.lora_add(y, x, a, b, ints(starts), ints(ids), out=out)
    assert qs.qs_device_error() == 5
    assert (out[8:] == -3).all()
    qs.lora_add(y, x, a, b, ints([0, 8, 8, 32]), ints([0, -1, 1]), out=out)
    assert qs.qs_device_error() == 0


# ----------------------------------------------------------------------------------- select

@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 128), (BF16, 64), (F16, 64)])
@pytest.mark.parametrize("B,L,H,lens", [(1, 1, 1, None), (2, 64, 3, None), (1, 65, 2, None), (3, 500, 5, [500, 0, 129]),
                                        (2, 1000, 1, [64, 999])])
def test_block_means(dtype, D, B, L, H, lens):
    x = randn(L, B, L, H, D, dtype=dtype)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = O.block_means(f64(x), lens)
    if lens is not None:  # what lies behind a length is never used
        for b, n in enumerate(lens):
            x[b, n:] = float("nan")
    got = qs.block_means(x, ln)
    assert np.array_equal(got.cpu().numpy(), want)
    nb = got.shape[2]
    kept = torch.full_like(got, 5.0)
    qs.block_means(x, ln, first_block=nb - 1, out=kept)
    assert (kept[:, :, : nb - 1] == 5).all() and torch.equal(kept[:, :, nb - 1 :], got[:, :, nb - 1 :])


def check_select(seed, B, Lq, Lk, Hq, Hkv, D, T, dtype=BF16, means=None, q=None, **kw):
    q = randn(seed, B, Lq, Hq, D, dtype=dtype) if q is None else q
    if means is None:
        means = randn(seed + 1, B, Hkv, -(-Lk // 64), D, dtype=F32)
    on_host = {k: v.tolist() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    want = O.block_select(f64(q), means.cpu().numpy(), T, Lk, **on_host)
    got = qs.block_select(q, means, T, Lk, **kw)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("first,last", [(0, 0), (1, 2), (3, 100)])
@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,D,T", [(1, 1, 1, 1, 1, 128, 1), (1, 1, 3000, 4, 4, 128, 9), (2, 300, 300, 4, 2, 64, 3),
                                                (1, 129, 1111, 2, 1, 128, 5), (1, 1100, 1100, 1, 1, 128, 7),
                                                (1, 70, 200, 2, 2, 64, 9)])
def test_block_select(causal, first, last, B, Lq, Lk, Hq, Hkv, D, T):
    check_select(Lq + T, B, Lq, Lk, Hq, Hkv, D, T, first=first, last=last, causal=causal)


@pytest.mark.parametrize("causal", [False, True])
def test_block_select_lengths(causal):
    ql = torch.tensor([300, 0, 130, 1], dtype=torch.int32, device="cuda")
    kl = torch.tensor([700, 64, 100, 0], dtype=torch.int32, device="cuda")
    q = randn(3, 4, 300, 2, 128, dtype=F16)
    for b in range(4):
        q[b, int(ql[b]):] = float("inf")
    check_select(3, 4, 300, 700, 2, 1, 128, 4, causal=causal, q_len=ql, k_len=kl, last=1, q=q)


def test_block_select_ties_and_special_scores():
    """Equal scores go to the lowest index; NaN ranks last; infinities in their places."""
    q = torch.ones(1, 1, 1, 64, dtype=BF16, device="cuda")
    m = torch.zeros(1, 1, 200, 64, device="cuda")
    m[0, 0, ::7, 0] = 1.0
    m[0, 0, 5] = float("nan")
    m[0, 0, 9, 3] = float("inf")
    m[0, 0, 11, 3] = -float("inf")
    m[0, 0, 13, 3] = -1e-300  # rounds to -0: the same as 0
    for T in (1, 2, 20, 31, 33, 150, 198, 199, 200, 230):
        check_select(0, 1, 1, 200 * 64, 1, 1, 64, T, means=m, q=q)


def test_block_select_many_blocks():
    """Rows of scores that leave room for one query block per CTA."""
    check_select(8, 1, 260, 24000 * 64, 1, 1, 64, 40)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,D,B,Lq,Lk,Hq,Hkv,T,ragged", [(BF16, 128, 1, 16645, 640, 8, 2, 4, False),
                                                              (F16, 64, 2, 9000, 9000, 8, 1, 23, True)])
def test_block_select_more_query_blocks_than_are_formed_on_the_way(causal, dtype, D, B, Lq, Lk, Hq, Hkv, T, ragged):
    """Above 1024 query blocks in all their means have a kernel of their own and a workspace."""
    ql, kl = ([torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([Lq, 7001], [Lk, 8200])] if ragged else (None, None))
    assert qs.qs_block_select_workspace_bytes(B, Lq, Hq, D) > 0
    q = randn(1, B, Lq, Hq, D, dtype=dtype)
    if ragged:
        q[1, 7001:] = float("nan")
    check_select(1, B, Lq, Lk, Hq, Hkv, D, T, q=q, causal=causal, first=1, last=1, q_len=ql, k_len=kl)


# -------------------------------------------------------------------------------- attention

def some_blocks(seed, B, Hq, Lq, Lk, T, holes=True):
    """Distinct blocks in any order, with -1 among them."""
    rng = np.random.default_rng(seed)
    nq, nk = -(-Lq // 128), -(-Lk // 64)
    out = np.full((B, Hq, nq, T), -1, dtype=np.int32)
    for at in np.ndindex(B, Hq, nq):
        n = min(T, nk)
        out[at][:n] = rng.permutation(nk)[:n]
        if holes and T > 2:
            out[at][rng.integers(0, T)] = -1
    return out


def check_attention(q, k, v, blocks, scale=None, causal=False, q_len=None, k_len=None, clean=None):
    """`clean`: what the oracle sees of (q, k, v), where the operator's hold something else behind the lengths."""
    B, Lq, Hq, D = q.shape
    dtype = q.dtype
    cq, ck, cv = clean or (q, k, v)
    hq, hk, hv = f64(cq), f64(ck), f64(cv)
    out = torch.full((B, Lq, Hq, D), 9.0, dtype=dtype, device="cuda")
    lse = torch.full((B, Hq, Lq), 9.0, device="cuda")
    ints = lambda t: None if t is None else torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    want, wlse, size = O.block_attention(hq, hk, hv, blocks, scale, causal, q_len, k_len, f64(out), f64(lse))
    got, glse = qs.block_attention(q, k, v, ints(blocks), scale, causal, ints(q_len), ints(k_len), out=out, lse=lse)
    s = D ** -0.5 if scale is None else scale
    c1 = s * np.abs(hq).sum(-1).max() * np.abs(hk).max()
    c = min(c1, s * np.linalg.norm(hq, axis=-1).max() * np.linalg.norm(hk, axis=-1).max())
    w = 2 * U * (D * c1 + 4 * c) + 2.0 ** -22
    n = 64 * blocks.shape[-1]
    e = half(dtype)
    valid = np.ones((B, Lq), dtype=bool) if q_len is None else np.arange(Lq) < np.array(q_len)[:, None]
    tol = e * np.abs(want) + (e + 2 * w + 2 * U * (n + 8)) * size
    if dtype is F16:
        tol += n * 2.0 ** -25 * np.abs(hv).max()
    tol[~valid] = 0.0
    close(got, want, tol, "out")
    ltol = np.where(np.isfinite(wlse), w + 2 * U * (n + 4) + 4 * U * np.abs(wlse), 0.0)
    ltol *= valid[:, None, :]
    close(glse, wlse, ltol, "lse")
    return got, glse


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 128), (BF16, 64), (F16, 64)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,T", [(1, 1, 1, 1, 1, 1), (1, 128, 128, 1, 1, 2), (1, 128, 192, 1, 1, 3),
                                              (2, 130, 300, 2, 1, 4), (1, 5, 1000, 3, 3, 16), (1, 300, 300, 4, 2, 5),
                                              (1, 1, 2000, 2, 2, 32)])
def test_attention(dtype, D, causal, B, Lq, Lk, Hq, Hkv, T):
    q = randn(Lq, B, Lq, Hq, D, dtype=dtype, by=2.0)
    k, v = randn(Lk, B, Lk, Hkv, D, dtype=dtype), randn(Lk + 1, B, Lk, Hkv, D, dtype=dtype)
    check_attention(q, k, v, some_blocks(T, B, Hq, Lq, Lk, T), causal=causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_lengths_hide_what_lies_behind(causal, bad, D):
    ql, kl = [200, 0, 130, 7, 3], [500, 300, 65, 0, 64]
    B, Lq, Lk, H = 5, 200, 500, 2
    q, k, v = randn(0, B, Lq, H, D), randn(1, B, Lk, H, D), randn(2, B, Lk, H, D)
    clean = (q.clone(), k.clone(), v.clone())
    for b in range(B):
        q[b, ql[b]:], k[b, kl[b]:], v[b, kl[b]:] = bad, bad, bad
    blocks = some_blocks(4, B, H, Lq, Lk, 8)
    check_attention(q, k, v, blocks, causal=causal, q_len=ql, k_len=kl, clean=clean)
    check_attention(q, k, v, blocks[..., ::-1].copy(), causal=causal, q_len=ql, k_len=kl, clean=clean)


def test_attention_growing_scores_move_the_maximum():
    """Scores that rise by far more than the lazy maximum's slack from tile to tile, and fall again."""
    D, Lk = 128, 64 * 12
    q, v = randn(0, 1, 130, 1, D), randn(1, 1, Lk, 1, D)
    k = randn(2, 1, Lk, 1, D)
    step = torch.arange(Lk, device="cuda") // 64
    k = (k * (1 + 3 * torch.where(step < 7, step, 12 - step)).view(1, Lk, 1, 1)).to(BF16)
    q, k = q.to(BF16), k
    check_attention(q, k, v, np.arange(12, dtype=np.int32).reshape(1, 1, 1, 12).repeat(2, 2))
    check_attention((q * 0.01).to(BF16), k, v, np.arange(12, dtype=np.int32)[::-1].reshape(1, 1, 1, 12).repeat(2, 2).copy())


def test_attention_lists():
    """No block, one block at the end of the list, a block twice, every block."""
    D, Lq, Lk = 64, 100, 640
    q, k, v = randn(0, 1, Lq, 1, D), randn(1, 1, Lk, 1, D), randn(2, 1, Lk, 1, D)
    for row in ([-1] * 6, [-1, -1, -1, -1, -1, 3], [4, 4, 2, 4, -1, 2], [9, 8, 0, 1, 2, 3]):
        check_attention(q, k, v, np.array(row, dtype=np.int32).reshape(1, 1, 1, 6))


def test_attention_bad_block_is_left_out():
    q, k, v = randn(0, 1, 10, 1, 64), randn(1, 1, 640, 1, 64), randn(2, 1, 640, 1, 64)
    ints = lambda r: torch.tensor(r, dtype=torch.int32, device="cuda").view(1, 1, 1, -1)  # noqa: E731
    got, lse = qs.block_attention(q, k, v, ints([1, 10, -2, 5, 2 ** 31 - 1, -2 ** 31]))
    assert qs.qs_device_error() == 5
    want, wlse = qs.block_attention(q, k, v, ints([1, 5, -1, -1, -1, -1]))
    assert torch.equal(got, want) and torch.equal(lse, wlse)
    n = torch.tensor([11], dtype=torch.int32, device="cuda")
    qs.block_attention(q, k, v, ints([1, 5]), q_len=n)
    assert qs.qs_device_error() == 5


def test_attention_views_and_shared_heads():
    """Views of one qkv row, heads-first caches, keys shared by stride 0, out into a wider row."""
    B, L, H, D, T = 2, 150, 3, 64, 3
    qkv = randn(0, B, L, 3 * H * D + 8)
    q, k, v = (qkv[..., 8 + i * H * D : 8 + (i + 1) * H * D].view(B, L, H, D) for i in range(3))
    blocks = some_blocks(1, B, H, L, L, T, holes=False)
    got, _ = check_attention(q, k, v, blocks)
    first = lambda t: t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)  # noqa: E731
    wide = torch.full((B, L, 2 * H, D), 4.0, dtype=BF16, device="cuda")
    ints = torch.tensor(blocks, device="cuda")
    qs.block_attention(first(q), first(k), first(v), ints, out=wide[:, :, 1::2])
    assert torch.equal(wide[:, :, 1::2], got) and (wide[:, :, ::2] == 4).all()
    one_k, one_v = k[:1, :, :1].expand(B, L, H, D), v[:1, :, :1].expand(B, L, H, D)
    check_attention(q, one_k, one_v, blocks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq,T", [(200, 6), (1, 6)])
def test_attention_nan_and_infinity_go_where_they_belong(D, Lq, T):
    """A NaN query row is NaN alone; a NaN key makes the rows that list its block NaN, wherever in
    the list it comes; a score of +inf makes its row NaN (inf - inf), as softmax does."""
    q, k, v = randn(0, 1, Lq, 3, D), randn(1, 1, 64 * T, 3, D), randn(2, 1, 64 * T, 3, D)
    blocks = torch.arange(T, dtype=torch.int32, device="cuda").expand(1, 3, -(-Lq // 128), T).contiguous()
    clean, clse = qs.block_attention(q, k, v, blocks)
    bad = q.clone()
    bad[0, 0, 0, 5] = float("nan")
    got, lse = qs.block_attention(bad, k, v, blocks)
    assert got[0, 0, 0].isnan().all() and lse[0, 0, 0].isnan()
    got[0, 0, 0], lse[0, 0, 0] = clean[0, 0, 0], clse[0, 0, 0]
    assert torch.equal(got, clean) and torch.equal(lse, clse)
    for row in (0, 64 * T - 1, 64 * (T // 2)):
        bad = k.clone()
        bad[0, row, 1, 0] = float("nan")
        got, lse = qs.block_attention(q, bad, v, blocks)
        assert got[:, :, 1].isnan().all() and lse[:, 1].isnan().all()
        assert torch.equal(got[:, :, ::2], clean[:, :, ::2]) and torch.equal(lse[:, ::2], clse[:, ::2])
    bad = k.clone()
    bad[0, 64:192, 1] = float("nan")  # two whole blocks, one tile
    got, lse = qs.block_attention(q, bad, v, blocks)
    assert got[:, :, 1].isnan().all() and lse[:, 1].isnan().all()
    bad, big = k.clone(), q.clone()
    bad[0, 70, 2, :], big[0, 0, 2, :] = float("inf"), 1.0
    got, lse = qs.block_attention(big, bad, v, blocks)
    assert got[0, 0, 2].isnan().all() and lse[0, 2, 0].isnan()
    assert torch.equal(got[:, :, :2], clean[:, :, :2])


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("causal,B,Lq,Lk,Hq,Hkv,T,ragged,copies", [
    (False, 1, 640, 300, 4, 2, 2, False, 40), (False, 1, 384, 512, 4, 4, 6, False, 60), (True, 2, 257, 500, 4, 2, 8, True, 30),
    (False, 3, 130, 900, 4, 1, 5, True, 30), (True, 1, 700, 700, 4, 4, 7, False, 30)])
def test_attention_more_items_than_processors(monkeypatch, dtype, D, causal, B, Lq, Lk, Hq, Hkv, T, ragged, copies):
    """Four and more items for each CTA, of one tile, three and others: O, both Q buffers, the sums and
    the rings serve one item after another, and again the same to the last bit.  The batch is `copies`
    of the same B sequences, which the oracle sees once."""
    again = lambda t: t.repeat(copies, 1, 1, 1)  # noqa: E731
    q = again(randn(Lq, B, Lq, Hq, D, dtype=dtype, by=2.0))
    k, v = again(randn(Lk, B, Lk, Hkv, D, dtype=dtype)), again(randn(Lk + 1, B, Lk, Hkv, D, dtype=dtype))
    ql = [Lq - 61 * b for b in range(B)] * copies if ragged else None
    kl = [Lk - 67 * b for b in range(B)] * copies if ragged else None
    blocks = np.tile(some_blocks(T, B, Hq, Lq, Lk, T, holes=ragged), (copies, 1, 1, 1))
    assert blocks.size // T >= 600
    real = O.block_attention

    def once(q, k, v, blocks, scale, causal, q_len, k_len, out, lse):
        n = [None if t is None else t[:B] for t in (q_len, k_len)]
        want = real(q[:B], k[:B], v[:B], blocks[:B], scale, causal, *n, out[:B], lse[:B])
        return [np.tile(t, (copies,) + (1,) * (t.ndim - 1)) for t in want]

    monkeypatch.setattr(O, "block_attention", once)
    got, lse = check_attention(q, k, v, blocks, causal=causal, q_len=ql, k_len=kl)
    for t in (got, lse):
        assert torch.equal(t, t[:B].repeat(copies, *[1] * (t.dim() - 1)))
    ints = lambda t: None if t is None else torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    dev = ints(blocks), ints(ql), ints(kl)
    for _ in range(10):
        o, z = qs.block_attention(q, k, v, dev[0], causal=causal, q_len=dev[1], k_len=dev[2], out=torch.full_like(got, 9.0),
                                  lse=torch.full_like(lse, 9.0))
        assert torch.equal(o, got) and torch.equal(z, lse)


@pytest.mark.parametrize("behind", [1.0, float("nan")])
@pytest.mark.parametrize("dtype,D", [(F16, 128), (BF16, 128), (BF16, 64)])
@pytest.mark.parametrize("kl", [[558, 20, 500, 97], [1279, 558, 64, 321]])
def test_attention_values_behind_a_length_beside_tiles_before_them(monkeypatch, dtype, D, behind, kl):
    """Rows of V behind a length become 0 in the tile that holds them and in no tile that had its place in
    shared memory before, however late that tile's V comes: the same to the last bit in every run.  The
    batch is 12 times the same sequences, of several items per CTA."""
    copies, H, Lk, T = 12, 4, 1280, 15
    again = lambda t: t.repeat(copies, 1, 1, 1)  # noqa: E731
    q, k, v = (randn(i, 4, Lk, H if i == 0 else 1, D, dtype=dtype) for i in range(3))
    clean = tuple(again(t.clone()) for t in (q, k, v))
    for b, n in enumerate(kl):
        k[b, n:], v[b, n:] = behind, behind
    seen = [-(-n // 64) for n in kl]
    blocks = np.full((4, H, 10, T), -1, dtype=np.int32)
    for b in range(4):
        blocks[b, ..., : min(T, seen[b])] = np.arange(max(0, seen[b] - T), seen[b])
    real = O.block_attention

    def once(q, k, v, blocks, scale, causal, q_len, k_len, out, lse):
        want = real(q[:4], k[:4], v[:4], blocks[:4], scale, causal, q_len[:4], k_len[:4], out[:4], lse[:4])
        return [np.tile(t, (copies,) + (1,) * (t.ndim - 1)) for t in want]

    monkeypatch.setattr(O, "block_attention", once)
    q, k, v, blocks, kl = again(q), again(k), again(v), np.tile(blocks, (copies, 1, 1, 1)), kl * copies
    got, lse = check_attention(q, k, v, blocks, q_len=kl, k_len=kl, clean=clean)
    dev, n = torch.tensor(blocks, device="cuda"), torch.tensor(kl, dtype=torch.int32, device="cuda")
    for _ in range(40):
        o, z = qs.block_attention(q, k, v, dev, q_len=n, k_len=n, out=torch.full_like(got, 9.0), lse=torch.full_like(lse, 9.0))
        assert torch.equal(o, got) and torch.equal(z, lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64), (BF16, 64), (F16, 128)])
@pytest.mark.parametrize("Lq,Lk,T", [(300, 300, 5), (300, 411, 7), (5, 900, 15), (64, 4096, 64)])
def test_attention_values_of_keys_that_a_row_does_not_see(dtype, D, bad, Lq, Lk, T):
    """Causal: a NaN or an infinity in v reaches the rows that see its key, and no other row of the
    block; with lists that are cut too (5 and 64 queries)."""
    q, k, v = randn(0, 2, Lq, 2, D, dtype=dtype), randn(1, 2, Lk, 1, D, dtype=dtype), randn(2, 2, Lk, 1, D, dtype=dtype)
    off = Lk - Lq
    for key in (off + 3, off + Lq // 2, Lk - 1):
        v[0, key, 0, 7] = bad
        v[1, key, 0] = bad
    v[0, off + 2, 0, 9], v[0, off + 3, 0, 9] = float("inf"), -float("inf")
    nq, nk = -(-Lq // 128), -(-Lk // 64)
    blocks = np.tile(np.arange(nk, dtype=np.int32)[::-1][:T], (2, 2, nq, 1))
    clean = torch.where(v.isfinite(), v, 0.0)
    with np.errstate(invalid="ignore"):
        want, wlse, _ = O.block_attention(f64(q), f64(k), f64(v), blocks, None, True)
    got, lse = qs.block_attention(q, k, v, torch.tensor(blocks, device="cuda"), causal=True)
    base, blse = check_attention(q, k, clean, blocks, causal=True)
    bad = ~np.isfinite(want)
    assert 0 < bad.sum() < bad.size
    assert np.array_equal(f64(got)[bad], want[bad], equal_nan=True)
    assert torch.equal(lse, blse)
    # finite elements: as with those values 0, but summed apart from the products, and P not rounded
    e = half(dtype)
    size = O.block_attention(f64(q), f64(k), f64(clean), blocks, None, True)[2]
    tol = 2 * (e * np.abs(f64(base)) + (e + 2.0 ** -12) * size) + Lk * 2.0 ** -23
    assert (np.abs(f64(got)[~bad] - f64(base)[~bad]) <= tol[~bad]).all()


def test_attention_at_once_on_two_streams():
    q, k, v = randn(0, 2, 300, 4, 128), randn(1, 2, 700, 2, 128), randn(2, 2, 700, 2, 128)
    blocks = torch.tensor(some_blocks(0, 2, 4, 300, 700, 7), device="cuda")
    one = torch.tensor(some_blocks(1, 2, 4, 1, 700, 11), device="cuda")
    want, token = qs.block_attention(q, k, v, blocks), qs.block_attention(q[:, :1], k, v, one)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [[qs.block_attention(q, k, v, blocks, stream=s), qs.block_attention(q[:, :1], k, v, one, stream=s)]
           for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    for a, b in got:
        for p, r in zip((*a, *b), (*want, *token)):
            assert torch.equal(p, r)


def test_attention_long_list_is_cut():
    """More entries than a CTA's list holds, and the split of a single token's."""
    D, Lk, T = 64, 64 * 40, 4500
    q, k, v = randn(0, 1, 3, 2, D), randn(1, 1, Lk, 1, D), randn(2, 1, Lk, 1, D)
    rng = np.random.default_rng(0)
    check_attention(q, k, v, rng.integers(-1, 40, (1, 2, 1, T)).astype(np.int32))


# ------------------------------------------------------------------------- a run of them together

def test_block_of_a_transformer():
    """qkv projection with adapters -> rotary positions -> choice of blocks -> attention -> out
    projection with adapters, as one sequence of calls and again on a side stream and from a graph."""
    L, H, D, K = 333, 4, 128, 512
    x = randn(0, L, K)
    qkv_l = qs.QuantLinear(randn(1, 3 * H * D, K, by=0.05), randn(2, 3 * H * D, by=0.01), bits=4, alpha=0.9)
    out_l = qs.QuantLinear(randn(3, K, H * D, by=0.05), None, bits=8)
    st = torch.tensor([0, 100, 333], dtype=torch.int32, device="cuda")
    ids = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    lora_in = qs.LoraBatch(randn(4, 2, 16, K, by=0.05), randn(5, 2, 3 * H * D, 16, by=0.1), st, ids)
    lora_out = qs.LoraBatch(randn(6, 2, 8, H * D, by=0.05), randn(7, 2, K, 8, by=0.1), st, ids,
                            torch.tensor([0.5, 2.0], device="cuda"))
    inv, axis, scale = qs.rope_frequencies(D, axes=(44, 42, 42))
    row = torch.arange(L, device="cuda")
    pos = torch.stack([row // 60, row // 10 % 6, row % 10], 1).contiguous()

    def run(stream=None):
        qkv = qkv_l(x, stream=stream, lora=lora_in)
        qk = qkv[:, : 2 * H * D].view(L, 2 * H, D)
        qs.rope(qk, pos, inv, axis, scale=scale, out=qk, stream=stream)
        q, k, v = (qkv[:, i * H * D : (i + 1) * H * D].view(1, L, H, D) for i in range(3))
        means = qs.block_means(k, stream=stream)
        blocks = qs.block_select(q, means, 3, L, stream=stream)
        o, lse = qs.block_attention(q, k, v, blocks, stream=stream)
        return qkv, blocks, o, lse, out_l(o.view(L, H * D), stream=stream, lora=lora_out)

    first = run()
    torch.cuda.synchronize()
    qkv, blocks, o, lse, y = first
    # the pieces against their binary64 forms, each on the values that reached it
    q, k, v = (qkv[:, i * H * D : (i + 1) * H * D].view(1, L, H, D) for i in range(3))
    means = O.block_means(f64(k))
    assert np.array_equal(blocks.cpu().numpy(), O.block_select(f64(q), means, 3, L))
    check_attention(q, k, v, blocks.cpu().numpy())
    plain = out_l(o.view(L, H * D))
    want, size = O.lora_add(f64(plain), f64(o.view(L, H * D)), f64(lora_out.a), f64(lora_out.b), [0, 100, 333], [1, 0],
                            [0.5, 2.0])
    close(y, want, half(BF16) * np.abs(want) + (2 * U * (H * D + 16) + 2.0 ** -17) * size, "lora")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run(side)
    side.synchronize()
    for p, r in zip(first, again):
        assert torch.equal(p, r)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for p in held:
        p.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    for p, r in zip(first, held):
        assert torch.equal(p, r)
