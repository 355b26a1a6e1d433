"""The binary64 forms of the operators around the projections against closed forms and against
other ways to the same numbers."""

import numpy as np
import pytest

from oracle import attn_oracle as O


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("inter", [True, False])
def test_rope_is_a_rotation_by_position(inter):
    x, inv = rnd(0, 5, 3, 16), 100.0 ** (-np.arange(6) / 6)
    pos = np.array([0, 1, 2, 7, 1000])
    y = O.rope(x, pos, inv, None, inter)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 12:], x[..., 12:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(O.rope(y, pos, inv, None, inter, inverse=True), x)
    # products of a query and a key depend on their distance alone
    q, k = rnd(1, 1, 1, 16).repeat(4, 0), rnd(2, 1, 1, 16).repeat(4, 0)
    at = np.array([0, 5, 11, 400])
    dots = (O.rope(q, at + 3, inv, None, inter) * O.rope(k, at, inv, None, inter)).sum(-1)
    assert np.allclose(dots, dots[0])
    # one pair, a quarter turn: (1, 0) -> (0, 1)
    one = np.zeros((1, 1, 2))
    one[..., 0] = 1
    assert np.allclose(O.rope(one, np.array([1]), np.array([np.pi / 2]), None, inter), [[[0, 1]]])


def test_rope_axes():
    x, inv = rnd(3, 4, 2, 8), np.array([1.0, 0.5, 1.0, 0.25])
    pos = np.array([[0, 9], [1, 0], [2, 3], [5, 5]])
    y = O.rope(x, pos, inv, [0, 0, 1, 1])
    assert np.allclose(y[..., :4], O.rope(x[..., :4], pos[:, 0], inv[:2]))
    assert np.allclose(y[..., 4:], O.rope(x[..., 4:], pos[:, 1], inv[2:]))


def test_lora_is_a_merged_weight():
    x, y, a, b = rnd(0, 9, 12), rnd(1, 9, 7), rnd(2, 2, 3, 12), rnd(3, 2, 7, 3)
    out, size = O.lora_add(y, x, a, b, [1, 4, 4, 8], [1, 0, -1], [2.0, 0.5])
    assert np.array_equal(out[[0, 8]], y[[0, 8]]) and np.array_equal(out[4:8], y[4:8])
    assert np.allclose(out[1:4], y[1:4] + x[1:4] @ (0.5 * b[1] @ a[1]).T)
    assert (np.abs(out - y) <= size + 1e-12).all()


def test_means_and_selection():
    k = rnd(0, 1, 200, 1, 64)
    m = O.block_means(k, [150])
    assert np.allclose(m[0, 0, 0], k[0, :64, 0].mean(0)) and np.allclose(m[0, 0, 2], k[0, 128:150, 0].mean(0))
    assert (m[0, 0, 3] == 0).all()
    q = np.zeros((1, 130, 1, 64))
    q[..., 0] = 1.0  # the scores are the means' first column
    means = np.zeros((1, 1, 5, 64), dtype=np.float32)
    means[0, 0, :, 0] = [3, 1, 3, 5, 4]
    assert O.block_select(q, means, 3, 300)[0, 0].tolist() == [[0, 3, 4], [0, 3, 4]]
    assert O.block_select(q, means, 2, 300, first=1, last=1)[0, 0, 0].tolist() == [0, 4]
    # causal over as many keys as queries: the first block's last row sees 128 keys, the second's 130
    got = O.block_select(q, means, 2, 130, causal=True)
    assert got[0, 0].tolist() == [[0, 1], [0, 2]]
    assert O.block_select(q, means, 4, 300, k_len=[70])[0, 0, 0].tolist() == [0, 1, -1, -1]


def test_attention_over_all_blocks_is_attention():
    q, k, v = rnd(0, 1, 70, 2, 64), rnd(1, 1, 130, 1, 64), rnd(2, 1, 130, 1, 64)
    blocks = np.array([2, 0, -1, 1]).reshape(1, 1, 1, 4).repeat(2, 1)
    o, lse, _ = O.block_attention(q, k, v, blocks)
    s = np.einsum("ihd,jd->hij", q[0], k[0, :, 0]) / 8
    p = np.exp(s)
    assert np.allclose(o[0], np.einsum("hij,jd->ihd", p / p.sum(-1, keepdims=True), v[0, :, 0]))
    assert np.allclose(lse[0], np.log(p.sum(-1)))
    o, lse, _ = O.block_attention(q, k, v, blocks, causal=True)
    # row i sees keys 0 .. i + 60
    p = np.where(np.arange(130)[None, None] <= np.arange(70)[None, :, None] + 60, p, 0.0)
    assert np.allclose(o[0], np.einsum("hij,jd->ihd", p / p.sum(-1, keepdims=True), v[0, :, 0]))
    # nothing seen: zero and -inf; behind the length: as it was
    o, lse, _ = O.block_attention(q, k, v, blocks, q_len=[10], k_len=[0], out=np.full_like(q, 5.0), lse=np.ones((1, 2, 70)))
    assert (o[0, :10] == 0).all() and (o[0, 10:] == 5).all()
    assert np.isneginf(lse[..., :10]).all() and (lse[..., 10:] == 1).all()
