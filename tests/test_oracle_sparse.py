"""The float64 definitions of oracle/sparse.py against other ways to the same
numbers: brute force, the dense oracle, central differences and torch's autograd
in float64.  CPU only."""
import numpy as np
import pytest
import torch

from oracle import reference as ref
from oracle import sparse as sp


def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def _mask(seed, B, H, nq, nk, keep=0.5):
    return np.random.default_rng(seed).random((B, H, nq, nk)) < keep


def test_select_brute_force():
    q, k = _rand(0, 2, 300, 2, 8), _rand(1, 2, 517, 2, 8)
    on = sp.select_blocks(q, k, 2)
    assert on.shape == (2, 2, 3, 5)
    for b in range(2):
        for h in range(2):
            for i in range(3):
                qm = q[b, 128 * i:128 * (i + 1), h].mean(0)
                score = [qm @ k[b, 128 * j:128 * (j + 1), h].mean(0) for j in range(5)]
                best = sorted(range(5), key=lambda j: (-score[j], j))[:2]
                assert sorted(np.flatnonzero(on[b, h, i])) == sorted(best)


def test_select_ties_and_nan_go_by_index():
    q = np.ones((1, 128, 1, 4))
    k = np.ones((1, 128 * 5, 1, 4))
    assert np.flatnonzero(sp.select_blocks(q, k, 3)[0, 0, 0]).tolist() == [0, 1, 2]
    k[0, 130] = np.nan                                         # block 1: NaN, behind every number
    assert np.flatnonzero(sp.select_blocks(q, k, 3)[0, 0, 0]).tolist() == [0, 2, 3]
    k[0, 256:384] = -np.inf
    assert np.flatnonzero(sp.select_blocks(q, k, 4)[0, 0, 0]).tolist() == [0, 2, 3, 4]


def test_attention_all_blocks_is_the_dense_oracle():
    q, k, v = _rand(0, 1, 200, 2, 16), _rand(1, 1, 333, 2, 16), _rand(2, 1, 333, 2, 16)
    o, lse = sp.attention(q, k, v, np.ones((1, 2, 2, 3), dtype=bool))
    eo, el = ref.attention(q, k, v)
    assert np.allclose(o, eo, rtol=0, atol=1e-13) and np.allclose(lse, el, rtol=0, atol=1e-13)


def test_attention_masked_rows_and_empty_rows():
    q, k, v = _rand(3, 1, 200, 1, 16), _rand(4, 1, 333, 1, 16), _rand(5, 1, 333, 1, 16)
    blocks = np.zeros((1, 1, 2, 3), dtype=bool)
    blocks[0, 0, 0, 1] = True
    k2, v2 = k.copy(), v.copy()
    k2[:, 256:], v2[:, 256:] = 7.0, 7.0                         # unmarked: must not matter
    o, lse = sp.attention(q, k2, v2, blocks)
    eo, el = ref.attention(q[:, :128], k[:, 128:256], v[:, 128:256])
    assert np.allclose(o[:, :128], eo, atol=1e-13) and np.allclose(lse[..., :128], el, atol=1e-13)
    assert np.all(o[:, 128:] == 0) and np.all(lse[..., 128:] == -np.inf)


@pytest.mark.parametrize("Lq,Lk", [(150, 150), (1, 300), (260, 40)])
def test_attention_bwd_is_autograd(Lq, Lk):
    B, H, D = 1, 2, 8
    q, k, v, g = (_rand(i, B, L, H, D) for i, L in enumerate((Lq, Lk, Lk, Lq)))
    blocks = _mask(7, B, H, sp.n_blocks(Lq), sp.n_blocks(Lk))
    blocks[:, 0, 0, 0] = True
    t = [torch.from_numpy(x).requires_grad_() for x in (q, k, v)]
    mask = torch.from_numpy(np.stack([[sp.token_mask(blocks[b, h], Lq, Lk) for h in range(H)] for b in range(B)]))
    s = torch.einsum("bihd,bjhd->bhij", t[0], t[1]) * D ** -0.5
    p = torch.softmax(s.masked_fill(~mask, -1e300), -1) * mask.any(-1, keepdim=True)
    torch.einsum("bhij,bjhd->bihd", p, t[2]).backward(torch.from_numpy(g))
    o, lse = sp.attention(q, k, v, blocks)
    for got, x in zip(sp.attention_bwd(q, k, v, blocks, o, lse, g), t):
        assert np.allclose(got, x.grad.numpy(), rtol=0, atol=1e-12)


def _difference(f, x, g, n, seed, h=1e-6):
    """Central differences of sum(f(x) * g) at n seeded elements of x: (indices, values)."""
    at = np.random.default_rng(seed).choice(x.size, n, replace=False)
    out = []
    for i in at:
        d = np.zeros(x.size)
        d[i] = h
        d = d.reshape(x.shape)
        out.append(((f(x + d) - f(x - d)) * g).sum() / (2 * h))
    return at, np.array(out)


def test_attention_bwd_is_the_difference_quotient():
    q, k, v, g = (_rand(i, 1, 140, 1, 8) for i in range(4))
    blocks = np.array([[[[True, False], [True, True]]]])
    o, lse = sp.attention(q, k, v, blocks)
    grads = sp.attention_bwd(q, k, v, blocks, o, lse, g)
    for i, got in enumerate(grads):
        def f(x, i=i):
            a = [q, k, v]
            a[i] = x
            return sp.attention(*a, blocks)[0]
        at, d = _difference(f, (q, k, v)[i], g, 12, seed=i)
        assert np.allclose(got.ravel()[at], d, rtol=0, atol=1e-7)


@pytest.mark.parametrize("group", [16, 48])
def test_norm_rope_bwd_is_the_difference_quotient(group):
    grid, split, H, D = (2, 3, 2), (8, 4, 4), 3, 16
    x, g, w = _rand(0, 2, 12, H, D), _rand(1, 2, 12, H, D), _rand(2, group)
    dx, dw = sp.qk_norm_rope_3d_bwd(x, g, grid, split, group, w, eps=1e-3)
    at, d = _difference(lambda a: ref.qk_norm_rope_3d(a, grid, split, group, w, eps=1e-3), x, g, 20, seed=3)
    assert np.allclose(dx.ravel()[at], d, rtol=0, atol=1e-7)
    at, d = _difference(lambda a: ref.qk_norm_rope_3d(x, grid, split, group, a, eps=1e-3), w, g, group, seed=4)
    assert np.allclose(dw.ravel()[at], d, rtol=0, atol=1e-7)


def test_rope_bwd_undoes_the_rotation():
    x = _rand(0, 1, 24, 2, 32)
    y = ref.rope_3d(x, (2, 3, 4), (12, 10, 10))
    assert np.allclose(sp.rope_3d_bwd(y, (2, 3, 4), (12, 10, 10)), x, rtol=0, atol=1e-13)
