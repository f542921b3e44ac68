"""Float64 definitions of attention over selected key blocks, and of the
gradients of the attention sub-layer's steps.

TEST INFRASTRUCTURE: imported only by tests and the smoke check.  Shares no code
with the CUDA library.

* Selection: the score of a block of queries and a block of keys is the product
  of their means; each query block takes the ``top_k`` key blocks of highest
  score, of equal ones the first.
* Attention over blocks: softmax over the keys of the marked blocks; a query
  with none gets zeros and a log-sum-exp of -inf.
* Gradients, with P = exp(scale q k^T - lse): dV = P^T dO, delta = rowsum(dO o O),
  dS = P o (dO V^T - delta), dQ = scale dS K, dK = scale dS^T Q.
* Rotation: its transpose, the rotation by the opposite angles.
* RMSNorm y = x r w with r = (mean(x^2) + eps)^(-1/2):
  dx = r (u w) - x r^3 mean(x u w), dw = sum u x r, u the gradient of y.

Every function that stands for a kernel with rounded intermediates can also
return the magnitudes its error bound is made of (``with_magnitudes``).
"""
from __future__ import annotations

import numpy as np

from .reference import default_scale, rope_tables

BLOCK = 128


def n_blocks(L: int) -> int:
    return (L + BLOCK - 1) // BLOCK


def block_means(x: np.ndarray) -> np.ndarray:
    """[B, L, H, D] -> the mean of each 128-token block, [B, H, n, D]."""
    parts = [x[:, i:i + BLOCK].astype(np.float64).mean(axis=1) for i in range(0, x.shape[1], BLOCK)]
    return np.stack(parts, axis=2)


def select_blocks(q: np.ndarray, k: np.ndarray, top_k: int) -> np.ndarray:
    """Truth values [B, H, nq, nk]."""
    score = np.einsum("bhid,bhjd->bhij", block_means(q), block_means(k))
    key = np.where(np.isnan(score), -np.inf, score)      # a NaN goes behind every number, -inf included
    order = np.lexsort((np.broadcast_to(np.arange(key.shape[-1]), key.shape), np.isnan(score), -key))
    on = np.zeros(score.shape, dtype=bool)
    np.put_along_axis(on, order[..., :top_k], True, axis=-1)
    return on


def token_mask(blocks: np.ndarray, Lq: int, Lk: int) -> np.ndarray:
    """One (batch, head)'s [nq, nk] block mask as a token mask [Lq, Lk]."""
    return blocks.astype(bool).repeat(BLOCK, axis=0)[:Lq].repeat(BLOCK, axis=1)[:, :Lk]


def attention(q, k, v, blocks, scale=None, with_magnitudes=False):
    """(o [B, Lq, H, D], lse [B, H, Lq]); with_magnitudes also sum_j p_j |v_j|."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    B, Lq, H, D = q.shape
    scale = scale if scale else default_scale(D)
    o, mag = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((B, H, Lq), -np.inf)
    for b in range(B):
        for h in range(H):
            m = token_mask(blocks[b, h], Lq, k.shape[1])
            rows = np.flatnonzero(m.any(axis=1))
            if rows.size == 0:
                continue
            s = np.where(m[rows], (q[b, rows, h] @ k[b, :, h].T) * scale, -np.inf)
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            l = p.sum(axis=1, keepdims=True)
            vv = np.where(m.any(axis=0)[:, None], v[b, :, h], 0.0)   # values no query attends to do not count
            o[b, rows, h] = (p @ vv) / l
            mag[b, rows, h] = (p @ np.abs(vv)) / l
            lse[b, h, rows] = (top + np.log(l))[:, 0]
    return (o, lse, mag) if with_magnitudes else (o, lse)


def attention_bwd(q, k, v, blocks, o, lse, d_o, scale=None, with_magnitudes=False, rel_p=0.0, rel_ds=0.0, acc=0.0):
    """(dq, dk, dv).  with_magnitudes also returns the bound on each one's error
    when P is off by the relative ``rel_p``, dS by the relative ``rel_ds`` and
    each dot product of D terms by ``acc`` times the sum of its terms' magnitudes."""
    q, k, v, o, d_o = (np.asarray(x, dtype=np.float64) for x in (q, k, v, o, d_o))
    B, Lq, H, D = q.shape
    scale = scale if scale else default_scale(D)
    grads = [np.zeros_like(x) for x in (q, k, v)]
    bounds = [np.zeros_like(x) for x in (q, k, v)]
    for b in range(B):
        for h in range(H):
            m = token_mask(blocks[b, h], Lq, k.shape[1])
            m &= np.isfinite(lse[b, h])[:, None]
            qq, kk, vv, oo, gg = q[b, :, h], k[b, :, h], v[b, :, h], o[b, :, h], d_o[b, :, h]
            stat = np.where(np.isfinite(lse[b, h]), lse[b, h], 0.0)
            p = np.where(m, np.exp(np.where(m, (qq @ kk.T) * scale, -np.inf) - stat[:, None]), 0.0)
            delta = (gg * oo).sum(axis=1, keepdims=True)
            ds = p * (gg @ vv.T - delta)
            grads[0][b, :, h] = scale * (ds @ kk)
            grads[1][b, :, h] = scale * (ds.T @ qq)
            grads[2][b, :, h] = p.T @ gg
            if with_magnitudes:
                e_dp = acc * (np.abs(gg) @ np.abs(vv).T + (np.abs(gg) * np.abs(oo)).sum(axis=1, keepdims=True))
                e_ds = rel_ds * np.abs(ds) + p * e_dp
                bounds[0][b, :, h] = scale * (e_ds @ np.abs(kk))
                bounds[1][b, :, h] = scale * (e_ds.T @ np.abs(qq))
                bounds[2][b, :, h] = rel_p * (p.T @ np.abs(gg))
    return (*grads, *bounds) if with_magnitudes else tuple(grads)


def rope_3d_bwd(g, grid, split, theta: float = 10000.0):
    """The transposed rotation of [B, L, H, D]."""
    g = np.asarray(g, dtype=np.float64)
    a = rope_tables(grid, split, theta)[None, :, None, :]
    c, s = np.cos(a), np.sin(a)
    out = np.empty_like(g)
    out[..., 0::2] = g[..., 0::2] * c + g[..., 1::2] * s
    out[..., 1::2] = g[..., 1::2] * c - g[..., 0::2] * s
    return out


def qk_norm_rope_3d_bwd(x, g, grid, split, group: int, weight=None, eps: float = 1e-6, theta: float = 10000.0,
                        with_magnitudes=False):
    """(dx, dw) of y = rope_3d(rms_norm(x) * weight) for the gradient g of y;
    with_magnitudes also (r (|u w| + |x| r^2 mean|x u w|), sum |u x r|) with |u| the
    sum of the two magnitudes the rotation adds."""
    x = np.asarray(x, dtype=np.float64)
    shape = x.shape
    w = np.ones(group) if weight is None else np.asarray(weight, dtype=np.float64)
    u = rope_3d_bwd(g, grid, split, theta).reshape(-1, group)
    xg = x.reshape(-1, group)
    r = 1.0 / np.sqrt((xg * xg).mean(axis=1, keepdims=True) + eps)
    uw = u * w
    dx = r * uw - xg * r ** 3 * (xg * uw).mean(axis=1, keepdims=True)
    dw = (u * xg * r).sum(axis=0)
    if not with_magnitudes:
        return dx.reshape(shape), dw
    a = np.abs(np.asarray(g, dtype=np.float64))
    au = (a[..., 0::2] + a[..., 1::2]).repeat(2, axis=-1).reshape(-1, group)
    aw, ax = np.abs(w), np.abs(xg)
    mx = r * (au * aw) + ax * r ** 3 * (ax * au * aw).mean(axis=1, keepdims=True)
    return dx.reshape(shape), dw, mx.reshape(shape), (au * ax * r).sum(axis=0)
