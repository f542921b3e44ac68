"""The sizes at the ends of what the sparse-attention and gradient calls take: rows of
6,144 key blocks, columns of 6,144 query blocks, heads that are not a power of two
wide, norm groups of several heads.

Bounds: those of test_gpu_block_sparse.py (for the long sums with the 2^-12 of
test_gpu_block_sparse_long.py) and of test_gpu_norm_rope_bwd.py."""
import numpy as np
import pytest
import torch

from oracle import sparse as sp
from tests.gpu_util import LSE_ABS, dev_f64, to_dev_bf16, watchdog_clear
from tests.test_gpu_block_sparse import E_P, HALF, _bits, f64
from tests.test_gpu_block_sparse_long import SUMS, _compare, _rows
from tests.test_gpu_norm_rope_bwd import _check_norm, test_rope_bwd as check_rope

pytestmark = pytest.mark.gpu

MOST = 6144


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    watchdog_clear()


def _marks(n, seed):
    """Some of n blocks, first, last and word boundaries among them."""
    on = np.random.default_rng(seed).random(n) < 0.02
    on[[0, 31, 32, n // 2, n - 1]] = True
    return on


@pytest.mark.parametrize("Lq", [1, 200, 128 * 300 + 5])
def test_rows_of_6144_key_blocks(Lq):
    """One query, two blocks (a cluster) and 301 blocks of one head (a CTA a pair)."""
    import spacetime_attention_vdit_b200 as vd
    D, Lk = 32, 128 * MOST - 60
    q, g, k, v = _bits(1, 1, Lq, 1, D), _bits(2, 1, Lq, 1, D), _bits(3, 1, Lk, 1, D), _bits(4, 1, Lk, 1, D)
    nq = sp.n_blocks(Lq)
    on = np.stack([_marks(MOST, 10 + i) for i in range(nq)])[None, None]
    t = [to_dev_bf16(x) for x in (q, k, v, g)]
    blocks = torch.from_numpy(on).cuda()
    o, lse = vd.attn_block_sparse(*t[:3], blocks, lse=True)
    dq, dk, dv = (dev_f64(x) for x in vd.attn_block_sparse_bwd(*t[:3], blocks, o, lse, t[3]))
    o64, lse64 = dev_f64(o), lse.cpu().numpy().astype(np.float64)
    for i in sorted({0, nq // 2, nq - 1}):
        cols, r = np.flatnonzero(on[0, 0, i]), _rows([i], Lq)
        c = _rows(cols, Lk)
        part = np.ones((1, 1, 1, cols.size), dtype=bool)
        eo, el, mag = sp.attention(f64(q)[:, r], f64(k)[:, c], f64(v)[:, c], part, with_magnitudes=True)
        err, bound = np.abs(o64[:, r] - eo), (HALF + 2 * E_P) * mag + HALF * np.abs(eo)
        assert np.all(err <= bound), (i, f"{(err - bound).max():.3e}")
        assert np.all(np.abs(lse64[..., r] - el) <= LSE_ABS)
        exp = sp.attention_bwd(f64(q)[:, r], f64(k)[:, c], f64(v)[:, c], part, o64[:, r], lse64[..., r], f64(g)[:, r],
                               with_magnitudes=True, rel_p=HALF + E_P + SUMS, rel_ds=HALF + E_P + SUMS,
                               acc=D * 2.0 ** -23)
        _compare(("dq", i), dq[:, r], exp[0], exp[3])
        if nq == 1:
            _compare("dk", dk[:, c], exp[1], exp[4])
            _compare("dv", dv[:, c], exp[2], exp[5])
    quiet = _rows(np.flatnonzero(~on[0, 0].any(axis=0)), Lk)
    assert not dk[:, quiet].any() and not dv[:, quiet].any()


def test_columns_of_6144_query_blocks():
    import spacetime_attention_vdit_b200 as vd
    D, Lq, Lk = 32, 128 * MOST - 60, 200
    q, g, k, v = _bits(1, 1, Lq, 1, D), _bits(2, 1, Lq, 1, D), _bits(3, 1, Lk, 1, D), _bits(4, 1, Lk, 1, D)
    on = np.stack([_marks(MOST, 10 + j) for j in range(2)], axis=-1)[None, None]
    t = [to_dev_bf16(x) for x in (q, k, v, g)]
    blocks = torch.from_numpy(on).cuda()
    o, lse = vd.attn_block_sparse(*t[:3], blocks, lse=True)
    dq, dk, dv = (dev_f64(x) for x in vd.attn_block_sparse_bwd(*t[:3], blocks, o, lse, t[3]))
    o64, lse64 = dev_f64(o), lse.cpu().numpy().astype(np.float64)
    for j in range(2):
        rows, c = np.flatnonzero(on[0, 0, :, j]), _rows([j], Lk)
        r = _rows(rows, Lq)
        exp = sp.attention_bwd(f64(q)[:, r], f64(k)[:, c], f64(v)[:, c], np.ones((1, 1, rows.size, 1), dtype=bool),
                               o64[:, r], lse64[..., r], f64(g)[:, r], with_magnitudes=True,
                               rel_p=HALF + E_P + SUMS, rel_ds=HALF + E_P + SUMS, acc=D * 2.0 ** -23)
        _compare(("dk", j), dk[:, c], exp[1], exp[4])
        _compare(("dv", j), dv[:, c], exp[2], exp[5])
    quiet = _rows(np.flatnonzero(~on[0, 0].any(axis=1)), Lq)
    assert not dq[:, quiet].any() and not o64[:, quiet].any() and np.all(lse64[..., quiet] == -np.inf)


def test_selection_of_6144_key_blocks():
    import spacetime_attention_vdit_b200 as vd
    q, k = _bits(5, 1, 129, 2, 32), _bits(6, 1, 128 * MOST - 60, 2, 32)
    for top_k in (1, 700, MOST):
        got = vd.attn_select_blocks(to_dev_bf16(q), to_dev_bf16(k), top_k).cpu().numpy()
        assert np.array_equal(got, sp.select_blocks(f64(q), f64(k), top_k)), top_k


def test_many_short_sequences():
    """40,000 single tokens, each over its own 130 keys."""
    import spacetime_attention_vdit_b200 as vd
    B, D = 40000, 32
    q, k, v = _bits(7, B, 1, 1, D), _bits(8, B, 130, 1, D), _bits(9, B, 130, 1, D)
    t = [to_dev_bf16(x) for x in (q, k, v)]
    on = vd.attn_select_blocks(t[0], t[1], 1)
    o, lse = vd.attn_block_sparse(*t, on, lse=True)
    grads = vd.attn_block_sparse_bwd(*t, on, o, lse, t[0])
    for b in (0, 1, B // 2, B - 1):
        one = slice(b, b + 1)
        on1 = sp.select_blocks(f64(q[one]), f64(k[one]), 1)
        assert np.array_equal(on[one].cpu().numpy(), on1)
        eo, _, mag = sp.attention(f64(q[one]), f64(k[one]), f64(v[one]), on1, with_magnitudes=True)
        assert np.all(np.abs(dev_f64(o[one]) - eo) <= (HALF + 2 * E_P) * mag + HALF * np.abs(eo))
        exp = sp.attention_bwd(f64(q[one]), f64(k[one]), f64(v[one]), on1, dev_f64(o[one]),
                               lse[one].cpu().numpy().astype(np.float64), f64(q[one]), with_magnitudes=True,
                               rel_p=HALF + E_P, rel_ds=HALF + E_P, acc=D * 2.0 ** -23)
        for name, a, e, bound in zip(("dq", "dk", "dv"), grads, exp[:3], exp[3:]):
            _compare((name, b), dev_f64(a[one]), e, bound)


@pytest.mark.parametrize("heads,D,split,group", [
    (5, 24, (8, 8, 8), 120),             # three vectors a head, the whole token
    (5, 24, (8, 8, 8), 8),
    (3, 40, (16, 12, 12), 120),
    (4, 96, (32, 32, 32), 384),
    (3, 200, (72, 64, 64), 600),         # 25 vectors a head
    (2, 256, (88, 84, 84), 256),         # the widest head, normed by itself
    (7, 256, (88, 84, 84), 1792),
    (32, 256, (88, 84, 84), 8192),
    (6, 64, (22, 20, 22), 128),          # a group of two heads
    (8, 32, (12, 10, 10), 256),          # the whole token, in one warp
    (12, 32, (12, 10, 10), 64),
    (41, 128, (44, 42, 42), 5248),       # an odd number of heads per token
])
def test_heads_and_groups_of_other_widths(heads, D, split, group):
    _check_norm(1, (2, 3, 29), heads, D, split, group)
    _check_norm(2, (1, 1, 3), heads, D, split, group)


@pytest.mark.parametrize("heads,D,split", [(5, 24, (8, 8, 8)), (3, 40, (16, 12, 12)), (3, 200, (72, 64, 64)),
                                           (2, 256, (88, 84, 84)), (1, 8, (8, 0, 0))])
def test_rotation_of_other_widths(heads, D, split):
    check_rope(1, (3, 5, 7), heads, D, split)
    check_rope(2, (1, 1, 1), heads, D, split)
