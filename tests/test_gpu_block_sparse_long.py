"""The gradients of block-sparse attention at 32,760 tokens against the float64
definition, on sampled blocks: mask rows and columns with up to 256 marked blocks
(eight words of their bits), the ragged last block among them.

dK and dV of a key block take part of every query block of its column and of
nothing else: they are compared with the definition on those query blocks and that
key block alone.  dQ of a query block is the same with its row.

Bounds: those of test_gpu_block_sparse.py, and for the sums over up to 2^15 rows,
taken 16 at a time in float32, 2^11 additions of at most 2^-23 of the sum of the
terms' magnitudes each: 2^-12 beside the relative error of P and dS."""
import numpy as np
import pytest
import torch

from oracle import sparse as sp
from tests.gpu_util import dev_f64, to_dev_bf16, watchdog_clear
from tests.test_gpu_block_sparse import E_P, HALF, _bits, _inputs, f64

pytestmark = pytest.mark.gpu

SUMS = 2.0 ** -12


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    watchdog_clear()


def _rows(blocks, L):
    return np.concatenate([np.arange(128 * i, min(L, 128 * (i + 1))) for i in blocks])


def _compare(what, got, exp, bound):
    bound = np.maximum(bound + HALF * (np.abs(exp) + bound), 1e-6)
    err = np.abs(got - exp)
    assert np.all(err <= bound), (what, f"max excess {(err - bound).max():.3e}")


@pytest.mark.parametrize("Lq,Lk,D", [(32760, 32760, 128), (32760, 4200, 64), (4200, 32760, 32)])
def test_sampled_blocks_of_long_rows_and_columns(Lq, Lk, D):
    import spacetime_attention_vdit_b200 as vd
    heads = 2
    q, k, v = _inputs(1, Lq, Lk, heads, D, seed=D)
    g = _bits(77, 1, Lq, heads, D)
    t = [to_dev_bf16(x) for x in (q, k, v, g)]
    on = vd.attn_select_blocks(t[0], t[1], 12)
    nq, nk = on.shape[2:]
    on[..., 0] = True                       # columns that every row marks: the first and the ragged last
    on[..., nk - 1] = True
    on[:, :, nq // 2] = True                # and a row that marks every column
    on[:, 1, 1] = False
    o, lse = vd.attn_block_sparse(*t[:3], on, lse=True)
    dq, dk, dv = (dev_f64(x) for x in vd.attn_block_sparse_bwd(*t[:3], on, o, lse, t[3]))
    host, o64, lse64 = on.cpu().numpy(), dev_f64(o), lse.cpu().numpy().astype(np.float64)

    def definition(h, query_blocks, key_blocks):
        r, c = _rows(query_blocks, Lq), _rows(key_blocks, Lk)
        part = host[:, h:h + 1][:, :, query_blocks][..., key_blocks]
        assert part.all()
        at = (slice(None), r, slice(h, h + 1))
        of = (slice(None), c, slice(h, h + 1))
        return r, c, sp.attention_bwd(f64(q)[at], f64(k)[of], f64(v)[of], part, o64[at], lse64[:, h:h + 1, r],
                                      f64(g)[at], with_magnitudes=True, rel_p=HALF + E_P + SUMS,
                                      rel_ds=HALF + E_P + SUMS, acc=D * 2.0 ** -23)

    for h, j in ((0, 0), (1, nk - 1), (0, nk // 3), (1, nk // 2)):
        rows = np.flatnonzero(host[0, h, :, j])
        _, c, exp = definition(h, rows, [j])
        _compare(("dk", h, j, rows.size), dk[0, c, h], exp[1][0, :, 0], exp[4][0, :, 0])
        _compare(("dv", h, j, rows.size), dv[0, c, h], exp[2][0, :, 0], exp[5][0, :, 0])
    for h, i in ((0, 0), (1, nq - 1), (0, nq // 2), (1, nq // 3)):
        r, _, exp = definition(h, [i], np.flatnonzero(host[0, h, i]))
        _compare(("dq", h, i), dq[0, r, h], exp[0][0, :, 0], exp[3][0, :, 0])
    assert np.all(dq[0, 128:256, 1] == 0)
