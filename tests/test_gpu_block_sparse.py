"""GPU parity of block selection, attention over selected blocks and its
gradients against the float64 definitions of oracle/sparse.py.

Bounds, from the arithmetic (bf16 rounding: half a step, 2^-8 relative):

* selection is float64 on both sides: whole masks must be equal (seeded normal
  data; where two scores agree to the last bits, both sides see the tie).
* O = sum_j P_j V_j / l with P rounded to bf16 as an operand (2^-8 P), and each P
  off by e_p relative: its score s is a float32 dot product of at most 128 terms
  (|ds| <= 128 * 2^-23 * sum|q k| scale <= 3e-4 for the data here), its
  exponential is good to 8e-5 (the cubic on the FMA pipe) and its argument's
  rounding to |s| 2^-22; e_p = 6e-4 covers the three.  l carries e_p too.  With
  mag = sum_j p_j |V_j|: |dO| <= (2^-8 + 2 e_p) mag + 2^-8 |O|.
* log-sum-exp: |dlse| <= 1e-3, the bound of the dense kernels' tests.
* gradients: P is formed once more from the given lse (e_p), dP and delta are
  float32 dot products of D terms (2^-23 D times the terms' magnitudes); dS is
  rounded to bf16 (2^-8), the gradients once more (2^-8 of the value), sums are
  float32: 2^-20 of the terms' magnitudes for up to 2^13 terms summed in chunks of
  16 is covered by the e_p of each term.  Elements whose bound is below 1e-6
  (float32's own dust next to values of order 1) get 1e-6.
"""
import numpy as np
import pytest
import torch

import synthetic
from oracle import sparse as sp
from tests.gpu_util import LSE_ABS, dev_f64, to_dev_bf16, watchdog_clear

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
E_P = 6e-4


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import spacetime_attention_vdit_b200 as v  # noqa: F401
    yield
    watchdog_clear()


def _bits(seed, *shape, scale=1.0):
    return synthetic.f32_to_bf16_bits((np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32))


def _inputs(B, Lq, Lk, heads, D, seed=0):
    return (_bits(seed, B, Lq, heads, D), _bits(seed + 1, B, Lk, heads, D), _bits(seed + 2, B, Lk, heads, D))


def _mask(B, Lq, Lk, heads, keep, seed):
    """Seeded marks; of every head's rows the second (if any) is left empty and
    of the columns the first."""
    on = np.random.default_rng(seed).random((B, heads, sp.n_blocks(Lq), sp.n_blocks(Lk))) < keep
    if on.shape[2] > 1:
        on[:, :, 1] = False
    if on.shape[3] > 1 and keep < 1:
        on[..., 0] = False
    return on


f64 = synthetic.bf16_bits_to_f64


def _check_forward(q, k, v, blocks, scale=0.0, got=None):
    import spacetime_attention_vdit_b200 as vd
    if got is None:
        got = vd.attn_block_sparse(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), torch.from_numpy(blocks).cuda(),
                                   lse=True, scale=scale)
    o, lse = dev_f64(got[0]), got[1].cpu().numpy().astype(np.float64)
    eo, el, mag = sp.attention(f64(q), f64(k), f64(v), blocks, scale, with_magnitudes=True)
    err, bound = np.abs(o - eo), (HALF + 2 * E_P) * mag + HALF * np.abs(eo)
    assert np.all(err <= bound), f"max excess {(err - bound).max():.3e} at {np.unravel_index((err - bound).argmax(), err.shape)}"
    empty = ~np.isfinite(el)
    assert np.array_equal(empty, lse == -np.inf)
    assert np.all(np.abs(lse[~empty] - el[~empty]) <= LSE_ABS)
    return got


def _check_backward(q, k, v, blocks, scale=0.0, seed=9):
    import spacetime_attention_vdit_b200 as vd
    on = torch.from_numpy(blocks).cuda()
    t = [to_dev_bf16(x) for x in (q, k, v)]
    o, lse = vd.attn_block_sparse(*t, on, lse=True, scale=scale)
    g = _bits(seed, *q.shape)
    got = vd.attn_block_sparse_bwd(*t, on, o, lse, to_dev_bf16(g), scale=scale)
    exp = sp.attention_bwd(f64(q), f64(k), f64(v), blocks, dev_f64(o), lse.cpu().numpy().astype(np.float64), f64(g),
                           scale, with_magnitudes=True, rel_p=HALF + E_P, rel_ds=HALF + E_P,
                           acc=q.shape[-1] * 2.0 ** -23)
    for name, a, e, b in zip(("dq", "dk", "dv"), got, exp[:3], exp[3:]):
        err, bound = np.abs(dev_f64(a) - e), np.maximum(b + HALF * (np.abs(e) + b), 1e-6)
        assert np.all(err <= bound), (name, f"max excess {(err - bound).max():.3e}",
                                      np.unravel_index((err - bound).argmax(), err.shape))
    return got


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("B,Lq,Lk,heads,D,top_k", [
    (1, 1, 1, 1, 32, 1), (1, 128, 128, 2, 64, 1), (2, 129, 640, 3, 32, 2), (1, 1000, 1000, 5, 128, 8),
    (1, 1, 4100, 2, 128, 33), (2, 777, 5000, 2, 64, 39), (1, 9000, 300, 1, 128, 3), (1, 300, 9000, 3, 32, 1),
    (1, 200, 9000, 1, 32, 71), (1, 300, 30000, 2, 32, 17), (1, 300, 82000, 1, 32, 100), (1, 140, 90000, 2, 32, 9),
])
def test_select_matches_oracle(B, Lq, Lk, heads, D, top_k):
    import spacetime_attention_vdit_b200 as vd
    q, k, _ = _inputs(B, Lq, Lk, heads, D, seed=Lq + Lk)
    got = vd.attn_select_blocks(to_dev_bf16(q), to_dev_bf16(k), top_k)
    assert got.dtype == torch.bool
    assert np.array_equal(got.cpu().numpy(), sp.select_blocks(f64(q), f64(k), top_k))


def test_select_ties_go_to_the_lower_block():
    import spacetime_attention_vdit_b200 as vd
    k = _bits(0, 1, 128, 2, 32).repeat(50, axis=0).reshape(1, 50 * 128, 2, 32)       # 50 equal blocks
    q = _bits(1, 1, 300, 2, 32)
    got = vd.attn_select_blocks(to_dev_bf16(q), to_dev_bf16(k), 7).cpu().numpy()
    assert np.all(got[..., :7]) and not got[..., 7:].any()
    zero = vd.attn_select_blocks(to_dev_bf16(q), to_dev_bf16(np.zeros_like(k)), 33).cpu().numpy()
    assert np.all(zero[..., :33]) and not zero[..., 33:].any()
    # scores of +0 and -0 are equal
    signs = np.zeros_like(k)
    signs[:, 128 * 40:] = 0x8000
    zero = vd.attn_select_blocks(to_dev_bf16(q), to_dev_bf16(signs), 33).cpu().numpy()
    assert np.all(zero[..., :33]) and not zero[..., 33:].any()


def test_select_nan_infinite_and_denormal_scores():
    import spacetime_attention_vdit_b200 as vd
    q = np.full((1, 200, 1, 32), 0x3f80, dtype=np.uint16)                  # ones
    k = _bits(3, 1, 128 * 9, 1, 32)
    k[0, 128 * 2 + 5, 0, 3] = 0x7fc0                                       # NaN: behind every number
    k[0, 128 * 3 + 5, 0, 3] = 0xff80                                       # -inf: before NaN only
    k[0, 128 * 4 + 5, 0, 3] = 0x7f80                                       # +inf: first
    k[0, 128 * 5:128 * 6] = 0x0001                                         # the least denormal
    k[0, 128 * 6:128 * 7] = 0x0000
    k[0, 128 * 7:128 * 8] = 0x7f7f                                         # the largest number: a finite score
    for top_k in range(1, 10):
        got = vd.attn_select_blocks(to_dev_bf16(q), to_dev_bf16(k), top_k).cpu().numpy()
        with np.errstate(all="ignore"):
            assert np.array_equal(got, sp.select_blocks(f64(q), f64(k), top_k)), top_k


@pytest.mark.parametrize("n", [40, 200, 300, 700])
def test_select_long_rows_decided_by_the_last_bits(n):
    """Means that agree in their leading 40 bits, and some that are equal: the
    threshold search has to go to the end, at every length of row."""
    import spacetime_attention_vdit_b200 as vd
    k = np.zeros((1, 128 * n, 1, 32), dtype=np.float32)
    k[:, 0::128, 0, 0] = 1024.0
    k[:, 1::128, 0, 0] = np.random.default_rng(n).integers(0, n // 3, n).astype(np.float32) * 2.0 ** -30
    kb = synthetic.f32_to_bf16_bits(k)
    q = np.full((1, 128, 1, 32), 0x3f80, dtype=np.uint16)
    for top_k in (1, 2, n // 4, n // 2, n - 1, n):
        got = vd.attn_select_blocks(to_dev_bf16(q), to_dev_bf16(kb), top_k).cpu().numpy()
        assert np.array_equal(got, sp.select_blocks(f64(q), f64(kb), top_k)), top_k


def test_select_values_next_to_a_border():
    """Blocks whose means differ by one part in 2^40: the choice needs float64."""
    import spacetime_attention_vdit_b200 as vd
    k = np.zeros((1, 128 * 6, 1, 32), dtype=np.float32)
    k[:, 0::128, 0, 0] = 1024.0
    k[:, 1::128, 0, 0] = np.array([3, 1, 5, 0, 2, 4], dtype=np.float32) * 2.0 ** -30
    kb = synthetic.f32_to_bf16_bits(k)
    q = np.full((1, 128, 1, 32), 0x3f80, dtype=np.uint16)
    for top_k, want in ((1, [2]), (2, [2, 5]), (3, [0, 2, 5]), (4, [0, 2, 4, 5]), (5, [0, 1, 2, 4, 5])):
        got = vd.attn_select_blocks(to_dev_bf16(q), to_dev_bf16(kb), top_k).cpu().numpy()
        assert np.flatnonzero(got[0, 0, 0]).tolist() == want


# -------------------------------------------------------------------- forward

SIZES = [
    # B, Lq, Lk, heads, D, keep
    (1, 1, 1, 1, 32, 1.0), (1, 1, 300, 2, 128, 1.0), (1, 128, 128, 1, 64, 1.0), (2, 129, 257, 3, 32, 0.7),
    (1, 300, 1000, 2, 64, 0.5), (2, 1000, 1000, 2, 128, 0.5), (1, 1100, 129, 3, 128, 0.6), (1, 77, 2100, 5, 32, 0.4),
    (1, 1, 4500, 12, 128, 0.6), (3, 5, 3001, 2, 64, 0.5), (1, 257, 4100, 40, 32, 0.3),
]


@pytest.mark.parametrize("B,Lq,Lk,heads,D,keep", SIZES)
def test_forward(B, Lq, Lk, heads, D, keep):
    _check_forward(*_inputs(B, Lq, Lk, heads, D, seed=Lk), _mask(B, Lq, Lk, heads, keep, seed=Lq))


@pytest.mark.parametrize("Lq", [3, 200])
@pytest.mark.parametrize("heads", [5, 24, 40, 80, 200])
def test_forward_at_each_split(heads, Lq):
    """Eight, four, two and one CTA per pair of query blocks, and for a single block."""
    q, k, v = _inputs(1, Lq, 2500, heads, 64, seed=heads)
    on = _mask(1, Lq, 2500, heads, 0.5, seed=1)
    on[:, 0, 0] = False                          # a head whose first block has nothing
    _check_forward(q, k, v, on)


@pytest.mark.parametrize("Lq,heads", [(1, 1), (256, 1), (256, 40), (5000, 8)])
def test_forward_nothing_marked(Lq, heads):
    import spacetime_attention_vdit_b200 as vd
    q, k, v = (to_dev_bf16(x) for x in _inputs(1, Lq, 2500, heads, 64))
    blocks = torch.zeros(1, heads, sp.n_blocks(Lq), 20, dtype=torch.bool, device="cuda")
    o, lse = vd.attn_block_sparse(q, k, v, blocks, out=torch.full_like(q, 7.0), lse=True)
    assert torch.all(o == 0) and torch.all(lse == -torch.inf)
    g = torch.randn_like(q)
    for x in vd.attn_block_sparse_bwd(q, k, v, blocks, o, lse, g, dq=torch.full_like(q, 7.0)):
        assert torch.all(x == 0)


@pytest.mark.parametrize("pattern", ["one", "last", "first_row_only", "second_row_only", "disjoint", "alternating"])
@pytest.mark.parametrize("heads", [1, 90])
def test_forward_patterns_of_two_rows(pattern, heads):
    """The ways two query blocks of a CTA can share key blocks, the ragged last
    one among them."""
    Lq, Lk, nk = 250, 128 * 9 - 50, 9
    on = np.zeros((1, heads, 2, nk), dtype=bool)
    if pattern == "one":
        on[..., 0, 4] = on[..., 1, 4] = True
    elif pattern == "last":
        on[..., nk - 1] = True
    elif pattern == "first_row_only":
        on[..., 0, :] = True
    elif pattern == "second_row_only":
        on[..., 1, 3:] = True
    elif pattern == "disjoint":
        on[..., 0, :2] = on[..., 1, 2:] = True
    else:
        on[..., 0, 0::2] = on[..., 1, 1::2] = True
        on[..., :, 6] = True
    q, k, v = _inputs(1, Lq, Lk, heads, 32, seed=4)
    _check_forward(q, k, v, on)
    _check_backward(q, k, v, on)


@pytest.mark.parametrize("heads", [2, 70])
def test_unmarked_blocks_may_hold_anything(heads):
    """NaN and infinities in key blocks that no row marks, and past the marked ones."""
    import spacetime_attention_vdit_b200 as vd
    q, k, v = _inputs(1, 384, 1000, heads, 64, seed=2)
    on = _mask(1, 384, 1000, heads, 0.5, seed=3)
    on[..., 4] = False
    clean = _check_forward(q, k, v, on)
    k[:, 512:640], v[:, 512:640] = 0x7fc0, 0x7f80
    t = [to_dev_bf16(x) for x in (q, k, v)]
    blocks = torch.from_numpy(on).cuda()
    dirty = vd.attn_block_sparse(*t, blocks, lse=True)
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
    grads = vd.attn_block_sparse_bwd(*t, blocks, *dirty, torch.randn_like(t[0]))
    assert all(torch.isfinite(x).all() for x in grads)
    assert torch.all(grads[1][:, 512:640] == 0) and torch.all(grads[2][:, 512:640] == 0)


@pytest.mark.parametrize("heads", [2, 70])
def test_forward_rising_scores(heads):
    """Later key blocks with far larger scores (the running max moves), at a large
    scale, and rows whose scores are all very negative.  The scores reach 300 in
    log2 units, where the float32 dot product's and argument's rounding is some
    1e-4 of P: the usual bound."""
    Lq, Lk = 256, 1300
    q = np.full((1, Lq, heads, 32), 0.25, dtype=np.float32)
    q[:, 1::2] *= -1
    k = np.random.default_rng(5).standard_normal((1, Lk, heads, 32)).astype(np.float32) * 0.25
    k += (np.arange(Lk) // 128).astype(np.float32)[None, :, None, None] * 4
    v = _bits(6, 1, Lk, heads, 32)
    qb, kb = synthetic.f32_to_bf16_bits(q), synthetic.f32_to_bf16_bits(k)
    on = np.ones((1, heads, 2, 11), dtype=bool)
    _check_forward(qb, kb, v, on)
    _check_forward(qb, kb, v, on, scale=0.5)


def test_all_blocks_marked_is_cross_attention():
    import spacetime_attention_vdit_b200 as vd
    q, k, v = (to_dev_bf16(x) for x in _inputs(2, 1000, 3000, 4, 128))
    on = torch.ones(2, 4, 8, 24, dtype=torch.bool, device="cuda")
    o, lse = vd.attn_block_sparse(q, k, v, on, lse=True)
    eo, el = vd.attn_cross(q, k, v, lse=True)
    # both within their bounds of one and the same value
    assert (lse - el).abs().max() <= 2 * LSE_ABS
    assert (o.float() - eo.float()).abs().max() <= 0.02


def test_masks_as_bytes_and_combined():
    import spacetime_attention_vdit_b200 as vd
    q, k, v = (to_dev_bf16(x) for x in _inputs(1, 512, 1024, 2, 64))
    a, b = (vd.attn_select_blocks(q, x, 3) for x in (k, v))
    o = vd.attn_block_sparse(q, k, v, a | b)
    assert torch.equal(o, vd.attn_block_sparse(q, k, v, (a | b).to(torch.uint8) * 200))


def test_forward_long_sampled():
    """32,760 keys, 12 heads x 128: sampled query blocks against the oracle."""
    import spacetime_attention_vdit_b200 as vd
    L, heads, D = 32760, 12, 128
    q, k, v = _inputs(1, L, L, heads, D, seed=11)
    t = [to_dev_bf16(x) for x in (q, k, v)]
    on = vd.attn_select_blocks(t[0], t[1], 20)
    o, lse = vd.attn_block_sparse(*t, on, lse=True)
    host = on.cpu().numpy()
    for i, h in ((0, 0), (1, 11), (127, 3), (254, 7), (255, 5)):
        rows = slice(128 * i, min(L, 128 * (i + 1)))
        _check_forward(q[:, rows, h:h + 1], k[:, :, h:h + 1], v[:, :, h:h + 1], host[:, h:h + 1, i:i + 1],
                       got=(o[:, rows, h:h + 1].contiguous(), lse[:, h:h + 1, rows].contiguous()))


def test_offsets_past_32_bits():
    """2.7e9 elements per tensor: the last clip's rows against a call on that clip alone."""
    import spacetime_attention_vdit_b200 as vd
    B, L, heads, D = 7, 75600, 40, 128
    gen = torch.Generator(device="cuda").manual_seed(0)

    def make():
        x = torch.empty(B, L, heads, D, dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            x[b] = torch.randn(L, heads, D, device="cuda", generator=gen)
        return x

    q, k, v = make(), make(), make()
    on = vd.attn_select_blocks(q, k, 2)
    last = slice(B - 1, B)
    on1 = vd.attn_select_blocks(q[last], k[last], 2)
    assert torch.equal(on[last], on1)
    o, lse = vd.attn_block_sparse(q, k, v, on, lse=True)
    o1, lse1 = vd.attn_block_sparse(q[last], k[last], v[last], on1, lse=True)
    assert torch.equal(o[last], o1) and torch.equal(lse[last], lse1)
    got = vd.attn_block_sparse_bwd(q, k, v, on, o, lse, v)
    one = vd.attn_block_sparse_bwd(q[last], k[last], v[last], on1, o1, lse1, v[last])
    for a, b in zip(got, one):
        assert torch.equal(a[last], b)


# ------------------------------------------------------------------ gradients

@pytest.mark.parametrize("B,Lq,Lk,heads,D,keep", SIZES)
def test_backward(B, Lq, Lk, heads, D, keep):
    _check_backward(*_inputs(B, Lq, Lk, heads, D, seed=Lk), _mask(B, Lq, Lk, heads, keep, seed=Lq))


def test_backward_scale():
    _check_backward(*_inputs(1, 300, 500, 2, 64, seed=1), np.ones((1, 2, 3, 4), dtype=bool), scale=0.3)


def test_backward_is_the_difference_quotient():
    """Differences of the float64 forward along seeded directions: sum(dO . dO/dx) =
    dx . direction.  Each gradient element is off by its bound at most, so their
    sum along a direction of signs is off by the sum of the bounds."""
    import spacetime_attention_vdit_b200 as vd
    q, k, v = _inputs(1, 200, 300, 2, 32, seed=20)
    on = _mask(1, 200, 300, 2, 0.8, seed=21)
    g = _bits(22, 1, 200, 2, 32)
    t = [to_dev_bf16(x) for x in (q, k, v)]
    blocks = torch.from_numpy(on).cuda()
    o, lse = vd.attn_block_sparse(*t, blocks, lse=True)
    got = vd.attn_block_sparse_bwd(*t, blocks, o, lse, to_dev_bf16(g))
    x = [f64(a) for a in (q, k, v)]
    eo, el = sp.attention(*x, on)
    bounds = sp.attention_bwd(*x, on, eo, el, f64(g), with_magnitudes=True, rel_p=HALF + E_P, rel_ds=HALF + E_P,
                              acc=32 * 2.0 ** -23)
    delta_err = (np.abs(f64(g)) * HALF * np.abs(eo)).sum(-1)                       # delta from the rounded O
    p_err = [HALF, HALF, 0.0]
    h = 1e-5
    for i, name in enumerate(("dq", "dk", "dv")):
        sign = np.where(np.random.default_rng(30 + i).random(x[i].shape) < 0.5, -1.0, 1.0)
        up, down = ([a + s * h * sign if j == i else a for j, a in enumerate(x)] for s in (1, -1))
        want = ((sp.attention(*up, on)[0] - sp.attention(*down, on)[0]) * f64(g)).sum() / (2 * h)
        value = (dev_f64(got[i]) * sign).sum()
        bound = (bounds[3 + i] + HALF * (np.abs(bounds[i]) + bounds[3 + i])).sum()
        if p_err[i]:
            # sum_j P delta_err |x_j| scale over all elements: at most delta_err * D * max|x| * scale per row
            other = x[1 - i]
            bound += delta_err.sum() * 32 * np.abs(other).max() * 32 ** -0.5
        assert abs(value - want) <= bound, (name, value, want, bound)


# ----------------------------------------------------------- how it is called

def test_runs_repeat_bit_for_bit():
    import spacetime_attention_vdit_b200 as vd
    q, k, v = (to_dev_bf16(x) for x in _inputs(1, 1500, 4000, 6, 128))
    on = vd.attn_select_blocks(q, k, 9)
    first = None
    for _ in range(3):
        o, lse = vd.attn_block_sparse(q, k, v, on, lse=True)
        out = (o, lse, *vd.attn_block_sparse_bwd(q, k, v, on, o, lse, q))
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, out))
        first = out


def test_other_stream_and_graphs():
    """The chain on a side stream (by argument), and two captured graphs replayed
    in turn and together, against the plain calls."""
    import spacetime_attention_vdit_b200 as vd
    sets = [[to_dev_bf16(x) for x in _inputs(1, 700, 1900, 3, 64, seed=s)] for s in (40, 50)]

    def chain(q, k, v, stream=None):
        on = vd.attn_select_blocks(q, k, 4, stream=stream)
        o, lse = vd.attn_block_sparse(q, k, v, on, lse=True, stream=stream)
        return on, o, lse, *vd.attn_block_sparse_bwd(q, k, v, on, o, lse, q, stream=stream)

    plain = [chain(*s) for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        got = chain(*sets[0], stream=handle)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(plain[0], got))
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(chain(*s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for together in (False, True):
        for o in outs:
            for x in o:
                x.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
            if not together:
                st.synchronize()
        torch.cuda.synchronize()
        for p, o in zip(plain, outs):
            assert all(torch.equal(a, b) for a, b in zip(p, o))


def test_outputs_given_and_rows_behind_the_last_left_alone():
    """Outputs inside a larger buffer: nothing past the sequence is touched."""
    import spacetime_attention_vdit_b200 as vd
    q, k, v = (to_dev_bf16(x) for x in _inputs(1, 200, 300, 2, 64))
    on = torch.ones(1, 2, 2, 3, dtype=torch.bool, device="cuda")

    def room(x):
        buf = torch.full((1, x.shape[1] + 56, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        return buf, buf[:, :x.shape[1]]

    (bo, o), (bq, dq), (bk, dk), (bv, dv) = room(q), room(q), room(k), room(v)
    o2, lse = vd.attn_block_sparse(q, k, v, on, out=o, lse=True)
    assert o2.data_ptr() == o.data_ptr()
    vd.attn_block_sparse_bwd(q, k, v, on, o, lse, q, dq=dq, dk=dk, dv=dv)
    for buf, n in ((bo, 200), (bq, 200), (bk, 300), (bv, 300)):
        assert torch.all(buf[:, n:] == 7.0) and torch.any(buf[:, :n] != 7.0)


def test_first_call_may_be_captured(tmp_path):
    """A fresh process whose first call of each new operator is inside a capture."""
    import subprocess
    import sys
    from tests.conftest import ROOT
    code = """
import torch, spacetime_attention_vdit_b200 as vd
q, k, v = (torch.randn(1, 512, 2, 64, device="cuda").bfloat16() for _ in range(3))
w = torch.ones(64, device="cuda")
def chain():
    qn, kn = q, k
    on = vd.attn_select_blocks(qn, kn, 2)
    o, lse = vd.attn_block_sparse(qn, kn, v, on, lse=True)
    dq, dk, dv = vd.attn_block_sparse_bwd(qn, kn, v, on, o, lse, v)
    a = vd.qk_norm_rope_3d_bwd(q, k, dq, dk, (2, 16, 16), 64, w, w)
    b = vd.rope_3d_bwd(dq, dk, (2, 16, 16))
    return (on, o, lse, dq, dk, dv, *a, *b)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = chain()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, chain()))
assert vd.device_status() == (0, 0)
print("captured first")
"""
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert res.returncode == 0 and "captured first" in res.stdout, res.stdout[-2000:] + res.stderr[-3000:]
