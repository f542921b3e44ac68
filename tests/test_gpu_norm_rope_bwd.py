"""GPU parity of the gradients of Q/K RMSNorm + 3D rotation, and of the rotation
alone, against the float64 definitions of oracle/sparse.py; and the whole chain
of a sub-layer's gradients.

Bounds (bf16 in, float32 arithmetic, one bf16 rounding of half a step, 2^-8):
* rotation back: two products and a sum of float32 values, (cos, sin) rounded to
  float32: |err| <= 2^-8 |dx| + 2^-21 (|g0| + |g1|);
* dx of the norm: u as above; r from a float32 sum of squares (at most 32 terms in
  sequence in a thread and 16 levels of adding threads: 48 * 2^-24) and rsqrtf
  (2^-22); mean(x u w) alike: each term of dx is good to 2e-5 of its magnitude
  (the magnitudes oracle/sparse.py returns): |err| <= 2^-8 |dx| + 2e-5 mag;
* dw: float32 sums, at most ceil(tokens / CTAs) * 4 + 300 terms in sequence:
  |err| <= ((tokens / CTAs + 1) * 4 + 300) * 2^-24 mag + 2e-5 mag, CTAs =
  min(tokens, 148)."""
import numpy as np
import pytest
import torch

import synthetic
from oracle import reference as ref
from oracle import sparse as sp
from tests.gpu_util import dev_f64, from_dev_bf16, to_dev_bf16, watchdog_clear

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
f64 = synthetic.bf16_bits_to_f64


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import spacetime_attention_vdit_b200 as v  # noqa: F401
    yield
    watchdog_clear()


def _bits(seed, *shape, scale=1.0):
    return synthetic.f32_to_bf16_bits((np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32))


def _weight(seed, group):
    return (np.random.default_rng(seed).standard_normal(group) * 0.5 + 1.0).astype(np.float32)


def _check_dx(got, exp, mag, what):
    err, bound = np.abs(dev_f64(got) - exp), HALF * np.abs(exp) + mag
    assert np.all(err <= bound), (what, f"max excess {(err - bound).max():.3e}")


GRIDS = [
    (1, (8, 8, 8), 2, 32, (12, 10, 10)), (2, (3, 4, 5), 3, 64, (22, 20, 22)), (1, (1, 1, 1), 4, 128, (44, 42, 42)),
    (1, (2, 3, 7), 2, 128, (44, 42, 42)), (2, (3, 5, 6), 2, 128, (0, 64, 64)), (1, (5, 30, 52), 12, 128, (44, 42, 42)),
]


@pytest.mark.parametrize("B,grid,heads,D,split", GRIDS)
def test_rope_bwd(B, grid, heads, D, split):
    import spacetime_attention_vdit_b200 as vd
    L = grid[0] * grid[1] * grid[2]
    bits = [_bits(i, B, L, heads, D) for i in range(2)]
    dev = [to_dev_bf16(x) for x in bits]
    got = vd.rope_3d_bwd(*dev, grid, split)
    for x, g in zip(bits, got):
        a = np.abs(f64(x))
        pair = (a[..., 0::2] + a[..., 1::2]).repeat(2, axis=-1)
        _check_dx(g, sp.rope_3d_bwd(f64(x), grid, split), 2.0 ** -21 * pair, "dx")
    only_k = vd.rope_3d_bwd(None, dev[1], grid, split)
    assert only_k[0] is None and torch.equal(only_k[1], got[1])
    vd.rope_3d_bwd(*dev, grid, split, dq=dev[0], dk=dev[1])            # in place
    assert torch.equal(dev[0], got[0]) and torch.equal(dev[1], got[1])


def test_rope_forward_is_unchanged_by_its_gradient():
    """The rotation turned back is the transpose: <R x, y> = <x, R^T y> on values
    whose products are exact, and the forward still equals the float32 restatement."""
    import spacetime_attention_vdit_b200 as vd
    grid, split = (3, 4, 5), (44, 42, 42)
    x = _bits(0, 1, 60, 2, 128)
    q, _ = vd.rope_3d(to_dev_bf16(x), to_dev_bf16(x), grid, split)
    exp = synthetic.f32_to_bf16_bits(ref.rope_3d_fp32(synthetic.bf16_bits_to_f32(x), grid, split))
    assert np.array_equal(from_dev_bf16(q), exp)


def _check_norm(B, grid, heads, D, split, group, eps=1e-6, weighted=True, seed=5, x_scale=3.0):
    import spacetime_attention_vdit_b200 as vd
    L = grid[0] * grid[1] * grid[2]
    q, k = _bits(seed, B, L, heads, D, scale=x_scale), _bits(seed + 1, B, L, heads, D)
    gq, gk = _bits(seed + 2, B, L, heads, D), _bits(seed + 3, B, L, heads, D)
    w = [_weight(seed + 4 + i, group) if weighted else None for i in range(2)]
    wd = [None if x is None else torch.from_numpy(x).cuda() for x in w]
    dev = [to_dev_bf16(x) for x in (q, k, gq, gk)]
    dq, dk, dwq, dwk = vd.qk_norm_rope_3d_bwd(*dev, grid, group, *wd, eps=eps, split=split)
    n = (B * L / min(B * L, 148) + 1) * 4 + 300
    for x, g, wt, dx, dw in ((q, gq, w[0], dq, dwq), (k, gk, w[1], dk, dwk)):
        edx, edw, mx, mw = sp.qk_norm_rope_3d_bwd(f64(x), f64(g), grid, split, group, wt, eps, with_magnitudes=True)
        _check_dx(dx, edx, 2e-5 * mx, "dx")
        if weighted:
            err = np.abs(dw.cpu().numpy().astype(np.float64) - edw)
            assert np.all(err <= (n * 2.0 ** -24 + 2e-5) * mw), f"dw max {err.max():.3e}"
        else:
            assert dw is None
    only_k = vd.qk_norm_rope_3d_bwd(None, dev[1], None, dev[3], grid, group, None, wd[1], eps=eps, split=split)
    assert only_k[0] is None and only_k[2] is None and torch.equal(only_k[1], dk)
    if weighted:
        # K alone is split over more CTAs, so its sums are taken in another order
        assert np.all(np.abs(only_k[3].cpu().numpy().astype(np.float64) - edw) <= (n * 2.0 ** -24 + 2e-5) * mw)
        again = vd.qk_norm_rope_3d_bwd(*dev, grid, group, *wd, eps=eps, split=split)
        assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dwq, dwk)))


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("B,grid,heads,D,split", GRIDS)
def test_norm_rope_bwd(B, grid, heads, D, split, per_token):
    _check_norm(B, grid, heads, D, split, heads * D if per_token else D)


@pytest.mark.parametrize("heads,D,split,group", [
    (64, 128, (44, 42, 42), 8192),       # the widest token
    (64, 128, (44, 42, 42), 128),
    (40, 128, (44, 42, 42), 5120),
    (2, 128, (44, 42, 42), 64),          # two groups per head
    (2, 64, (22, 20, 22), 8),            # one vector per group
    (1, 8, (2, 2, 4), 8),
])
def test_norm_rope_bwd_widths(heads, D, split, group):
    _check_norm(1, (2, 5, 31), heads, D, split, group)


def test_norm_rope_bwd_unweighted_and_large_eps():
    _check_norm(1, (3, 5, 6), 4, 128, (44, 42, 42), 512, eps=0.75, weighted=False)
    _check_norm(1, (3, 5, 6), 4, 128, (44, 42, 42), 128, eps=0.75)


def test_norm_rope_bwd_one_weight_only():
    """A weight on K alone: dwk is as with both, Q's slot stays empty."""
    import spacetime_attention_vdit_b200 as vd
    x = [to_dev_bf16(_bits(i, 1, 60, 2, 64)) for i in range(4)]
    w = torch.from_numpy(_weight(9, 64)).cuda()
    both = vd.qk_norm_rope_3d_bwd(*x, (3, 4, 5), 64, w, w, split=(22, 20, 22))
    one = vd.qk_norm_rope_3d_bwd(*x, (3, 4, 5), 64, None, w, split=(22, 20, 22))
    assert one[2] is None and torch.equal(one[1], both[1]) and torch.equal(one[3], both[3])


def test_norm_rope_bwd_zero_rows():
    """Tokens of zeros (padding): r = eps^-1/2, dx = r u w, finite."""
    import spacetime_attention_vdit_b200 as vd
    x = torch.zeros(1, 60, 2, 64, dtype=torch.bfloat16, device="cuda")
    g = to_dev_bf16(_bits(1, 1, 60, 2, 64))
    w = torch.ones(64, device="cuda")
    dq, dk, dwq, dwk = vd.qk_norm_rope_3d_bwd(x, x, g, g, (3, 4, 5), 64, w, w, eps=1e-6, split=(22, 20, 22))
    exp = sp.rope_3d_bwd(f64(from_dev_bf16(g)), (3, 4, 5), (22, 20, 22)) * 1e3
    _check_dx(dq, exp, 1e-5 * 1e3 * 10, "dx")
    assert torch.equal(dq, dk) and torch.all(dwq == 0) and torch.all(dwk == 0)


@pytest.mark.parametrize("stream", [False, True])
def test_sub_layer_chain(stream):
    """Norm + rotation -> selection -> sparse attention, and the gradients back to
    the projected Q, K, V and the norm weights.  Each step is checked by itself
    above; here every gradient is compared with the float64 gradient of the
    whole chain at the GPU's own selection.  The chain rounds q', k', O, dq', dk' to
    bf16, each off by half a step (2^-8): to first order the relative error of
    each gradient in the l2 norm is below the sum of what each rounding does to it.
    A rounding of q' and k' moves a score by 2^-8 sqrt(2 sum q^2 k^2) scale <= 2^-8
    * 1.5 (normalised q', k' have unit mean square), that is P by 6e-3, and the
    rounding of P, dS, O (in delta), dq' and dk' by 2^-8 each: below 0.03 in all."""
    import spacetime_attention_vdit_b200 as vd
    grid, split, heads, D = (4, 10, 16), (44, 42, 42), 2, 128
    L = 640
    q, k, v, g = (_bits(60 + i, 1, L, heads, D) for i in range(4))
    w = [_weight(70 + i, D) for i in range(2)]
    dev = [to_dev_bf16(x) for x in (q, k, v, g)]
    wd = [torch.from_numpy(x).cuda() for x in w]
    st = torch.cuda.Stream() if stream else None
    if st:
        st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st) if st else torch.cuda.stream(torch.cuda.current_stream()):
        qn, kn = vd.qk_norm_rope_3d(dev[0], dev[1], grid, D, *wd, split=split)
        on = vd.attn_select_blocks(qn, kn, 2)
        o, lse = vd.attn_block_sparse(qn, kn, dev[2], on, lse=True)
        gqn, gkn, gv = vd.attn_block_sparse_bwd(qn, kn, dev[2], on, o, lse, dev[3])
        gq, gk, gwq, gwk = vd.qk_norm_rope_3d_bwd(dev[0], dev[1], gqn, gkn, grid, D, *wd, split=split)
    torch.cuda.synchronize()
    host = on.cpu().numpy()
    assert np.array_equal(host, sp.select_blocks(dev_f64(qn), dev_f64(kn), 2))
    x = [f64(a) for a in (q, k, v)]
    n = [ref.qk_norm_rope_3d(a, grid, split, D, wt, 1e-6) for a, wt in zip(x, w)]
    eo, el = sp.attention(*n, x[2], host)
    en = sp.attention_bwd(*n, x[2], host, eo, el, f64(g))
    eq, ewq = sp.qk_norm_rope_3d_bwd(x[0], en[0], grid, split, D, w[0])
    ek, ewk = sp.qk_norm_rope_3d_bwd(x[1], en[1], grid, split, D, w[1])
    for name, a, b in (("o", dev_f64(o), eo), ("dv", dev_f64(gv), en[2]), ("dq", dev_f64(gq), eq), ("dk", dev_f64(gk), ek),
                       ("dwq", gwq.cpu().numpy(), ewq), ("dwk", gwk.cpu().numpy(), ewk)):
        rel = np.linalg.norm(a - b) / np.linalg.norm(b)
        assert rel <= 0.03, (name, rel)
