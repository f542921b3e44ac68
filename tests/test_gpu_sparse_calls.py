"""How the sparse-attention and gradient calls are made on the GPU."""
import pytest
import torch

from tests.gpu_util import watchdog_clear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    watchdog_clear()


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _every_call(q, k, v, stream):
    import spacetime_attention_vdit_b200 as vd
    grid, w = (2, 16, 16), torch.ones(64, device="cuda")
    on = vd.attn_select_blocks(q, k, 2, stream=stream)
    o, lse = vd.attn_block_sparse(q, k, v, on, lse=True, stream=stream)
    grads = vd.attn_block_sparse_bwd(q, k, v, on, o, lse, v, stream=stream)
    return (on, o, lse, *grads, *vd.rope_3d_bwd(q, k, grid, stream=stream),
            *vd.qk_norm_rope_3d_bwd(q, k, v, v, grid, 64, w, w, stream=stream))


def test_the_default_streams_handle():
    """Handle 0: the calls run in order with the work queued on the default stream
    before them (a fill that is still running when they are made)."""
    import spacetime_attention_vdit_b200 as vd
    handle = torch.cuda.default_stream().cuda_stream
    q, k, v = (_randn(s, 1, 512, 2, 64) for s in range(3))
    assert handle == 0 and vd._launch_stream(q, "q", handle)[1] == 0
    plain = _every_call(q, k, v, None)
    late = [torch.zeros_like(x) for x in (q, k, v)]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)                # some 25 ms
    for a, b in zip(late, (q, k, v)):
        a.copy_(b)
    got = _every_call(*late, handle)
    assert all(torch.equal(a, b) for a, b in zip(plain, got))
