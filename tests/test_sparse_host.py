"""Host-side checks of the sparse-attention and gradient calls (no GPU needed):
every refusal returns before CUDA is touched."""
import ctypes

import pytest
import torch

from tests.test_abi_host import ALIGN, FAKE, L, MIS, NULL, SHAPE, UNSUP  # noqa: F401  (L: fixture)

F = ctypes.c_float


def select(L, q=FAKE, k=FAKE, out=FAKE, ws=FAKE, B=1, Lq=500, Lk=700, heads=2, D=128, top_k=3):
    return L.vdit_attn_select_blocks(q, k, out, ws, B, Lq, Lk, heads, D, top_k, None)


def test_select_validation(L):
    for name in ("q", "k", "out", "ws"):
        assert select(L, **{name: None}) == NULL
    assert select(L, D=48) == UNSUP
    assert select(L, Lq=0) == SHAPE
    assert select(L, Lk=-1) == SHAPE
    assert select(L, B=0) == SHAPE
    assert select(L, heads=0) == SHAPE
    assert select(L, top_k=0) == SHAPE
    assert select(L, top_k=7) == SHAPE                 # six key blocks
    assert select(L, Lk=6144 * 128 + 1) == UNSUP
    assert select(L, q=MIS) == ALIGN
    assert select(L, ws=MIS) == ALIGN
    assert select(L, B=70000) == SHAPE                 # past the grid's extent


def test_workspaces(L):
    f = L.vdit_attn_select_blocks_workspace
    assert f(1, 500, 700, 2, 128) >= 8 * 2 * (4 + 6) * 128
    assert f(0, 500, 700, 2, 128) == -1 and f(1, 500, 0, 2, 128) == -1
    g = L.vdit_attn_block_sparse_bwd_workspace
    assert g(2, 500, 3) == 2 * 2 * 3 * 512 * 4
    assert g(2, 0, 3) == -1
    h = L.vdit_qk_norm_rope_3d_bwd_workspace
    assert h(128) > 0 and h(0) == -1
    # sizes past 32 bits are counted in 64
    assert g(1000, 75600, 40) == 2 * 1000 * 40 * 591 * 128 * 4
    assert f(100, 75600, 75600, 40, 128) > 2 ** 32


def sparse(L, q=FAKE, k=FAKE, v=FAKE, blocks=FAKE, o=FAKE, lse=None, B=1, Lq=500, Lk=700, heads=2, D=128):
    return L.vdit_attn_block_sparse(q, k, v, blocks, o, lse, B, Lq, Lk, heads, D, F(0.0), None)


def test_block_sparse_validation(L):
    for name in ("q", "k", "v", "blocks", "o"):
        assert sparse(L, **{name: None}) == NULL
    for name in ("q", "k", "v", "o"):
        assert sparse(L, **{name: MIS}) == ALIGN
    assert sparse(L, lse=FAKE + 2) == ALIGN
    assert sparse(L, D=48) == UNSUP
    assert sparse(L, Lk=6144 * 128 + 1) == UNSUP
    for name in ("B", "Lq", "Lk", "heads"):
        assert sparse(L, **{name: 0}) == SHAPE
        assert sparse(L, **{name: -3}) == SHAPE


def sparse_bwd(L, B=1, Lq=500, Lk=700, heads=2, D=128, **kw):
    a = {n: kw.get(n, FAKE) for n in ("q", "k", "v", "blocks", "o", "lse", "d_o", "dq", "dk", "dv", "ws")}
    return L.vdit_attn_block_sparse_bwd(*a.values(), B, Lq, Lk, heads, D, F(0.0), None)


def test_block_sparse_bwd_validation(L):
    for name in ("q", "k", "v", "blocks", "o", "lse", "d_o", "dq", "dk", "dv", "ws"):
        assert sparse_bwd(L, **{name: None}) == NULL
        if name not in ("blocks", "lse"):
            assert sparse_bwd(L, **{name: MIS}) == ALIGN
    assert sparse_bwd(L, lse=FAKE + 2) == ALIGN
    assert sparse_bwd(L, D=96) == UNSUP
    assert sparse_bwd(L, Lq=6144 * 128 + 1) == UNSUP
    assert sparse_bwd(L, Lk=6144 * 128 + 1) == UNSUP
    assert sparse_bwd(L, Lk=0) == SHAPE
    assert sparse_bwd(L, heads=-1) == SHAPE


def rope_bwd(L, gq=FAKE, gk=FAKE, dq=FAKE, dk=FAKE, B=1, Tg=2, Hg=3, Wg=4, heads=2, D=128, split=(44, 42, 42),
             theta=10000.0):
    return L.vdit_rope_3d_bwd(gq, gk, dq, dk, B, Tg, Hg, Wg, heads, D, *split, F(theta), None)


def test_rope_bwd_validation(L):
    assert rope_bwd(L, gq=None) == NULL
    assert rope_bwd(L, dk=None) == NULL
    assert rope_bwd(L, gq=None, dq=None, gk=None) == NULL
    assert rope_bwd(L, split=(44, 42, 40)) == SHAPE
    assert rope_bwd(L, Hg=0) == SHAPE
    assert rope_bwd(L, theta=-1.0) == SHAPE
    assert rope_bwd(L, D=36, split=(12, 12, 12)) == UNSUP
    assert rope_bwd(L, dq=MIS) == ALIGN


def norm_bwd(L, group=128, eps=1e-6, B=1, grid=(2, 3, 4), heads=2, D=128, split=(44, 42, 42), theta=10000.0, **kw):
    names = ("q", "k", "gq", "gk", "dq", "dk", "wq", "wk", "dwq", "dwk", "ws")
    a = [kw.get(n, FAKE) for n in names]
    return L.vdit_qk_norm_rope_3d_bwd(*a, group, F(eps), B, *grid, heads, D, *split, F(theta), None)


def test_norm_rope_bwd_validation(L):
    for name in ("q", "k", "gq", "gk", "dq", "dk", "ws"):
        assert norm_bwd(L, **{name: None}) == NULL
        assert norm_bwd(L, **{name: MIS}) == ALIGN
    assert norm_bwd(L, q=None, gq=None, dq=None, k=None) == NULL
    assert norm_bwd(L, wk=MIS) == ALIGN
    assert norm_bwd(L, group=0) == SHAPE
    assert norm_bwd(L, group=96) == SHAPE
    assert norm_bwd(L, eps=-1.0) == SHAPE
    assert norm_bwd(L, eps=float("nan")) == SHAPE
    assert norm_bwd(L, split=(44, 42, 40)) == SHAPE
    assert norm_bwd(L, grid=(2, 0, 4)) == SHAPE
    assert norm_bwd(L, B=0) == SHAPE
    assert norm_bwd(L, group=12, D=24, split=(8, 8, 8)) == UNSUP
    assert norm_bwd(L, heads=3, D=32, split=(12, 10, 10), group=48) == UNSUP
    assert norm_bwd(L, heads=72) == UNSUP
    assert norm_bwd(L, grid=(400, 1, 1)) == UNSUP      # 8,800 table entries


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals(L):
    """Shapes, types and the device are checked before any pointer is taken."""
    import spacetime_attention_vdit_b200 as vd
    q, k = _t(1, 200, 2, 32), _t(1, 300, 2, 32)
    on = _t(1, 2, 2, 3, dtype=torch.bool)
    lse = _t(1, 2, 200, dtype=torch.float32)
    calls = {
        "select": lambda **a: vd.attn_select_blocks(a.get("q", q), a.get("k", k), 1),
        "sparse": lambda **a: vd.attn_block_sparse(a.get("q", q), a.get("k", k), a.get("k", k), a.get("on", on)),
        "bwd": lambda **a: vd.attn_block_sparse_bwd(a.get("q", q), a.get("k", k), a.get("k", k), a.get("on", on),
                                                    a.get("q", q), lse, a.get("q", q)),
        "rope": lambda **a: vd.rope_3d_bwd(a.get("q", q), a.get("q", q), (2, 10, 10)),
        "norm": lambda **a: vd.qk_norm_rope_3d_bwd(*[a.get("q", q)] * 4, (2, 10, 10), 32),
    }
    for f in calls.values():
        with pytest.raises(ValueError, match="CUDA"):
            f()
    for name in ("select", "sparse", "bwd"):
        with pytest.raises(ValueError, match="heads"):
            calls[name](k=_t(1, 300, 3, 32))
        with pytest.raises(ValueError, match="head_dim"):
            calls[name](q=_t(200, 2, 32))
    for name in ("rope", "norm"):
        with pytest.raises(ValueError, match="grid"):
            calls[name](q=_t(1, 201, 2, 32))


class _Pretend:
    """A stand-in that calls itself a CUDA tensor (no GPU here): only what the
    argument checks look at."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16, device="cuda:0", contiguous=True):
        self.shape, self.dtype, self.device, self._c = torch.Size(shape), dtype, torch.device(device), contiguous

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._c

    def data_ptr(self):
        return FAKE


@pytest.fixture
def pretend(monkeypatch):
    import spacetime_attention_vdit_b200 as vd

    def dev(t, name, dtype=None):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        return t.data_ptr()

    def same(device, **tensors):
        for name, t in tensors.items():
            if t is not None and t.device != device:
                raise ValueError(f"{name} is on {t.device}, not on {device}")

    monkeypatch.setattr(vd, "_dev", dev)
    monkeypatch.setattr(vd, "_same_device", same)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    return vd


def test_block_masks_are_checked(pretend):
    q, k = _Pretend(1, 200, 2, 32), _Pretend(1, 300, 2, 32)
    for bad, text in ((_Pretend(1, 2, 3, 2, dtype=torch.bool), "ceil"), (_Pretend(1, 1, 2, 3, dtype=torch.bool), "ceil"),
                      (_Pretend(1, 2, 2, 3, dtype=torch.int32), "uint8"),
                      (_Pretend(1, 2, 2, 3, dtype=torch.bool, contiguous=False), "contiguous")):
        with pytest.raises(ValueError, match=text):
            pretend.attn_block_sparse(q, k, k, bad)


def test_tensors_of_another_device_are_refused(pretend):
    """Inputs of two devices, and a device that is not the current one."""
    on = _Pretend(1, 2, 2, 3, dtype=torch.bool)
    q, k = _Pretend(1, 200, 2, 32), _Pretend(1, 300, 2, 32)
    with pytest.raises(ValueError, match="not on cuda:0"):
        pretend.attn_block_sparse(q, _Pretend(1, 300, 2, 32, device="cuda:1"), k, on)
    with pytest.raises(ValueError, match="current device"):
        pretend.attn_block_sparse(q, k, k, on)
    with pytest.raises(ValueError, match="current device"):
        pretend.attn_select_blocks(q, k, 1)
    with pytest.raises(ValueError, match="current device"):
        pretend.rope_3d_bwd(q, q, (2, 10, 10))


def test_a_stream_of_another_device_is_refused(pretend, monkeypatch):
    class Stream:
        device, cuda_stream = torch.device("cuda:1"), 0

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    q = _Pretend(1, 200, 2, 32)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        pretend.attn_select_blocks(q, q, 1, stream=Stream())
