"""Operators of sparse and trainable spacetime attention, as cases to be timed.

Four operators, each in a plain form (elementary torch operations) and through
the library's public calls:

* ``select``         a cheap score (the product of the mean query and the mean
                     key of two 128-token blocks) picks each query block's
                     ``top_k`` key blocks;
* ``sparse``         attention of each query block over its picked key blocks;
* ``sparse_bwd``     the gradients of that attention;
* ``norm_rope_bwd``  the gradients of Q/K RMSNorm followed by the 3D rotation
                     (of the rotation alone where ``group`` is 0).

Tokens are [B, L, heads, head_dim] bfloat16, block masks [B, heads,
ceil(Lq/128), ceil(Lk/128)] truth values.  All arithmetic of the plain forms is
float32, apart from the block scores and the rotation's angles (float64: a
selection is decided by values next to a border, and far positions need their
whole angle).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128                 # tokens of a query block and of a key block
EPS = 1e-6
THETA = 10000.0
MOST_ELEMENTS = 1 << 28     # elements of one intermediate of the plain forms


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # the tiny clip of the unit tests and the smoke check: launch latency
        dict(name="select_tiny", op="select", B=1, Lq=512, Lk=512, heads=2, D=32, top_k=2),
        # 81 frames of 832x480 (21 x 30 x 52 tokens), width 5120
        dict(name="select_480p81", op="select", B=1, Lq=32760, Lk=32760, heads=40, D=128, top_k=32),
        # 81 frames of 1280x720 (21 x 45 x 80 tokens)
        dict(name="select_720p81", op="select", B=1, Lq=75600, Lk=75600, heads=40, D=128, top_k=74),
        # one query token over a long cache of keys: the work is one long row
        dict(name="sparse_one_token", op="sparse", B=1, Lq=1, Lk=32760, heads=12, D=128, top_k=64, mask="top"),
        # the next latent frame of a streamed 480p clip over what came before it
        dict(name="sparse_one_frame", op="sparse", B=1, Lq=1560, Lk=14040, heads=12, D=128, top_k=20, mask="top"),
        # two clips of unequal length in one padded batch, a window over time
        # and the first frame; the padding's rows are empty
        dict(name="sparse_window_padded", op="sparse", B=2, Lq=7001, Lk=7001, heads=20, D=64, top_k=11,
             mask="window"),
        # one forward pass of the 720p clip at an eighth of the blocks
        dict(name="sparse_720p81", op="sparse", B=1, Lq=75600, Lk=75600, heads=40, D=128, top_k=74, mask="top"),
        # training on short clips: 17 frames of 832x480 (5 x 30 x 52 tokens)
        dict(name="sparse_bwd_480p17", op="sparse_bwd", B=1, Lq=7800, Lk=7800, heads=12, D=128, top_k=12, mask="top"),
        # the padded batch, trained
        dict(name="sparse_bwd_window_padded", op="sparse_bwd", B=2, Lq=7001, Lk=7001, heads=20, D=64, top_k=11,
             mask="window"),
        # one training pass of the 81-frame 480p clip
        dict(name="sparse_bwd_480p81", op="sparse_bwd", B=1, Lq=32760, Lk=32760, heads=40, D=128, top_k=32,
             mask="top"),
        # per-head norm at the 17-frame clip
        dict(name="norm_rope_bwd_480p17", op="norm_rope_bwd", B=1, T=5, H=30, W=52, heads=12, D=128, group=128),
        # the token-wide norm at the 720p clip
        dict(name="norm_rope_bwd_720p81", op="norm_rope_bwd", B=1, T=21, H=45, W=80, heads=40, D=128, group=5120),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "sparse", "sparse", "sparse_bwd", "sparse_bwd", "norm_rope_bwd"])
    heads = rng.choice([1, 2, 3, 5, 8, 12, 20, 40])
    D = rng.choice([32, 64, 128, 128])
    if op == "norm_rope_bwd":
        while True:
            T, H, W = _spread(rng, 1, 24), _spread(rng, 1, 48), _spread(rng, 1, 80)
            B = rng.choice([1, 1, 2])
            if B * T * H * W * heads * D <= 21 * 45 * 80 * 40 * 128:
                break
        group = rng.choice([0, D, heads * D])
        return dict(op=op, B=B, T=T, H=H, W=W, heads=heads, D=D, group=group)
    most = 75600 if op != "sparse_bwd" else 32760
    B = rng.choice([1, 1, 2])
    while True:
        Lk = _spread(rng, 64, most)
        Lq = Lk if rng.random() < 0.6 else _spread(rng, 1, most)
        if op == "select":
            if B * (Lq + Lk) * heads * D <= 2 * 75600 * 40 * 128 and B * heads * Lq * Lk <= 75600 ** 2 * 40:
                break
            continue
        top_k = _spread(rng, 1, _ceil(Lk))
        cap = (75600 * 74 * 40 if op == "sparse" else 32760 * 32 * 40) * 128
        if B * heads * (Lq + BLOCK) * top_k * D <= cap and B * (Lq + Lk) * heads * D <= 2 * most * 40 * 128:
            break
    if op == "select":
        return dict(op=op, B=B, Lq=Lq, Lk=Lk, heads=heads, D=D, top_k=_spread(rng, 1, _ceil(Lk)))
    return dict(op=op, B=B, Lq=Lq, Lk=Lk, heads=heads, D=D, top_k=top_k, mask=rng.choice(["top", "top", "window"]))


def _ceil(n):
    return (n + BLOCK - 1) // BLOCK


def _window(case):
    """The window masks' blocks, [B, nqb, nkb] on the host: `top_k` neighbouring
    key blocks around the query block's own place and the first key block; the
    last clip of a batch of two is a third shorter, and its padding (queries
    and keys) takes no part."""
    B, nq, nk, w = case["B"], _ceil(case["Lq"]), _ceil(case["Lk"]), min(case["top_k"], _ceil(case["Lk"]))
    on = np.zeros((B, nq, nk), dtype=bool)
    for b in range(B):
        keep = 2 / 3 if b > 0 else 1.0
        vq, vk = max(1, int(nq * keep)), max(1, int(nk * keep))
        for i in range(vq):
            at = i * vk // vq
            lo = max(0, min(at - w // 2, vk - w))
            on[b, i, lo:min(vk, lo + w)] = True
            on[b, i, 0] = True
    return on


# ------------------------------------------------------------------ the inputs

def _normed(gen, B, L, heads, D, spread=200):
    """Projected and RMS-normalised tokens: a part that changes slowly along the
    sequence (what neighbouring patches share) and a part of each token's own."""
    n = L // spread + 2
    slow = torch.randn(B, n, heads, D, device="cuda", generator=gen)
    at = torch.arange(L, device="cuda", dtype=torch.float32) / spread
    i = at.long()
    f = (at - i).view(1, L, 1, 1)
    x = torch.lerp(slow[:, i], slow[:, i + 1], f).mul_(0.7)
    x += torch.randn(B, L, heads, D, device="cuda", generator=gen).mul_(0.7)
    x *= torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x.to(torch.bfloat16)


def _randn16(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, heads, D = case["B"], case["heads"], case["D"]
    if case["op"] == "norm_rope_bwd":
        grid = (case["T"], case["H"], case["W"])
        L = grid[0] * grid[1] * grid[2]
        st = dict(case=case, grid=grid)
        if case["group"]:
            st["q"], st["k"] = (_randn16(gen, B, L, heads, D) for _ in range(2))
            st["wq"], st["wk"] = (1 + 0.2 * torch.randn(case["group"], device="cuda", generator=gen) for _ in range(2))
        st["gq"], st["gk"] = (_randn16(gen, B, L, heads, D) for _ in range(2))
        return st
    Lq, Lk = case["Lq"], case["Lk"]
    st = dict(case=case, k=_normed(gen, B, Lk, heads, D))
    if Lq == Lk:
        # tokens of one clip: the slow parts of queries and keys are related
        st["q"] = (st["k"].float() * 0.5 + _normed(gen, B, Lq, heads, D).float()).to(torch.bfloat16)
    else:
        st["q"] = _normed(gen, B, Lq, heads, D)
    if case["op"] == "select":
        return st
    st["v"] = _randn16(gen, B, Lk, heads, D)
    if case["mask"] == "top":
        st["blocks"] = _select(st["q"], st["k"], case["top_k"])
        st["most"] = min(case["top_k"], _ceil(Lk))
    else:
        on = _window(case)
        st["most"] = int(on.sum(-1).max())
        st["blocks"] = torch.from_numpy(on).cuda()[:, None].expand(-1, heads, -1, -1).contiguous()
    if case["op"] == "sparse_bwd":
        st["o"], st["lse"] = _sparse(st["q"], st["k"], st["v"], st["blocks"], st["most"])
        st["do"] = _randn16(gen, B, Lq, heads, D)
    return st


# -------------------------------------------------------------- the plain forms

def _means(x):
    """Mean of each 128-token block of one head, float64 [n, D] from [L, D]."""
    L, D = x.shape
    n = _ceil(L)
    s = torch.nn.functional.pad(x.double(), (0, 0, 0, n * BLOCK - L)).view(n, BLOCK, D).sum(1)
    size = torch.full((n, 1), float(BLOCK), dtype=torch.float64, device=x.device)
    size[-1] = L - (n - 1) * BLOCK
    return s / size


def _select(q, k, top_k):
    B, Lq, heads, _ = q.shape
    nq, nk = _ceil(Lq), _ceil(k.shape[1])
    on = torch.zeros(B, heads, nq, nk, dtype=torch.bool, device=q.device)
    for b in range(B):
        for h in range(heads):
            score = _means(q[b, :, h]) @ _means(k[b, :, h]).T
            best = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :top_k]
            on[b, h].scatter_(1, best, True)
    return on


def _blocks(x):
    """One head's tokens as float32 blocks, [n, 128, D], zeros past the end."""
    L, D = x.shape
    n = _ceil(L)
    return torch.nn.functional.pad(x.float(), (0, 0, 0, n * BLOCK - L)).view(n, BLOCK, D)


def _picked(blocks, most, Lk):
    """For one head: the picked key blocks of each query block, [nq, most], and
    which of their keys take part, [nq, most * 128]."""
    order = torch.sort(blocks.to(torch.uint8), dim=-1, descending=True, stable=True)
    idx, on = order.indices[:, :most], order.values[:, :most] > 0
    key = idx[..., None] * BLOCK + torch.arange(BLOCK, device=blocks.device)
    return idx, (on[..., None] & (key < Lk)).reshape(idx.shape[0], -1)


def _sparse(q, k, v, blocks, most):
    B, Lq, heads, D = q.shape
    Lk = k.shape[1]
    scale = 1.0 / math.sqrt(D)
    o = torch.empty_like(q)
    lse = torch.empty(B, heads, Lq, dtype=torch.float32, device=q.device)
    step = max(1, MOST_ELEMENTS // (BLOCK * most * BLOCK))
    for b in range(B):
        for h in range(heads):
            qb, kb, vb = (_blocks(x[b, :, h]) for x in (q, k, v))
            idx, part = _picked(blocks[b, h], most, Lk)
            out, stat = torch.empty_like(qb), torch.empty(qb.shape[:2], device=q.device)
            for i in range(0, qb.shape[0], step):
                at = idx[i:i + step]
                n = at.shape[0]
                s = torch.bmm(qb[i:i + step] * scale, kb[at].view(n, -1, D).transpose(1, 2))
                s.masked_fill_(~part[i:i + step, None], -math.inf)
                m = s.amax(-1, keepdim=True)
                m = torch.where(m == -math.inf, torch.zeros_like(m), m)
                p = torch.exp(s - m)
                l = p.sum(-1, keepdim=True)
                out[i:i + step] = torch.bmm(p, vb[at].view(n, -1, D)) / torch.where(l == 0, torch.ones_like(l), l)
                stat[i:i + step] = (m + torch.log(l))[..., 0]
            o[b, :, h] = out.view(-1, D)[:Lq].to(o.dtype)
            lse[b, h] = stat.view(-1)[:Lq]
    return o, lse


def _sparse_bwd(q, k, v, blocks, most, o, lse, do):
    B, Lq, heads, D = q.shape
    Lk = k.shape[1]
    scale = 1.0 / math.sqrt(D)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    step = max(1, MOST_ELEMENTS // (BLOCK * most * BLOCK))
    for b in range(B):
        for h in range(heads):
            qb, kb, vb, ob, gb = (_blocks(x[b, :, h]) for x in (q, k, v, o, do))
            stat = _blocks(lse[b, h][:, None])
            stat = torch.where(stat == -math.inf, torch.zeros_like(stat), stat)
            idx, part = _picked(blocks[b, h], most, Lk)
            dqb, dkb, dvb = torch.empty_like(qb), torch.zeros_like(kb), torch.zeros_like(vb)
            for i in range(0, qb.shape[0], step):
                at = idx[i:i + step]
                n = at.shape[0]
                qi, gi = qb[i:i + step], gb[i:i + step]
                ki, vi = kb[at].view(n, -1, D), vb[at].view(n, -1, D)
                s = torch.bmm(qi * scale, ki.transpose(1, 2)).masked_fill_(~part[i:i + step, None], -math.inf)
                p = torch.exp(s - stat[i:i + step])
                dvb.index_add_(0, at.reshape(-1), torch.bmm(p.transpose(1, 2), gi).view(-1, BLOCK, D))
                delta = (gi * ob[i:i + step]).sum(-1, keepdim=True)
                ds = p * (torch.bmm(gi, vi.transpose(1, 2)) - delta) * scale
                dqb[i:i + step] = torch.bmm(ds, ki)
                dkb.index_add_(0, at.reshape(-1), torch.bmm(ds.transpose(1, 2), qi).view(-1, BLOCK, D))
            dq[b, :, h] = dqb.view(-1, D)[:Lq].to(dq.dtype)
            dk[b, :, h] = dkb.view(-1, D)[:Lk].to(dk.dtype)
            dv[b, :, h] = dvb.view(-1, D)[:Lk].to(dv.dtype)
    return dq, dk, dv


def _split(D):
    s = 2 * (D // 6)
    return D - 2 * s, s, s


def _angles(grid, D):
    """float64 [L, D/2]: the angle of every pair at every token."""
    T, H, W = grid
    t = torch.arange(T * H * W, device="cuda")
    out = []
    for pos, d in zip((t // (H * W), t // W % H, t % W), _split(D)):
        out.append(pos.double()[:, None] * THETA ** (-torch.arange(0, d, 2, device="cuda").double() / d))
    return torch.cat(out, -1)


def _norm_rope_bwd(x, w, g, group, cos, sin):
    """(dx, dw) of y = rotation(x / rms * w) for the gradient g of y."""
    g = g.float()
    g0, g1 = g[..., 0::2], g[..., 1::2]
    u = torch.stack((g0 * cos + g1 * sin, g1 * cos - g0 * sin), -1).flatten(-2)
    if x is None:
        return u.to(torch.bfloat16), None
    shape = x.shape
    x = x.float().view(-1, group)
    u = u.view(-1, group)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    dw = (u * x * r).sum(0)
    u = u * w
    dx = r * u - x * (r ** 3 * (x * u).mean(-1, keepdim=True))
    return dx.view(shape).to(torch.bfloat16), dw


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "select":
        return _select(state["q"], state["k"], case["top_k"])
    if case["op"] == "sparse":
        return _sparse(state["q"], state["k"], state["v"], state["blocks"], state["most"])
    if case["op"] == "sparse_bwd":
        return _sparse_bwd(state["q"], state["k"], state["v"], state["blocks"], state["most"], state["o"],
                           state["lse"], state["do"])
    a = _angles(state["grid"], case["D"])
    cos, sin = (f(a).float()[None, :, None] for f in (torch.cos, torch.sin))
    dq, dwq = _norm_rope_bwd(state.get("q"), state.get("wq"), state["gq"], case["group"], cos, sin)
    dk, dwk = _norm_rope_bwd(state.get("k"), state.get("wk"), state["gk"], case["group"], cos, sin)
    return (dq, dk, dwq, dwk) if case["group"] else (dq, dk)


def _run_own(st):
    import spacetime_attention_vdit_b200 as vd
    case = st["case"]
    if case["op"] == "select":
        return vd.attn_select_blocks(st["q"], st["k"], min(case["top_k"], _ceil(case["Lk"])))
    if case["op"] == "sparse":
        return vd.attn_block_sparse(st["q"], st["k"], st["v"], st["blocks"], lse=True)
    if case["op"] == "sparse_bwd":
        return vd.attn_block_sparse_bwd(st["q"], st["k"], st["v"], st["blocks"], st["o"], st["lse"], st["do"])
    if case["group"] == 0:
        return vd.rope_3d_bwd(st["gq"], st["gk"], st["grid"], theta=THETA)
    return vd.qk_norm_rope_3d_bwd(st["q"], st["k"], st["gq"], st["gk"], st["grid"], case["group"], st["wq"], st["wk"],
                                  eps=EPS, theta=THETA)


# ---------------------------------------------------------------- what it takes

def _pairs(case):
    """(query, key) pairs of one head, summed over the batch."""
    B, Lq, Lk = case["B"], case["Lq"], case["Lk"]
    if case["mask"] == "top":
        return B * Lq * min(case["top_k"] * BLOCK, Lk)
    on = _window(case)
    rows = np.minimum(BLOCK, Lq - BLOCK * np.arange(on.shape[1]))
    keys = np.minimum(BLOCK, Lk - BLOCK * np.arange(on.shape[2]))
    return int(np.einsum("bij,i,j->", on.astype(np.int64), rows, keys))


def work(case):
    B, heads, D = case["B"], case["heads"], case["D"]
    if case["op"] == "norm_rope_bwd":
        n = B * case["T"] * case["H"] * case["W"] * heads * D
        if case["group"] == 0:
            return {"bytes": 4 * n * 2, "flops": 2 * 3 * n}
        return {"bytes": 6 * n * 2 + 4 * 4 * case["group"], "flops": 2 * 12 * n}
    Lq, Lk = case["Lq"], case["Lk"]
    cells = B * heads * _ceil(Lq) * _ceil(Lk)
    if case["op"] == "select":
        return {"bytes": B * (Lq + Lk) * heads * D * 2 + cells, "flops": B * (Lq + Lk) * heads * D + cells * D * 2}
    pairs = heads * _pairs(case)
    # keys and values that some query may have picked; a short run of queries picks few
    keys = min(B * heads * Lk, B * heads * _ceil(Lq) * case["top_k"] * BLOCK)
    q_bytes, k_bytes, stat = B * heads * Lq * D * 2, keys * D * 2, B * heads * Lq * 4
    if case["op"] == "sparse":
        return {"bytes": 2 * q_bytes + 2 * k_bytes + stat + cells, "flops": 4 * pairs * D}
    # q, o, do and dq; k and v read, dk and dv written whole
    return {"bytes": 4 * q_bytes + 2 * k_bytes + 2 * B * heads * Lk * D * 2 + stat + cells, "flops": 10 * pairs * D}


# -------------------------------------------------------- the definition, 64 bits

def _exact_select(st):
    q, k, top_k = st["q"], st["k"], st["case"]["top_k"]

    def block_means(x):                                   # [B, L, heads, D] -> [B, heads, n, D]
        parts = [x[:, i:i + BLOCK].double().mean(1) for i in range(0, x.shape[1], BLOCK)]
        return torch.stack(parts, 2)

    qm, km = block_means(q), block_means(k)
    out = []
    for b in range(q.shape[0]):
        for h in range(q.shape[2]):
            rows = []
            for qi in qm[b, h].split(16):
                s = (qi[:, None] * km[b, h][None]).sum(-1)                     # [rows, nk]
                ahead = s[:, None, :] > s[:, :, None]                         # i ahead of j: [row, j, i]
                tie = torch.ones(s.shape[1], s.shape[1], dtype=torch.bool, device=s.device).tril(-1)
                ahead |= (s[:, None, :] == s[:, :, None]) & tie
                rows.append(ahead.sum(-1) < top_k)
            out.append(torch.cat(rows))
    return torch.stack(out).view(q.shape[0], q.shape[2], *out[0].shape)


def _each_block(st):
    """(b, h, query rows, key rows) of every query block, keys as an index tensor."""
    blocks, Lq, Lk = st["blocks"].cpu().numpy(), st["case"]["Lq"], st["case"]["Lk"]
    tokens = torch.arange(Lk, device="cuda")
    of = [tokens[i:i + BLOCK] for i in range(0, Lk, BLOCK)]
    for b in range(blocks.shape[0]):
        for h in range(blocks.shape[1]):
            for i in range(blocks.shape[2]):
                on = np.flatnonzero(blocks[b, h, i])
                yield b, h, slice(i * BLOCK, min(Lq, (i + 1) * BLOCK)), (
                    torch.cat([of[j] for j in on]) if len(on) else None)


def _exact_sparse(st):
    q, k, v = st["q"], st["k"], st["v"]
    scale = q.shape[-1] ** -0.5
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st_shape(q), -math.inf, dtype=torch.float64, device="cuda")
    at = None
    for b, h, rows, keys in _each_block(st):
        if keys is None:
            continue
        if at != (b, h):
            at, kh, vh = (b, h), k[b, :, h].double(), v[b, :, h].double()
        s = (q[b, rows, h].double() @ kh[keys].T) * scale
        stat = torch.logsumexp(s, -1)
        o[b, rows, h] = torch.exp(s - stat[:, None]) @ vh[keys]
        lse[b, h, rows] = stat
    return o, lse


def st_shape(q):
    return (q.shape[0], q.shape[2], q.shape[1])


def _exact_sparse_bwd(st):
    q, k, v, o, do, lse = (st[x] for x in ("q", "k", "v", "o", "do", "lse"))
    scale = q.shape[-1] ** -0.5
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v))
    at = None
    for b, h, rows, keys in _each_block(st):
        if keys is None:
            continue
        if at != (b, h):
            if at:
                dk[at[0], :, at[1]], dv[at[0], :, at[1]] = dkh, dvh
            at, kh, vh = (b, h), k[b, :, h].double(), v[b, :, h].double()
            dkh, dvh = torch.zeros_like(kh), torch.zeros_like(vh)
        qi, gi, kj, vj = q[b, rows, h].double(), do[b, rows, h].double(), kh[keys], vh[keys]
        p = torch.exp((qi @ kj.T) * scale - lse[b, h, rows].double()[:, None])
        dvh[keys] += p.T @ gi
        ds = p * (gi @ vj.T - (gi * o[b, rows, h].double()).sum(-1, keepdim=True)) * scale
        dq[b, rows, h] = ds @ kj
        dkh[keys] += ds.T @ qi
    if at:
        dk[at[0], :, at[1]], dv[at[0], :, at[1]] = dkh, dvh
    return dq, dk, dv


def _exact_norm_rope_bwd(st):
    case = st["case"]
    T, H, W = st["grid"]
    D, group = case["D"], case["group"]
    d_t, d_h, d_w = _split(D)
    where = torch.cartesian_prod(*(torch.arange(n, dtype=torch.float64, device="cuda") for n in (T, H, W)))
    where = where.view(-1, 3)
    turn = []
    for axis, d in enumerate((d_t, d_h, d_w)):
        for i in range(d // 2):
            turn.append(where[:, axis] / THETA ** (2 * i / d))
    phasor = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.stack(turn, -1)).conj()

    def one(x, w, g):
        dx = torch.empty(g.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(max(group, 1), dtype=torch.float64, device="cuda")
        L = g.shape[1]
        for b in range(g.shape[0]):
            for i in range(0, L, 8192):
                part = slice(i, min(L, i + 8192))
                z = torch.view_as_complex(g[b, part].double().unflatten(-1, (-1, 2)).contiguous())
                u = torch.view_as_real(z * phasor[part, None]).flatten(-2)
                if group == 0:
                    dx[b, part] = u
                    continue
                xs = x[b, part].double().reshape(-1, group)
                us = u.reshape(-1, group)
                rms = torch.sqrt(xs.pow(2).sum(-1, keepdim=True) / group + EPS)
                hat = xs / rms
                dw += (us * hat).sum(0)
                gw = us * w.double()
                dx[b, part] = ((gw - hat * (gw * hat).sum(-1, keepdim=True) / group) / rms).view(u.shape)
        return dx, dw

    dq, dwq = one(st.get("q"), st.get("wq"), st["gq"])
    dk, dwk = one(st.get("k"), st.get("wk"), st["gk"])
    return (dq, dk, dwq, dwk) if group else (dq, dk)


def exact(case, seed):
    st = prepare(case, seed)
    return {"select": _exact_select, "sparse": _exact_sparse, "sparse_bwd": _exact_sparse_bwd,
            "norm_rope_bwd": _exact_norm_rope_bwd}[case["op"]](st)
