// attn_block_sparse_bwd.cuh - the gradients of attn_block_sparse.cuh's
// attention, on the 5th-generation tensor cores.
//
// With S = scale * Q K^T over the marked blocks, P = exp(S - lse) and the
// gradient dO of O:
//   delta = rowsum(dO o O)
//   dS = P o (dO V^T - delta)
//   dV = P^T dO      dK = scale * dS^T Q      dQ = scale * dS K
// Two kernels, each of which owns the rows it writes, so no sum crosses CTAs:
// no atomics, the same result on every run.  That costs seven products per
// marked pair of blocks instead of five (S and dO V^T are formed twice); a
// single kernel would add dQ tiles of 64 KB in float32 to memory for every
// pair, in an order that changes from run to run.
//   dq:  one CTA per query block, over the key blocks of its mask row; it
//        also forms delta, and leaves (lse, delta) of its rows for
//   dkv: one CTA per key block, over the query blocks of its mask column, with
//        every product transposed (rows are keys), so that P^T and dS^T are the
//        left operands of their products straight out of TMEM.
// Both have the dense kernel's roles: warps 0..7 the elementwise work, warp 8
// the TMA producer, warp 9 the one issuer of UMMAs.  Two warpgroups share each
// 128 x 128 tile: thread = (row, half of the columns).  P and dS are rounded to
// bfloat16 (nearest even) as operands of the products, as P is in the forward
// pass (that, beside the last rounding, is the error against float64: 0.0025
// relative, of which the rounding of the result is 0.0017); scores, sums and
// accumulators are float32.
//
// Measured: 32,760 tokens, 40 heads x 128, 32 of 256 blocks 8.7 to 9.1 ms (1.06 to
// 1.11 PFLOP/s of the seven products), 43 % of it dq; a tile takes 1.3 us (dq) and 1.5
// (dkv), a CTA's start and end 6 us.  Bound at head_dim 128 by the tensor pipe and its
// changes of operand form: two a tile (dq), four (dkv).  With half and a quarter of the
// products a marked pair of blocks takes 2.6 us (head_dim 64) and 2.4 (32) in both
// kernels together instead of 3.1 (148 x 4 blocks, 8 to 32 marked): there it is the chain
// of a tile, S -> P -> dP -> dS -> product, one after another.
//
// A CTA per block, however many blocks its row or column marks: few query blocks (dq)
// or few key blocks (dkv) leave SMs idle, and one column that every row marks is walked
// by one CTA.  128 queries over 256 marked blocks, 12 heads x 128: 514 us; 128 keys
// under 256 blocks of queries: 602; a window of 11 blocks at 32,760 tokens 966, with the
// first key block marked by every row 1,405.  (The names carry the dense kernel's stem:
// same CTA, same registers at launch.)
#pragma once

#include "attn_block_sparse.cuh"

namespace vdit {

struct SparseBwdParams {
  const float* lse;        // [B, heads, Lq], natural log
  float* stats;            // [2][B * heads][nqb * 128]: lse in log2 units (+inf where no key counts), then delta
  const uint8_t* blocks;   // [B, heads, nqb, nkb]
  int Lq, Lk, heads, nqb, nkb;
  long long stats_n;       // B * heads * nqb * 128
  float scale, scale_log2;
};

enum : int {
  kSiteBwdIn = 48, kSiteBwdRow, kSiteBwdCol, kSiteBwdRowFree, kSiteBwdColFree, kSiteBwdS, kSiteBwdDp, kSiteBwdP,
  kSiteBwdDs, kSiteBwdStat, kSiteBwdStatFree, kSiteBwdDone
};

template <int D>
struct SparseBwdCfg : AttnCfg<D> {
  using A = AttnCfg<D>;
  // registers: at the dense kernel's 56 the issuing thread spills
  static constexpr int REGS_ELEMENT = 208, REGS_CTRL = 88;
  static_assert(2 * 128 * REGS_ELEMENT + 128 * REGS_CTRL <= A::THREADS * A::REGS_LAUNCH, "register split");
  // dq: Q and dO stay, K and V stream (K is needed once more, for dQ, after V)
  static constexpr int NA = 3, NB = 2;
  static constexpr int TILES = 2 + NA + NB;
  static constexpr int BITS_OFF = TILES * A::TILE_BYTES;
  static constexpr int DQ_PART_OFF = BITS_OFF + kSparseWords * 4;   // halves of delta, [2][128] floats
  static constexpr int DQ_BARS_OFF = DQ_PART_OFF + 1024;
  static constexpr int DQ_NBARS = 1 + 2 * NA + 2 * NB + 2 + 1 + 1 + 1;
  static constexpr int DQ_SMEM = 1024 + DQ_BARS_OFF + DQ_NBARS * 8 + 16;
  // dkv: K and V stay, Q, dO and the rows' statistics stream
  static constexpr int NST = 2;
  static constexpr int DKV_STAT_OFF = BITS_OFF + kSparseWords * 4;  // [NST][lse 128, delta 128] floats
  static constexpr int DKV_BARS_OFF = DKV_STAT_OFF + NST * 1024;
  static constexpr int DKV_NBARS = 1 + 2 * NA + 2 * NB + 2 * NST + 4 + 1;
  static constexpr int DKV_SMEM = DKV_BARS_OFF + DKV_NBARS * 8 + 16;
  static_assert(DQ_SMEM <= 232448 && DKV_SMEM <= 232448, "shared memory");
  // TMEM columns
  static constexpr uint32_t DQ_S = 0, DQ_DP = 256, DQ_ACC = 384;         // S double-buffered
  static constexpr uint32_t KV_S = 0, KV_DP = 128, KV_DV = 256, KV_DK = 384;
};

// acc [128 x D] += A [128 x 128, bf16 in TMEM] * B [128 rows of D, MN-major in
// shared memory, `b` bytes behind the descriptor].  A's packed columns: the first 64
// of its columns at a, the others 64 TMEM columns further (each warpgroup packs over
// its own scores).
template <int D>
__device__ __forceinline__ void bwd_accumulate(uint32_t acc, uint32_t a, const UmmaDesc& db, uint32_t b, bool first) {
  using C = AttnCfg<D>;
  umma_ts_at(acc, a, db, b, C::IDESC_PV, first ? 0u : 1u);
#pragma unroll
  for (int kk = 1; kk < 8; ++kk)
    umma_ts_at(acc, a + (kk >> 2) * 64 + (kk & 3) * 8, db, b + kk * 16 * C::ROWB, C::IDESC_PV, 1u);
}

// Load one 128-row tile of (head h, batch b) starting at token `row`.
template <int D>
__device__ __forceinline__ void bwd_load_tile(unsigned char* dst, const CUtensorMap* map, uint64_t* bar, int h, int row,
                                              int b) {
  using C = AttnCfg<D>;
#pragma unroll
  for (int db = 0; db < C::NDB; ++db)
    tma_load_5d(dst + db * C::DB_BYTES, map, bar, db * C::DBLK, h, 0, row, b);
}

// 64 TMEM columns of this thread's lane.
__device__ __forceinline__ void bwd_ld64(uint32_t t, uint32_t (&r)[2][32]) {
  tmem_ld32(t, r[0]);
  tmem_ld32(t + 32, r[1]);
  tmem_ld_wait();
  tmem_ld_fence(r[0]);
  tmem_ld_fence(r[1]);
}

// 32 accumulator columns, times `f`, rounded to bf16, staged as columns c0 .. c0+31
// of row `row` in the swizzled layout of the tile's tensor map.
template <int D>
__device__ __forceinline__ void bwd_stage32(unsigned char* stage, int row, int c0, const uint32_t (&o)[32], float f) {
  using C = AttnCfg<D>;
  const int key = C::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
  constexpr int CPB = C::ROWB / 16;
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    uint4 v;
    v.x = pack_bf16x2(__uint_as_float(o[e + 0]) * f, __uint_as_float(o[e + 1]) * f);
    v.y = pack_bf16x2(__uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f);
    v.z = pack_bf16x2(__uint_as_float(o[e + 4]) * f, __uint_as_float(o[e + 5]) * f);
    v.w = pack_bf16x2(__uint_as_float(o[e + 6]) * f, __uint_as_float(o[e + 7]) * f);
    const int cc = c0 / 8 + e / 8;
    *reinterpret_cast<uint4*>(stage + (cc / CPB) * C::DB_BYTES + row * C::ROWB + (((cc % CPB) ^ key) << 4)) = v;
  }
}

// ---------------------------------------------------------------------------
// dQ, delta
// ---------------------------------------------------------------------------
//
// S is double-buffered in TMEM, so S of the next key block is ready when the
// elementwise warps get to it; dO V^T of the next block runs while they
// exponentiate.  dS overwrites the scores it came from.

template <int D>
__global__ void __launch_bounds__(384, 1)
    grad_attn_fwd_tcgen05_sparse_dq_kernel(const __grid_constant__ CUtensorMap tmQ,
                                           const __grid_constant__ CUtensorMap tmK,
                                           const __grid_constant__ CUtensorMap tmV,
                                           const __grid_constant__ CUtensorMap tmO,
                                           const __grid_constant__ CUtensorMap tmDO,
                                           const __grid_constant__ CUtensorMap tmDQ, const SparseBwdParams p) {
  using C = SparseBwdCfg<D>;
  unsigned char* sQ = smem_base_1024();
  unsigned char* sDO = sQ + C::TILE_BYTES;
  unsigned char* sK = sDO + C::TILE_BYTES;               // NA tiles
  unsigned char* sV = sK + C::NA * C::TILE_BYTES;        // NB tiles
  uint32_t* bits = reinterpret_cast<uint32_t*>(sQ + C::BITS_OFF);
  float* part = reinterpret_cast<float*>(sQ + C::DQ_PART_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sQ + C::DQ_BARS_OFF);
  uint64_t* in_full = bars;
  uint64_t* k_full = in_full + 1;
  uint64_t* k_empty = k_full + C::NA;
  uint64_t* v_full = k_empty + C::NA;
  uint64_t* v_empty = v_full + C::NB;
  uint64_t* s_full = v_empty + C::NB;                    // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* ds_ready = dp_full + 1;
  uint64_t* drain = ds_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int qb = blockIdx.x % p.nqb;
  const int bh = blockIdx.x / p.nqb;
  const int h = bh % p.heads;
  const int b = bh / p.heads;
  const int q0 = qb * C::BM;
  const int nw = (p.nkb + 31) / 32;

  if (threadIdx.x == 0) {
    mbar_init(in_full, 1);
    for (int s = 0; s < C::NA; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
    for (int s = 0; s < C::NB; ++s) { mbar_init(&v_full[s], 1); mbar_init(&v_empty[s], 1); }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(dp_full, 1);
    mbar_init(ds_ready, 8);              // one elected lane per elementwise warp
    mbar_init(drain, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(in_full, 3 * C::TILE_BYTES);
    bwd_load_tile<D>(sQ, &tmQ, in_full, h, q0, b);
    bwd_load_tile<D>(sDO, &tmDO, in_full, h, q0, b);
    bwd_load_tile<D>(sK + (C::NA - 1) * C::TILE_BYTES, &tmO, in_full, h, q0, b);
  }
  mask_words(bits, p.blocks + ((long long)bh * p.nqb + qb) * p.nkb, 1, p.nkb, warp, 12, lane);
  if (warp == C::MMA_WARP) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  int n = 0;                                             // key blocks of this mask row
  for (int w = lane; w < nw; w += 32) n += __popc(bits[w]);
  n = warp_sum(n);

  if (warp >= 8) {
    regs_decrease<C::REGS_CTRL>();
    if (warp == C::TMA_WARP) {
      if (lane == 0) {
        int word = -1;
        uint32_t left = 0u;
        int k_issued = 0, v_issued = 0;
        bool ok = true;
        for (int x = 0; x < n && ok; ++x) {
          while (left == 0u) left = bits[++word];
          const int kb = word * 32 + __ffs(left) - 1;
          left &= left - 1u;
          const int sk = x % C::NA, sv = x % C::NB;
          // the last stage holds O first, which the elementwise warps release
          if (sk == C::NA - 1) ok = mbar_wait(&k_empty[sk], (x / C::NA) & 1, kSiteBwdRowFree);
          else if (x >= C::NA) ok = mbar_wait(&k_empty[sk], ((x / C::NA) - 1) & 1, kSiteBwdRowFree);
          if (!ok) break;
          mbar_arrive_expect_tx(&k_full[sk], C::TILE_BYTES);
          bwd_load_tile<D>(sK + sk * C::TILE_BYTES, &tmK, &k_full[sk], h, kb * C::BN, b);
          k_issued = x + 1;
          if (x >= C::NB) ok = mbar_wait(&v_empty[sv], ((x / C::NB) - 1) & 1, kSiteBwdColFree);
          if (!ok) break;
          mbar_arrive_expect_tx(&v_full[sv], C::TILE_BYTES);
          bwd_load_tile<D>(sV + sv * C::TILE_BYTES, &tmV, &v_full[sv], h, kb * C::BN, b);
          v_issued = x + 1;
        }
        // no copy may still be landing in shared memory when the CTA exits
        mbar_drain(in_full, 0);
        for (int j = k_issued - C::NA < 0 ? 0 : k_issued - C::NA; j < k_issued; ++j)
          mbar_drain(&k_full[j % C::NA], (j / C::NA) & 1);
        for (int j = v_issued - C::NB < 0 ? 0 : v_issued - C::NB; j < v_issued; ++j)
          mbar_drain(&v_full[j % C::NB], (j / C::NB) & 1);
      }
    } else if (warp == C::MMA_WARP) {
      if (lane == 0) {
        constexpr uint32_t SBO = 8 * C::ROWB;
        const UmmaDesc dQ(sQ, 16, SBO, C::SWZ), dG(sDO, 16, SBO, C::SWZ), dK(sK, 16, SBO, C::SWZ),
            dV(sV, 16, SBO, C::SWZ), dKt(sK, C::DB_BYTES, SBO, C::SWZ);
        RingPos<C::NA> ks, ka;                           // K: as S's operand, and later as dQ's
        RingPos<C::NB> vr;
        auto scores = [&](int j) -> bool {               // S_j = Q K_j^T
          if (!mbar_wait(&k_full[ks.st], ks.phase, kSiteBwdRow)) return false;
          tc_fence_after();
          umma_scores<D>(tmem + C::DQ_S + (j & 1) * 128, dQ, 0, dK, ks.st * C::TILE_BYTES);
          umma_commit(&s_full[j & 1]);
          ks.step();
          return true;
        };
        auto dprob = [&]() -> bool {                     // dP_j = dO V_j^T
          if (!mbar_wait(&v_full[vr.st], vr.phase, kSiteBwdCol)) return false;
          tc_fence_after();
          umma_scores<D>(tmem + C::DQ_DP, dG, 0, dV, vr.st * C::TILE_BYTES);
          umma_commit(dp_full);
          umma_commit(&v_empty[vr.st]);
          vr.step();
          return true;
        };
        bool ok = mbar_wait(in_full, 0, kSiteBwdIn);
        if (ok && n > 0) ok = scores(0) && dprob();
        if (ok && n > 1) ok = scores(1);
        for (int j = 0; j < n && ok; ++j) {
          ok = mbar_wait(ds_ready, j & 1, kSiteBwdDs);
          if (!ok) break;
          tc_fence_after();
          if (j + 1 < n) ok = dprob();
          if (!ok) break;
          bwd_accumulate<D>(tmem + C::DQ_ACC, tmem + C::DQ_S + (j & 1) * 128, dKt, ka.st * C::TILE_BYTES, j == 0);
          // S_{j+2} takes the columns dQ's product above reads: UMMAs of one
          // thread execute in issue order
          if (j + 2 < n) {
            const int st = ka.st;
            ok = scores(j + 2);
            umma_commit(&k_empty[st]);
          } else {
            umma_commit(&k_empty[ka.st]);
          }
          ka.step();
        }
        umma_commit(drain);
        mbar_drain(drain, 0);
      }
      __syncwarp();
    }
  } else {
    regs_increase<C::REGS_ELEMENT>();
    const int half = warp >> 2;                          // columns 64 half .. 64 half + 63
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const int i = q0 + row;
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    // Delta of the row, from the tiles of O and dO in shared memory: this thread's
    // half of the channels, then the halves' sum.  (From global memory, a row per
    // thread, it took 6 us of a CTA's 27 at 12 key blocks and head_dim 128.)
    float l = i < p.Lq ? __ldg(p.lse + (long long)bh * p.Lq + i) : -INFINITY;
    bool ok = warp_wait(in_full, 0, kSiteBwdIn);
    {
      float a = 0.f;
      const unsigned char* tO = sK + (C::NA - 1) * C::TILE_BYTES;
      const int key = C::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
      constexpr int CPB = C::ROWB / 16;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const int cc = half * (D / 16) + c;
        const int off = (cc / CPB) * C::DB_BYTES + row * C::ROWB + (((cc % CPB) ^ key) << 4);
        const uint4 x = *reinterpret_cast<const uint4*>(tO + off), y = *reinterpret_cast<const uint4*>(sDO + off);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          a = fmaf(__uint_as_float(xs[m] << 16), __uint_as_float(ys[m] << 16), a);
          a = fmaf(__uint_as_float(xs[m] & 0xffff0000u), __uint_as_float(ys[m] & 0xffff0000u), a);
        }
      }
      part[half * 128 + row] = a;
    }
    // every warp comes here, also one whose wait ran out
    named_bar_sync(1, 256);
    if (threadIdx.x == 0) mbar_arrive(&k_empty[C::NA - 1]);
    const float delta = part[row] + part[128 + row], ndelta = -delta;
    // -lse in log2 units; a row without keys (lse = -inf) gets P = 0, as a row past the sequence
    const float nlse = l != -INFINITY ? -l * 1.4426950408889634f : -INFINITY;
    p.stats[(half ? p.stats_n : 0) + (long long)bh * p.nqb * 128 + q0 + row] = half ? delta : -nlse;
    const int last = p.nkb - 1, tail_keys = p.Lk - last * C::BN;
    const bool tail = tail_keys < C::BN && ((bits[last >> 5] >> (last & 31)) & 1u) != 0u;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nl2 = make_float2(nlse, nlse),
                 nd2 = make_float2(ndelta, ndelta);
    for (int j = 0; j < n && ok; ++j) {
      ok = warp_wait(&s_full[j & 1], (j >> 1) & 1, kSiteBwdS);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_s = tl + C::DQ_S + (j & 1) * 128 + half * 64;
      uint32_t s[2][32];
      bwd_ld64(t_s, s);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = ffma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), sc2, nl2);
          s[c][e] = __float_as_uint(ex2_approx(x.x));
          s[c][e + 1] = __float_as_uint(ex2_approx(x.y));
        }
      if (tail && j + 1 == n) {                          // ascending order: the ragged block comes last
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (half * 64 + c * 32 + e >= tail_keys) s[c][e] = 0u;
      }
      ok = warp_wait(dp_full, j & 1, kSiteBwdDp);
      if (!ok) break;
      tc_fence_after();
      uint32_t d[2][32];
      bwd_ld64(tl + C::DQ_DP + half * 64, d);
      uint32_t pk[32];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x =
              fmul2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                    fadd2(make_float2(__uint_as_float(d[c][e]), __uint_as_float(d[c][e + 1])), nd2));
          pk[c * 16 + e / 2] = pack_bf16x2(x.x, x.y);
        }
      tmem_st32(t_s, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_ready);
    }
    // dQ, scaled once, leaves through the Q buffer (every UMMA has finished)
    if (ok && n > 0) ok = warp_wait(drain, 0, kSiteBwdDone);
    if (ok) {
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        if (c % 2 != half) continue;                     // the warpgroups take turns
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(tl + C::DQ_ACC + c * 32, o);
          tmem_ld_wait();
          tmem_ld_fence(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        bwd_stage32<D>(sQ, row, c * 32, o, p.scale);
      }
    }
    fence_proxy_async_smem();
    const bool all_good = named_bar_and(2, 256, ok);
    if (all_good && threadIdx.x == 0) {
#pragma unroll
      for (int db = 0; db < C::NDB; ++db)
        tma_store_5d(&tmDQ, sQ + db * C::DB_BYTES, db * C::DBLK, h, 0, q0, b);
      bulk_commit_group();
      bulk_wait_group_read<0>();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// dK, dV
// ---------------------------------------------------------------------------
//
// Rows are keys.  TMEM is full at head_dim 128 (S^T, dP^T, dV and dK of 128 columns
// each), so nothing is double-buffered; smaller heads use the same places and leave
// 128 (64) or 192 (32) columns idle.  The issue order
//   dV_j, S_{j+1}, dK_j, dP_{j+1}
// lets the elementwise warps exponentiate S_{j+1} under dK_j and dP_{j+1}, and
// form dS_j under dV_j and S_{j+1}.

template <int D>
__global__ void __launch_bounds__(384, 1)
    grad_attn_fwd_tcgen05_sparse_dkv_kernel(const __grid_constant__ CUtensorMap tmQ,
                                            const __grid_constant__ CUtensorMap tmK,
                                            const __grid_constant__ CUtensorMap tmV,
                                            const __grid_constant__ CUtensorMap tmDO,
                                            const __grid_constant__ CUtensorMap tmDK,
                                            const __grid_constant__ CUtensorMap tmDV, const SparseBwdParams p) {
  using C = SparseBwdCfg<D>;
  // the shared-memory budget leaves no room to round the base up: it is
  // declared 1024-byte aligned
  unsigned char* sK = dyn_smem;
  unsigned char* sV = sK + C::TILE_BYTES;
  unsigned char* sQ = sV + C::TILE_BYTES;                // NA tiles
  unsigned char* sDO = sQ + C::NA * C::TILE_BYTES;       // NB tiles
  uint32_t* bits = reinterpret_cast<uint32_t*>(sK + C::BITS_OFF);
  float* stat = reinterpret_cast<float*>(sK + C::DKV_STAT_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sK + C::DKV_BARS_OFF);
  uint64_t* in_full = bars;
  uint64_t* q_full = in_full + 1;
  uint64_t* q_empty = q_full + C::NA;
  uint64_t* do_full = q_empty + C::NA;
  uint64_t* do_empty = do_full + C::NB;
  uint64_t* st_full = do_empty + C::NB;                  // [NST]
  uint64_t* st_empty = st_full + C::NST;                 // [NST]
  uint64_t* s_full = st_empty + C::NST;
  uint64_t* p_ready = s_full + 1;
  uint64_t* dp_full = p_ready + 1;
  uint64_t* ds_ready = dp_full + 1;
  uint64_t* drain = ds_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  if ((smem_u32(dyn_smem) & 1023u) != 0u) {              // the swizzled tiles would be misread
    watchdog_trip(kSiteBwdIn);
    return;
  }

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int kb = blockIdx.x % p.nkb;
  const int bh = blockIdx.x / p.nkb;
  const int h = bh % p.heads;
  const int b = bh / p.heads;
  const int k0 = kb * C::BN;
  const int nw = (p.nqb + 31) / 32;

  if (threadIdx.x == 0) {
    mbar_init(in_full, 1);
    for (int s = 0; s < C::NA; ++s) { mbar_init(&q_full[s], 1); mbar_init(&q_empty[s], 1); }
    for (int s = 0; s < C::NB; ++s) { mbar_init(&do_full[s], 1); mbar_init(&do_empty[s], 1); }
    for (int s = 0; s < C::NST; ++s) { mbar_init(&st_full[s], 1); mbar_init(&st_empty[s], 8); }
    mbar_init(s_full, 1);
    mbar_init(p_ready, 8);
    mbar_init(dp_full, 1);
    mbar_init(ds_ready, 8);
    mbar_init(drain, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(in_full, 2 * C::TILE_BYTES);
    bwd_load_tile<D>(sK, &tmK, in_full, h, k0, b);
    bwd_load_tile<D>(sV, &tmV, in_full, h, k0, b);
  }
  mask_words(bits, p.blocks + (long long)bh * p.nqb * p.nkb + kb, p.nkb, p.nqb, warp, 12, lane);
  if (warp == C::MMA_WARP) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  int n = 0;                                             // query blocks of this mask column
  for (int w = lane; w < nw; w += 32) n += __popc(bits[w]);
  n = warp_sum(n);

  if (warp >= 8) {
    regs_decrease<C::REGS_CTRL>();
    if (warp == C::TMA_WARP) {
      if (lane == 0) {
        int word = -1;
        uint32_t left = 0u;
        int q_issued = 0, st_issued = 0, do_issued = 0;
        bool ok = true;
        for (int x = 0; x < n && ok; ++x) {
          while (left == 0u) left = bits[++word];
          const int qb = word * 32 + __ffs(left) - 1;
          left &= left - 1u;
          const int sa = x % C::NA, sb = x % C::NB, ss = x % C::NST;
          if (x >= C::NA) ok = mbar_wait(&q_empty[sa], ((x / C::NA) - 1) & 1, kSiteBwdRowFree);
          if (!ok) break;
          mbar_arrive_expect_tx(&q_full[sa], C::TILE_BYTES);
          bwd_load_tile<D>(sQ + sa * C::TILE_BYTES, &tmQ, &q_full[sa], h, qb * C::BM, b);
          q_issued = x + 1;
          if (x >= C::NST) ok = mbar_wait(&st_empty[ss], ((x / C::NST) - 1) & 1, kSiteBwdStatFree);
          if (!ok) break;
          const float* from = p.stats + ((long long)bh * p.nqb + qb) * 128;
          mbar_arrive_expect_tx(&st_full[ss], 1024);
          bulk_load(stat + ss * 256, from, 512, &st_full[ss]);
          bulk_load(stat + ss * 256 + 128, from + p.stats_n, 512, &st_full[ss]);
          st_issued = x + 1;
          if (x >= C::NB) ok = mbar_wait(&do_empty[sb], ((x / C::NB) - 1) & 1, kSiteBwdColFree);
          if (!ok) break;
          mbar_arrive_expect_tx(&do_full[sb], C::TILE_BYTES);
          bwd_load_tile<D>(sDO + sb * C::TILE_BYTES, &tmDO, &do_full[sb], h, qb * C::BM, b);
          do_issued = x + 1;
        }
        mbar_drain(in_full, 0);
        for (int j = q_issued - C::NA < 0 ? 0 : q_issued - C::NA; j < q_issued; ++j)
          mbar_drain(&q_full[j % C::NA], (j / C::NA) & 1);
        for (int j = st_issued - C::NST < 0 ? 0 : st_issued - C::NST; j < st_issued; ++j)
          mbar_drain(&st_full[j % C::NST], (j / C::NST) & 1);
        for (int j = do_issued - C::NB < 0 ? 0 : do_issued - C::NB; j < do_issued; ++j)
          mbar_drain(&do_full[j % C::NB], (j / C::NB) & 1);
      }
    } else if (warp == C::MMA_WARP) {
      if (lane == 0) {
        constexpr uint32_t SBO = 8 * C::ROWB;
        const UmmaDesc dK(sK, 16, SBO, C::SWZ), dV(sV, 16, SBO, C::SWZ), dQ(sQ, 16, SBO, C::SWZ),
            dG(sDO, 16, SBO, C::SWZ), dQt(sQ, C::DB_BYTES, SBO, C::SWZ), dGt(sDO, C::DB_BYTES, SBO, C::SWZ);
        RingPos<C::NA> qs, qa;                           // Q: as S's operand, and later as dK's
        RingPos<C::NB> gs, ga;                           // dO: as dP's operand, and as dV's
        auto scores = [&]() -> bool {                    // S_j^T = K Q_j^T
          if (!mbar_wait(&q_full[qs.st], qs.phase, kSiteBwdRow)) return false;
          tc_fence_after();
          umma_scores<D>(tmem + C::KV_S, dK, 0, dQ, qs.st * C::TILE_BYTES);
          umma_commit(s_full);
          qs.step();
          return true;
        };
        auto dprob = [&]() -> bool {                     // dP_j^T = V dO_j^T
          if (!mbar_wait(&do_full[gs.st], gs.phase, kSiteBwdCol)) return false;
          tc_fence_after();
          umma_scores<D>(tmem + C::KV_DP, dV, 0, dG, gs.st * C::TILE_BYTES);
          umma_commit(dp_full);
          gs.step();
          return true;
        };
        bool ok = mbar_wait(in_full, 0, kSiteBwdIn);
        if (ok && n > 0) ok = scores() && dprob();
        for (int j = 0; j < n && ok; ++j) {
          ok = mbar_wait(p_ready, j & 1, kSiteBwdP);
          if (!ok) break;
          tc_fence_after();
          bwd_accumulate<D>(tmem + C::KV_DV, tmem + C::KV_S, dGt, ga.st * C::TILE_BYTES, j == 0);
          // S_{j+1} takes the columns of P_j, dP_{j+1} those of dS_j: UMMAs of
          // one thread execute in issue order
          if (j + 1 < n) ok = scores();
          umma_commit(&do_empty[ga.st]);
          ga.step();
          if (ok) ok = mbar_wait(ds_ready, j & 1, kSiteBwdDs);
          if (!ok) break;
          tc_fence_after();
          bwd_accumulate<D>(tmem + C::KV_DK, tmem + C::KV_DP, dQt, qa.st * C::TILE_BYTES, j == 0);
          if (j + 1 < n) ok = dprob();
          umma_commit(&q_empty[qa.st]);
          qa.step();
        }
        umma_commit(drain);
        mbar_drain(drain, 0);
      }
      __syncwarp();
    }
  } else {
    regs_increase<C::REGS_ELEMENT>();
    const int half = warp >> 2;                          // columns (queries) 64 half .. 64 half + 63
    const int quad = warp & 3;
    const int row = quad * 32 + lane;                    // key within the block
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t t_s = tl + C::KV_S + half * 64, t_dp = tl + C::KV_DP + half * 64;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int ss = j % C::NST;
      const float4* lse4 = reinterpret_cast<const float4*>(stat + ss * 256 + half * 64);
      const float4* del4 = reinterpret_cast<const float4*>(stat + ss * 256 + 128 + half * 64);
      ok = warp_wait(&st_full[ss], (j / C::NST) & 1, kSiteBwdStat) && warp_wait(s_full, j & 1, kSiteBwdS);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[2][32];
      bwd_ld64(t_s, s);
      uint32_t pk[32];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l = lse4[c * 8 + e / 4];
          const float2 x = ffma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), sc2,
                                 make_float2(-l.x, -l.y));
          const float2 y = ffma2(make_float2(__uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3])), sc2,
                                 make_float2(-l.z, -l.w));
          const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y), p2 = ex2_approx(y.x), p3 = ex2_approx(y.y);
          pk[c * 16 + e / 2] = pack_bf16x2(p0, p1);
          pk[c * 16 + e / 2 + 1] = pack_bf16x2(p2, p3);
          s[c][e] = __float_as_uint(p0);
          s[c][e + 1] = __float_as_uint(p1);
          s[c][e + 2] = __float_as_uint(p2);
          s[c][e + 3] = __float_as_uint(p3);
        }
      tmem_st32(t_s, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready);

      ok = warp_wait(dp_full, j & 1, kSiteBwdDp);
      if (!ok) break;
      tc_fence_after();
      uint32_t d[2][32];
      bwd_ld64(t_dp, d);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 dl = del4[c * 8 + e / 4];
          const float2 x = fmul2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                 fadd2(make_float2(__uint_as_float(d[c][e]), __uint_as_float(d[c][e + 1])),
                                       make_float2(-dl.x, -dl.y)));
          const float2 y = fmul2(make_float2(__uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3])),
                                 fadd2(make_float2(__uint_as_float(d[c][e + 2]), __uint_as_float(d[c][e + 3])),
                                       make_float2(-dl.z, -dl.w)));
          pk[c * 16 + e / 2] = pack_bf16x2(x.x, x.y);
          pk[c * 16 + e / 2 + 1] = pack_bf16x2(y.x, y.y);
        }
      tmem_st32(t_dp, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ds_ready);
        mbar_arrive(&st_empty[ss]);
      }
    }
    // warps 0..3 write dV through V's buffer, warps 4..7 dK (scaled once)
    // through K's; every UMMA has finished
    if (ok) ok = n > 0 ? warp_wait(drain, 0, kSiteBwdDone) : warp_wait(in_full, 0, kSiteBwdIn);
    unsigned char* stage = half == 0 ? sV : sK;
    if (ok) {
      tc_fence_after();
      const float f = half == 0 ? 1.f : p.scale;
      const uint32_t acc = tl + (half == 0 ? C::KV_DV : C::KV_DK);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(acc + c * 32, o);
          tmem_ld_wait();
          tmem_ld_fence(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        bwd_stage32<D>(stage, row, c * 32, o, f);
      }
    }
    fence_proxy_async_smem();
    const bool all_good = named_bar_and(1 + half, 128, ok);
    if (all_good && quad == 0 && lane == 0) {
#pragma unroll
      for (int db = 0; db < C::NDB; ++db)
        tma_store_5d(half == 0 ? &tmDV : &tmDK, stage + db * C::DB_BYTES, db * C::DBLK, h, 0, k0, b);
      bulk_commit_group();
      bulk_wait_group_read<0>();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace vdit
