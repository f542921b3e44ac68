// attn_block_sparse.cuh - attention of each 128-query block over the 128-key
// blocks a mask marks for it, on the 5th-generation tensor cores.
//
//   O[i] = sum_j softmax_j(scale * Q[i] . K[j]) V[j],  j over the keys of the
//   blocks kb with blocks[b, h, i / 128, kb] != 0
//
// The products, the softmax and the register split are those of the dense
// kernel (attn_tcgen05.cuh): two 128-row query tiles per CTA, one softmax
// warpgroup each, S and P in TMEM, one thread issuing every UMMA.  What differs
// is which key tiles a CTA sweeps.  Its two query blocks have a mask row each;
// the rows are turned into bit words in shared memory and swept in this order:
//   1. the key blocks both rows mark, in ascending order: one K and one V tile
//      serve both query tiles, as in the dense kernel;
//   2. the blocks only one row marks, each row's in ascending order, the two
//      tiles taking turns (so the tensor core always has the other tile's
//      products to run while one tile exponentiates).
// Neighbouring query blocks of a clip mostly pick the same key blocks, so most
// of a CTA's traffic is of the first kind (64 KB of K and V for two tile steps;
// the second kind takes 64 KB per step).  A mask row is a set: no block can be
// listed twice, none can be out of range, and the order is fixed, so the result
// does not depend on how the mask was made.
//
// A few query blocks (a single token, a small chunk of a stream) would leave
// most SMs idle while a few CTAs walk a long row of keys.  Then (kSplit) a
// cluster of CTAs shares the two query blocks: CTA r of S takes every S-th
// marked key block, and the partial results - unnormalised O in float32, the
// max in use and the sum of P of each row - meet in distributed shared memory:
// each CTA joins every S-th row from its peers' copies, in the order of their
// ranks.  No workspace, no second launch, no atomics.  A sequence of one query
// block has no second one to take turns with: there both tiles of a CTA hold the
// same queries and share its key blocks too.
//
// Measured: 75,600 tokens, 40 heads x 128, 74 of 591 blocks 14.3 to 14.8 ms (1.0
// PFLOP/s; the dense kernel with as many keys 13.5 ms); one token over 32,760 keys, 12
// heads, 64 blocks 18 us in a graph (22 by a call: the host's work is longer).  Bound as
// the dense kernel is, by the tensor pipe's changes of operand form and the
// exponentials; a CTA's start (mask, first copies) and end take 7 us of its 28 at 11
// blocks.
#pragma once

#include "attn_tcgen05.cuh"

namespace vdit {

constexpr int kSparseBlock = 128;        // tokens per query block and per key block
constexpr int kSparseMaxBlocks = 6144;   // key blocks a mask row may have: its bit words sit in shared memory
constexpr int kSparseWords = kSparseMaxBlocks / 32;

struct SparseParams {
  __nv_bfloat16* o;
  float* lse;              // may be null
  const uint8_t* blocks;   // [B, heads, nqb, nkb], nonzero: attend
  int Lq, Lk, heads;
  int nqb, nkb;            // query blocks and key blocks per sequence
  int n_pairs;             // ceil(nqb / 2): CTAs (kSplit: clusters) per (batch, head)
  int splits;              // CTAs of a cluster (kSplit)
  float scale_log2;        // scale * log2(e)
};

template <int D>
struct SparseCfg : AttnCfg<D> {
  using A = AttnCfg<D>;
  // more registers for the issuing thread than the dense kernel's (+1 %)
  static constexpr int REGS_SOFT = 208, REGS_CTRL = 88;
  static_assert(2 * 128 * REGS_SOFT + 128 * REGS_CTRL <= A::THREADS * A::REGS_LAUNCH, "register split");
  static constexpr int NBARS = 1 + 2 * A::NK + 2 * A::NV + 3 * A::NQ + 1;
  static constexpr int BITS_OFF = (A::NQ + A::NK + A::NV) * A::TILE_BYTES;
  static constexpr int BARS_OFF = BITS_OFF + A::NQ * kSparseWords * 4;
  static constexpr int SMEM_BYTES = 1024 + BARS_OFF + NBARS * 8 + 16;
  static_assert(SMEM_BYTES <= 232448, "shared memory");
  // kSplit: partial O of both tiles (float32) over Q and the rings, then
  // (max, sum) of each row of both tiles
  static constexpr int PART_BYTES = A::BM * D * 4;
  static constexpr int STAT_OFF = A::NQ * PART_BYTES;
  static_assert(STAT_OFF + A::NQ * A::BM * 8 <= BITS_OFF, "partial results");
};

// Walks the set bits of a mask-row combination in ascending order.
struct BitWalk {
  int word;        // index of the word held
  uint32_t bits;   // its bits not yet walked
};

// One mask row (n bytes, `stride` bytes apart) as bit words, a word per warp in
// turn, four words' loads in flight.
__device__ __forceinline__ void mask_words(uint32_t* words, const uint8_t* row, long long stride, int n, int warp,
                                           int nwarps, int lane) {
  for (int w0 = warp; w0 * 32 < n; w0 += 4 * nwarps) {
    bool on[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = (w0 + u * nwarps) * 32 + lane;
      on[u] = i < n && __ldg(row + i * stride) != 0;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t m = __ballot_sync(0xffffffffu, on[u]);
      if (lane == 0 && (w0 + u * nwarps) * 32 < n) words[w0 + u * nwarps] = m;
    }
  }
}

// ---- UMMAs from precomputed descriptors
//
// One thread issues every UMMA, and at 16 per tile step what it computes for each
// weighs.  So the words of a descriptor are built once per operand, and a UMMA's own
// is an addition to the address field of the low word (14 bits of 16 bytes: shared
// memory never carries out of it): 75,600 tokens x 40 heads 15.7 -> 14.7 ms; with the
// tile known at compile time and ring positions stepped instead of divided, 15.4 ->
// 14.3 (another box).

struct UmmaDesc {
  uint32_t lo, hi;
  __device__ __forceinline__ UmmaDesc(const void* at, uint32_t lbo_bytes, uint32_t sbo_bytes, uint32_t swizzle) {
    const uint64_t d = umma_sdesc(smem_u32(at), lbo_bytes, sbo_bytes, swizzle);
    lo = (uint32_t)d;
    hi = (uint32_t)(d >> 32);
  }
};

// D[tmem] (+)= A[smem] * B[smem], operands `a` and `b` bytes behind their descriptors.
template <bool kAccumulate>
__device__ __forceinline__ void umma_ss_at(uint32_t d, const UmmaDesc& da, uint32_t a, const UmmaDesc& db, uint32_t b,
                                           uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %6, 0;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
      "r"(da.lo + (a >> 4)), "r"(da.hi), "r"(db.lo + (b >> 4)), "r"(db.hi), "r"(idesc), "n"(kAccumulate ? 1 : 0)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem].
__device__ __forceinline__ void umma_ts_at(uint32_t d, uint32_t a, const UmmaDesc& db, uint32_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(db.lo + (b >> 4)), "r"(db.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One 128 x 128 product of two K-major tiles of D columns, `a` and `b` bytes
// behind the descriptors of their buffers.
template <int D>
__device__ __forceinline__ void umma_scores(uint32_t acc, const UmmaDesc& da, uint32_t a, const UmmaDesc& db,
                                            uint32_t b) {
  using C = AttnCfg<D>;
  umma_ss_at<false>(acc, da, a, db, b, C::IDESC_QK);
#pragma unroll
  for (int kk = 1; kk < D / 16; ++kk) {
    const uint32_t off = (kk / (C::DBLK / 16)) * C::DB_BYTES + (kk % (C::DBLK / 16)) * 32;
    umma_ss_at<true>(acc, da, a + off, db, b + off, C::IDESC_QK);
  }
}

// A ring's stage and the parity of its barriers.
template <int N>
struct RingPos {
  int st = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++st == N) { st = 0; phase ^= 1u; }
  }
};

// ---- thread-block clusters and distributed shared memory

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// All threads of all CTAs of the cluster meet; shared-memory writes before it
// are visible cluster-wide after it.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address of `p` (own shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

__device__ __forceinline__ float cluster_ld(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float4 cluster_ld4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Sum over one warp.
__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D, bool kSplit>
__global__ void __launch_bounds__(384, 1)
    attn_fwd_tcgen05_sparse_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                                   const SparseParams p) {
  using C = SparseCfg<D>;
  unsigned char* sQ = smem_base_1024();                            // NQ tiles
  unsigned char* sK = sQ + C::NQ * C::TILE_BYTES;                  // NK tiles
  unsigned char* sV = sK + C::NK * C::TILE_BYTES;                  // NV tiles
  uint32_t* bits = reinterpret_cast<uint32_t*>(sQ + C::BITS_OFF);  // [NQ][kSparseWords]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sQ + C::BARS_OFF);
  uint64_t* q_full = bars;
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + C::NK;
  uint64_t* v_full = k_empty + C::NK;
  uint64_t* v_empty = v_full + C::NV;
  uint64_t* s_full = v_empty + C::NV;      // [NQ]
  uint64_t* p_full = s_full + C::NQ;       // [NQ]
  uint64_t* o_done = p_full + C::NQ;       // [NQ] the tile's last P.V (and all before it) finished
  uint64_t* drain = o_done + C::NQ;        // every UMMA of the CTA has finished
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  const int unit = kSplit ? blockIdx.x / p.splits : blockIdx.x;   // a cluster's CTAs are consecutive
  const int rank = kSplit ? (int)cluster_rank() : 0;
  const int pair = unit % p.n_pairs;
  const int bh = unit / p.n_pairs;
  const int h = bh % p.heads;
  const int b = bh / p.heads;
  const int q0 = pair * (C::NQ * C::BM);
  const bool solo = kSplit && p.nqb == 1;          // both tiles hold the one query block
  const int nq = solo || 2 * pair + 1 < p.nqb ? 2 : 1;   // query tiles holding rows of the sequence
  const int nw = (p.nkb + 31) / 32;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < C::NK; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
    for (int s = 0; s < C::NV; ++s) { mbar_init(&v_full[s], 1); mbar_init(&v_empty[s], 1); }
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);           // one elected lane per softmax warp
      mbar_init(&o_done[i], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(q_full, nq * C::TILE_BYTES);
    for (int i = 0; i < nq; ++i)
#pragma unroll
      for (int db = 0; db < C::NDB; ++db)
        tma_load_5d(sQ + i * C::TILE_BYTES + db * C::DB_BYTES, &tmQ, q_full, db * C::DBLK, h, 0,
                    solo ? q0 : q0 + i * C::BM, b);
  }
  {
    const uint8_t* row = p.blocks + ((long long)bh * p.nqb + 2 * pair) * p.nkb;
    mask_words(bits, row, 1, p.nkb, warp, 12, lane);
    if (nq == 2)
      mask_words(bits + kSparseWords, solo ? row : row + p.nkb, 1, p.nkb, warp, 12, lane);
    else
      for (int w = threadIdx.x; w < nw; w += 384) bits[kSparseWords + w] = 0u;
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if constexpr (kSplit) {
    // keep every splits-th block of the two rows' union (one word per thread), or
    // for one query block every 2 * splits-th for each tile
    static_assert(kSparseWords <= 384, "one word per thread");
    const int w = threadIdx.x;
    uint32_t keep[2] = {0u, 0u}, a = 0u, c = 0u;
    if (w < nw) {
      int at = 0;
      for (int u = 0; u < w; ++u) at += __popc(bits[u] | bits[kSparseWords + u]);
      a = bits[w];
      c = bits[kSparseWords + w];
      for (uint32_t left = a | c; left != 0u; left &= left - 1u, ++at) {
        const uint32_t bit = left & (0u - left);
        const int turn = at % (solo ? 2 * p.splits : p.splits);
        if (turn == (solo ? 2 * rank : rank)) keep[0] |= bit;
        if (turn == (solo ? 2 * rank + 1 : rank)) keep[1] |= bit;
      }
    }
    __syncthreads();
    if (w < nw) {
      bits[w] = a & keep[0];
      bits[kSparseWords + w] = c & keep[1];
    }
    __syncthreads();
  }

  // blocks marked by both rows, and by each row alone (every warp counts for itself)
  int n_both = 0, n_own0 = 0, n_own1 = 0;
  for (int w = lane; w < nw; w += 32) {
    const uint32_t a = bits[w], c = bits[kSparseWords + w];
    n_both += __popc(a & c);
    n_own0 += __popc(a & ~c);
    n_own1 += __popc(c & ~a);
  }
  n_both = warp_sum(n_both);
  n_own0 = warp_sum(n_own0);
  n_own1 = warp_sum(n_own1);
  const int steps0 = n_both + n_own0, steps1 = n_both + n_own1;   // key tiles of tile 0 and of tile 1

  if (warp >= 8) {
    regs_decrease<C::REGS_CTRL>();
    if (warp == C::TMA_WARP) {
      // ---------------------------------------------------------------- TMA
      if (lane == 0) {
        const int n_items = n_both + n_own0 + n_own1;
        // K and V tiles are loaded in one and the same order of items; the key
        // block of item x is remembered until V follows, kLead items later
        constexpr int kLead = 2;
        int recent[kLead] = {0, 0};
        BitWalk both{-1, 0u}, own0{-1, 0u}, own1{-1, 0u};
        auto next = [&](BitWalk& k, int which) -> int {   // which: 0 both, 1 row 0 alone, 2 row 1 alone
          while (k.bits == 0u) {
            ++k.word;
            const uint32_t a = bits[k.word], c = bits[kSparseWords + k.word];
            k.bits = which == 0 ? (a & c) : (which == 1 ? (a & ~c) : (c & ~a));
          }
          const int kb = k.word * 32 + __ffs(k.bits) - 1;
          k.bits &= k.bits - 1u;
          return kb;
        };
        int left0 = n_own0, left1 = n_own1;
        bool turn0 = true;
        auto item_block = [&](int x) -> int {             // called for x = 0, 1, 2, ... in turn
          if (x < n_both) return next(both, 0);
          const bool zero = left1 == 0 || (turn0 && left0 > 0);
          turn0 = !zero;
          if (zero) { --left0; return next(own0, 1); }
          --left1;
          return next(own1, 2);
        };
        int k_issued = 0, v_issued = 0;
        bool ok = true;
        auto load = [&](unsigned char* ring, const CUtensorMap* map, uint64_t* full, uint64_t* empty, int stages,
                        int x, int kb, int site) -> bool {
          const int st = x % stages;
          if (x >= stages && !mbar_wait(&empty[st], ((x / stages) - 1) & 1, site)) return false;
          mbar_arrive_expect_tx(&full[st], C::TILE_BYTES);
#pragma unroll
          for (int db = 0; db < C::NDB; ++db)
            tma_load_5d(ring + st * C::TILE_BYTES + db * C::DB_BYTES, map, &full[st], db * C::DBLK, h, 0,
                        kb * C::BN, b);
          return true;
        };
        for (int x = 0; x < n_items + kLead && ok; ++x) {
          int kb = 0;
          if (x < n_items) {
            kb = item_block(x);
            ok = load(sK, &tmK, k_full, k_empty, C::NK, x, kb, kSiteKEmpty);
            if (ok) k_issued = x + 1;
          }
          const int old = recent[kLead - 1];
#pragma unroll
          for (int r = kLead - 1; r > 0; --r) recent[r] = recent[r - 1];
          recent[0] = kb;
          if (ok && x >= kLead) {
            ok = load(sV, &tmV, v_full, v_empty, C::NV, x - kLead, old, kSiteVEmpty);
            if (ok) v_issued = x - kLead + 1;
          }
        }
        // No copy may still be landing in shared memory when the CTA exits.
        mbar_drain(q_full, 0);
        for (int j = k_issued - C::NK < 0 ? 0 : k_issued - C::NK; j < k_issued; ++j)
          mbar_drain(&k_full[j % C::NK], (j / C::NK) & 1);
        for (int j = v_issued - C::NV < 0 ? 0 : v_issued - C::NV; j < v_issued; ++j)
          mbar_drain(&v_full[j % C::NV], (j / C::NV) & 1);
      }
    } else if (warp == C::MMA_WARP) {
      // ---------------------------------------------------------------- MMA
      if (lane == 0) {
        constexpr uint32_t SBO = 8 * C::ROWB;       // 8-row core-matrix group stride
        const UmmaDesc dQ(sQ, 16, SBO, C::SWZ), dK(sK, 16, SBO, C::SWZ), dV(sV, C::DB_BYTES, SBO, C::SWZ);
        RingPos<C::NK> kr;                          // K and V items consumed so far
        RingPos<C::NV> vr;
        // Step j of tile i takes its j-th key tile.  Of a tile that serves
        // both, tile 0's product waits for the copy and tile 1's releases it.
        auto scores = [&](auto tile, int j) -> bool {
          constexpr int i = decltype(tile)::value;
          const bool shared = j < n_both;
          if (!shared || i == 0)
            if (!mbar_wait(&k_full[kr.st], kr.phase, kSiteKFull)) return false;
          tc_fence_after();
          umma_scores<D>(tmem + C::S_COL + i * C::BN, dQ, i * C::TILE_BYTES, dK, kr.st * C::TILE_BYTES);
          umma_commit(&s_full[i]);
          if (!shared || i == 1) { umma_commit(&k_empty[kr.st]); kr.step(); }
          return true;
        };
        auto turn = [&](auto tile, int j) -> bool {     // O_i += P_i V of step j, then S_i of step j + 1
          constexpr int i = decltype(tile)::value;
          const int mine = i == 0 ? steps0 : steps1;
          if (j >= mine) return true;
          const bool shared = j < n_both;
          if (!shared || i == 0)
            if (!mbar_wait(&v_full[vr.st], vr.phase, kSiteVFull)) return false;
          if (!mbar_wait(&p_full[i], j & 1, kSitePFull)) return false;
          tc_fence_after();
          const uint32_t v_at = vr.st * C::TILE_BYTES;
          umma_ts_at(tmem + C::O_COL + i * C::BM, tmem + C::S_COL + i * C::BN, dV, v_at, C::IDESC_PV, j > 0 ? 1u : 0u);
#pragma unroll
          for (int kk = 1; kk < C::BN / 16; ++kk)
            umma_ts_at(tmem + C::O_COL + i * C::BM, tmem + C::S_COL + i * C::BN + kk * 8, dV, v_at + kk * 16 * C::ROWB,
                       C::IDESC_PV, 1u);
          if (j + 1 == mine) umma_commit(&o_done[i]);
          if (j + 1 < mine && !scores(tile, j + 1)) return false;
          if (!shared || i == 1) { umma_commit(&v_empty[vr.st]); vr.step(); }
          return true;
        };
        constexpr std::integral_constant<int, 0> tile0{};
        constexpr std::integral_constant<int, 1> tile1{};
        bool ok = mbar_wait(q_full, 0, kSiteQFull);
        if (ok && steps0 > 0) ok = scores(tile0, 0);
        if (ok && steps1 > 0) ok = scores(tile1, 0);
        const int steps = max(steps0, steps1);
        for (int j = 0; j < steps && ok; ++j) ok = turn(tile0, j) && turn(tile1, j);
        // every UMMA issued above has finished before TMEM is released
        umma_commit(drain);
        mbar_drain(drain, 0);
      }
      __syncwarp();
    }
  } else {
    regs_increase<C::REGS_SOFT>();
    // -------------------------------------------------------------- softmax
    const int tile = warp >> 2;                   // warps 0..3 -> tile 0, 4..7 -> tile 1
    const int quad = warp & 3;                    // TMEM lanes this warp may touch
    const int row = quad * 32 + lane;             // query row within the tile
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t t_s = tl + C::S_COL + tile * C::BN;
    const uint32_t t_o = tl + C::O_COL + tile * C::BM;
    const int mine = tile == 0 ? steps0 : steps1;
    // the step whose key tile is the sequence's last, if that one is ragged:
    // ascending order puts it at the end of its group
    const int last = p.nkb - 1, tail_keys = p.Lk - last * C::BN;
    int tail_step = -1;
    if (tail_keys < C::BN) {
      const uint32_t bit = 1u << (last & 31);
      const bool a = (bits[tile * kSparseWords + (last >> 5)] & bit) != 0u;
      const bool c = (bits[(tile ^ 1) * kSparseWords + (last >> 5)] & bit) != 0u;
      if (a) tail_step = c ? n_both - 1 : mine - 1;
    }
    float m_use = -INFINITY;                      // max used for the exponentials (log2 units)
    float l_sum = 0.f;
    bool ok = tile < nq;
    for (int j = 0; j < mine && ok; ++j) {
      if (!warp_wait(&s_full[tile], j & 1, kSiteSFull)) { ok = false; break; }
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_s + c * 32, s[c]);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_fence(s[c]);
      if (j == tail_step) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e >= tail_keys) s[c][e] = __float_as_uint(-INFINITY);
      }
      auto tile_max = [&]() -> float {
        float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mp[(e >> 1) & 3] = fmax3(mp[(e >> 1) & 3], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
        return fmaxf(fmax3(mp[0], mp[1], mp[2]), mp[3]) * p.scale_log2;
      };
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
      auto exps = [&]() -> float {
        float2 sp[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
        exp_tile(s, t_s, sc2, make_float2(-m_use, -m_use), sp);
        const float2 s01 = fadd2(fadd2(sp[0], sp[1]), fadd2(sp[2], sp[3]));
        return s01.x + s01.y;
      };
      // the dense kernel's rule: the max in use moves only when a tile raises
      // it by more than 8 (log2 units), and is looked at only when the tile's
      // sum of P reaches 2^7
      float alpha = 1.f;
      if (j == 0) m_use = tile_max();
      float lt = exps();
      if (j > 0 && __any_sync(0xffffffffu, !(lt < 128.f))) {
        const float m_new = tile_max();
        const bool rescale = m_new > m_use + 8.f;
        if (__any_sync(0xffffffffu, rescale)) {
          if (rescale) {
            alpha = ex2_approx(m_use - m_new);
            m_use = m_new;
          }
          tmem_st_wait();       // the first stores of P have landed before they are overwritten
          lt = exps();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(t_o + c * 32, o);
            tmem_ld_wait();
            tmem_ld_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(t_o + c * 32, o);
          }
        }
      }
      l_sum = l_sum * alpha + lt;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[tile]);
    }

    if constexpr (kSplit) {
      // Partial results for the cluster: every UMMA of the CTA has finished, so
      // nothing reads or writes Q and the rings any more.  16-byte chunks are
      // swizzled by the row so that neighbouring rows hit different banks.
      if (ok) ok = warp_wait(drain, 0, kSiteODone);
      if (ok) {
        tc_fence_after();
        float2* stat = reinterpret_cast<float2*>(sQ + C::STAT_OFF) + tile * C::BM;
        stat[row] = make_float2(m_use, l_sum);
        if (mine > 0) {
          unsigned char* part = sQ + tile * C::PART_BYTES + row * (D * 4);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(t_o + c * 32, o);
            tmem_ld_wait();
            tmem_ld_fence(o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(part + (((c * 8 + e) ^ (row & 7)) << 4)) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      }
    } else {
      // Epilogue: O / l is staged in the tile's Q buffer (no UMMA reads it any
      // more) in the layout of the O tensor map and leaves by TMA stores, which
      // clip the rows past the sequence.  A tile whose mask row is empty writes
      // zeros, with a log-sum-exp of -inf.
      bool good = ok;
      if (good) good = mine > 0 ? warp_wait(&o_done[tile], 0, kSiteODone) : warp_wait(q_full, 0, kSiteQFull);
      if (good) {
        tc_fence_after();
        const int i = q0 + tile * C::BM + row;      // position in the sequence
        const float inv_l = mine > 0 ? 1.f / l_sum : 0.f;
        unsigned char* stage = sQ + tile * C::TILE_BYTES;
        const int key = C::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
        constexpr int CPB = C::ROWB / 16;           // 16-byte chunks per staged row
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (mine > 0) {
            tmem_ld32(t_o + c * 32, o);
            tmem_ld_wait();
            tmem_ld_fence(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 v;
            v.x = pack_bf16x2(__uint_as_float(o[e + 0]) * inv_l, __uint_as_float(o[e + 1]) * inv_l);
            v.y = pack_bf16x2(__uint_as_float(o[e + 2]) * inv_l, __uint_as_float(o[e + 3]) * inv_l);
            v.z = pack_bf16x2(__uint_as_float(o[e + 4]) * inv_l, __uint_as_float(o[e + 5]) * inv_l);
            v.w = pack_bf16x2(__uint_as_float(o[e + 6]) * inv_l, __uint_as_float(o[e + 7]) * inv_l);
            const int cc = c * 4 + e / 8;           // 16-byte chunk of the row
            *reinterpret_cast<uint4*>(stage + (cc / CPB) * C::DB_BYTES + row * C::ROWB + (((cc % CPB) ^ key) << 4)) = v;
          }
        }
        if (p.lse != nullptr && i < p.Lq)
          p.lse[(long long)bh * p.Lq + i] =
              mine > 0 ? (m_use + __log2f(l_sum)) * 0.69314718055994531f : -INFINITY;
      }
      fence_proxy_async_smem();
      const bool all_good = named_bar_and(1 + tile, 128, good);
      if (all_good && quad == 0 && lane == 0) {
#pragma unroll
        for (int db = 0; db < C::NDB; ++db)
          tma_store_5d(&tmO, sQ + tile * C::TILE_BYTES + db * C::DB_BYTES, db * C::DBLK, h, 0, q0 + tile * C::BM, b);
        bulk_commit_group();
        bulk_wait_group_read<0>();                  // the buffer is read before the CTA exits
      }
    }
  }

  if constexpr (kSplit) {
    __syncwarp();
    cluster_sync_all();
    if (warp < 8) {
      // thread = one 16-byte chunk of a row; this CTA joins rows rank, rank + splits, ...
      constexpr int CH = D / 4;
      const int rows = min(solo ? C::BM : nq * C::BM, p.Lq - q0);
      const int my_rows = rows > rank ? (rows - 1 - rank) / p.splits + 1 : 0;
      const int tiles = solo ? 2 : 1;             // partial results of a row in each CTA
      for (int x = threadIdx.x; x < my_rows * CH; x += 256) {
        const int r = (x / CH) * p.splits + rank, ch = x % CH;
        const float2* stat = reinterpret_cast<const float2*>(sQ + C::STAT_OFF) + r;
        const unsigned char* part = sQ + r * (D * 4) + ((ch ^ (r & 7)) << 4);
        float m = -INFINITY;
        for (int s = 0; s < tiles * p.splits; ++s) {
          const uint32_t at = cluster_addr(stat + (s % tiles) * C::BM, s / tiles);
          if (cluster_ld(at + 4) != 0.f) m = fmaxf(m, cluster_ld(at));
        }
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < tiles * p.splits; ++s) {
          const uint32_t at = cluster_addr(stat + (s % tiles) * C::BM, s / tiles);
          const float ls = cluster_ld(at + 4);
          if (ls == 0.f) continue;                // the tile had no key block of the row
          const float f = ex2_approx(cluster_ld(at) - m);
          const float4 v = cluster_ld4(cluster_addr(part + (s % tiles) * C::PART_BYTES, s / tiles));
          l = fmaf(ls, f, l);
          o.x = fmaf(v.x, f, o.x);
          o.y = fmaf(v.y, f, o.y);
          o.z = fmaf(v.z, f, o.z);
          o.w = fmaf(v.w, f, o.w);
        }
        const float inv_l = l != 0.f ? 1.f / l : 0.f;
        const long long i = q0 + r;
        *reinterpret_cast<uint2*>(p.o + ((((long long)b * p.Lq + i) * p.heads + h) * D + ch * 4)) =
            make_uint2(pack_bf16x2(o.x * inv_l, o.y * inv_l), pack_bf16x2(o.z * inv_l, o.w * inv_l));
        if (p.lse != nullptr && ch == 0)
          p.lse[(long long)bh * p.Lq + i] = l != 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
    }
    __syncwarp();
    cluster_sync_all();                           // no CTA leaves while a peer reads its shared memory
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace vdit
