// block_select.cu - the cheap score that picks each query block's key blocks
// for attn_block_sparse.cuh, and its entry points.
//
//   score[i, j] = mean of Q over query block i . mean of K over key block j
//   blocks[i, j] = 1 for the top_k highest scores of row i; of equal scores the
//                  lower index goes first; a NaN score goes behind every number
// A ragged last block's mean is over its own tokens.  Which block is picked is
// decided by values next to a border, so means and scores are float64: sums of
// 128 bfloat16 values are then exact unless their exponents span more than 38
// bits, and two scores are told apart down to a relative 1e-15.
//
// These kernels have no waits.  They are a translation unit of their own (the
// tensor-core kernels' compile flags and register budgets do not apply), and
// take the watchdog's flag by address.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "vdit.h"
#include "vdit_internal.h"

namespace vdit {
namespace {

constexpr int kBlock = 128;               // tokens per block
constexpr int kMaxKeyBlocks = 6144;       // what one row of attn_block_sparse takes

struct SelectShape {
  int B, Lq, Lk, heads, D, nqb, nkb, top_k;
};

__device__ __forceinline__ bool tripped(const unsigned int* flag) {
  return *reinterpret_cast<const volatile unsigned int*>(flag) != 0u;
}

// Means of every 128-token block of Q (blockIdx.x < nqb) and K: a CTA takes 256
// channels of one block, a thread 8 channels of every 8th token.  Bound by the
// bytes of Q and K (240 us for twice 75,600 x 40 x 128: 6.45 TB/s); a conversion instruction to float64 per value would take
// longer than they do (16 per clock and SM), so a bfloat16's bits are moved into
// a float64's high word as they are: exponent field e stands for 2^(e - 1023)
// there and 2^(e - 127) in the bfloat16, denormals alike, so the float64 is the
// value times 2^-896, and the sum is scaled back once.  Exponent 255 (infinities
// and NaN) would not survive: a thread that meets one sums again by conversions.
__device__ __forceinline__ double bits_to_double(uint32_t f32_bits) {
  return __hiloint2double(((int)f32_bits >> 3) & 0x8fffffff, 0);
}

__global__ void __launch_bounds__(256) block_means_kernel(const __nv_bfloat16* __restrict__ q,
                                                          const __nv_bfloat16* __restrict__ k, double* qm, double* km,
                                                          SelectShape s, const unsigned int* flag) {
  __shared__ double part[8][32][9];
  let_next_start();
  if (tripped(flag)) return;
  const bool is_q = (int)blockIdx.x < s.nqb;
  const int blk = is_q ? blockIdx.x : blockIdx.x - s.nqb;
  const int L = is_q ? s.Lq : s.Lk, n = is_q ? s.nqb : s.nkb;
  const int b = blockIdx.z;
  const int width = s.heads * s.D;
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int c0 = (blockIdx.y * 32 + lane) * 8;
  const int rows = min(kBlock, L - blk * kBlock);
  double a[8] = {0., 0., 0., 0., 0., 0., 0., 0.};
  if (c0 < width) {
    const __nv_bfloat16* src = (is_q ? q : k) + ((long long)b * L + (long long)blk * kBlock) * width + c0;
    uint32_t most = 0u;                                  // the largest magnitudes met, as 16-bit halves
    auto add = [&](const uint4& v) {
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        a[2 * m] += bits_to_double(u[m] << 16);
        a[2 * m + 1] += bits_to_double(u[m] & 0xffff0000u);
        most = __vmaxu2(most, u[m] & 0x7fff7fffu);
      }
    };
    if (rows == kBlock) {                                // a whole block: 16 tokens, 8 loads in flight
#pragma unroll
      for (int r0 = 0; r0 < 16; r0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          v[r] = __ldcs(reinterpret_cast<const uint4*>(src + (long long)(sub + 8 * (r0 + r)) * width));
#pragma unroll
        for (int r = 0; r < 8; ++r) add(v[r]);
      }
    } else {
      for (int r = sub; r < rows; r += 8) add(__ldcs(reinterpret_cast<const uint4*>(src + (long long)r * width)));
    }
    if ((most & 0xffffu) >= 0x7f80u || (most >> 16) >= 0x7f80u) {
#pragma unroll
      for (int m = 0; m < 8; ++m) a[m] = 0.;
      for (int r = sub; r < rows; r += 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + (long long)r * width));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          a[2 * m] += (double)__uint_as_float(u[m] << 16) * 0x1p-896;
          a[2 * m + 1] += (double)__uint_as_float(u[m] & 0xffff0000u) * 0x1p-896;
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 8; ++m) part[sub][lane][m] = a[m];
  __syncthreads();
  // 256 threads, one channel each
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c < width) {
    double t = 0.;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += part[i][threadIdx.x >> 3][threadIdx.x & 7];
    const int h = c / s.D, d = c - h * s.D;
    (is_q ? qm : km)[(((long long)b * s.heads + h) * n + blk) * s.D + d] = t * 0x1p896 / (double)rows;
  }
}

// A float64 as an unsigned integer of the same order; both zeros alike, NaN lowest.
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return 0ull;
  const long long v = __double_as_longlong(x + 0.0);
  return v < 0 ? ~(unsigned long long)v : (unsigned long long)v | 0x8000000000000000ull;
}

// Scores of 64 query blocks x 64 key blocks of one head: 128 threads, 4 x 8 each,
// the means fetched 16 channels at a time into two buffers with asynchronous
// copies (rows of 144 bytes: the eight rows that eight lanes read 16 bytes of fall
// into different banks).  Bound by issuing float64 multiply-adds (60 % of its
// instructions; 45 us for 40 x 256 x 256 scores of 128 channels, 35 % of the float64
// units' rate); 64 threads of 8 x 8 take 4 % longer.  The ordered scores leave as
// two arrays of 32-bit words: the second is hardly ever read.
constexpr int kScoreRow = 18;                            // doubles per staged row: 16 channels and padding

__device__ __forceinline__ void copy16(void* dst, const void* src, bool on) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(on ? 16 : 0) : "memory");
}

__global__ void __launch_bounds__(128, 4) block_scores_kernel(const double* qm, const double* km, uint32_t* hi,
                                                              uint32_t* lo, SelectShape s, const unsigned int* flag) {
  __shared__ __align__(16) double st[2][2][64 * kScoreRow];
  let_next_start();
  wait_for_previous();
  if (tripped(flag)) return;
  const long long bh = blockIdx.z;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  const int ty = threadIdx.x >> 3, tx = threadIdx.x & 7;
  auto fetch = [&](int buf, int d0) {                    // 2 x 64 rows x 8 chunks of 16 bytes
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int r = ty + 16 * (c & 3), which = c >> 2;
      const int row = (which ? j0 : i0) + r, n = which ? s.nkb : s.nqb;
      const double* from = (which ? km : qm) + (bh * n + min(row, n - 1)) * s.D + d0 + tx * 2;
      copy16(&st[buf][which][r * kScoreRow + tx * 2], from, row < n);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  double acc[4][8] = {};
  const int steps = s.D / 16;
  fetch(0, 0);
  for (int x = 0; x < steps; ++x) {
    if (x + 1 < steps) {
      fetch((x + 1) & 1, (x + 1) * 16);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const double* sq = &st[x & 1][0][ty * kScoreRow];
    const double* sk = &st[x & 1][1][tx * kScoreRow];
#pragma unroll 2
    for (int d = 0; d < 16; ++d) {
      double q[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) q[m] = sq[16 * m * kScoreRow + d];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const double k = sk[8 * n * kScoreRow + d];
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[m][n] = fma(q[m], k, acc[m][n]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int i = i0 + ty + 16 * m, j = j0 + tx + 8 * n;
      if (i < s.nqb && j < s.nkb) {
        const unsigned long long key = order_key(acc[m][n]);
        hi[(bh * s.nqb + i) * s.nkb + j] = (uint32_t)(key >> 32);
        lo[(bh * s.nqb + i) * s.nkb + j] = (uint32_t)key;
      }
    }
}

// One warp per row: a threshold t with exactly top_k keys at or above it, bit by
// bit from the first bit in which the row's high words differ; the search ends
// as soon as the count fits (some 20 of 64 bits).  Only rows whose high words
// leave it open read the low words.  Only where keys are equal can the search end
// with more than top_k at or above t: of those equal to t the first ones are
// marked.  N > 0: the high words of a row of at most 32 N keys are held in
// registers (zeros past its end, which no threshold of the search counts); N = 0:
// longer rows are read again for each bit.  40 x 591 rows of 591 keys take 66 us.
template <int N>
__global__ void __launch_bounds__(256) block_pick_kernel(const uint32_t* hi_words, const uint32_t* lo_words,
                                                         unsigned char* blocks, long long rows, SelectShape s,
                                                         const unsigned int* flag) {
  wait_for_previous();
  if (tripped(flag)) return;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const uint32_t* hw = hi_words + row * s.nkb;
  const uint32_t* lw = lo_words + row * s.nkb;
  unsigned char* out = blocks + row * s.nkb;
  uint32_t held[N > 0 ? N : 1];
#pragma unroll
  for (int i = 0; i < N; ++i) held[i] = i * 32 + lane < s.nkb ? __ldcs(hw + i * 32 + lane) : 0u;
  // the keys of this lane: f(high word, index); `padded`: those past the row's end too, as zeros
  auto each = [&](bool padded, auto f) {
    if constexpr (N > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (padded || i * 32 + lane < s.nkb) f(held[i], i * 32 + lane);
    } else {
      for (int j = lane; j < s.nkb; j += 32) f(hw[j], j);
    }
  };
  uint32_t least = 0xffffffffu, most = 0u;
  each(false, [&](uint32_t h, int) {
    least = min(least, h);
    most = max(most, h);
  });
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  int above = s.nkb;                                     // keys at or above the threshold
  const int top = 31 - __clz((int)(least ^ most));       // -1: all high words are equal
  uint32_t t = top < 0 ? most : (top < 31 ? most & ~((2u << top) - 1u) : 0u);
  for (int bit = top; bit >= 0 && above != s.top_k; --bit) {
    const uint32_t cand = t | (1u << bit);
    int n = 0;
    each(true, [&](uint32_t h, int) { n += h >= cand; });
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= s.top_k) { t = cand; above = n; }
  }
  if (above == s.top_k) {
    each(false, [&](uint32_t h, int j) { out[j] = h >= t ? 1 : 0; });
    return;
  }
  // the low words of the keys whose high word is t decide
  auto sure = [&](uint32_t h) { return h > t; };
  uint32_t tl = 0u;
  for (int bit = 31; bit >= 0 && above != s.top_k; --bit) {
    const uint32_t cand = tl | (1u << bit);
    int n = 0;
    each(false, [&](uint32_t h, int j) { n += sure(h) || (h == t && lw[j] >= cand); });
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= s.top_k) { tl = cand; above = n; }
  }
  int n = 0;
  each(false, [&](uint32_t h, int j) { n += sure(h) || (h == t && lw[j] > tl); });
  int ties = s.top_k - (int)__reduce_add_sync(0xffffffffu, n);   // of the keys equal to (t, tl), the first so many
  for (int j0 = 0; j0 < s.nkb; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t h = j < s.nkb ? hw[j] : 0u, l = j < s.nkb ? lw[j] : 0u;
    const bool eq = j < s.nkb && h == t && l == tl;
    const unsigned int eqs = __ballot_sync(0xffffffffu, eq);
    const bool on = sure(h) || (h == t && l > tl) || (eq && __popc(eqs & ((1u << lane) - 1u)) < ties);
    ties -= min(ties, __popc(eqs));
    if (j < s.nkb) out[j] = on ? 1 : 0;
  }
}

bool select_shape(SelectShape& s, int B, int Lq, int Lk, int heads, int D, int top_k) {
  if (B <= 0 || Lq <= 0 || Lk <= 0 || heads <= 0 || D <= 0) return false;
  s = SelectShape{B, Lq, Lk, heads, D, sparse_blocks(Lq), sparse_blocks(Lk), top_k};
  return (double)B * heads * ((double)Lq + Lk + 256.) * D < 1.0e17 &&
         (double)B * heads * s.nqb * (double)s.nkb < 1.0e17;
}

long long mean_count(const SelectShape& s) { return (long long)s.B * s.heads * ((long long)s.nqb + s.nkb) * s.D; }

}  // namespace
}  // namespace vdit

using namespace vdit;

extern "C" {

long long vdit_attn_select_blocks_workspace(int B, int Lq, int Lk, int heads, int head_dim) {
  SelectShape s;
  if (!select_shape(s, B, Lq, Lk, heads, head_dim, 1)) return -1;
  return 8 * (mean_count(s) + (long long)B * heads * s.nqb * s.nkb);
}

int vdit_attn_select_blocks(const void* q, const void* k, void* blocks, void* workspace, int B, int Lq, int Lk,
                            int heads, int head_dim, int top_k, vdit_stream_t stream) {
  if (!q || !k || !blocks || !workspace) return VDIT_ERR_NULL;
  SelectShape s;
  if (!select_shape(s, B, Lq, Lk, heads, head_dim, top_k)) return VDIT_ERR_SHAPE;
  if (head_dim != 32 && head_dim != 64 && head_dim != 128) return VDIT_ERR_UNSUPPORTED;
  if (top_k < 1 || top_k > s.nkb) return VDIT_ERR_SHAPE;
  if (s.nkb > kMaxKeyBlocks) return VDIT_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k, workspace};
  for (const void* x : ptrs)
    if ((reinterpret_cast<uintptr_t>(x) & 15u) != 0) return VDIT_ERR_ALIGN;
  const long long width = (long long)heads * head_dim, bh = (long long)B * heads;
  const long long chunks = (width + 255) / 256, qt = (s.nqb + 63) / 64, kt = (s.nkb + 63) / 64;
  const long long rows = bh * s.nqb;
  if (chunks > 65535 || B > 65535 || bh > 65535 || qt > 65535 || (rows + 7) / 8 > 0x7fffffffLL) return VDIT_ERR_SHAPE;
  const unsigned int* flag = watchdog_flag();
  if (flag == nullptr) return VDIT_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* qm = static_cast<double*>(workspace);
  double* km = qm + bh * s.nqb * head_dim;
  uint32_t* hi = reinterpret_cast<uint32_t*>(qm + mean_count(s));
  uint32_t* lo = hi + rows * s.nkb;
  block_means_kernel<<<dim3((unsigned)(s.nqb + s.nkb), (unsigned)chunks, (unsigned)B), 256, 0, st>>>(
      static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), qm, km, s, flag);
  if (cudaGetLastError() != cudaSuccess) return VDIT_ERR_CUDA;
  unsigned char* out = static_cast<unsigned char*>(blocks);
  const auto pick = s.nkb <= 128   ? block_pick_kernel<4>
                    : s.nkb <= 256 ? block_pick_kernel<8>
                    : s.nkb <= 640 ? block_pick_kernel<20>
                                   : block_pick_kernel<0>;
  if (!launch_early(block_scores_kernel, dim3((unsigned)kt, (unsigned)qt, (unsigned)bh), 128, st, qm, km, hi, lo, s, flag) ||
      !launch_early(pick, dim3((unsigned)((rows + 7) / 8)), 256, st, hi, lo, out, rows, s, flag)) {
    cudaGetLastError();
    return VDIT_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? VDIT_OK : VDIT_ERR_CUDA;
}

}  // extern "C"
