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
// channels of one block, a thread 8 channels of every 8th token.  bound by the
// bytes of Q and K; a conversion instruction to float64 per value would take
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

// Scores of 64 query blocks x 64 key blocks of one head: 64 threads, 8 x 8 each
// (two shared-memory loads per eight multiply-adds).  Bound by the float64 units.
__global__ void __launch_bounds__(64) block_scores_kernel(const double* __restrict__ qm, const double* __restrict__ km,
                                                          unsigned long long* keys, SelectShape s,
                                                          const unsigned int* flag) {
  __shared__ double sq[16][65], sk[16][65];
  if (tripped(flag)) return;
  const long long bh = blockIdx.z;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  const int ty = threadIdx.x >> 3, tx = threadIdx.x & 7;
  double acc[8][8] = {};
  for (int d0 = 0; d0 < s.D; d0 += 16) {
#pragma unroll 8
    for (int e = threadIdx.x; e < 64 * 16; e += 64) {
      const int r = e >> 4, d = e & 15;
      sq[d][r] = i0 + r < s.nqb ? qm[(bh * s.nqb + i0 + r) * s.D + d0 + d] : 0.;
      sk[d][r] = j0 + r < s.nkb ? km[(bh * s.nkb + j0 + r) * s.D + d0 + d] : 0.;
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 16; ++d) {
      double x[8], y[8];
#pragma unroll
      for (int m = 0; m < 8; ++m) { x[m] = sq[d][ty + 8 * m]; y[m] = sk[d][tx + 8 * m]; }
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < 8; ++n) acc[m][n] = fma(x[m], y[n], acc[m][n]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int i = i0 + ty + 8 * m, j = j0 + tx + 8 * n;
      if (i < s.nqb && j < s.nkb) keys[(bh * s.nqb + i) * s.nkb + j] = order_key(acc[m][n]);
    }
}

// One warp per row: a threshold t with exactly top_k keys at or above it, bit by
// bit from the first bit in which the row's keys differ (the search ends as soon
// as the count fits: some 20 of 64 bits); then the row's marks.  Only where keys
// are equal can the search end with more than top_k at or above t; of those equal
// to t the first ones are marked.  N > 0: a row of at most 32 N keys is held in
// registers; N = 0: longer rows are read again for each bit.
template <int N>
__global__ void __launch_bounds__(256) block_pick_kernel(const unsigned long long* __restrict__ keys,
                                                         unsigned char* blocks, long long rows, SelectShape s,
                                                         const unsigned int* flag) {
  if (tripped(flag)) return;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const unsigned long long* key = keys + row * s.nkb;
  unsigned long long held[N > 0 ? N : 1];
#pragma unroll
  for (int i = 0; i < N; ++i) held[i] = i * 32 + lane < s.nkb ? __ldcs(key + i * 32 + lane) : 0ull;
  auto each = [&](auto f) {                              // f(key) over this lane's keys
    if constexpr (N > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i * 32 + lane < s.nkb) f(held[i]);
    } else {
      for (int j = lane; j < s.nkb; j += 32) f(key[j]);
    }
  };
  // the bits all keys of the row share, by the high words' extremes
  uint32_t lo = 0xffffffffu, hi = 0u;
  each([&](unsigned long long x) {
    const uint32_t h = (uint32_t)(x >> 32);
    lo = min(lo, h);
    hi = max(hi, h);
  });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  uint32_t t = 0u;                                       // the threshold's high word
  int above = s.nkb;                                     // keys at or above the threshold
  const int top = 31 - __clz((int)(lo ^ hi));            // -1: all high words are equal
  t = top < 0 ? hi : (top < 31 ? hi & ~((2u << top) - 1u) : 0u);
  for (int bit = top; bit >= 0 && above != s.top_k; --bit) {
    const uint32_t cand = t | (1u << bit);
    int n = 0;
    each([&](unsigned long long x) { n += (uint32_t)(x >> 32) >= cand; });
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= s.top_k) { t = cand; above = n; }
  }
  unsigned long long thr = (unsigned long long)t << 32;
  for (int bit = 31; bit >= 0 && above != s.top_k; --bit) {
    const unsigned long long cand = thr | (1ull << bit);
    int n = 0;
    each([&](unsigned long long x) { n += x >= cand; });
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= s.top_k) { thr = cand; above = n; }
  }
  int ties = s.nkb;                                      // marks left for keys equal to thr
  if (above != s.top_k) {
    int n = 0;
    each([&](unsigned long long x) { n += x > thr; });
    ties = s.top_k - (int)__reduce_add_sync(0xffffffffu, n);
  }
  auto mark = [&](int j, unsigned long long x) {
    const bool eq = j < s.nkb && x == thr;
    const unsigned int eqs = __ballot_sync(0xffffffffu, eq);
    const bool on = x > thr || (eq && __popc(eqs & ((1u << lane) - 1u)) < ties);
    ties -= min(ties, __popc(eqs));
    if (j < s.nkb) blocks[row * s.nkb + j] = on ? 1 : 0;
  };
  if constexpr (N > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) mark(i * 32 + lane, held[i]);
  } else {
    for (int j0 = 0; j0 < s.nkb; j0 += 32) mark(j0 + lane, j0 + lane < s.nkb ? key[j0 + lane] : 0ull);
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
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(qm + mean_count(s));
  block_means_kernel<<<dim3((unsigned)(s.nqb + s.nkb), (unsigned)chunks, (unsigned)B), 256, 0, st>>>(
      static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), qm, km, s, flag);
  block_scores_kernel<<<dim3((unsigned)kt, (unsigned)qt, (unsigned)bh), 64, 0, st>>>(qm, km, keys, s, flag);
  unsigned char* out = static_cast<unsigned char*>(blocks);
  const unsigned picks = (unsigned)((rows + 7) / 8);
  if (s.nkb <= 128) block_pick_kernel<4><<<picks, 256, 0, st>>>(keys, out, rows, s, flag);
  else if (s.nkb <= 256) block_pick_kernel<8><<<picks, 256, 0, st>>>(keys, out, rows, s, flag);
  else if (s.nkb <= 640) block_pick_kernel<20><<<picks, 256, 0, st>>>(keys, out, rows, s, flag);
  else block_pick_kernel<0><<<picks, 256, 0, st>>>(keys, out, rows, s, flag);
  return cudaGetLastError() == cudaSuccess ? VDIT_OK : VDIT_ERR_CUDA;
}

}  // extern "C"
