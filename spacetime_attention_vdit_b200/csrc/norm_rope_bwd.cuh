// norm_rope_bwd.cuh - the gradients of qk_norm_rope3d_kernel: RMSNorm of Q and
// K, then the 3D rotation.
//
// Forward, for one group of N channels with weight w and r = rsqrt(mean(x^2) + eps):
//   y = R (x r w),  R the rotation of the token's position.
// With g the gradient of y:
//   u  = R^T g                                    (each pair turned back)
//   dx = r (u w) - x r^3 mean(x u w)
//   dw = sum over tokens (and the groups of a token) of u x r
// One HBM pass: x and g are read once, dx written once, per tensor.  A CTA
// walks the tokens of one tensor (blockIdx.y: Q or K), blockIdx.x + k *
// gridDim.x; thread 0 streams each token's rows of x and g into a ring of
// shared-memory stages with bulk copies, several tokens ahead; thread t takes
// the 16-byte vectors t, t + 256, ...  A thread meets the same channels in every
// token, so it keeps its part of dw in float32 registers to the end; the CTA's
// part goes to the workspace and a second kernel adds the CTAs' parts in a
// fixed order (no atomics: the same result on every run).
#pragma once

#include "patchify_rope.cuh"

namespace vdit {

constexpr int kNormBwdThreads = 256;
constexpr int kNormBwdVecs = 4;          // vectors per thread: heads * head_dim <= 256 * 8 * 4 = 8,192
constexpr int kNormBwdMaxStages = 4;
constexpr int kNormBwdMaxCtas = 160;     // CTAs per tensor (rows of the workspace)
constexpr int kSiteNormBwdFull = 32, kSiteNormBwdDrain = 33;

struct NormBwdParams {
  const __nv_bfloat16 *q, *k, *gq, *gk;
  __nv_bfloat16 *dq, *dk;
  const float *wq, *wk;
  float* parts;            // [2][kNormBwdMaxCtas][group], or null when no weight gradient is wanted
  int group, stages;
  float eps;
  double theta;
};

template <bool kWide>   // the group is the token's whole heads*D vector
__global__ void __launch_bounds__(kNormBwdThreads, 2) bwd_qk_norm_rope3d_kernel(const NormBwdParams p, RopeShape s) {
  __shared__ float wsum[2][2][8];                       // [token parity][sum][warp]
  __shared__ float2 cs[2][kRopeMaxPairs];               // the token's pairs, by token parity
  __shared__ __align__(8) uint64_t full[kNormBwdMaxStages];
  if (__syncthreads_or(watchdog_tripped())) return;     // all threads of the CTA decide alike

  const int tensor = s.ntens == 2 ? (int)blockIdx.y : 1;
  const __nv_bfloat16* x_in = tensor ? p.k : p.q;
  const __nv_bfloat16* g_in = tensor ? p.gk : p.gq;
  __nv_bfloat16* d_out = tensor ? p.dk : p.dq;
  const float* w = tensor ? p.wk : p.wq;

  const int vec_per_head = s.D / 8;
  const int nv = s.heads * vec_per_head;                // vectors per token
  uint4* ring = reinterpret_cast<uint4*>(dyn_smem);     // [stage][x row, g row] of nv vectors each
  // per-axis tables: time [Tg][d_t/2], then height [Hg][d_h/2], then width [Wg][d_w/2]
  float2* tab = reinterpret_cast<float2*>(ring + (size_t)p.stages * 2 * nv);
  const int pt = s.d_t / 2, ph = s.d_h / 2, pw = s.d_w / 2;
  const int Tg = (int)(s.L / ((long long)s.Hg * s.Wg));
  const int off_h = Tg * pt, off_w = off_h + s.Hg * ph, n_tab = off_w + s.Wg * pw;
  if (threadIdx.x == 0) {
    for (int st = 0; st < p.stages; ++st) mbar_init(&full[st], 1);
    fence_mbar_init();
  }
  __syncthreads();

  const uint32_t row_bytes = (uint32_t)nv * 16u;
  const long long n_my = (s.ntok - 1 - blockIdx.x) / gridDim.x + 1;   // grid <= ntok
  auto issue = [&](long long k) {                       // thread 0: token k of this CTA into its stage
    const int st = (int)(k % p.stages);
    const long long tok = blockIdx.x + k * gridDim.x;
    mbar_arrive_expect_tx(&full[st], 2 * row_bytes);
    bulk_load(ring + (size_t)st * 2 * nv, x_in + tok * nv * 8, row_bytes, &full[st]);
    bulk_load(ring + (size_t)st * 2 * nv + nv, g_in + tok * nv * 8, row_bytes, &full[st]);
  };
  long long issued = n_my < p.stages ? n_my : p.stages;
  if (threadIdx.x == 0)
    for (long long k = 0; k < issued; ++k) issue(k);
  // the table is built while the first rows land
  for (int x = threadIdx.x; x < n_tab; x += blockDim.x)
    tab[x] = rope_axis_entry(x, off_h, off_w, s.d_t, s.d_h, s.d_w, p.theta);
  __syncthreads();

  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int gv = p.group / 8;                           // vectors per group
  const float inv_group = 1.f / (float)p.group;
  float dw[kWide ? kNormBwdVecs : 1][8];
#pragma unroll
  for (int r = 0; r < (kWide ? kNormBwdVecs : 1); ++r)
#pragma unroll
    for (int m = 0; m < 8; ++m) dw[r][m] = 0.f;
  auto load_w = [&](int e, float (&wv)[8]) {            // the vector's weights
    if (w != nullptr) {
      const int c0 = (e * 8) % p.group;
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + c0));
      const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + c0 + 4));
      wv[0] = w0.x; wv[1] = w0.y; wv[2] = w0.z; wv[3] = w0.w;
      wv[4] = w1.x; wv[5] = w1.y; wv[6] = w1.z; wv[7] = w1.w;
    } else {
#pragma unroll
      for (int m = 0; m < 8; ++m) wv[m] = 1.f;
    }
  };
  auto unpack = [](const uint4& v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const __nv_bfloat162 pr = *reinterpret_cast<const __nv_bfloat162*>(&u[m]);
      f[2 * m] = __low2float(pr);
      f[2 * m + 1] = __high2float(pr);
    }
  };

  long long k = 0;
  for (; k < n_my; ++k) {
    const long long tok = blockIdx.x + k * gridDim.x;
    const int l = (int)(tok % s.L);
    const int par = (int)(k & 1);
    if (t < pt + ph + pw) {                             // the token's row of pairs, from the axis tables
      float2 c;
      if (t < pt) c = tab[(l / (s.Hg * s.Wg)) * pt + t];
      else if (t < pt + ph) c = tab[off_h + ((l / s.Wg) % s.Hg) * ph + (t - pt)];
      else c = tab[off_w + (l % s.Wg) * pw + (t - pt - ph)];
      cs[par][t] = c;
    }
    const int st = (int)(k % p.stages);
    const bool okw = mbar_wait(&full[st], (uint32_t)((k / p.stages) & 1), kSiteNormBwdFull);
    if (!__syncthreads_and(okw)) break;                 // also publishes cs[par]
    const uint4* sx = ring + (size_t)st * 2 * nv;
    const uint4* sg = sx + nv;
    // u = R^T g of vector e: (g0, g1) -> (g0 cos + g1 sin, g1 cos - g0 sin)
    auto turned = [&](int e, float (&u)[8]) {
      unpack(sg[e], u);
      const int p0 = (e % vec_per_head) * 4;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 c = cs[par][p0 + m];
        const float g0 = u[2 * m], g1 = u[2 * m + 1];
        u[2 * m] = fmaf(g0, c.x, g1 * c.y);
        u[2 * m + 1] = fmaf(g1, c.x, -(g0 * c.y));
      }
    };
    // sums of x^2 and of x u w over this thread's vectors of a group
    auto sums = [&](int e, float& sq, float& dot) {
      float x[8], u[8], wv[8];
      unpack(sx[e], x);
      turned(e, u);
      load_w(e, wv);
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        sq = fmaf(x[m], x[m], sq);
        dot = fmaf(x[m], u[m] * wv[m], dot);
      }
    };
    float sq = 0.f, dot = 0.f;
    if (kWide) {
#pragma unroll
      for (int r = 0; r < kNormBwdVecs; ++r)
        if (t + 256 * r < nv) sums(t + 256 * r, sq, dot);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      if (lane == 0) { wsum[par][0][warp] = sq; wsum[par][1][warp] = dot; }
      __syncthreads();
      sq = 0.f; dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) { sq += wsum[par][0][i]; dot += wsum[par][1][i]; }
    }
    uint4* dst = reinterpret_cast<uint4*>(d_out) + tok * nv;
#pragma unroll
    for (int r = 0; r < kNormBwdVecs; ++r) {
      const int e = t + 256 * r;
      if (!kWide) {                                     // the group's gv vectors: gv consecutive lanes
        sq = 0.f; dot = 0.f;
        if (e < nv) sums(e, sq, dot);
        for (int o = gv >> 1; o >= 1; o >>= 1) {
          sq += __shfl_xor_sync(0xffffffffu, sq, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
      }
      if (e < nv) {
        const float rr = rsqrtf(fmaf(sq, inv_group, p.eps));
        const float back = -(rr * rr) * (dot * inv_group);   // dx = rr (u w + x back)
        float x[8], u[8], wv[8];
        unpack(sx[e], x);
        turned(e, u);
        load_w(e, wv);
        uint32_t o[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float a = rr * fmaf(x[2 * m], back, u[2 * m] * wv[2 * m]);
          const float c = rr * fmaf(x[2 * m + 1], back, u[2 * m + 1] * wv[2 * m + 1]);
          o[m] = pack_bf16x2(a, c);
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) dw[kWide ? r : 0][m] = fmaf(u[m], x[m] * rr, dw[kWide ? r : 0][m]);
        dst[e] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    __syncthreads();                                    // the stage is free
    if (t == 0 && issued < n_my) issue(issued++);
  }
  const bool whole = k == n_my;
  // No copy may still be landing in shared memory when the CTA exits (only
  // when a wait above ran out can tokens k .. issued-1 still be in flight).
  if (t == 0)
    for (long long k2 = k; k2 < issued; ++k2)
      mbar_drain_site(&full[k2 % p.stages], (uint32_t)((k2 / p.stages) & 1), kSiteNormBwdDrain);
  if (p.parts == nullptr || !whole) return;
  float* out = p.parts + ((long long)tensor * kNormBwdMaxCtas + blockIdx.x) * p.group;
  if (kWide) {
#pragma unroll
    for (int r = 0; r < kNormBwdVecs; ++r) {
      const int e = t + 256 * r;
      if (e < nv) {
        float4* to = reinterpret_cast<float4*>(out + e * 8);
        to[0] = make_float4(dw[r][0], dw[r][1], dw[r][2], dw[r][3]);
        to[1] = make_float4(dw[r][4], dw[r][5], dw[r][6], dw[r][7]);
      }
    }
  } else {
    // threads t, t + gv, t + 2 gv, ... hold the same channels
    float* all = reinterpret_cast<float*>(dyn_smem);    // [256][8], over the ring
#pragma unroll
    for (int m = 0; m < 8; ++m) all[t * 8 + m] = dw[0][m];
    __syncthreads();
    for (int c = t; c < p.group; c += blockDim.x) {
      float a = 0.f;
      for (int i = c >> 3; i < kNormBwdThreads; i += gv) a += all[i * 8 + (c & 7)];
      out[c] = a;
    }
  }
}

// dw[c] = the CTAs' parts of channel c, added in a fixed order: a CTA takes 32
// channels of one tensor, its eight warps the CTAs w, w + 8, ...
__global__ void __launch_bounds__(256) bwd_weights_qk_norm_rope3d_kernel(const float* __restrict__ parts, float* dwq,
                                                                         float* dwk, int group, int n_parts) {
  __shared__ float sum[8][32];
  if (watchdog_tripped()) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* dw = blockIdx.y ? dwk : dwq;
  const float* from = parts + (long long)blockIdx.y * kNormBwdMaxCtas * group;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (dw != nullptr && c < group) {
#pragma unroll 4
    for (int i = warp; i < n_parts; i += 8) a += from[(long long)i * group + c];
  }
  sum[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && dw != nullptr && c < group) {
    float b = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) b += sum[i][lane];
    dw[c] = b;
  }
}

}  // namespace vdit
