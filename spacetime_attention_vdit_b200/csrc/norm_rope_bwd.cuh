// norm_rope_bwd.cuh - the gradients of qk_norm_rope3d_kernel: RMSNorm of Q and
// K, then the 3D rotation.
//
// Forward, for one group of N channels with weight w and r = rsqrt(mean(x^2) + eps):
//   y = R (x r w),  R the rotation of the token's position.
// With g the gradient of y:
//   u  = R^T g                                    (each pair turned back)
//   dx = r (u w) - x r^3 mean(x u w)
//   dw = sum over tokens (and the groups of a token) of u x r
// One HBM pass: x and g are read once, dx written once, per tensor (blockIdx.y: Q
// or K).  A CTA walks chunks of `groups` consecutive tokens, blockIdx.x + k *
// gridDim.x; thread 0 streams the chunks' rows of x and g into a ring of
// shared-memory stages with bulk copies, several chunks ahead.  `warps` warps
// share a token; a thread takes its 16-byte vectors lane, lane + 32 * warps, ...
// (V of them), holds x and u in registers from the sums to the result, and meets
// the same channels in every token, so that it keeps its weights and its part
// of dw in float32 registers to the end.  One barrier per chunk: it publishes the
// warps' sums and the next chunk's (cos, sin) rows, and frees the stage, which
// every thread has read by then.  The CTA's part of dw goes to the workspace and
// a second kernel adds the CTAs' parts in a fixed order (no atomics: the same
// result on every run).
#pragma once

#include "patchify_rope.cuh"

namespace vdit {

constexpr int kNormBwdThreads = 320;     // at most: warps * groups * 32 (256 with V = 4)
constexpr int kNormBwdVecs = 4;          // V at most: heads * head_dim <= 8,192
constexpr int kNormBwdMaxStages = 8;
constexpr int kNormBwdMaxCtas = 320;     // CTAs per tensor (rows of the workspace)
constexpr int kSiteNormBwdFull = 32, kSiteNormBwdDrain = 33;

struct NormBwdParams {
  const __nv_bfloat16 *q, *k, *gq, *gk;
  __nv_bfloat16 *dq, *dk;
  const float *wq, *wk;
  float* parts;            // [2][kNormBwdMaxCtas][group], or null when no weight gradient is wanted
  int group, stages;
  int warps, groups;       // warps per token, tokens per chunk
  float eps;
  double theta;
};

// kWide: the group is the token's whole heads*D vector; else a group is 1 .. 32
// neighbouring lanes of one vector each.
template <bool kWide, int V>
__global__ void __launch_bounds__(V == 4 ? 256 : kNormBwdThreads, V == 1 ? 3 : 2)
    bwd_qk_norm_rope3d_kernel(const NormBwdParams p, RopeShape s) {
  __shared__ float2 wsum[2][kNormBwdThreads / 32];      // [chunk parity][warp]: sums of x^2 and of x u w
  __shared__ double inv_freq[kRopeMaxPairs];
  __shared__ __align__(8) uint64_t full[kNormBwdMaxStages];
  if (__syncthreads_or(watchdog_tripped())) return;     // all threads of the CTA decide alike

  const int tensor = s.ntens == 2 ? (int)blockIdx.y : 1;
  const __nv_bfloat16* x_in = tensor ? p.k : p.q;
  const __nv_bfloat16* g_in = tensor ? p.gk : p.gq;
  __nv_bfloat16* d_out = tensor ? p.dk : p.dq;
  const float* w = tensor ? p.wk : p.wq;

  const int T = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int G = p.groups, span = 32 * p.warps;          // threads of one token
  const int gi = warp / p.warps, li = t - gi * span;
  const int vph = s.D / 8, P = s.D / 2;                 // vectors and pairs per head
  const int nv = s.heads * vph;                         // vectors per token
  uint4* ring = reinterpret_cast<uint4*>(dyn_smem);     // [stage][G x rows, G g rows] of nv vectors each
  // the chunk's pairs, by chunk parity: [2][G][2][vph] float4, pairs 0 and 1 of
  // every vector, then pairs 2 and 3 (neighbouring lanes read neighbouring 16 bytes)
  float4* cs = reinterpret_cast<float4*>(ring + (size_t)p.stages * 2 * G * nv);
  // per-axis tables: time [Tg][d_t/2], then height [Hg][d_h/2], then width [Wg][d_w/2]
  float2* tab = reinterpret_cast<float2*>(cs + 4 * G * vph);
  const int pt = s.d_t / 2, ph = s.d_h / 2, pw = s.d_w / 2;
  const int Tg = (int)(s.L / ((long long)s.Hg * s.Wg));
  const int off_h = Tg * pt, off_w = off_h + s.Hg * ph, n_tab = off_w + s.Wg * pw;
  if (t == 0) {
    for (int st = 0; st < p.stages; ++st) mbar_init(&full[st], 1);
    fence_mbar_init();
  }
  for (int x = t; x < P; x += T) {
    int i, d;
    if (x < pt) { i = x; d = s.d_t; }
    else if (x < pt + ph) { i = x - pt; d = s.d_h; }
    else { i = x - pt - ph; d = s.d_w; }
    inv_freq[x] = 1.0 / pow(p.theta, (double)(2 * i) / (double)d);
  }
  __syncthreads();

  const uint32_t row_bytes = (uint32_t)nv * 16u;
  const long long n_chunks = (s.ntok + G - 1) / G;
  const long long n_my = (n_chunks - 1 - blockIdx.x) / gridDim.x + 1;   // grid <= n_chunks
  auto issue = [&](long long k) {                       // thread 0: chunk k of this CTA into its stage
    const int st = (int)(k % p.stages);
    const long long tok = (blockIdx.x + k * gridDim.x) * G;
    const uint32_t bytes = (uint32_t)min((long long)G, s.ntok - tok) * row_bytes;
    uint4* to = ring + (size_t)st * 2 * G * nv;
    mbar_arrive_expect_tx(&full[st], 2 * bytes);
    bulk_load(to, x_in + tok * nv * 8, bytes, &full[st]);
    bulk_load(to + (size_t)G * nv, g_in + tok * nv * 8, bytes, &full[st]);
  };
  long long issued = n_my < p.stages ? n_my : p.stages;
  if (t == 0)
    for (long long k = 0; k < issued; ++k) issue(k);
  // the tables are built while the first rows land: rope_phasor's arithmetic
  for (int x = t; x < n_tab; x += T) {
    int pos, pi;
    if (x < off_h) { pos = x / pt; pi = x - pos * pt; }
    else if (x < off_w) { pos = (x - off_h) / ph; pi = x - off_h - pos * ph + pt; }
    else { pos = (x - off_w) / pw; pi = x - off_w - pos * pw + pt + ph; }
    double sn, cn;
    sincos((double)pos * inv_freq[pi], &sn, &cn);
    tab[x] = make_float2((float)cn, (float)sn);
  }
  __syncthreads();
  // the pairs of chunk k's tokens, from the axis tables
  auto pairs = [&](long long k) {
    const long long tok0 = (blockIdx.x + k * gridDim.x) * G;
    float2* to = reinterpret_cast<float2*>(cs + (k & 1) * 2 * G * vph);
    for (int x = t; x < G * P; x += T) {
      const int j = x / P, pi = x - j * P;
      if (tok0 + j >= s.ntok) break;
      const int l = (int)((tok0 + j) % s.L);
      float2 c;
      if (pi < pt) c = tab[(l / (s.Hg * s.Wg)) * pt + pi];
      else if (pi < pt + ph) c = tab[off_h + ((l / s.Wg) % s.Hg) * ph + (pi - pt)];
      else c = tab[off_w + (l % s.Wg) * pw + (pi - pt - ph)];
      to[((j * 2 + ((pi >> 1) & 1)) * vph + (pi >> 2)) * 2 + (pi & 1)] = c;
    }
  };
  pairs(0);

  constexpr int NW = kWide ? V : 1;                     // vectors of a thread with channels of their own
  constexpr bool kHoldW = NW <= 2;                      // their weights fit the registers too
  const int gv = p.group / 8;                           // vectors per group
  const float inv_group = 1.f / (float)p.group;
  float2 dw[NW][4], wv[NW][4];
  auto load_w = [&](int e, float2 (&to)[4]) {           // the vector's weights
    if (w != nullptr) {
      const float* at = w + (e * 8) % p.group;
      const float4 a = __ldg(reinterpret_cast<const float4*>(at));
      const float4 b = __ldg(reinterpret_cast<const float4*>(at + 4));
      to[0] = make_float2(a.x, a.y); to[1] = make_float2(a.z, a.w);
      to[2] = make_float2(b.x, b.y); to[3] = make_float2(b.z, b.w);
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) to[m] = make_float2(1.f, 1.f);
    }
  };
#pragma unroll
  for (int r = 0; r < NW; ++r) {
#pragma unroll
    for (int m = 0; m < 4; ++m) dw[r][m] = make_float2(0.f, 0.f);
    if (kHoldW && li + span * r < nv) load_w(li + span * r, wv[r]);
  }
  auto pair_of = [](uint32_t b) { return make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)); };
  __syncthreads();                                      // pairs(0)

  long long k = 0;
  for (; k < n_my; ++k) {
    const long long tok = (blockIdx.x + k * gridDim.x) * G + gi;
    const int par = (int)(k & 1);
    const int st = (int)(k % p.stages);
    const bool live = gi < G && tok < s.ntok;
    const bool okw = mbar_wait(&full[st], (uint32_t)((k / p.stages) & 1), kSiteNormBwdFull);
    const uint4* sx = ring + ((size_t)st * 2 * G + gi) * nv;
    const uint4* sg = sx + (size_t)G * nv;
    const float4* c4 = cs + (par * G + gi) * 2 * vph;
    uint4 x[V];
    float2 u[V][4];
    float2 sum[kWide ? 1 : V];                          // x^2 and x u w
#pragma unroll
    for (int r = 0; r < V; ++r) {
      const int e = li + span * r;
      float2 a = make_float2(0.f, 0.f), d = a;
      if (live && okw && e < nv) {
        x[r] = sx[e];
        const uint4 g = sg[e];
        const int vi = e % vph;
        const float4 ca = c4[vi], cb = c4[vph + vi];
        // u = R^T g: (g0, g1) -> (g0 cos + g1 sin, g1 cos - g0 sin)
        auto back = [&](uint32_t b, float c, float sn) {
          const float2 y = pair_of(b);
          return make_float2(fmaf(y.x, c, y.y * sn), fmaf(y.y, c, -(y.x * sn)));
        };
        u[r][0] = back(g.x, ca.x, ca.y);
        u[r][1] = back(g.y, ca.z, ca.w);
        u[r][2] = back(g.z, cb.x, cb.y);
        u[r][3] = back(g.w, cb.z, cb.w);
        float2 we[4];
        if (!kHoldW) load_w(e, we);
        const uint32_t xs[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 y = pair_of(xs[m]);
          a = ffma2(y, y, a);
          d = ffma2(y, fmul2(u[r][m], kHoldW ? wv[kWide ? r : 0][m] : we[m]), d);
        }
      }
      const float2 one = make_float2(a.x + a.y, d.x + d.y);
      if (kWide && r > 0) sum[0] = fadd2(sum[0], one);
      else sum[kWide ? 0 : r] = one;
    }
    auto add_lanes = [&](float2& v, int o) {
      v = fadd2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    };
    if (kWide) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) add_lanes(sum[0], o);
      if (lane == 0) wsum[par][warp] = sum[0];
    } else {
#pragma unroll
      for (int r = 0; r < V; ++r)
        for (int o = gv >> 1; o >= 1; o >>= 1) add_lanes(sum[kWide ? 0 : r], o);
    }
    if (k + 1 < n_my) pairs(k + 1);
    if (!__syncthreads_and(okw)) break;                 // the stage is free; the sums and the next pairs are out
    if (t == 0 && issued < n_my) issue(issued++);
    if (kWide) {
      sum[0] = wsum[par][gi * p.warps];
      for (int i = 1; i < p.warps; ++i) sum[0] = fadd2(sum[0], wsum[par][gi * p.warps + i]);
    }
    uint4* dst = reinterpret_cast<uint4*>(d_out) + tok * nv;
#pragma unroll
    for (int r = 0; r < V; ++r) {
      const int e = li + span * r;
      if (live && e < nv) {
        const float2 sm = sum[kWide ? 0 : r];
        const float rr = rsqrtf(fmaf(sm.x, inv_group, p.eps));
        const float back = -(rr * rr) * (sm.y * inv_group);   // dx = rr (u w + x back)
        const float2 rr2 = make_float2(rr, rr), bk2 = make_float2(back, back);
        float2 we[4];
        if (!kHoldW) load_w(e, we);
        const uint32_t xs[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
        uint32_t o[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int rw = kWide ? r : 0;
          const float2 y = pair_of(xs[m]);
          const float2 dx = fmul2(rr2, ffma2(y, bk2, fmul2(u[r][m], kHoldW ? wv[rw][m] : we[m])));
          dw[rw][m] = ffma2(u[r][m], fmul2(y, rr2), dw[rw][m]);
          o[m] = pack_bf16x2(dx.x, dx.y);
        }
        dst[e] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  const bool whole = k == n_my;
  // No copy may still be landing in shared memory when the CTA exits (only
  // when a wait above ran out can chunks k .. issued-1 still be in flight).
  if (t == 0)
    for (long long k2 = k; k2 < issued; ++k2)
      mbar_drain_site(&full[k2 % p.stages], (uint32_t)((k2 / p.stages) & 1), kSiteNormBwdDrain);
  if (p.parts == nullptr || !whole) return;
  float* out = p.parts + ((long long)tensor * kNormBwdMaxCtas + blockIdx.x) * p.group;
  if (kWide && V > 1) {                                 // one token per chunk: a channel is one thread's
#pragma unroll
    for (int r = 0; r < V; ++r) {
      const int e = li + span * r;
      if (e < nv) {
        float4* to = reinterpret_cast<float4*>(out + e * 8);
        to[0] = make_float4(dw[kWide ? r : 0][0].x, dw[kWide ? r : 0][0].y, dw[kWide ? r : 0][1].x, dw[kWide ? r : 0][1].y);
        to[1] = make_float4(dw[kWide ? r : 0][2].x, dw[kWide ? r : 0][2].y, dw[kWide ? r : 0][3].x, dw[kWide ? r : 0][3].y);
      }
    }
    return;
  }
  // threads t, t + step, t + 2 step, ... hold the same channels
  const int step = kWide ? span : gv;
  float* all = reinterpret_cast<float*>(dyn_smem);      // [T][8], over the ring
  float2* mine = reinterpret_cast<float2*>(all + t * 8);
#pragma unroll
  for (int m = 0; m < 4; ++m) mine[m] = dw[0][m];
  __syncthreads();
  for (int c = t; c < p.group; c += T) {
    float a = 0.f;
    for (int i = c >> 3; i < T; i += step) a += all[i * 8 + (c & 7)];
    out[c] = a;
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
