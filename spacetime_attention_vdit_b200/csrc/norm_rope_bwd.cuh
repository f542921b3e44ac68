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

constexpr int kNormBwdThreads = 256;     // at most: warps * groups * 32
constexpr int kNormBwdSumRow = 8;        // a token's warps at most: 8,192 / 8 / 32 / V with V = 4
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
// neighbouring lanes of one vector each.  kThreads: the CTA's threads at most,
// which sets the registers a thread may have (kThreads * registers: half of an
// SM's, except for the widest tokens).
template <bool kWide, int V, int kThreads>
__global__ void __launch_bounds__(kThreads, V == 4 && kThreads > 160 ? 1 : 2)
    bwd_qk_norm_rope3d_kernel(const NormBwdParams p, RopeShape s) {
  // [chunk parity][token of the chunk][x^2, x u w][warp]: the warps' sums, zeros past them
  __shared__ __align__(16) float wsum[2][kNormBwdThreads / 32][2][kNormBwdSumRow];
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
  const long long n_my = (n_chunks - 1 - blockIdx.x) / gridDim.x + 1;   // grid <= n_chunks; below 2^31 (host)
  auto issue = [&](long long k, int st) {               // thread 0: chunk k of this CTA into stage st = k mod stages
    const long long tok = (blockIdx.x + k * gridDim.x) * G;
    const uint32_t bytes = (uint32_t)min((long long)G, s.ntok - tok) * row_bytes;
    uint4* to = ring + (size_t)st * 2 * G * nv;
    mbar_arrive_expect_tx(&full[st], 2 * bytes);
    bulk_load(to, x_in + tok * nv * 8, bytes, &full[st]);
    bulk_load(to + (size_t)G * nv, g_in + tok * nv * 8, bytes, &full[st]);
  };
  long long issued = n_my < p.stages ? n_my : p.stages;
  if (t == 0)
    for (int k = 0; k < (int)issued; ++k) issue(k, k);
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
  // the pairs of a chunk's tokens, from the axis tables: thread x < G * P takes
  // pair x % P of token x / P (P <= 128 and G <= 8 fit in the CTA four times), at
  // positions that are stepped from chunk to chunk without a 64-bit division
  const unsigned L = (unsigned)s.L, hw = (unsigned)(s.Hg * s.Wg), Wg = (unsigned)s.Wg;
  unsigned l0 = (unsigned)((unsigned long long)blockIdx.x * G % L);          // the chunk's first token in its clip
  const unsigned l_step = (unsigned)((unsigned long long)gridDim.x * G % L);
  auto pairs = [&](int parity) {
    float2* to = reinterpret_cast<float2*>(cs + parity * 2 * G * vph);
    for (int x = t; x < G * P; x += T) {
      const int j = x / P, pi = x - j * P;
      const unsigned l = (l0 + j) % L;                   // rows past the last token are filled too, and not read
      int at;
      if (pi < pt) {
        at = (int)(l / hw) * pt + pi;
      } else {
        const unsigned r = l % hw, y = r / Wg;
        at = pi < pt + ph ? off_h + (int)y * ph + (pi - pt) : off_w + (int)(r - y * Wg) * pw + (pi - pt - ph);
      }
      to[((j * 2 + ((pi >> 1) & 1)) * vph + (pi >> 2)) * 2 + (pi & 1)] = tab[at];
    }
    l0 += l_step;
    if (l0 >= L) l0 -= L;
  };
  pairs(0);

  for (int x = t; x < (int)(sizeof(wsum) / 4); x += T) (&wsum[0][0][0][0])[x] = 0.f;

  constexpr int NW = kWide ? V : 1;                     // vectors of a thread with channels of their own
  const int gv = p.group / 8;                           // vectors per group
  const float inv_group = 1.f / (float)p.group;
  float dw[NW][8], wv[NW][8];
#pragma unroll
  for (int r = 0; r < NW; ++r) {
    const int e = li + span * r;
    const bool have = w != nullptr && e < nv;
    const float* at = w + (e * 8) % p.group;
    const float4 a = have ? __ldg(reinterpret_cast<const float4*>(at)) : make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 b = have ? __ldg(reinterpret_cast<const float4*>(at + 4)) : a;
    wv[r][0] = a.x; wv[r][1] = a.y; wv[r][2] = a.z; wv[r][3] = a.w;
    wv[r][4] = b.x; wv[r][5] = b.y; wv[r][6] = b.z; wv[r][7] = b.w;
#pragma unroll
    for (int m = 0; m < 8; ++m) dw[r][m] = 0.f;
  }
  auto lo = [](uint32_t b) { return __uint_as_float(b << 16); };
  auto hi = [](uint32_t b) { return __uint_as_float(b & 0xffff0000u); };
  // What a thread reads and writes steps from chunk to chunk by constants.  Only
  // the last chunk can have fewer than G tokens, and only a CTA's last vectors can
  // lie past the token.
  bool in[V];
  int cs_at[V];
#pragma unroll
  for (int r = 0; r < V; ++r) {
    const int e = li + span * r;
    in[r] = gi < G && e < nv;
    cs_at[r] = gi * 2 * vph + e % vph;
  }
  const bool last_live = (blockIdx.x + (n_my - 1) * gridDim.x) * G + gi < s.ntok;
  uint4* dst = reinterpret_cast<uint4*>(d_out) + ((long long)blockIdx.x * G + gi) * nv + li;
  const long long dst_step = (long long)gridDim.x * G * nv;
  const int sg_off = G * nv, stage_vecs = 2 * G * nv, cs_step = 2 * G * vph;
  const uint4* sx = ring + gi * nv + li;
  const int my = (int)n_my;
  __syncthreads();                                      // pairs(0), the zeros

  int k = 0, st = 0, par = 0;                           // k mod stages, k mod 2
  uint32_t phase = 0;
  for (; k < my; ++k) {
    const bool live = k + 1 < my || last_live;
    const bool okw = mbar_wait(&full[st], phase, kSiteNormBwdFull);
    const float4* c4 = cs + par * cs_step;
    uint4 x[V];
    float u[V][8];
    float sq[kWide ? 1 : V], dot[kWide ? 1 : V];        // sums of x^2 and of x u w
#pragma unroll
    for (int r = 0; r < V; ++r) {
      float a = 0.f, d = 0.f;
      if (in[r] && live && okw) {
        x[r] = sx[st * stage_vecs + span * r];
        const uint4 g = sx[st * stage_vecs + sg_off + span * r];
        const float4 ca = c4[cs_at[r]], cb = c4[cs_at[r] + vph];
        // u = R^T g: (g0, g1) -> (g0 cos + g1 sin, g1 cos - g0 sin)
        auto back = [&](uint32_t b, float c, float sn, float& u0, float& u1) {
          const float g0 = lo(b), g1 = hi(b);
          u0 = fmaf(g0, c, g1 * sn);
          u1 = fmaf(g1, c, -(g0 * sn));
        };
        back(g.x, ca.x, ca.y, u[r][0], u[r][1]);
        back(g.y, ca.z, ca.w, u[r][2], u[r][3]);
        back(g.z, cb.x, cb.y, u[r][4], u[r][5]);
        back(g.w, cb.z, cb.w, u[r][6], u[r][7]);
        const uint32_t xs[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float x0 = lo(xs[m]), x1 = hi(xs[m]);
          const float* wr = wv[kWide ? r : 0];
          a = fmaf(x0, x0, a);
          d = fmaf(x0, u[r][2 * m] * wr[2 * m], d);
          a = fmaf(x1, x1, a);
          d = fmaf(x1, u[r][2 * m + 1] * wr[2 * m + 1], d);
        }
      }
      if (kWide && r > 0) {
        sq[0] += a;
        dot[0] += d;
      } else {
        sq[kWide ? 0 : r] = a;
        dot[kWide ? 0 : r] = d;
      }
    }
    if (kWide) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        sq[0] += __shfl_xor_sync(0xffffffffu, sq[0], o);
        dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], o);
      }
      if (lane == 0) {
        wsum[par][gi][0][warp - gi * p.warps] = sq[0];
        wsum[par][gi][1][warp - gi * p.warps] = dot[0];
      }
    } else {
      for (int o = gv >> 1; o >= 1; o >>= 1) {
#pragma unroll
        for (int r = 0; r < V; ++r) {
          sq[kWide ? 0 : r] += __shfl_xor_sync(0xffffffffu, sq[kWide ? 0 : r], o);
          dot[kWide ? 0 : r] += __shfl_xor_sync(0xffffffffu, dot[kWide ? 0 : r], o);
        }
      }
    }
    if (k + 1 < my) pairs(par ^ 1);
    if (!__syncthreads_and(okw)) break;                 // the stage is free; the sums and the next pairs are out
    if (t == 0 && issued < my) issue(issued++, st);
    if (kWide) {
      float* both[2] = {&sq[0], &dot[0]};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4* at = reinterpret_cast<const float4*>(wsum[par][gi][i]);
        const float4 a = at[0], b = at[1];
        *both[i] = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
      }
    }
#pragma unroll
    for (int r = 0; r < V; ++r) {
      if (in[r] && live) {
        const float rr = rsqrtf(fmaf(sq[kWide ? 0 : r], inv_group, p.eps));
        const float back = -(rr * rr) * (dot[kWide ? 0 : r] * inv_group);   // dx = rr (u w + x back)
        const uint32_t xs[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
        const float* wr = wv[kWide ? r : 0];
        float* dwr = dw[kWide ? r : 0];
        uint32_t o[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float x0 = lo(xs[m]), x1 = hi(xs[m]);
          const float u0 = u[r][2 * m], u1 = u[r][2 * m + 1];
          o[m] = pack_bf16x2(rr * fmaf(x0, back, u0 * wr[2 * m]), rr * fmaf(x1, back, u1 * wr[2 * m + 1]));
          dwr[2 * m] = fmaf(u0, x0 * rr, dwr[2 * m]);
          dwr[2 * m + 1] = fmaf(u1, x1 * rr, dwr[2 * m + 1]);
        }
        dst[span * r] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    dst += dst_step;
    par ^= 1;
    if (++st == p.stages) { st = 0; phase ^= 1u; }
  }
  const bool whole = k == my;
  // No copy may still be landing in shared memory when the CTA exits (only
  // when a wait above ran out can chunks k .. issued-1 still be in flight).
  if (t == 0)
    for (long long k2 = k; k2 < issued; ++k2)
      mbar_drain_site(&full[k2 % p.stages], (uint32_t)((k2 / p.stages) & 1), kSiteNormBwdDrain);
  if (p.parts == nullptr || !whole) return;
  float* out = p.parts + ((long long)tensor * kNormBwdMaxCtas + blockIdx.x) * p.group;
  // threads t, t + step, t + 2 step, ... hold the same channels
  const int step = kWide ? span : gv;
  float* all = reinterpret_cast<float*>(dyn_smem);      // [T][8], over the ring
#pragma unroll
  for (int r = 0; r < NW; ++r) {
    if (r > 0) __syncthreads();
#pragma unroll
    for (int m = 0; m < 8; ++m) all[t * 8 + m] = dw[r][m];
    __syncthreads();
    for (int c = t; c < min(step * 8, p.group - r * span * 8); c += T) {
      float a = 0.f;
      for (int i = c >> 3; i < T; i += step) a += all[i * 8 + (c & 7)];
      out[r * span * 8 + c] = a;
    }
  }
}

// dw[c] = the CTAs' parts of channel c, added in a fixed order: a CTA takes 32
// channels of one tensor, its 32 warps the CTAs w, w + 32, ... (at most ten loads
// each, all in flight at once).
__global__ void __launch_bounds__(1024) bwd_weights_qk_norm_rope3d_kernel(const float* __restrict__ parts, float* dwq,
                                                                          float* dwk, int group, int n_parts) {
  __shared__ float sum[32][33];
  if (watchdog_tripped()) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* dw = blockIdx.y ? dwk : dwq;
  if (dw == nullptr) return;
  const float* from = parts + (long long)blockIdx.y * kNormBwdMaxCtas * group;
  const int c = blockIdx.x * 32 + lane;
  constexpr int kEach = kNormBwdMaxCtas / 32;
  float v[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int row = warp + 32 * i;
    v[i] = c < group && row < n_parts ? __ldg(from + (long long)row * group + c) : 0.f;
  }
  float a = v[0];
#pragma unroll
  for (int i = 1; i < kEach; ++i) a += v[i];
  sum[warp][lane] = a;
  __syncthreads();
  // warp w adds channel w's 32 parts
  float b = sum[lane][warp];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
  const int ch = blockIdx.x * 32 + warp;
  if (lane == 0 && ch < group) dw[ch] = b;
}

}  // namespace vdit
