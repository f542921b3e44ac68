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
// or K).  A CTA is `groups` groups of `warps` warps; each group walks tokens of
// its own (group g of CTA c: c * groups + g, then steps of all groups of the
// grid) and shares with the others only the (cos, sin) tables and the weights.
// One thread of a group streams its tokens' rows of x and g into the group's ring
// of shared-memory stages with bulk copies, several tokens ahead.  A thread takes
// the 16-byte vectors lane, lane + 32 * warps, ... of a token (V of them), holds x
// and u in registers from the sums to the result, and meets the same channels in
// every token, so that it keeps its part of dw in float32 registers to the end.
// One barrier of the group per token: it publishes the warps' sums and the next
// token's (cos, sin) rows, and frees the stage, which every thread has read by
// then.  The CTA's part of dw goes to the workspace and a second kernel adds the
// CTAs' parts in a fixed order (no atomics: the same result on every run).
//
// Measured: 75,600 tokens x 5,120 channels, one group per token, Q and K: 912 to 972
// us (4.8 to 5.1 TB/s, 0.73 to 0.78 of the copy rate); 7,800 x 12 x 128 per head: 41 us.
// Bound by latency: a group has one token in flight, whose ten dependent shuffles,
// barrier and shared-memory round trip leave about half of the issue slots empty.  What
// had to be pared down before is instructions: a vector takes some 100 (half of them
// the formula's multiply-adds), and a warp some 150 more per token for the sums, the
// barrier and the loop, which is why a thread takes up to four vectors.
#pragma once

#include "patchify_rope.cuh"
#include "vdit_internal.h"

namespace vdit {

constexpr int kNormBwdVecs = 4;          // V at most
constexpr int kNormBwdWarps = 8;         // warps per token at most: 8,192 channels / 8 / 32 / V with V = 4
constexpr int kNormBwdGroups = 24;       // groups of a CTA at most
constexpr int kNormBwdMaxStages = 8;
constexpr int kNormBwdMaxCtas = 160;     // CTAs per tensor (rows of the workspace)
constexpr int kSiteNormBwdFull = 32, kSiteNormBwdDrain = 33;

// Threads of a CTA at most: one CTA takes an SM, and its registers with it.
constexpr int norm_bwd_threads(int V) { return V >= 3 ? 512 : (V == 2 ? 640 : 768); }

struct NormBwdParams {
  const __nv_bfloat16 *q, *k, *gq, *gk;
  __nv_bfloat16 *dq, *dk;
  const float *wq, *wk;
  float* parts;            // [2][kNormBwdMaxCtas][group], or null when no weight gradient is wanted
  int group, stages;
  int warps, groups;       // warps per token, tokens a CTA works on at a time
  float eps;
  double theta;
};

// What a group steps from token to token; in shared memory, since only a few of its
// threads use it and all of them would hold it in registers.
struct NormBwdGroup {
  const __nv_bfloat16 *x, *g;   // the rows to be copied next
  long long row_step;           // elements between the rows of two of its tokens
  int pos[2][3];                // grid position (t, h, w) of the next token, by parity
  int pos_step[3];
};

// kWide: the group is the token's whole heads*D vector; else a group is 1 .. 32
// neighbouring lanes of one vector each.
template <bool kWide, int V>
__global__ void __launch_bounds__(norm_bwd_threads(V), 1)
    bwd_qk_norm_rope3d_kernel(const NormBwdParams p, RopeShape s) {
  // [group][token parity][x^2, x u w][warp]: the warps' sums, zeros past them
  __shared__ __align__(16) float wsum[kNormBwdGroups][2][2][kNormBwdWarps];
  __shared__ double inv_freq[kRopeMaxPairs];
  __shared__ NormBwdGroup state[kNormBwdGroups];
  __shared__ __align__(8) uint64_t bars[kNormBwdGroups][kNormBwdMaxStages];
  let_next_start();
  if (__syncthreads_or(watchdog_tripped())) return;     // all threads of the CTA decide alike

  const int tensor = s.ntens == 2 ? (int)blockIdx.y : 1;
  const float* w = tensor ? p.wk : p.wq;

  const int T = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int G = p.groups, span = 32 * p.warps;          // threads of one group
  const int gi = warp / p.warps, li = t - gi * span;
  const int vph = s.D / 8, P = s.D / 2;                 // vectors and pairs per head
  const int nv = s.heads * vph;                         // vectors per token
  uint4* ring = reinterpret_cast<uint4*>(dyn_smem) + (size_t)gi * p.stages * 2 * nv;   // [stage][x row, g row]
  // each group's pairs, by token parity: [G][2][2][vph] float4, pairs 0 and 1 of
  // every vector, then pairs 2 and 3 (neighbouring lanes read neighbouring 16 bytes)
  float4* cs_all = reinterpret_cast<float4*>(dyn_smem) + (size_t)G * p.stages * 2 * nv;
  float4* cs = cs_all + gi * 4 * vph;
  // the weights (kWide: one thread's channels are too many for its registers)
  float4* wsm = cs_all + G * 4 * vph;
  // per-axis tables: time [Tg][d_t/2], then height [Hg][d_h/2], then width [Wg][d_w/2]
  float2* tab = reinterpret_cast<float2*>(wsm + (kWide ? nv * 2 : 0));
  uint64_t* full = bars[gi];
  const int pt = s.d_t / 2, ph = s.d_h / 2, pw = s.d_w / 2;
  const int Tg = (int)(s.L / ((long long)s.Hg * s.Wg));
  const int off_h = Tg * pt, off_w = off_h + s.Hg * ph, n_tab = off_w + s.Wg * pw;
  NormBwdGroup& mine = state[gi];
  // the group's tokens: first, first + step, ... (none, if there are more groups than tokens)
  const long long first = (long long)blockIdx.x * G + gi, step = (long long)gridDim.x * G;
  const int my = first < s.ntok ? (int)((s.ntok - 1 - first) / step + 1) : 0;   // below 2^31 (host)
  if (li == 0) {
    for (int st = 0; st < p.stages; ++st) mbar_init(&full[st], 1);
    fence_mbar_init();
    mine.x = (tensor ? p.k : p.q) + first * nv * 8;
    mine.g = (tensor ? p.gk : p.gq) + first * nv * 8;
    mine.row_step = step * nv * 8;
    const int hw = s.Hg * s.Wg, l = (int)(first % s.L), ls = (int)(step % s.L);
    mine.pos[0][0] = l / hw; mine.pos[0][1] = l % hw / s.Wg; mine.pos[0][2] = l % s.Wg;
    mine.pos_step[0] = ls / hw; mine.pos_step[1] = ls % hw / s.Wg; mine.pos_step[2] = ls % s.Wg;
  }
  for (int x = t; x < P; x += T) {
    int i, d;
    if (x < pt) { i = x; d = s.d_t; }
    else if (x < pt + ph) { i = x - pt; d = s.d_h; }
    else { i = x - pt - ph; d = s.d_w; }
    inv_freq[x] = 1.0 / pow(p.theta, (double)(2 * i) / (double)d);
  }
  for (int x = t; x < (int)(sizeof(wsum) / 4); x += T) (&wsum[0][0][0][0])[x] = 0.f;
  if (kWide)
    for (int x = t; x < nv * 2; x += T)
      wsm[x] = w != nullptr ? __ldg(reinterpret_cast<const float4*>(w) + x) : make_float4(1.f, 1.f, 1.f, 1.f);
  __syncthreads();

  auto issue = [&](int st) {                            // thread 0 of the group: its next token into a stage
    const uint32_t row_bytes = (uint32_t)nv * 16u;
    uint4* to = ring + (size_t)st * 2 * nv;
    mbar_arrive_expect_tx(&full[st], 2 * row_bytes);
    bulk_load(to, mine.x, row_bytes, &full[st]);
    bulk_load(to + nv, mine.g, row_bytes, &full[st]);
    mine.x += mine.row_step;
    mine.g += mine.row_step;
  };
  int issued = my < p.stages ? my : p.stages;
  if (li == 0)
    for (int k = 0; k < issued; ++k) issue(k);
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
  // The pairs of the group's next token, from the tables; its grid position is
  // stepped from token to token (thread 0 writes the one after next), so that
  // nothing is divided.
  auto pairs = [&](int parity) {
    float2* to = reinterpret_cast<float2*>(cs + parity * 2 * vph);
    for (int pi = li; pi < P; pi += span) {
      const int at = pi < pt        ? mine.pos[parity][0] * pt + pi
                     : pi < pt + ph ? off_h + mine.pos[parity][1] * ph + (pi - pt)
                                    : off_w + mine.pos[parity][2] * pw + (pi - pt - ph);
      to[(((pi >> 1) & 1) * vph + (pi >> 2)) * 2 + (pi & 1)] = tab[at];
    }
    if (li == 0) {
      int pos_t = mine.pos[parity][0] + mine.pos_step[0], pos_h = mine.pos[parity][1] + mine.pos_step[1],
          pos_w = mine.pos[parity][2] + mine.pos_step[2];
      if (pos_w >= s.Wg) { pos_w -= s.Wg; ++pos_h; }
      if (pos_h >= s.Hg) { pos_h -= s.Hg; ++pos_t; }
      if (pos_t >= Tg) pos_t -= Tg;
      mine.pos[parity ^ 1][0] = pos_t; mine.pos[parity ^ 1][1] = pos_h; mine.pos[parity ^ 1][2] = pos_w;
    }
  };
  pairs(0);

  constexpr int NW = kWide ? V : 1;                     // vectors of a thread with channels of their own
  const int gv = p.group / 8;                           // vectors per group of the norm
  const float inv_group = 1.f / (float)p.group;
  float dw[NW][8], wv[8];                               // wv: a per-head norm's weights, the same for all V vectors
#pragma unroll
  for (int r = 0; r < NW; ++r)
#pragma unroll
    for (int m = 0; m < 8; ++m) dw[r][m] = 0.f;
  if (!kWide) {
    const float* at = w + (li * 8) % p.group;
    const float4 a = w != nullptr ? __ldg(reinterpret_cast<const float4*>(at)) : make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 b = w != nullptr ? __ldg(reinterpret_cast<const float4*>(at + 4)) : a;
    wv[0] = a.x; wv[1] = a.y; wv[2] = a.z; wv[3] = a.w;
    wv[4] = b.x; wv[5] = b.y; wv[6] = b.z; wv[7] = b.w;
  }
  auto weights = [&](int r) {                           // vector r's weights
    if (kWide) {
      const float4 a = wsm[(li + span * r) * 2], b = wsm[(li + span * r) * 2 + 1];
      wv[0] = a.x; wv[1] = a.y; wv[2] = a.z; wv[3] = a.w;
      wv[4] = b.x; wv[5] = b.y; wv[6] = b.z; wv[7] = b.w;
    }
  };
  auto lo = [](uint32_t b) { return __uint_as_float(b << 16); };
  auto hi = [](uint32_t b) { return __uint_as_float(b & 0xffff0000u); };
  // where a vector lies in its head: the same for all V where 32 * warps is a
  // whole number of heads, and then its pairs are read once
  const bool same = span % vph == 0;
  const int vi0 = li % vph;
  uint4* dst = reinterpret_cast<uint4*>(tensor ? p.dk : p.dq) + first * nv + li;
  const int bar_id = 1 + (gi < 15 ? gi : 0);            // a hardware barrier per group; one-warp groups need none
  __syncthreads();                                      // pairs(0), the zeros

  int k = 0, st = 0, par = 0;                           // k mod stages, k mod 2
  uint32_t phase = 0;
  for (; k < my; ++k) {
    const bool okw = mbar_wait(&full[st], phase, kSiteNormBwdFull);
    const uint4* sx = ring + st * 2 * nv + li;
    const float4* c4 = cs + par * 2 * vph;
    uint4 x[V];
    float u[V][8];
    float sq[kWide ? 1 : V], dot[kWide ? 1 : V];        // sums of x^2 and of x u w
    float4 ca = make_float4(0.f, 0.f, 0.f, 0.f), cb = ca;
#pragma unroll
    for (int r = 0; r < V; ++r) {
      float a = 0.f, d = 0.f;
      if (li + span * r < nv && okw) {
        x[r] = sx[span * r];
        const uint4 g = sx[nv + span * r];
        if (r == 0 || !same) {
          const int vi = r == 0 ? vi0 : (li + span * r) % vph;
          ca = c4[vi];
          cb = c4[vph + vi];
        }
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
        weights(r);
        const uint32_t xs[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float x0 = lo(xs[m]), x1 = hi(xs[m]);
          a = fmaf(x0, x0, a);
          d = fmaf(x0, u[r][2 * m] * wv[2 * m], d);
          a = fmaf(x1, x1, a);
          d = fmaf(x1, u[r][2 * m + 1] * wv[2 * m + 1], d);
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
        wsum[gi][par][0][li >> 5] = sq[0];
        wsum[gi][par][1][li >> 5] = dot[0];
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
    // the stage is free; the sums and the next pairs are out
    bool all;
    if (p.warps == 1) {
      __syncwarp();
      all = __all_sync(0xffffffffu, okw);
    } else {
      all = named_bar_and(bar_id, span, okw);
    }
    if (!all) break;
    if (li == 0 && issued < my) issue(st);
    ++issued;
    if (kWide) {
      const float4* at = reinterpret_cast<const float4*>(wsum[gi][par][0]);
      const float4 a = at[0], b = at[1], c = at[2], d = at[3];
      sq[0] = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
      dot[0] = ((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w));
    }
    // dx = (u r) w - x r^3 mean(x u w); (u r) x is dw's term.  r^3 is never formed by
    // itself: it leaves float32 above r = 7e12 and below 1e-13, where r mean(x u w) is
    // of u's size and its products with r are not.  (r once more on the sum instead,
    // which would take r past 1e18 too, costs two multiplications a pair: 1 % at 75,600
    // tokens x 5,120.)
    float rr = 0.f, back = 0.f;
    auto factors = [&](float a, float d) {
      rr = rsqrtf(fmaf(a, inv_group, p.eps));
      back = -(rr * (rr * (d * inv_group))) * rr;
    };
    if (kWide) factors(sq[0], dot[0]);
#pragma unroll
    for (int r = 0; r < V; ++r) {
      if (li + span * r < nv) {
        if (!kWide) factors(sq[kWide ? 0 : r], dot[kWide ? 0 : r]);
        const uint32_t xs[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
        float* dwr = dw[kWide ? r : 0];
        weights(r);
        uint32_t o[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float x0 = lo(xs[m]), x1 = hi(xs[m]);
          const float u0 = u[r][2 * m] * rr, u1 = u[r][2 * m + 1] * rr;
          o[m] = pack_bf16x2(fmaf(u0, wv[2 * m], x0 * back), fmaf(u1, wv[2 * m + 1], x1 * back));
          dwr[2 * m] = fmaf(u0, x0, dwr[2 * m]);
          dwr[2 * m + 1] = fmaf(u1, x1, dwr[2 * m + 1]);
        }
        dst[span * r] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    dst += mine.row_step / 8;
    par ^= 1;
    if (++st == p.stages) { st = 0; phase ^= 1u; }
  }
  // No copy may still be landing in shared memory when the CTA exits (only
  // when a wait above ran out can tokens k .. issued-1 still be in flight).
  if (li == 0)
    for (int k2 = k; k2 < min(issued, my); ++k2)
      mbar_drain_site(&full[k2 % p.stages], (uint32_t)((k2 / p.stages) & 1), kSiteNormBwdDrain);
  if (!__syncthreads_and(k == my) || p.parts == nullptr) return;
  float* out = p.parts + ((long long)tensor * kNormBwdMaxCtas + blockIdx.x) * p.group;
  // threads t, t + every, t + 2 every, ... hold the same channels
  const int every = kWide ? span : gv;
  float* all = reinterpret_cast<float*>(dyn_smem);      // [T][8], over the rings
#pragma unroll
  for (int r = 0; r < NW; ++r) {
    if (r > 0) __syncthreads();
#pragma unroll
    for (int m = 0; m < 8; ++m) all[t * 8 + m] = dw[r][m];
    __syncthreads();
    for (int c = t; c < min(every * 8, p.group - r * span * 8); c += T) {
      float a = 0.f;
      for (int i = c >> 3; i < T; i += every) a += all[i * 8 + (c & 7)];
      out[r * span * 8 + c] = a;
    }
  }
}

// dw[c] = the CTAs' parts of channel c, added in a fixed order: a CTA takes 32
// channels of one tensor, its 32 warps the CTAs w, w + 32, ... (at most five loads
// each, all in flight at once).
__global__ void __launch_bounds__(1024) bwd_weights_qk_norm_rope3d_kernel(const float* parts, float* dwq, float* dwk,
                                                                          int group, int n_parts) {
  __shared__ float sum[32][33];
  wait_for_previous();
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
    v[i] = c < group && row < n_parts ? __ldcg(from + (long long)row * group + c) : 0.f;
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
