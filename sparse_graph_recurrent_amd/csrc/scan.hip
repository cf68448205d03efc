// scan.hip -- selective state space scan: forward, backward and single-token
// step.
//
//   dt_t = softplus(delta_t + bias)      a_t = exp(dt_t A)
//   h_t  = a_t h_{t-1} + dt_t B_t u_t    y_t = C_t . h_t + D u_t    out = y silu(z)
//
// Work split.  Four adjacent lanes (a quad) own one channel, each of them NL
// of its N states, and walk the steps in tiles of K.  The per-channel work of
// a step (loads, softplus, gate, store) is done by one lane of the quad: lane
// q takes step 4i + q of a tile and the quad reads dt and dt u of the others
// through DPP, so that work is not repeated four times.  What bounds the
// kernels is the vector ALU: per step and state an exponential, five multiply
// or add slots forward and about twice that backward, against 8 bytes per
// step and channel of 16-bit tensors.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ck.h"
#include "ck_internal.h"
#include "sequence.h"

namespace ckhip {
namespace {

constexpr int kScanThreads = 256;                // 4 waves
constexpr int kScanChan = kScanThreads / 4;      // channels per workgroup
constexpr int64_t kScanMaxN = 64;

// Steps per tile: a lane of the backward holds a_t and h_{t-1} of a whole
// tile in registers (2 K NL values).
constexpr int scan_tile(int NL) { return NL <= 4 ? 16 : 64 / NL; }

// Sizes that both directions share.
struct ScanDims {
  int64_t T, B, D, N, G;
  int NL, NP, K;    // states per lane, padded states (4 NL), steps per tile
  int64_t Dg, P;    // channels per group, workgroups per group
  int64_t tiles;    // tiles of the window
};

ScanDims scan_dims(const ck_scan_shape& s) {
  ScanDims d;
  d.T = s.T; d.B = s.B; d.D = s.D; d.N = s.N; d.G = s.G;
  d.NL = s.N <= 4 ? 1 : s.N <= 8 ? 2 : s.N <= 16 ? 4 : s.N <= 32 ? 8 : 16;
  d.NP = 4 * d.NL;
  d.K = scan_tile(d.NL);
  d.Dg = s.D / s.G;
  d.P = (d.Dg + kScanChan - 1) / kScanChan;
  d.tiles = (s.T + d.K - 1) / d.K;
  return d;
}

template <typename E>
struct ScanArgs {
  Seq<const E> u, delta, b, c, z;
  const float *a, *d, *delta_bias, *state0;
  const int32_t* lengths;
  int T, B, D, N, G, Dg, P;
  int softplus;
  // forward
  Seq<E> out;
  float* state;
  float* saved;
  // backward
  Seq<const E> go;
  const float* gstate;
  Seq<E> gu, gdelta, gz;
  float* gstate0;
  float *part_bc, *part_a;
};

// What a workgroup computes: channels [g Dg + blk 64, ...) of row b.
struct Place {
  int b, g, blk, len;
  int q;        // lane of the quad
  int d;        // channel (clamped to the group's last)
  bool active;  // the channel exists
};

template <typename E>
__device__ __forceinline__ Place scan_place(const ScanArgs<E>& s) {
  Place p;
  unsigned i = blockIdx.x;
  p.blk = i % s.P;
  i /= s.P;
  p.g = i % s.G;
  p.b = i / s.G;
  p.q = threadIdx.x & 3;
  const int dg = p.blk * kScanChan + (int)(threadIdx.x >> 2);
  p.active = dg < s.Dg;
  p.d = p.g * s.Dg + min(dg, s.Dg - 1);
  p.len = s.T;
  if (s.lengths) p.len = min(max(s.lengths[p.b], 0), s.T);
  return p;
}

// The lane's steps t0 + 4i + q of a tile; steps past `last` read step `last`
// (their values are replaced by 0 afterwards).
template <typename E, int KQ>
__device__ __forceinline__ void tile_load(E (&v)[KQ], const Seq<const E>& s, int b, int d, int q,
                                          int t0, int last) {
  const E* base = s.row(t0, b);
  const uint32_t st = (uint32_t)s.st * (uint32_t)sizeof(E), d0 = (uint32_t)d * (uint32_t)sizeof(E);
#pragma unroll
  for (int i = 0; i < KQ; ++i) {
    const uint32_t off = (uint32_t)min(4 * i + q, last - t0) * st + d0;
    v[i] = *reinterpret_cast<const E*>(reinterpret_cast<const char*>(base) + off);
  }
}

// Stages B_t and C_t of steps t0 .. t0 + K - 1 as fp32 [K][NP] (0 past `last`
// or N); a thread loads its element with tile_bc_load and writes it with
// tile_bc_store.
template <typename E, int K, int NP>
__device__ __forceinline__ void tile_bc_load(float& vb, float& vc, const ScanArgs<E>& s,
                                             const Place& p, int t0, int last) {
  const int t = t0 + (int)threadIdx.x / NP, n = (int)threadIdx.x % NP;
  if ((int)threadIdx.x >= K * NP) return;
  const int64_t at = (int64_t)p.g * s.N + min(n, s.N - 1);
  const float x = (float)s.b.row(min(t, last), p.b)[at], y = (float)s.c.row(min(t, last), p.b)[at];
  const bool in = t <= last && n < s.N;
  vb = in ? x : 0.0f;
  vc = in ? y : 0.0f;
}
template <int K, int NP>
__device__ __forceinline__ void tile_bc_store(float* sb, float* sc, float vb, float vc) {
  if ((int)threadIdx.x >= K * NP) return;
  sb[threadIdx.x] = vb;
  sc[threadIdx.x] = vc;
}

template <int NL>
__device__ __forceinline__ void lds_row(float (&v)[NL], const float* p) {
#pragma unroll
  for (int k = 0; k < NL; ++k) v[k] = p[k];
}

template <int NL>
__device__ __forceinline__ void load_a(float (&a)[NL], const float* A, int d, int q, int N) {
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    const int n = q * NL + k;
    a[k] = n < N ? A[(int64_t)d * N + n] : 0.0f;
  }
}

template <int NL>
__device__ __forceinline__ void load_state(float (&h)[NL], const float* s, int64_t row, int q,
                                           int N) {
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    const int n = q * NL + k;
    h[k] = s && n < N ? s[row * N + n] : 0.0f;
  }
}
template <int NL>
__device__ __forceinline__ void store_state(const float (&h)[NL], float* s, int64_t row, int q,
                                            int N) {
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    const int n = q * NL + k;
    if (n < N) s[row * N + n] = h[k];
  }
}

template <typename E>
__device__ __forceinline__ void zero_steps(const Seq<E>& s, const Place& p, int t0, int t1) {
  if (!p.active) return;
  for (int t = t0 + p.q; t < t1; t += 4) s.row(t, p.b)[p.d] = (E)0.0f;
}

template <typename E, int NL>
__global__ __launch_bounds__(kScanThreads) void scan_fwd(const ScanArgs<E> s) {
  constexpr int K = scan_tile(NL), KQ = K / 4, NP = 4 * NL;
  __shared__ float sb[2][K * NP], sc[2][K * NP];
  const Place p = scan_place(s);
  const int q = p.q;
  const int64_t row = (int64_t)p.b * s.D + p.d;
  float a2[NL], h[NL];
  load_a<NL>(a2, s.a, p.d, q, s.N);
#pragma unroll
  for (int k = 0; k < NL; ++k) a2[k] *= kLog2e;
  load_state<NL>(h, s.state0, row, q, s.N);
  const float bias = s.delta_bias ? s.delta_bias[p.d] : 0.0f;
  const float skip = s.d ? s.d[p.d] : 0.0f;
  const bool gate = s.z.p != nullptr;
  const int last = p.len - 1;

  E u[KQ], de[KQ], z[KQ];
  float vb = 0.0f, vc = 0.0f;
  if (p.len > 0) {
    tile_load(u, s.u, p.b, p.d, q, 0, last);
    tile_load(de, s.delta, p.b, p.d, q, 0, last);
    if (gate) tile_load(z, s.z, p.b, p.d, q, 0, last);
    tile_bc_load<E, K, NP>(vb, vc, s, p, 0, last);
  }
  int buf = 0;
  for (int t0 = 0; t0 < p.len; t0 += K, buf ^= 1) {
    tile_bc_store<K, NP>(sb[buf], sc[buf], vb, vc);
    float dt[KQ], x[KQ], uf[KQ], zf[KQ];
#pragma unroll
    for (int i = 0; i < KQ; ++i) {
      const bool in = t0 + 4 * i + q <= last;
      const float raw = (float)de[i] + bias;
      dt[i] = in ? (s.softplus ? softplus_hw(raw) : raw) : 0.0f;
      uf[i] = in ? (float)u[i] : 0.0f;
      x[i] = dt[i] * uf[i];
      zf[i] = gate ? (float)z[i] : 0.0f;
    }
    __syncthreads();
    if (t0 + K < p.len) {
      tile_load(u, s.u, p.b, p.d, q, t0 + K, last);
      tile_load(de, s.delta, p.b, p.d, q, t0 + K, last);
      if (gate) tile_load(z, s.z, p.b, p.d, q, t0 + K, last);
      tile_bc_load<E, K, NP>(vb, vc, s, p, t0 + K, last);
    }
    if (s.saved && p.active) {
      float* at = s.saved + (((int64_t)(t0 / K) * s.B + p.b) * s.D + p.d) * NP + q * NL;
#pragma unroll
      for (int k = 0; k < NL; ++k) at[k] = h[k];
    }
#pragma unroll
    for (int i = 0; i < KQ; ++i) {
      float acc[4];
      auto step = [&](auto jc) {
        constexpr int j = decltype(jc)::value;
        const float dj = quad_get<j>(dt[i]), xj = quad_get<j>(x[i]);
        float bb[NL], cc[NL];
        lds_row<NL>(bb, &sb[buf][(4 * i + j) * NP + q * NL]);
        lds_row<NL>(cc, &sc[buf][(4 * i + j) * NP + q * NL]);
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < NL; ++k) {
          h[k] = fmaf(exp2_hw(dj * a2[k]), h[k], xj * bb[k]);
          y = fmaf(cc[k], h[k], y);
        }
        acc[j] = y;
      };
      step(std::integral_constant<int, 0>());
      step(std::integral_constant<int, 1>());
      step(std::integral_constant<int, 2>());
      step(std::integral_constant<int, 3>());
      float y = fmaf(skip, uf[i], quad_reduce4(acc[0], acc[1], acc[2], acc[3], q));
      if (gate) y *= zf[i] * sigmoid_hw(zf[i]);
      const int t = t0 + 4 * i + q;
      if (p.active && t <= last) s.out.row(t, p.b)[p.d] = (E)y;
    }
  }
  zero_steps(s.out, p, p.len, s.T);
  if (s.state && p.active) store_state<NL>(h, s.state, row, q, s.N);
}

// x + y after the swap of their halves (rows): lanes of the lower half (even
// rows) get x summed over a pair of lanes 32 (16) apart, the others y.
__device__ __forceinline__ float swap32_add(float x, float y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x),
                                                  __builtin_bit_cast(unsigned, y), false, false);
  const unsigned lo = r[0], hi = r[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}
__device__ __forceinline__ float swap16_add(float x, float y) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x),
                                                  __builtin_bit_cast(unsigned, y), false, false);
  const unsigned lo = r[0], hi = r[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}

// Sums v[0..15] over the 16 channels of a wave: the lanes of channel slot s
// (lane >> 2) receive the total of v[s].  Halving exchanges: 15 adds and about
// as many moves, where 16 butterflies over 16 lanes would take 64 of each.
__device__ __forceinline__ float channel_reduce16(float (&v)[16], int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = swap32_add(v[i], v[i + 8]);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = swap16_add(v[i], v[i + 4]);
  const bool b3 = lane & 8, b2 = lane & 4;
  const float r0 = (b3 ? v[2] : v[0]) + dpp<0x128>(b3 ? v[0] : v[2]);  // row_ror:8
  const float r1 = (b3 ? v[3] : v[1]) + dpp<0x128>(b3 ? v[1] : v[3]);
  // exchange with lane ^ 4: reverse the quad, then mirror each half row
  const float x = dpp<0x141>(dpp<0x1B>(b2 ? r0 : r1));
  return (b2 ? r1 : r0) + x;
}

template <typename E, int NL>
__global__ __launch_bounds__(kScanThreads) void scan_bwd(const ScanArgs<E> s) {
  constexpr int K = scan_tile(NL), KQ = K / 4, NP = 4 * NL;
  __shared__ float sb[K * NP], sc[K * NP];
  __shared__ float red[4][K * 2 * NP];
  const Place p = scan_place(s);
  const int q = p.q, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)p.b * s.D + p.d;
  float a1[NL], ga[NL], g[NL];
  load_a<NL>(a1, s.a, p.d, q, s.N);
#pragma unroll
  for (int k = 0; k < NL; ++k) ga[k] = 0.0f;
  load_state<NL>(g, s.gstate, row, q, s.N);
  const float bias = s.delta_bias ? s.delta_bias[p.d] : 0.0f;
  const float skip = s.d ? s.d[p.d] : 0.0f;
  const bool gate = s.z.p != nullptr;
  const int last = p.len - 1;
  float gskip = 0.0f, gbias = 0.0f;
  // slot of channel_reduce16 this lane ends with: step tt of a flush, B or C, state k
  const int slot = lane >> 2;

  for (int tile = (p.len + K - 1) / K - 1; tile >= 0; --tile) {
    const int t0 = tile * K;
    E eu[KQ], ede[KQ], ez[KQ], ego[KQ];
    float vb = 0.0f, vc = 0.0f;
    tile_load(eu, s.u, p.b, p.d, q, t0, last);
    tile_load(ede, s.delta, p.b, p.d, q, t0, last);
    tile_load(ego, s.go, p.b, p.d, q, t0, last);
    if (gate) tile_load(ez, s.z, p.b, p.d, q, t0, last);
    tile_bc_load<E, K, NP>(vb, vc, s, p, t0, last);
    float h[NL];
    const float* at = s.saved + (((int64_t)tile * s.B + p.b) * s.D + p.d) * NP + q * NL;
#pragma unroll
    for (int k = 0; k < NL; ++k) h[k] = at[k];
    tile_bc_store<K, NP>(sb, sc, vb, vc);
    float dt[KQ], x[KQ], u[KQ], dy[KQ], raw[KQ], gzf[KQ];
#pragma unroll
    for (int i = 0; i < KQ; ++i) {
      const bool in = t0 + 4 * i + q <= last;
      raw[i] = (float)ede[i] + bias;
      dt[i] = in ? (s.softplus ? softplus_hw(raw[i]) : raw[i]) : 0.0f;
      u[i] = in ? (float)eu[i] : 0.0f;
      x[i] = dt[i] * u[i];
      dy[i] = in ? (float)ego[i] : 0.0f;
      gzf[i] = 0.0f;
      if (gate) {
        const float zf = (float)ez[i], sg = sigmoid_hw(zf);
        gzf[i] = dy[i] * (sg * fmaf(zf, 1.0f - sg, 1.0f));
        dy[i] = in ? dy[i] * (zf * sg) : 0.0f;
      }
    }
    __syncthreads();

    // the tile's states again, from its first
    float a[K][NL], hp[K][NL];
#pragma unroll
    for (int i = 0; i < KQ; ++i) {
      float acc[4];
      auto step = [&](auto jc) {
        constexpr int j = decltype(jc)::value;
        const int t = 4 * i + j;
        const float dj = quad_get<j>(dt[i]), xj = quad_get<j>(x[i]);
        float bb[NL], cc[NL];
        lds_row<NL>(bb, &sb[t * NP + q * NL]);
        lds_row<NL>(cc, &sc[t * NP + q * NL]);
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < NL; ++k) {
          a[t][k] = exp2_hw(dj * (kLog2e * a1[k]));
          hp[t][k] = h[k];
          h[k] = fmaf(a[t][k], h[k], xj * bb[k]);
          y = fmaf(cc[k], h[k], y);
        }
        acc[j] = y;
      };
      step(std::integral_constant<int, 0>());
      step(std::integral_constant<int, 1>());
      step(std::integral_constant<int, 2>());
      step(std::integral_constant<int, 3>());
      if (gate) {
        const float y = fmaf(skip, u[i], quad_reduce4(acc[0], acc[1], acc[2], acc[3], q));
        const int t = t0 + 4 * i + q;
        if (p.active && t <= last) s.gz.row(t, p.b)[p.d] = (E)(gzf[i] * y);
      }
    }

    // and backwards: g enters a step as a_{t+1} dL/dh_{t+1}
    float v[16];
#pragma unroll
    for (int i = KQ - 1; i >= 0; --i) {
      float sx[4], sa[4];
      auto step = [&](auto jc) {
        constexpr int j = decltype(jc)::value;
        const int t = 4 * i + j;
        const float dj = quad_get<j>(dt[i]), xj = quad_get<j>(x[i]), yj = quad_get<j>(dy[i]);
        float bb[NL], cc[NL];
        lds_row<NL>(bb, &sb[t * NP + q * NL]);
        lds_row<NL>(cc, &sc[t * NP + q * NL]);
        float s1 = 0.0f, s2 = 0.0f;
        [[maybe_unused]] float v2[16];
#pragma unroll
        for (int k = 0; k < NL; ++k) {
          const float gh = fmaf(cc[k], yj, g[k]);
          const float ht = t + 1 < K ? hp[t + 1 < K ? t + 1 : t][k] : h[k];
          // inactive lanes repeat the group's last channel: they add nothing
          const float vgb = p.active ? gh * xj : 0.0f, vgc = p.active ? ht * yj : 0.0f;
          if constexpr (NL <= 8) {
            const int tt = t % (8 / NL);
            v[tt * 2 * NL + k] = vgb;
            v[tt * 2 * NL + NL + k] = vgc;
          } else {
            v[k] = vgb;
            v2[k] = vgc;
          }
          s1 = fmaf(gh, bb[k], s1);
          g[k] = a[t][k] * gh;
          const float w = g[k] * hp[t][k];
          ga[k] = fmaf(w, dj, ga[k]);
          s2 = fmaf(w, a1[k], s2);
        }
        sx[j] = s1;
        sa[j] = s2;
        if constexpr (NL <= 8) {
          if (t % (8 / NL) == 0) {
            const float r = channel_reduce16(v, lane);
            const int tt = slot / (2 * NL), kind = slot / NL % 2, k = slot % NL;
            red[wave][((t + tt) * 2 + kind) * NP + q * NL + k] = r;
          }
        } else {
          red[wave][(t * 2) * NP + q * NL + slot] = channel_reduce16(v, lane);
          red[wave][(t * 2 + 1) * NP + q * NL + slot] = channel_reduce16(v2, lane);
        }
      };
      step(std::integral_constant<int, 3>());
      step(std::integral_constant<int, 2>());
      step(std::integral_constant<int, 1>());
      step(std::integral_constant<int, 0>());
      const float gx = quad_reduce4(sx[0], sx[1], sx[2], sx[3], q);  // dL/d(dt u)
      const float gl = quad_reduce4(sa[0], sa[1], sa[2], sa[3], q);  // sum_n dL/d(dt A) A
      const int t = t0 + 4 * i + q;
      const bool in = t <= last;
      float gdt = fmaf(u[i], gx, gl);
      if (s.softplus) gdt *= sigmoid_hw(raw[i]);
      gdt = in ? gdt : 0.0f;
      gbias += gdt;
      gskip = fmaf(dy[i], u[i], gskip);
      if (p.active && in) {
        s.gu.row(t, p.b)[p.d] = (E)fmaf(dt[i], gx, skip * dy[i]);
        s.gdelta.row(t, p.b)[p.d] = (E)gdt;
      }
    }
    __syncthreads();
    // the four waves' sums over their channels
    for (int e = threadIdx.x; e < K * 2 * NP; e += kScanThreads) {
      const int t = t0 + e / (2 * NP);
      if (t <= last)
        s.part_bc[((((int64_t)p.blk * s.T + t) * s.B + p.b) * s.G + p.g) * (2 * NP) +
                  e % (2 * NP)] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
    }
  }
  zero_steps(s.gu, p, p.len, s.T);
  zero_steps(s.gdelta, p, p.len, s.T);
  if (gate) zero_steps(s.gz, p, p.len, s.T);
  if (!p.active) return;
  if (s.gstate0) store_state<NL>(g, s.gstate0, row, q, s.N);
  float* pa = s.part_a + row * (NP + 2);
#pragma unroll
  for (int k = 0; k < NL; ++k) pa[q * NL + k] = ga[k];
  gskip = quad_sum(gskip);
  gbias = quad_sum(gbias);
  if (q == 0) {
    pa[NP] = gskip;
    pa[NP + 1] = gbias;
  }
}

// Gradients of B and C: the workgroups' partial sums of a group, in order.
template <typename E>
__global__ __launch_bounds__(256) void scan_sum_bc(const float* part, int T, int B, int G, int N,
                                                   int NP, int P, const int32_t* lengths,
                                                   Seq<E> gb, Seq<E> gc) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t rows = (int64_t)T * B * G, stride = rows * 2 * NP;
  if (i >= stride) return;
  const int e = (int)(i % (2 * NP)), kind = e / NP, n = e % NP;
  int64_t r = i / (2 * NP);
  const int g = (int)(r % G);
  r /= G;
  const int b = (int)(r % B), t = (int)(r / B);
  if (n >= N) return;
  float sum = 0.0f;
  if (!lengths || t < lengths[b])
    for (int k = 0; k < P; ++k) sum += part[k * stride + i];
  (kind ? gc : gb).row(t, b)[(int64_t)g * N + n] = (E)sum;
}

// Gradients of A, D and the bias: the rows' sums, in order.
__global__ __launch_bounds__(256) void scan_sum_a(const float* part, int64_t D, int N, int NP,
                                                  int rows, float* ga, float* gd, float* gbias) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= D * (NP + 2)) return;
  const int n = (int)(i % (NP + 2));
  const int64_t d = i / (NP + 2);
  float* out = n < N ? ga + d * N + n : n < NP ? nullptr : n == NP ? gd : gbias;
  if (!out) return;
  if (n >= NP) out += d;
  float sum = 0.0f;
  for (int r = 0; r < rows; ++r) sum += part[r * D * (NP + 2) + i];
  *out = sum;
}

template <typename E, int NL>
__global__ __launch_bounds__(kScanThreads) void scan_one(const ScanArgs<E> s) {
  const Place p = scan_place(s);
  if (!p.active) return;  // whole quads
  const int64_t row = (int64_t)p.b * s.D + p.d;
  float a[NL], h[NL];
  load_a<NL>(a, s.a, p.d, p.q, s.N);
  load_state<NL>(h, s.state0, row, p.q, s.N);
  const float raw = (float)s.delta.row(0, p.b)[p.d] + (s.delta_bias ? s.delta_bias[p.d] : 0.0f);
  const float dt = s.softplus ? softplus_hw(raw) : raw;
  const float u = (float)s.u.row(0, p.b)[p.d], x = dt * u;
  const E *pb = s.b.row(0, p.b) + (int64_t)p.g * s.N, *pc = s.c.row(0, p.b) + (int64_t)p.g * s.N;
  float y = 0.0f;
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    const int n = p.q * NL + k;
    if (n < s.N) {
      h[k] = fmaf(exp2_hw(dt * (kLog2e * a[k])), h[k], x * (float)pb[n]);
      y = fmaf((float)pc[n], h[k], y);
    }
  }
  y = quad_sum(y);
  if (s.d) y = fmaf(s.d[p.d], u, y);
  if (s.z.p) {
    const float zf = (float)s.z.row(0, p.b)[p.d];
    y *= zf * sigmoid_hw(zf);
  }
  if (p.q == 0) s.out.row(0, p.b)[p.d] = (E)y;
  store_state<NL>(h, s.state, row, p.q, s.N);
}

// Workspace byte offsets of a backward.
struct ScanWs {
  size_t part_bc, part_a, total;
};
ScanWs scan_bwd_ws(const ScanDims& d) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  ScanWs w;
  w.part_bc = 0;
  w.part_a = up((size_t)(d.P * d.T * d.B * d.G) * 2 * d.NP * 4);
  w.total = w.part_a + up((size_t)(d.B * d.D) * (d.NP + 2) * 4);
  return w;
}
size_t scan_saved(const ScanDims& d) { return (size_t)(d.tiles * d.B * d.D) * d.NP * 4; }

ck_status scan_check_shape(const ck_scan_shape* s) {
  if (!s) {
    set_error("shape is NULL");
    return CK_ERR_NULL_ARG;
  }
  const ck_status rc = seq_check_shape(s->T, s->B, s->D, s->dtype);
  if (rc != CK_OK) return rc;
  if (s->N < 1 || s->N > kScanMaxN || s->G < 1 || s->G > s->D || s->D % s->G != 0) {
    set_error("N must be in [1, 64] and G must divide D (N=%lld G=%lld D=%lld)", (long long)s->N,
              (long long)s->G, (long long)s->D);
    return CK_ERR_BAD_SIZE;
  }
  const ScanDims d = scan_dims(*s);
  if (d.P * d.G * d.B >= INT_MAX || d.D * d.NP >= INT_MAX ||
      (d.T > 0 && d.B * d.G * d.NP >= (int64_t(1) << 36) / d.T)) {
    set_error("B=%lld, D=%lld or T=%lld is too large", (long long)d.B, (long long)d.D,
              (long long)d.T);
    return CK_ERR_TOO_LARGE;
  }
  return CK_OK;
}

ck_status scan_check_inputs(const ck_scan_shape& s, const ck_scan_inputs* in) {
  if (!in || !in->a) {
    set_error("inputs or A is NULL");
    return CK_ERR_NULL_ARG;
  }
  const bool none = s.T == 0;
  ck_status rc = seq_check(in->u, s.dtype, none, "u");
  if (rc == CK_OK) rc = seq_check(in->delta, s.dtype, none, "delta");
  if (rc == CK_OK) rc = seq_check(in->b, s.dtype, none, "B");
  if (rc == CK_OK) rc = seq_check(in->c, s.dtype, none, "C");
  if (rc == CK_OK) rc = seq_check(in->z, s.dtype, true, "z");
  return rc;
}

template <typename E>
ScanArgs<E> scan_args(const ck_scan_shape& s, const ScanDims& d, const ck_scan_inputs& in) {
  ScanArgs<E> a = {};
  a.u = seq_of<const E>(in.u);
  a.delta = seq_of<const E>(in.delta);
  a.b = seq_of<const E>(in.b);
  a.c = seq_of<const E>(in.c);
  a.z = seq_of<const E>(in.z);
  a.a = in.a;
  a.d = in.d;
  a.delta_bias = in.delta_bias;
  a.state0 = in.state0;
  a.lengths = in.lengths;
  a.T = (int)d.T; a.B = (int)d.B; a.D = (int)d.D; a.N = (int)d.N; a.G = (int)d.G;
  a.Dg = (int)d.Dg; a.P = (int)d.P;
  a.softplus = s.delta_softplus;
  return a;
}

template <typename F>
void scan_by_states(int NL, F&& fn) {
  switch (NL) {
    case 1: fn(std::integral_constant<int, 1>()); break;
    case 2: fn(std::integral_constant<int, 2>()); break;
    case 4: fn(std::integral_constant<int, 4>()); break;
    case 8: fn(std::integral_constant<int, 8>()); break;
    default: fn(std::integral_constant<int, 16>()); break;
  }
}

}  // namespace
}  // namespace ckhip

using namespace ckhip;

extern "C" ck_status ck_scan_sizes(const ck_scan_shape* shape, size_t* saved_bytes,
                                   size_t* forward_bytes, size_t* backward_bytes) {
  clear_error();
  const ck_status rc = scan_check_shape(shape);
  if (rc != CK_OK) return rc;
  const ScanDims d = scan_dims(*shape);
  if (saved_bytes) *saved_bytes = scan_saved(d);
  if (forward_bytes) *forward_bytes = 0;
  if (backward_bytes) *backward_bytes = scan_bwd_ws(d).total;
  return CK_OK;
}

extern "C" ck_status ck_scan_forward(const ck_scan_shape* shape, const ck_scan_inputs* in,
                                     ck_seq out, float* state, void* saved, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  ck_status rc = scan_check_shape(shape);
  if (rc == CK_OK) rc = scan_check_inputs(*shape, in);
  if (rc == CK_OK) rc = seq_check(out, shape->dtype, shape->T == 0, "out");
  if (rc != CK_OK) return rc;
  const ScanDims d = scan_dims(*shape);
  rc = seq_check_ws(workspace, workspace_bytes, 0);
  if (rc == CK_OK && saved) rc = check_aligned(saved, "saved");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    ScanArgs<E> a = scan_args<E>(*shape, d, *in);
    a.out = seq_of<E>(out);
    a.state = state;
    a.saved = static_cast<float*>(saved);
    scan_by_states(d.NL, [&](auto nl) {
      scan_fwd<E, decltype(nl)::value>
          <<<(unsigned)(d.P * d.G * d.B), kScanThreads, 0, stream>>>(a);
    });
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}

extern "C" ck_status ck_scan_backward(const ck_scan_shape* shape, const ck_scan_inputs* in,
                                      const void* saved, ck_seq grad_out, const float* grad_state,
                                      const ck_scan_grads* grads, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  ck_status rc = scan_check_shape(shape);
  if (rc == CK_OK) rc = scan_check_inputs(*shape, in);
  if (rc != CK_OK) return rc;
  const bool none = shape->T == 0;
  if (!grads || !grads->a || (!saved && !none)) {
    set_error("grads, the gradient of A or saved is NULL");
    return CK_ERR_NULL_ARG;
  }
  rc = seq_check(grad_out, shape->dtype, none, "grad_out");
  if (rc == CK_OK) rc = seq_check(grads->u, shape->dtype, none, "the gradient of u");
  if (rc == CK_OK) rc = seq_check(grads->delta, shape->dtype, none, "the gradient of delta");
  if (rc == CK_OK) rc = seq_check(grads->b, shape->dtype, none, "the gradient of B");
  if (rc == CK_OK) rc = seq_check(grads->c, shape->dtype, none, "the gradient of C");
  if (rc == CK_OK)
    rc = seq_check(grads->z, shape->dtype, none || !in->z.data, "the gradient of z");
  if (rc != CK_OK) return rc;
  const ScanDims d = scan_dims(*shape);
  const ScanWs ws = scan_bwd_ws(d);
  rc = seq_check_ws(workspace, workspace_bytes, ws.total);
  if (rc == CK_OK && saved) rc = check_aligned(saved, "saved");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    ScanArgs<E> a = scan_args<E>(*shape, d, *in);
    a.saved = static_cast<float*>(const_cast<void*>(saved));
    a.go = seq_of<const E>(grad_out);
    a.gstate = grad_state;
    a.gu = seq_of<E>(grads->u);
    a.gdelta = seq_of<E>(grads->delta);
    a.gz = seq_of<E>(grads->z);
    a.gstate0 = grads->state0;
    a.part_bc = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.part_bc);
    a.part_a = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.part_a);
    scan_by_states(d.NL, [&](auto nl) {
      scan_bwd<E, decltype(nl)::value>
          <<<(unsigned)(d.P * d.G * d.B), kScanThreads, 0, stream>>>(a);
    });
    CK_HIP_TRY(hipGetLastError());
    const int64_t bc = d.T * d.B * d.G * 2 * d.NP, ae = d.D * (d.NP + 2);
    if (bc > 0)
      scan_sum_bc<E><<<(unsigned)((bc + 255) / 256), 256, 0, stream>>>(
          a.part_bc, a.T, a.B, a.G, a.N, d.NP, a.P, a.lengths, seq_of<E>(grads->b),
          seq_of<E>(grads->c));
    scan_sum_a<<<(unsigned)((ae + 255) / 256), 256, 0, stream>>>(
        a.part_a, d.D, a.N, d.NP, a.B, grads->a, grads->d, grads->delta_bias);
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}

extern "C" ck_status ck_scan_step(const ck_scan_shape* shape, const ck_scan_inputs* in, ck_seq out,
                                  float* state, hipStream_t stream) {
  clear_error();
  ck_status rc = scan_check_shape(shape);
  if (rc != CK_OK) return rc;
  if (shape->T != 1) {
    set_error("a step takes T = 1 (got %lld)", (long long)shape->T);
    return CK_ERR_BAD_SIZE;
  }
  rc = scan_check_inputs(*shape, in);
  if (rc == CK_OK) rc = seq_check(out, shape->dtype, false, "out");
  if (rc != CK_OK) return rc;
  if (!state || in->lengths) {
    set_error(state ? "a step takes no lengths" : "state is NULL");
    return state ? CK_ERR_BAD_VALUE : CK_ERR_NULL_ARG;
  }
  const ScanDims d = scan_dims(*shape);
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    ScanArgs<E> a = scan_args<E>(*shape, d, *in);
    a.out = seq_of<E>(out);
    a.state = state;
    scan_by_states(d.NL, [&](auto nl) {
      scan_one<E, decltype(nl)::value>
          <<<(unsigned)(d.P * d.G * d.B), kScanThreads, 0, stream>>>(a);
    });
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}
