// scan_backward.hip -- gradients of the selective scan (see scan.h).
//
//   gh_t = C_t gy_t + a_{t+1} gh_{t+1}          gy = go silu(z)
//   gC_t = sum_d gy_t h_t                       gB_t = sum_d gh_t dt_t u_t
//   gA   = sum gh_t dt_t a_t h_{t-1}            g(dt_t u_t) = sum_n gh_t B_t
//   gdt_t = sum_n gh_t a_t h_{t-1} A + u_t g(dt_t u_t)
//
// Tiles are walked from the last: the forward left the state at each tile's
// start, from which the tile's states are computed again into registers (a
// step back through h_{t-1} = (h_t - x) / a_t would lose everything where a_t
// is small), then the adjoint runs down through them.  As the forward, it is
// bound by the vector ALU.  The sums over channels of gB and gC cost most of
// the rest: 16 values are summed over a wave's 16 channels by halving
// exchanges, the four waves' sums are added in LDS and the workgroups' by a
// last launch, all in a fixed order.
#include "scan.h"

#include <type_traits>

namespace ckhip {
namespace {

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

// The adjoint's share of a chunk: what it hands to the chunk before, given
// nothing from the one behind, and the sum of the chunk's dt.
template <typename E, int NL, bool GATE>
__global__ __launch_bounds__(kScanThreads, 2) void scan_bwd_part(const ScanArgs<E> s) {
  constexpr int K = scan_tile(NL), KQ = K / 4, NP = 4 * NL;
  __shared__ float sb[2][K * NP], sc[2][K * NP];
  Place p = scan_place(s);
  // chunk 0 hands nothing on: the grid covers chunks 1 ..
  p.chunk += 1;
  p.t0 += s.chunk_steps;
  p.t1 = min(p.t0 + s.chunk_steps, s.T);
  p.te = min(p.t1, p.len);
  const int q = p.q;
  const int64_t row = (int64_t)p.b * s.D + p.d;
  float a2[NL], g[NL];
  load_a<NL>(a2, s.a, p.d, q, s.N);
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    a2[k] *= kLog2e;
    g[k] = 0.0f;
  }
  const float bias = s.delta_bias ? s.delta_bias[p.d] : 0.0f;
  float dtsum = 0.0f;
  if (p.t0 < p.te) {
    const int tl = p.t0 + (p.te - 1 - p.t0) / K * K;
    Walk<const E> wd(s.delta, tl, p.b, q, p.d), wg(s.go, tl, p.b, q, p.d);
    Walk<const E> wz(GATE ? s.z : s.go, tl, p.b, q, p.d);
    TileBC<E, K, NP> bc(s, p, tl);
    E de[KQ], go[KQ], z[KQ];
    auto fetch = [&](int last) {
      const uint32_t ld = walk_limit(wd, q, last), lg = walk_limit(wg, q, last);
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        de[i] = wd.load(4 * i, ld);
        go[i] = wg.load(4 * i, lg);
      }
      if constexpr (GATE) {
        const uint32_t lz = walk_limit(wz, q, last);
#pragma unroll
        for (int i = 0; i < KQ; ++i) z[i] = wz.load(4 * i, lz);
      }
      bc.load(s, last);
    };
    fetch(p.te - 1 - tl);
    int buf = 0;
    for (int t0 = tl; t0 >= p.t0; t0 -= K, buf ^= 1) {
      const int last = p.te - 1 - t0;
      bc.store(sb[buf], sc[buf]);
      __syncthreads();
      float dt[KQ], dy[KQ];
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        const bool in = 4 * i + q <= last;
        const float raw = (float)de[i] + bias, sp = softplus_hw(raw);
        dt[i] = in ? (s.softplus ? sp : raw) : 0.0f;
        dtsum += dt[i];
        float y = (float)go[i];
        if constexpr (GATE) {
          const float zf = (float)z[i];
          y *= zf * sigmoid_hw(zf);
        }
        dy[i] = in ? y : 0.0f;
      }
      if (t0 > p.t0) {
        wd.advance(-K);
        wg.advance(-K);
        if constexpr (GATE) wz.advance(-K);
        bc.advance(-K);
        fetch(last + K);
      }
      const float* lc = &sc[buf][q * NL];
#pragma unroll
      for (int i = KQ - 1; i >= 0; --i) {
        auto step = [&](auto jc) {
          constexpr int j = decltype(jc)::value;
          const float dj = quad_get<j>(dt[i]), yj = quad_get<j>(dy[i]);
          float cc[NL];
          load_vec<NL>(cc, lc + (4 * i + j) * NP);
#pragma unroll
          for (int k = 0; k < NL; ++k) g[k] = exp2_hw(dj * a2[k]) * fmaf(cc[k], yj, g[k]);
        };
        step(std::integral_constant<int, 3>());
        step(std::integral_constant<int, 2>());
        step(std::integral_constant<int, 1>());
        step(std::integral_constant<int, 0>());
      }
    }
  }
  dtsum = quad_sum(dtsum);
  if (!p.active) return;
  const int64_t at = (int64_t)p.chunk * s.B * s.D + row;
  store_vec<NL>(s.edge + at * NP + q * NL, g);
  if (q == 0) s.dtsum[at] = dtsum;
}

template <typename E, int NL, bool GATE>
__global__ __launch_bounds__(kScanThreads, 1) void scan_bwd(const ScanArgs<E> s) {
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
  if (s.chunks > 1)
    load_vec<NL>(g, s.edge + ((int64_t)p.chunk * s.B * s.D + row) * NP + q * NL);
  else
    load_state<NL>(g, s.gstate, row, q, s.N);
  const float bias = s.delta_bias ? s.delta_bias[p.d] : 0.0f;
  const float skip = s.d ? s.d[p.d] : 0.0f;
  float gskip = 0.0f, gbias = 0.0f;
  // what this lane ends channel_reduce16 with: a step of the flush, B or C, a state
  const int slot = lane >> 2;

  if (p.t0 < p.te) {
    const int tl = p.t0 + (p.te - 1 - p.t0) / K * K;
    Walk<const E> wu(s.u, tl, p.b, q, p.d), wd(s.delta, tl, p.b, q, p.d);
    Walk<const E> wg(s.go, tl, p.b, q, p.d), wz(GATE ? s.z : s.u, tl, p.b, q, p.d);
    Walk<E> ou(s.gu, tl, p.b, q, p.d), od(s.gdelta, tl, p.b, q, p.d);
    Walk<E> oz(GATE ? s.gz : s.gu, tl, p.b, q, p.d);
    TileBC<E, K, NP> bc(s, p, tl);
    const int64_t ck_step = (int64_t)s.B * s.D * NP;
    const float* ck = s.saved + (int64_t)(tl / K) * ck_step + row * NP + q * NL;
    E eu[KQ], ede[KQ], ez[KQ], ego[KQ];
    float h[NL];
    auto fetch = [&](int last) {
      const uint32_t lu = walk_limit(wu, q, last), ld = walk_limit(wd, q, last);
      const uint32_t lg = walk_limit(wg, q, last);
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        eu[i] = wu.load(4 * i, lu);
        ede[i] = wd.load(4 * i, ld);
        ego[i] = wg.load(4 * i, lg);
      }
      if constexpr (GATE) {
        const uint32_t lz = walk_limit(wz, q, last);
#pragma unroll
        for (int i = 0; i < KQ; ++i) ez[i] = wz.load(4 * i, lz);
      }
      bc.load(s, last);
      load_vec<NL>(h, ck);
    };
    fetch(p.te - 1 - tl);

    for (int t0 = tl; t0 >= p.t0; t0 -= K) {
      const int last = p.te - 1 - t0;
      bc.store(sb, sc);
      float dt[KQ], x[KQ], u[KQ], dy[KQ], raw[KQ], gzf[KQ];
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        const bool in = 4 * i + q <= last;
        raw[i] = (float)ede[i] + bias;
        const float sp = softplus_hw(raw[i]);
        dt[i] = in ? (s.softplus ? sp : raw[i]) : 0.0f;
        u[i] = in ? (float)eu[i] : 0.0f;
        x[i] = dt[i] * u[i];
        dy[i] = in ? (float)ego[i] : 0.0f;
        if constexpr (GATE) {
          const float zf = in ? (float)ez[i] : 0.0f, sg = sigmoid_hw(zf);
          gzf[i] = dy[i] * (sg * fmaf(zf, 1.0f - sg, 1.0f));
          dy[i] *= zf * sg;
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
          load_vec<NL>(bb, &sb[t * NP + q * NL]);
          if constexpr (GATE) load_vec<NL>(cc, &sc[t * NP + q * NL]);
          float y = 0.0f;
#pragma unroll
          for (int k = 0; k < NL; ++k) {
            a[t][k] = exp2_hw(dj * (kLog2e * a1[k]));
            hp[t][k] = h[k];
            h[k] = fmaf(a[t][k], h[k], xj * bb[k]);
            if constexpr (GATE) y = k ? fmaf(cc[k], h[k], y) : cc[k] * h[k];
          }
          acc[j] = y;
        };
        step(std::integral_constant<int, 0>());
        step(std::integral_constant<int, 1>());
        step(std::integral_constant<int, 2>());
        step(std::integral_constant<int, 3>());
        if constexpr (GATE)
          gzf[i] *= fmaf(skip, u[i], quad_reduce4(acc[0], acc[1], acc[2], acc[3], q));
      }

      // and backwards: g enters a step as a_{t+1} dL/dh_{t+1}
      float v[16], gu[KQ], gd[KQ];
#pragma unroll
      for (int i = KQ - 1; i >= 0; --i) {
        float sx[4], sa[4];
        auto step = [&](auto jc) {
          constexpr int j = decltype(jc)::value;
          const int t = 4 * i + j;
          const float dj = quad_get<j>(dt[i]), xj = quad_get<j>(x[i]), yj = quad_get<j>(dy[i]);
          float bb[NL], cc[NL];
          load_vec<NL>(bb, &sb[t * NP + q * NL]);
          load_vec<NL>(cc, &sc[t * NP + q * NL]);
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
        const float sg = sigmoid_hw(raw[i]), gr = fmaf(u[i], gx, gl);
        gd[i] = 4 * i + q <= last ? (s.softplus ? gr * sg : gr) : 0.0f;
        gu[i] = fmaf(dt[i], gx, skip * dy[i]);
        gbias += gd[i];
        gskip = fmaf(dy[i], u[i], gskip);
      }
      // the tile before, while the waves' sums are joined
      if (t0 > p.t0) {
        wu.advance(-K);
        wd.advance(-K);
        wg.advance(-K);
        if constexpr (GATE) wz.advance(-K);
        bc.advance(-K);
        ck -= ck_step;
        fetch(last + K);
      }
      if (p.active) {
#pragma unroll
        for (int i = 0; i < KQ; ++i)
          if (4 * i + q <= last) {
            *ou.at(4 * i) = (E)gu[i];
            *od.at(4 * i) = (E)gd[i];
            if constexpr (GATE) *oz.at(4 * i) = (E)gzf[i];
          }
      }
      ou.advance(-K);
      od.advance(-K);
      if constexpr (GATE) oz.advance(-K);
      __syncthreads();
      for (int e = threadIdx.x; e < K * 2 * NP; e += kScanThreads) {
        const int t = e / (2 * NP);
        if (t <= last)
          s.part_bc[((((int64_t)p.blk * s.T + t0 + t) * s.B + p.b) * s.G + p.g) * (2 * NP) +
                    e % (2 * NP)] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
      }
    }
  }
  zero_steps(s.gu, p);
  zero_steps(s.gdelta, p);
  if constexpr (GATE) zero_steps(s.gz, p);
  if (!p.active) return;
  if (s.gstate0 && p.chunk == 0) store_state<NL>(g, s.gstate0, row, q, s.N);
  float* pa = s.part_a + ((int64_t)p.chunk * s.B * s.D + row) * (NP + 2);
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

// Gradients of A, D and the bias: the sums of all rows and chunks, in order.
__global__ __launch_bounds__(256) void scan_sum_a(const float* part, int64_t D, int N, int NP,
                                                  int64_t rows, float* ga, float* gd,
                                                  float* gbias) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= D * (NP + 2)) return;
  const int n = (int)(i % (NP + 2));
  const int64_t d = i / (NP + 2);
  float* out = n < N ? ga + d * N + n : n < NP ? nullptr : n == NP ? gd : gbias;
  if (!out) return;
  if (n >= NP) out += d;
  float sum = 0.0f;
  for (int64_t r = 0; r < rows; ++r) sum += part[r * D * (NP + 2) + i];
  *out = sum;
}

template <typename E, int NL>
void launch(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream) {
  const unsigned wgs = (unsigned)(d.P * d.G * d.B);
  if (d.chunks > 1) {
    const unsigned grid = wgs * (unsigned)(d.chunks - 1);
    if (a.z.p)
      scan_bwd_part<E, NL, true><<<grid, kScanThreads, 0, stream>>>(a);
    else
      scan_bwd_part<E, NL, false><<<grid, kScanThreads, 0, stream>>>(a);
    const int64_t n = d.B * d.D * d.NP;
    scan_join<false><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(
        a.edge, a.dtsum, a.a, a.gstate, d.B * d.D, a.D, a.N, d.NP, a.chunks);
  }
  const unsigned grid = wgs * (unsigned)d.chunks;
  if (a.z.p)
    scan_bwd<E, NL, true><<<grid, kScanThreads, 0, stream>>>(a);
  else
    scan_bwd<E, NL, false><<<grid, kScanThreads, 0, stream>>>(a);
  const int64_t bc = d.T * d.B * d.G * 2 * d.NP, ae = d.D * (d.NP + 2);
  if (bc > 0)
    scan_sum_bc<E><<<(unsigned)((bc + 255) / 256), 256, 0, stream>>>(
        a.part_bc, a.T, a.B, a.G, a.N, d.NP, a.P, a.lengths, a.gb, a.gc);
  scan_sum_a<<<(unsigned)((ae + 255) / 256), 256, 0, stream>>>(
      a.part_a, d.D, a.N, d.NP, d.chunks * d.B, a.ga, a.gd, a.gbias);
}

}  // namespace

template <typename E>
void scan_launch_backward(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream) {
  switch (d.NL) {
    case 1: return launch<E, 1>(d, a, stream);
    case 2: return launch<E, 2>(d, a, stream);
    case 4: return launch<E, 4>(d, a, stream);
    case 8: return launch<E, 8>(d, a, stream);
    default: return launch<E, 16>(d, a, stream);
  }
}
template void scan_launch_backward<float>(const ScanDims&, const ScanArgs<float>&, hipStream_t);
template void scan_launch_backward<bf16_t>(const ScanDims&, const ScanArgs<bf16_t>&, hipStream_t);
template void scan_launch_backward<f16_t>(const ScanDims&, const ScanArgs<f16_t>&, hipStream_t);

}  // namespace ckhip
