// scan_forward.hip -- the selective scan over a window (see scan.h).
//
// What bounds it is the vector ALU: per step and state an exponential, two
// products and two multiply-adds, against 6 to 8 bytes per step and channel of
// 16-bit tensors.  A wave's steps depend on each other only through h, one
// multiply-add a step, so a single wave per SIMD keeps its ALU busy as long as
// nothing else is waited for: the next tile's global loads are issued a tile
// ahead and B, C come from LDS four steps ahead of their use.
#include "scan.h"

#include <type_traits>

namespace ckhip {
namespace {

// PART: only the chunk's summary (what it makes of a zero state, sum of dt).
template <typename E, int NL, bool GATE, bool PART>
__global__ __launch_bounds__(kScanThreads, 2) void scan_fwd(const ScanArgs<E> s) {
  constexpr int K = scan_tile(NL), KQ = K / 4, NP = 4 * NL;
  __shared__ float sb[2][K * NP], sc[2][K * NP];
  const Place p = scan_place(s);
  const int q = p.q;
  const int64_t row = (int64_t)p.b * s.D + p.d;
  const int64_t edge = ((int64_t)p.chunk * s.B * s.D + row) * NP + q * NL;
  float a2[NL], h[NL];
  load_a<NL>(a2, s.a, p.d, q, s.N);
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    a2[k] *= kLog2e;
    h[k] = 0.0f;
  }
  if constexpr (!PART) {
    if (s.chunks > 1)
      load_vec<NL>(h, s.edge + edge);
    else
      load_state<NL>(h, s.state0, row, q, s.N);
  }
  const float bias = s.delta_bias ? s.delta_bias[p.d] : 0.0f;
  const float skip = s.d ? s.d[p.d] : 0.0f;
  float dtsum = 0.0f;

  if (p.t0 < p.te) {
    Walk<const E> wu(s.u, p.t0, p.b, q, p.d), wd(s.delta, p.t0, p.b, q, p.d);
    Walk<const E> wz(GATE ? s.z : s.u, p.t0, p.b, q, p.d);
    Walk<E> wo(s.out, p.t0, p.b, q, p.d);
    TileBC<E, K, NP> bc(s, p, p.t0);
    E u[KQ], de[KQ], z[KQ];
    auto fetch = [&](int last) {
      const uint32_t lu = walk_limit(wu, q, last), ld = walk_limit(wd, q, last);
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        u[i] = wu.load(4 * i, lu);
        de[i] = wd.load(4 * i, ld);
      }
      if constexpr (GATE && !PART) {
        const uint32_t lz = walk_limit(wz, q, last);
#pragma unroll
        for (int i = 0; i < KQ; ++i) z[i] = wz.load(4 * i, lz);
      }
      bc.load(s, last);
    };
    fetch(p.te - 1 - p.t0);
    float* ck = s.saved;
    const int64_t ck_step = (int64_t)s.B * s.D * NP;
    if (ck) ck += (int64_t)(p.t0 / K) * ck_step + row * NP + q * NL;

    int buf = 0;
    for (int t0 = p.t0; t0 < p.te; t0 += K, buf ^= 1) {
      const int last = p.te - 1 - t0;  // of the tile's steps, the last with text
      bc.store(sb[buf], sc[buf]);
      __syncthreads();
      float bb[4][NL], cc[4][NL];
      const float *lb = &sb[buf][q * NL], *lc = &sc[buf][q * NL];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        load_vec<NL>(bb[j], lb + j * NP);
        if constexpr (!PART) load_vec<NL>(cc[j], lc + j * NP);
      }
      float dt[KQ], x[KQ], y0[KQ], gt[KQ];
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        const bool in = 4 * i + q <= last;
        const float raw = (float)de[i] + bias, sp = softplus_hw(raw);
        dt[i] = in ? (s.softplus ? sp : raw) : 0.0f;
        const float uf = in ? (float)u[i] : 0.0f;
        x[i] = dt[i] * uf;
        if constexpr (PART) {
          dtsum += dt[i];
        } else {
          y0[i] = skip * uf;
          gt[i] = 1.0f;
          if constexpr (GATE) {
            const float zf = (float)z[i];
            gt[i] = zf * sigmoid_hw(zf);
          }
        }
      }
      if (t0 + K < p.te) {
        wu.advance(K);
        wd.advance(K);
        if constexpr (GATE) wz.advance(K);
        bc.advance(K);
        fetch(last - K);
      }
      if constexpr (!PART) {
        if (ck) {
          if (p.active) store_vec<NL>(ck, h);
          ck += ck_step;
        }
      }
      float yo[KQ];
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        float nb[4][NL], nc[4][NL];
        if (i + 1 < KQ) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            load_vec<NL>(nb[j], lb + (4 * i + 4 + j) * NP);
            if constexpr (!PART) load_vec<NL>(nc[j], lc + (4 * i + 4 + j) * NP);
          }
        }
        float acc[4];
        auto step = [&](auto jc) {
          constexpr int j = decltype(jc)::value;
          const float dj = quad_get<j>(dt[i]), xj = quad_get<j>(x[i]);
          float y = 0.0f;
#pragma unroll
          for (int k = 0; k < NL; ++k) {
            h[k] = fmaf(exp2_hw(dj * a2[k]), h[k], xj * bb[j][k]);
            if constexpr (!PART) y = k ? fmaf(cc[j][k], h[k], y) : cc[j][k] * h[k];
          }
          acc[j] = y;
        };
        step(std::integral_constant<int, 0>());
        step(std::integral_constant<int, 1>());
        step(std::integral_constant<int, 2>());
        step(std::integral_constant<int, 3>());
        if constexpr (!PART)
          yo[i] = (y0[i] + quad_reduce4(acc[0], acc[1], acc[2], acc[3], q)) * gt[i];
        if (i + 1 < KQ) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < NL; ++k) {
              bb[j][k] = nb[j][k];
              if constexpr (!PART) cc[j][k] = nc[j][k];
            }
        }
      }
      if constexpr (!PART) {
        if (p.active) {
#pragma unroll
          for (int i = 0; i < KQ; ++i)
            if (4 * i + q <= last) *wo.at(4 * i) = (E)yo[i];
        }
        wo.advance(K);
      }
    }
  }
  if constexpr (PART) {
    dtsum = quad_sum(dtsum);
    if (p.active) {
      store_vec<NL>(s.edge + edge, h);
      if (q == 0) s.dtsum[(int64_t)p.chunk * s.B * s.D + row] = dtsum;
    }
  } else {
    zero_steps(s.out, p);
    // the chunk in which the text ends has the final state
    if (s.state && p.active && p.chunk == min(p.len / s.chunk_steps, s.chunks - 1))
      store_state<NL>(h, s.state, row, q, s.N);
  }
}

template <typename E, int NL>
void launch(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream) {
  const unsigned wgs = (unsigned)(d.P * d.G * d.B);
  if (d.chunks > 1) {
    scan_fwd<E, NL, false, true>
        <<<wgs * (unsigned)(d.chunks - 1), kScanThreads, 0, stream>>>(a);
    const int64_t n = d.B * d.D * d.NP;
    scan_join<true><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(
        a.edge, a.dtsum, a.a, a.state0, d.B * d.D, a.D, a.N, d.NP, a.chunks);
  }
  const unsigned grid = wgs * (unsigned)d.chunks;
  if (a.z.p)
    scan_fwd<E, NL, true, false><<<grid, kScanThreads, 0, stream>>>(a);
  else
    scan_fwd<E, NL, false, false><<<grid, kScanThreads, 0, stream>>>(a);
}

}  // namespace

template <typename E>
void scan_launch_forward(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream) {
  switch (d.NL) {
    case 1: return launch<E, 1>(d, a, stream);
    case 2: return launch<E, 2>(d, a, stream);
    case 4: return launch<E, 4>(d, a, stream);
    case 8: return launch<E, 8>(d, a, stream);
    default: return launch<E, 16>(d, a, stream);
  }
}
template void scan_launch_forward<float>(const ScanDims&, const ScanArgs<float>&, hipStream_t);
template void scan_launch_forward<bf16_t>(const ScanDims&, const ScanArgs<bf16_t>&, hipStream_t);
template void scan_launch_forward<f16_t>(const ScanDims&, const ScanArgs<f16_t>&, hipStream_t);

}  // namespace ckhip
