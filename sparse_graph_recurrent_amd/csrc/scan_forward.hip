// scan_forward.hip -- the selective scan over a window (see scan.h).
//
// Bound by the vector ALU: per step and state an exponential (8.5 cycles a
// wave), two products and two multiply-adds (4 each where they mix with
// others), and a fifth of that again for the per-channel work.  Measured, 16
// states, bf16, gated: a training window of 2048 steps x 8 rows x 2048 channels
// in 210 us (vector ALU 83 % busy; 550 MB, half of it the states left for the
// backward, at 2.6 TB/s); a prompt of 16384 steps, one row, in 95 (summaries, ALU
// 87 % busy) + 9 (join) + 125 us (95 %; 2.3 TB/s).  For 64 states of a step a wave
// executes 7.8 vector instructions on one tile, 11.5 on several, whose decays it
// keeps but whose products it forms twice.
#include "scan.h"

#include <type_traits>

namespace ckhip {
namespace {

// PART: only the chunk's summary (what it makes of a zero state, sum of dt).
template <typename E, int NP, int TW, bool GATE, bool PART>
__global__ __launch_bounds__(kScanThreads * TW) void scan_fwd(const ScanArgs<E> s) {
  constexpr int M = scan_blocks(NP), K = scan_tile(NP), KQ = K / 4, KT = K * TW;
  constexpr int kBufs = TW > 1 ? 3 : 2;  // (with one barrier amid the tile's work)
  __shared__ __align__(16) float lds_dt[4 * TW][StepsLds::kFloats];
  __shared__ __align__(16) float lds_x[4 * TW][StepsLds::kFloats];
  __shared__ __align__(16) float lds_bc[kBufs][2 * KT * NP];
  // what each tile makes of a zero state, and its decay
  __shared__ __align__(16) float made[2][TW > 1 ? TW * kScanChan * NP : 4];
  __shared__ __align__(16) float decay[2][TW > 1 ? TW * kScanChan * NP : 4];
  const Place p = scan_place(s);
  const int q = p.q, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float *ldt = lds_dt[wave], *lx = lds_x[wave];
  const int64_t row = (int64_t)p.b * s.D + p.d;
  float* edge = s.edge + ((int64_t)p.chunk * s.B * s.D + row) * NP;
  States<NP> a2[M], h[M];  // h: the state the workgroup's tiles start from
  load_rates<NP>(a2, s.a, p.d, q, s.N);
#pragma unroll
  for (int m = 0; m < M; ++m) {
    a2[m] *= kLog2e;
    h[m] = 0.0f;
  }
  if constexpr (!PART) {
    if (s.chunks > 1 && !s.fold) {
      load_rows<NP>(h, edge, q);
    } else {
      load_states<NP>(h, s.state0, row, q, s.N);
      if (TW == 1 && s.chunks > 1) fold_chunks<NP, true>(h, a2, s, p, row);
    }
  }
  const float bias = s.delta_bias ? s.delta_bias[p.d] : 0.0f;
  const float skip = s.d ? s.d[p.d] : 0.0f;
  float dtsum = 0.0f;

  if (p.t0 < p.te) {
    const int tw0 = p.t0 + p.tw * K;
    Walk<const E> wu(s.u, tw0, p.b, q, p.d), wd(s.delta, tw0, p.b, q, p.d);
    Walk<const E> wz(GATE ? s.z : s.u, tw0, p.b, q, p.d);
    Walk<E> wo(s.out, tw0, p.b, q, p.d);
    TileBC<E, NP, TW> bc(s, p, p.t0);
    E u[KQ], de[KQ], z[KQ];
    // the wave's tile, whose last step with text is `last` (negative: none)
    auto fetch = [&](int last) {
      if (TW > 1 && last < 0) return;
      wu.load(u, q, last);
      wd.load(de, q, last);
      if constexpr (GATE && !PART) wz.load(z, q, last);
    };
    fetch(p.te - 1 - tw0);
    bc.load(p.te - 1 - p.t0);
    // (asked only here: it waits for A, and the first tiles' loads are on their way)
    const bool grows = TW > 1 && scan_grows<NP>(a2, s.softplus);
    bc.store(lds_bc[0]);
    const int64_t ck_step = (int64_t)s.B * s.D * NP;
    float* ck = nullptr;
    if (s.saved) ck = s.saved + (int64_t)(tw0 / K) * ck_step + row * NP;
    __syncthreads();

    int buf = 0, par = 0;
    for (int t0 = p.t0; t0 < p.te; t0 += KT, par ^= 1) {
      const int last = p.te - 1 - t0 - p.tw * K;  // of the tile's steps, the last with text
      const int nbuf = buf + 1 < kBufs ? buf + 1 : 0;
      const bool more = t0 + KT < p.te;
      float dt[KQ], x[KQ], y0[KQ], gt[KQ];
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        const float raw = (float)de[i] + bias, sp = softplus_hw(raw).value;
        dt[i] = s.softplus ? sp : raw;
        y0[i] = (float)u[i];
      }
      if (last < K - 1) {
#pragma unroll
        for (int i = 0; i < KQ; ++i) {
          const bool in = 4 * i + q <= last;
          dt[i] = in ? dt[i] : 0.0f;
          y0[i] = in ? y0[i] : 0.0f;
        }
      }
      wave_sync();  // the tile before has read its rows
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        x[i] = dt[i] * y0[i];
        if constexpr (PART) dtsum += dt[i];
        StepsLds::put(ldt, p.c, q, i, dt[i]);
        StepsLds::put(lx, p.c, q, i, x[i]);
        y0[i] *= skip;
        gt[i] = 1.0f;
        if constexpr (GATE && !PART) {
          const float zf = (float)z[i];
          gt[i] = zf * sigmoid_hw(zf);
        }
      }
      wave_sync();
      if (more) {
        wu.advance(KT);
        wd.advance(KT);
        if constexpr (GATE) wz.advance(KT);
        bc.advance(KT);
        fetch(last - KT);
        bc.load(p.te - 1 - t0 - KT);
      }
      const float *lb = lds_bc[buf] + p.tw * K * NP, *lc = lb + KT * NP;

      States<NP> a[TW > 1 ? K : 1][M], next[M];
      if constexpr (TW > 1) {
        // decays, and what the tile makes of a zero state
        States<NP> mk[M], e[M];
        float sum = 0.0f;
#pragma unroll
        for (int m = 0; m < M; ++m) mk[m] = 0.0f;
#pragma unroll
        for (int i = 0; i < KQ; ++i) {
          const f32x4 d4 = StepsLds::get(ldt, p.c, i), x4 = StepsLds::get(lx, p.c, i);
          sum += (d4[0] + d4[1]) + (d4[2] + d4[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            States<NP> b4[M];
            load_rows<NP>(b4, lb + (4 * i + j) * NP, q);
#pragma unroll
            for (int m = 0; m < M; ++m) {
              a[4 * i + j][m] = exp2_v(d4[j] * a2[m]);
              mk[m] = fma_v(a[4 * i + j][m], mk[m], x4[j] * b4[m]);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < M; ++m) e[m] = tile_decay(sum, a2[m], grows);
        const int at = (p.tw * kScanChan + p.wc) * NP;
        store_rows<NP>(&made[par][at], mk, q);
        store_rows<NP>(&decay[par][at], e, q);
        if (more) bc.store(lds_bc[nbuf]);
        __syncthreads();
        fold_tiles<NP, TW, true>(h, next, made[par], decay[par], p, grows);
      }

      if constexpr (!PART)
        if (ck && p.active && (TW == 1 || last >= 0)) store_rows<NP>(ck, h, q);
      float yo[KQ];
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        float acc[4];
        const f32x4 d4 = StepsLds::get(ldt, p.c, i), x4 = StepsLds::get(lx, p.c, i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          States<NP> b4[M], c4[M];
          float y = 0.0f;
          load_rows<NP>(b4, lb + (4 * i + j) * NP, q);
          if constexpr (!PART) load_rows<NP>(c4, lc + (4 * i + j) * NP, q);
#pragma unroll
          for (int m = 0; m < M; ++m) {
            States<NP> am;
            if constexpr (TW > 1)
              am = a[4 * i + j][m];
            else
              am = exp2_v(d4[j] * a2[m]);
            h[m] = fma_v(am, h[m], x4[j] * b4[m]);
            if constexpr (!PART) y = dot_add(c4[m], h[m], y);
          }
          acc[j] = y;
        }
        if constexpr (!PART) yo[i] = (y0[i] + rows_reduce4(acc)) * gt[i];
      }
      if constexpr (!PART) {
        if (p.active) {
#pragma unroll
          for (int i = 0; i < KQ; ++i)
            if (4 * i + q <= last) *wo.at(4 * i) = (E)yo[i];
        }
        wo.advance(KT);
        if (ck) ck += TW * ck_step;
      }
      if constexpr (TW > 1) {
#pragma unroll
        for (int m = 0; m < M; ++m) h[m] = next[m];
      } else {
        if (more) bc.store(lds_bc[nbuf]);
        __syncthreads();
      }
      buf = nbuf;
    }
  }
  if constexpr (PART) {
    dtsum = rows_sum(dtsum);
    if (p.active) {
      store_rows<NP>(edge, h, q);
      if (q == 0) s.dtsum[(int64_t)p.chunk * s.B * s.D + row] = dtsum;
    }
  } else if (p.tw == 0) {
    zero_steps(s.out, p);
    // the chunk in which the text ends has the final state
    if (s.state && p.active && p.chunk == min(p.len / s.chunk_steps, s.chunks - 1))
      store_states<NP>(h, s.state, row, q, s.N);
  }
}

template <typename E, int NP, int TW>
void launch_main(unsigned grid, const ScanArgs<E>& a, hipStream_t stream) {
  if (a.z.p)
    scan_fwd<E, NP, TW, true, false><<<grid, kScanThreads * TW, 0, stream>>>(a);
  else
    scan_fwd<E, NP, TW, false, false><<<grid, kScanThreads * TW, 0, stream>>>(a);
}

template <typename E, int NP>
void launch(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream) {
  const unsigned wgs = (unsigned)(d.P * d.G * d.B), grid = wgs * (unsigned)d.chunks;
  if (d.chunks > 1) {
    // (nothing follows the last chunk)
    scan_fwd<E, NP, 1, false, true><<<grid - wgs, kScanThreads, 0, stream>>>(a);
    if (!d.fold) {
      const int64_t n = d.B * d.D * d.NP;
      scan_join<true><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(
          a.edge, a.dtsum, a.a, a.state0, d.B * d.D, a.D, a.N, d.NP, a.chunks, a.softplus);
    }
  }
  if constexpr (NP <= 16) {
    if (d.waves) return launch_main<E, NP, kScanFwdTW>(grid, a, stream);
  }
  launch_main<E, NP, 1>(grid, a, stream);
}

}  // namespace

template <typename E>
void scan_launch_forward(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream) {
  switch (d.NP) {
    case 8: return launch<E, 8>(d, a, stream);
    case 16: return launch<E, 16>(d, a, stream);
    case 32: return launch<E, 32>(d, a, stream);
    default: return launch<E, 64>(d, a, stream);
  }
}
template void scan_launch_forward<float>(const ScanDims&, const ScanArgs<float>&, hipStream_t);
template void scan_launch_forward<bf16_t>(const ScanDims&, const ScanArgs<bf16_t>&, hipStream_t);
template void scan_launch_forward<f16_t>(const ScanDims&, const ScanArgs<f16_t>&, hipStream_t);

}  // namespace ckhip
