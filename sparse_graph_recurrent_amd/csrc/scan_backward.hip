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
// is small), then the adjoint runs down through them.  Bound by the vector ALU
// as the forward, with eleven products and multiply-adds a step and state.  The
// sums over channels of gB and gC are a fifth of its work: 16 values are summed
// over a wave's 16 channels by halving exchanges (through LDS instead: 500 to
// 715 us, the waves wait), the four waves' sums are added in LDS and the
// workgroups' by a last launch, all in a fixed order.  Registers allow two
// waves a SIMD; a third cost 16 spilled registers and a fifth of the speed.
// Measured at 2048 steps x 8 rows x 2048 channels x 16 states, bf16, gated:
// 459 us (ALU 81 % busy, 820 MB at 1.8 TB/s; 25.8 vector instructions for 64 states
// of a step, of which the formulas are 13 and an exponential) and 18 us for the sums.
#include "scan.h"

#include <type_traits>

namespace ckhip {
namespace {

// v[i] of the channels' lanes 0-7 of each row, v[i + 8] of lanes 8-15, summed
// over lanes 8 apart.  (DPP operands need two wait states behind a write; outputs
// written before the last operand is read are early-clobbered.)
__device__ __forceinline__ void halve8(float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; i += 4)
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %1, %1, %1 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %2, %2, %2 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %3, %3, %3 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %0, %4, %4 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %1, %5, %5 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %3, %7, %7 row_ror:8 row_mask:0xf bank_mask:0xc"
        : "+&v"(v[i]), "+&v"(v[i + 1]), "+&v"(v[i + 2]), "+&v"(v[i + 3])
        : "v"(v[i + 8]), "v"(v[i + 9]), "v"(v[i + 10]), "v"(v[i + 11]));
}
// The same for v[i] and v[i + 4] and lanes n and n ^ 7.
__device__ __forceinline__ void halve4(float (&v)[16]) {
  asm("s_nop 1\n\t"
      "v_add_f32_dpp %0, %0, %0 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %1, %1, %1 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %2, %2, %2 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %3, %3, %3 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %0, %4, %4 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %1, %5, %5 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %2, %6, %6 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %3, %7, %7 row_half_mirror row_mask:0xf bank_mask:0xa"
      : "+&v"(v[0]), "+&v"(v[1]), "+&v"(v[2]), "+&v"(v[3])
      : "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]));
}

// Sums v[0..15] over a wave's 16 channels (the lanes of a row): lane c of each
// row gets the total of v[c].  Halving exchanges with lanes c ^ 8, c ^ 7,
// c ^ 2 and c ^ 1 (each one DPP): 33 operations, where 16 butterflies take 64.
__device__ __forceinline__ float channel_reduce16(float (&v)[16], int c) {
  halve8(v);
  halve4(v);
  const bool b1 = c & 2, b0 = c & 1;
  const float r0 = (b1 ? v[2] : v[0]) + quad_xor2(b1 ? v[0] : v[2]);
  const float r1 = (b1 ? v[3] : v[1]) + quad_xor2(b1 ? v[1] : v[3]);
  return (b0 ? r1 : r0) + quad_xor1(b0 ? r0 : r1);
}

// The adjoint's share of a chunk: what it hands to the chunk before, given
// nothing from the one behind, and the sum of the chunk's dt.
template <typename E, int NP, bool GATE>
__global__ __launch_bounds__(kScanThreads) void scan_bwd_part(const ScanArgs<E> s) {
  constexpr int M = scan_blocks(NP), K = scan_tile(NP), KQ = K / 4;
  __shared__ __align__(16) float lds_dt[4][StepsLds::kFloats], lds_dy[4][StepsLds::kFloats];
  __shared__ __align__(16) float lds_bc[2][2 * K * NP];
  Place p = scan_place(s);
  // chunk 0 hands nothing on: the grid covers chunks 1 ..
  p.chunk += 1;
  p.t0 += s.chunk_steps;
  p.t1 = min(p.t0 + s.chunk_steps, s.T);
  p.te = min(p.t1, p.len);
  const int q = p.q, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float *ldt = lds_dt[wave], *ldy = lds_dy[wave];
  const int64_t row = (int64_t)p.b * s.D + p.d;
  States<NP> a2[M], g[M];
  load_rates<NP>(a2, s.a, p.d, q, s.N);
#pragma unroll
  for (int m = 0; m < M; ++m) {
    a2[m] *= kLog2e;
    g[m] = 0.0f;
  }
  const float bias = s.delta_bias ? s.delta_bias[p.d] : 0.0f;
  float dtsum = 0.0f;
  if (p.t0 < p.te) {
    const int tl = p.t0 + (p.te - 1 - p.t0) / K * K;
    Walk<const E> wd(s.delta, tl, p.b, q, p.d), wg(s.go, tl, p.b, q, p.d);
    Walk<const E> wz(GATE ? s.z : s.go, tl, p.b, q, p.d);
    TileBC<E, NP, 1> bc(s, p, tl);
    E de[KQ], go[KQ], z[KQ];
    auto fetch = [&](int last) {
      wd.load(de, q, last);
      wg.load(go, q, last);
      if constexpr (GATE) wz.load(z, q, last);
    };
    fetch(p.te - 1 - tl);
    bc.load(p.te - 1 - tl);
    bc.store(lds_bc[0]);
    __syncthreads();
    int buf = 0;
    for (int t0 = tl; t0 >= p.t0; t0 -= K, buf ^= 1) {
      const int last = p.te - 1 - t0;
      const bool more = t0 > p.t0;
      wave_sync();
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        const bool in = 4 * i + q <= last;
        const float raw = (float)de[i] + bias, sp = softplus_hw(raw).value;
        const float dt = in ? (s.softplus ? sp : raw) : 0.0f;
        dtsum += dt;
        StepsLds::put(ldt, p.c, q, i, dt);
        float y = (float)go[i];
        if constexpr (GATE) {
          const float zf = (float)z[i];
          y *= zf * sigmoid_hw(zf);
        }
        StepsLds::put(ldy, p.c, q, i, in ? y : 0.0f);
      }
      wave_sync();
      if (more) {
        wd.advance(-K);
        wg.advance(-K);
        if constexpr (GATE) wz.advance(-K);
        bc.advance(-K);
        fetch(last + K);
        bc.load(last + K);
      }
      const float* lc = lds_bc[buf] + K * NP;
#pragma unroll
      for (int i = KQ - 1; i >= 0; --i) {
        const f32x4 d4 = StepsLds::get(ldt, p.c, i), y4 = StepsLds::get(ldy, p.c, i);
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          States<NP> c4[M];
          load_rows<NP>(c4, lc + (4 * i + j) * NP, q);
#pragma unroll
          for (int m = 0; m < M; ++m)
            g[m] = exp2_v(d4[j] * a2[m]) * fma_v(c4[m], States<NP>(y4[j]), g[m]);
        }
      }
      if (more) bc.store(lds_bc[buf ^ 1]);
      __syncthreads();
    }
  }
  dtsum = rows_sum(dtsum);
  if (!p.active) return;
  const int64_t at = (int64_t)p.chunk * s.B * s.D + row;
  store_rows<NP>(s.edge + at * NP, g, q);
  if (q == 0) s.dtsum[at] = dtsum;
}

template <typename E, int NP, int TW, bool GATE>
__global__ __launch_bounds__(kScanThreads * TW, NP < 64 && TW == 1 ? 2 : 1) void scan_bwd(const ScanArgs<E> s) {
  constexpr int M = scan_blocks(NP), K = scan_tile(NP), KQ = K / 4, KT = K * TW;
  constexpr int R = scan_lane(NP), S = 8 / R;
  __shared__ __align__(16) float lds_dt[4 * TW][StepsLds::kFloats];
  __shared__ __align__(16) float lds_x[4 * TW][StepsLds::kFloats];
  __shared__ __align__(16) float lds_dy[4 * TW][StepsLds::kFloats];
  __shared__ __align__(16) float lds_bc[2][2 * KT * NP];
  __shared__ __align__(16) float red[4 * TW][K * 2 * NP];
  // what each tile hands on of a zero adjoint, and its decay
  __shared__ __align__(16) float made[TW > 1 ? TW * kScanChan * NP : 4];
  __shared__ __align__(16) float decay[TW > 1 ? TW * kScanChan * NP : 4];
  const Place p = scan_place(s);
  const int q = p.q, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float *ldt = lds_dt[wave], *lx = lds_x[wave], *ldy = lds_dy[wave];
  const int64_t row = (int64_t)p.b * s.D + p.d;
  States<NP> a1[M], ga[M], g[M];  // g: the adjoint the workgroup's tiles start from
  load_rates<NP>(a1, p.active ? s.a : nullptr, p.d, q, s.N);
#pragma unroll
  for (int m = 0; m < M; ++m) ga[m] = g[m] = 0.0f;
  // Lanes without a channel hold zeros throughout, so they add nothing to gB, gC.
  if (p.active) {
    if (s.chunks > 1 && !s.fold) {
      load_rows<NP>(g, s.edge + ((int64_t)p.chunk * s.B * s.D + row) * NP, q);
    } else {
      load_states<NP>(g, s.gstate, row, q, s.N);
      if (TW == 1 && s.chunks > 1) {
        States<NP> a2[M];
#pragma unroll
        for (int m = 0; m < M; ++m) a2[m] = kLog2e * a1[m];
        fold_chunks<NP, false>(g, a2, s, p, row);
      }
    }
  }
  const float bias = s.delta_bias ? s.delta_bias[p.d] : 0.0f;
  const float skip = s.d ? s.d[p.d] : 0.0f;
  float gskip = 0.0f, gbias = 0.0f;
  const bool part_wg = (p.blk + 1) * kScanChan > s.Dg;  // some lanes have no channel

  if (p.t0 < p.te) {
    const int tl = p.t0 + (p.te - 1 - p.t0) / KT * KT, tw0 = tl + p.tw * K;
    Walk<const E> wu(s.u, tw0, p.b, q, p.d), wd(s.delta, tw0, p.b, q, p.d);
    Walk<const E> wg(s.go, tw0, p.b, q, p.d), wz(GATE ? s.z : s.u, tw0, p.b, q, p.d);
    Walk<E> ou(s.gu, tw0, p.b, q, p.d), od(s.gdelta, tw0, p.b, q, p.d);
    Walk<E> oz(GATE ? s.gz : s.gu, tw0, p.b, q, p.d);
    TileBC<E, NP, TW> bc(s, p, tl);
    const int64_t ck_step = (int64_t)s.B * s.D * NP;
    const float* ck = s.saved + (int64_t)(tw0 / K) * ck_step + row * NP;
    E eu[KQ], ede[KQ], ez[KQ], ego[KQ];
    States<NP> h[M], hn[M];  // states; those the next tile starts from
#pragma unroll
    for (int m = 0; m < M; ++m) hn[m] = 0.0f;
    // the wave's tile, whose last step with text is `last` (negative: none)
    auto fetch = [&](int last) {
      if (TW > 1 && last < 0) return;
      wu.load(eu, q, last);
      wd.load(ede, q, last);
      wg.load(ego, q, last);
      if constexpr (GATE) wz.load(ez, q, last);
      if (p.active) load_rows<NP>(hn, ck, q);
    };
    fetch(p.te - 1 - tw0);
    bc.load(p.te - 1 - tl);
    const bool grows = TW > 1 && scan_grows<NP>(a1, s.softplus);  // (waits for A)
    bc.store(lds_bc[0]);
    __syncthreads();

    int buf = 0;
    for (int t0 = tl; t0 >= p.t0; t0 -= KT, buf ^= 1) {
      const int last = p.te - 1 - t0 - p.tw * K;  // of the tile's steps, the last with text
      const bool more = t0 > p.t0;
      float dt[KQ], u[KQ], dy[KQ], sg[KQ], gzf[KQ];
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        const float raw = (float)ede[i] + bias;
        const Softplus sp = softplus_hw(raw);
        sg[i] = s.softplus ? sp.slope : 1.0f;
        dt[i] = s.softplus ? sp.value : raw;
        u[i] = (float)eu[i];
        dy[i] = (float)ego[i];
        if constexpr (GATE) {
          const float zf = (float)ez[i], sz = sigmoid_hw(zf);
          gzf[i] = dy[i] * (sz * fmaf(zf, 1.0f - sz, 1.0f));
          dy[i] *= zf * sz;
        }
      }
      if (last < K - 1 || part_wg) {
#pragma unroll
        for (int i = 0; i < KQ; ++i) {
          const bool in = 4 * i + q <= last && p.active;
          sg[i] = in ? sg[i] : 0.0f;
          dt[i] = in ? dt[i] : 0.0f;
          u[i] = in ? u[i] : 0.0f;
          dy[i] = in ? dy[i] : 0.0f;
        }
      }
      wave_sync();
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        StepsLds::put(ldt, p.c, q, i, dt[i]);
        StepsLds::put(lx, p.c, q, i, dt[i] * u[i]);
        StepsLds::put(ldy, p.c, q, i, dy[i]);
      }
      wave_sync();
#pragma unroll
      for (int m = 0; m < M; ++m) h[m] = hn[m];
      // the tile before, a whole tile's work ahead of its use
      if (more) {
        wu.advance(-KT);
        wd.advance(-KT);
        wg.advance(-KT);
        if constexpr (GATE) wz.advance(-KT);
        bc.advance(-KT);
        ck -= TW * ck_step;
        fetch(last + KT);
        bc.load(p.te - 1 - t0 + KT);
      }
      const float *lb = lds_bc[buf] + p.tw * K * NP, *lc = lb + KT * NP;

      // the tile's states again, from its first
      States<NP> a[K][M], before[K][M];  // decays, and the states before each step
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        const f32x4 d4 = StepsLds::get(ldt, p.c, i), x4 = StepsLds::get(lx, p.c, i);
        if constexpr (TW > 1) sum += (d4[0] + d4[1]) + (d4[2] + d4[3]);
        float acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          States<NP> b4[M], c4[M];
          float y = 0.0f;
          load_rows<NP>(b4, lb + (4 * i + j) * NP, q);
          if constexpr (GATE) load_rows<NP>(c4, lc + (4 * i + j) * NP, q);
#pragma unroll
          for (int m = 0; m < M; ++m) {
            a[4 * i + j][m] = exp2_v(d4[j] * (kLog2e * a1[m]));
            before[4 * i + j][m] = h[m];
            h[m] = fma_v(a[4 * i + j][m], h[m], x4[j] * b4[m]);
            if constexpr (GATE) y = dot_add(c4[m], h[m], y);
          }
          acc[j] = y;
        }
        if constexpr (GATE) gzf[i] *= fmaf(skip, u[i], rows_reduce4(acc));
      }

      States<NP> next[M];
      if constexpr (TW > 1) {
        // what the tile hands on of a zero adjoint
        States<NP> mk[M], e[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          mk[m] = 0.0f;
          e[m] = tile_decay(sum, kLog2e * a1[m], grows);
        }
#pragma unroll
        for (int i = KQ - 1; i >= 0; --i) {
          const f32x4 y4 = StepsLds::get(ldy, p.c, i);
#pragma unroll
          for (int j = 3; j >= 0; --j) {
            States<NP> c4[M];
            load_rows<NP>(c4, lc + (4 * i + j) * NP, q);
#pragma unroll
            for (int m = 0; m < M; ++m)
              mk[m] = a[4 * i + j][m] * fma_v(c4[m], States<NP>(y4[j]), mk[m]);
          }
        }
        const int at = (p.tw * kScanChan + p.wc) * NP;
        store_rows<NP>(&made[at], mk, q);
        store_rows<NP>(&decay[at], e, q);
      }
      if (more) bc.store(lds_bc[buf ^ 1]);
      __syncthreads();  // (and the waves' sums of the tiles before are read)
      if constexpr (TW > 1) fold_tiles<NP, TW, false>(g, next, made, decay, p, grows);

      // and backwards: g enters a step as a_{t+1} dL/dh_{t+1}
      float v[16], gu[KQ], gd[KQ];
#pragma unroll
      for (int i = KQ - 1; i >= 0; --i) {
        const f32x4 d4 = StepsLds::get(ldt, p.c, i), x4 = StepsLds::get(lx, p.c, i);
        const f32x4 y4 = StepsLds::get(ldy, p.c, i);
        float sx[4], sa[4];
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          const int t = 4 * i + j;
          States<NP> b4[M], c4[M];
          float s1 = 0.0f, s2 = 0.0f;
          load_rows<NP>(b4, lb + t * NP, q);
          load_rows<NP>(c4, lc + t * NP, q);
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const States<NP> gh = fma_v(c4[m], States<NP>(y4[j]), g[m]);
            const States<NP> vb = gh * x4[j], vc = h[m] * y4[j];
            h[m] = before[t][m];
            s1 = dot_add(gh, b4[m], s1);
            g[m] = a[t][m] * gh;
            const States<NP> w = g[m] * h[m];
            ga[m] = fma_v(w, States<NP>(d4[j]), ga[m]);
            s2 = dot_add(w, a1[m], s2);
            // values of S (step, block) pairs make 16 sums over the channels
            const int part = (t * M + m) % S;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              v[part * 2 * R + r] = vb[r];
              v[part * 2 * R + R + r] = vc[r];
            }
            if constexpr (M > 1) {
              // pairs are the blocks 2 k, 2 k + 1 of a step
              if (part == 1) {
                const int kind = p.c / 4 % 2, blk = m - 1 + p.c / 8;
                red[wave][(t * 2 + kind) * NP + 16 * blk + 4 * q + p.c % 4] =
                    channel_reduce16(v, p.c);
              }
            }
          }
          if constexpr (M == 1) {
            // the steps t .. t + S - 1
            if (t % S == 0) {
              const int kind = p.c / R % 2;
              red[wave][((t + p.c / (2 * R)) * 2 + kind) * NP + R * q + p.c % R] =
                  channel_reduce16(v, p.c);
            }
          }
          sx[j] = s1;
          sa[j] = s2;
        }
        const float gx = rows_reduce4(sx);  // dL/d(dt u)
        const float gl = rows_reduce4(sa);  // sum_n dL/d(dt A) A
        // (past the text gl, with a decay of 1, may be anything)
        gd[i] = 4 * i + q <= last ? fmaf(u[i], gx, gl) * sg[i] : 0.0f;
        gu[i] = fmaf(dt[i], gx, skip * dy[i]);
        gbias += gd[i];
        gskip = fmaf(dy[i], u[i], gskip);
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
      ou.advance(-KT);
      od.advance(-KT);
      if constexpr (GATE) oz.advance(-KT);
      if constexpr (TW > 1) {
#pragma unroll
        for (int m = 0; m < M; ++m) g[m] = next[m];
      }
      __syncthreads();
      for (int e = threadIdx.x; e < KT * 2 * NP; e += kScanThreads * TW) {
        const int t = t0 + e / (2 * NP), w = e / (K * 2 * NP) * 4, i = e % (K * 2 * NP);
        if (t < p.te)
          s.part_bc[((((int64_t)p.blk * s.T + t) * s.B + p.b) * s.G + p.g) * (2 * NP) +
                    e % (2 * NP)] =
              (red[w][i] + red[w + 1][i]) + (red[w + 2][i] + red[w + 3][i]);
      }
    }
  }
  if (p.tw == 0) {
    zero_steps(s.gu, p);
    zero_steps(s.gdelta, p);
    if constexpr (GATE) zero_steps(s.gz, p);
    if (s.gstate0 && p.chunk == 0 && p.active) store_states<NP>(g, s.gstate0, row, q, s.N);
  }
  if (!p.active) return;
  // (with several tiles a workgroup there is one chunk, and tw in its place)
  float* pa = s.part_a + ((int64_t)(p.chunk + p.tw) * s.B * s.D + row) * (NP + 2);
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < R; ++r) pa[16 * m + R * q + r] = ga[m][r];
  gskip = rows_sum(gskip);
  gbias = rows_sum(gbias);
  if (q == 0) {
    pa[NP] = gskip;
    pa[NP + 1] = gbias;
  }
}

// Gradients of B and C: the workgroups' partial sums of a group, in order.
template <typename E>
__device__ __forceinline__ void sum_bc(const ScanArgs<E>& s, int NP, int64_t i) {
  const int64_t stride = (int64_t)s.T * s.B * s.G * 2 * NP;
  if (i >= stride) return;
  const int e = (int)(i % (2 * NP)), kind = e / NP, n = e % NP;
  int64_t r = i / (2 * NP);
  const int g = (int)(r % s.G);
  r /= s.G;
  const int b = (int)(r % s.B), t = (int)(r / s.B);
  if (n >= s.N) return;
  float sum = 0.0f;
  if (!s.lengths || t < s.lengths[b]) {
#pragma unroll 8
    for (int k = 0; k < s.P; ++k) sum += s.part_bc[k * stride + i];
  }
  (kind ? s.gc : s.gb).row(t, b)[(int64_t)g * s.N + n] = (E)sum;
}

// Gradients of A, D and the bias: the sums of all rows and chunks in a fixed
// order.  A workgroup takes 32 sums, eight threads each one a stretch of them.
template <typename E>
__device__ __forceinline__ void sum_a(const ScanArgs<E>& s, int NP, int parts, int64_t first) {
  __shared__ float red[8][32];
  const int64_t all = (int64_t)s.D * (NP + 2), i = first + (threadIdx.x & 31);
  const int y = threadIdx.x >> 5;
  const int64_t rows = (int64_t)parts * s.B;
  const int64_t each = (rows + 7) / 8, r0 = each * y, r1 = min(r0 + each, rows);
  float sum = 0.0f;
  if (i < all) {
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) sum += s.part_a[r * all + i];
  }
  red[y][threadIdx.x & 31] = sum;
  __syncthreads();
  if (y != 0 || i >= all) return;
  sum = 0.0f;
  for (int j = 0; j < 8; ++j) sum += red[j][threadIdx.x];
  const int n = (int)(i % (NP + 2));
  const int64_t d = i / (NP + 2);
  if (n < s.N)
    s.ga[d * s.N + n] = sum;
  else if (n == NP && s.gd)
    s.gd[d] = sum;
  else if (n == NP + 1 && s.gbias)
    s.gbias[d] = sum;
}

// The last launch: both kinds of sums, the first a_wgs workgroups those of A.
template <typename E>
__global__ __launch_bounds__(256) void scan_sums(const ScanArgs<E> s, int NP, int parts,
                                                  unsigned a_wgs) {
  const int64_t wg = seq_block();
  if (wg < a_wgs)
    sum_a(s, NP, parts, wg * 32);
  else
    sum_bc(s, NP, (wg - a_wgs) * 256 + threadIdx.x);
}

template <typename E, int NP, int TW>
void launch_main(unsigned grid, const ScanArgs<E>& a, hipStream_t stream) {
  if (a.z.p)
    scan_bwd<E, NP, TW, true><<<grid, kScanThreads * TW, 0, stream>>>(a);
  else
    scan_bwd<E, NP, TW, false><<<grid, kScanThreads * TW, 0, stream>>>(a);
}

template <typename E, int NP>
void launch(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream) {
  const unsigned wgs = (unsigned)(d.P * d.G * d.B), grid = wgs * (unsigned)d.chunks;
  if (d.chunks > 1) {
    if (a.z.p)
      scan_bwd_part<E, NP, true><<<grid - wgs, kScanThreads, 0, stream>>>(a);
    else
      scan_bwd_part<E, NP, false><<<grid - wgs, kScanThreads, 0, stream>>>(a);
    if (!d.fold) {
      const int64_t n = d.B * d.D * d.NP;
      scan_join<false><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(
          a.edge, a.dtsum, a.a, a.gstate, d.B * d.D, a.D, a.N, d.NP, a.chunks, a.softplus);
    }
  }
  int parts = a.chunks;  // partial sums of A's gradient a row
  if constexpr (NP <= 16) {
    if (d.waves) parts = kScanBwdTW;
    if (d.waves) launch_main<E, NP, kScanBwdTW>(grid, a, stream);
  }
  if (!d.waves) launch_main<E, NP, 1>(grid, a, stream);
  const int64_t bc = d.T * d.B * d.G * 2 * d.NP, ae = d.D * (d.NP + 2);
  const unsigned a_wgs = (unsigned)((ae + 31) / 32);
  scan_sums<E><<<seq_grid(a_wgs + (bc + 255) / 256), 256, 0, stream>>>(a, d.NP, parts, a_wgs);
}

}  // namespace

template <typename E>
void scan_launch_backward(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream) {
  switch (d.NP) {
    case 8: return launch<E, 8>(d, a, stream);
    case 16: return launch<E, 16>(d, a, stream);
    case 32: return launch<E, 32>(d, a, stream);
    default: return launch<E, 64>(d, a, stream);
  }
}
template void scan_launch_backward<float>(const ScanDims&, const ScanArgs<float>&, hipStream_t);
template void scan_launch_backward<bf16_t>(const ScanDims&, const ScanArgs<bf16_t>&, hipStream_t);
template void scan_launch_backward<f16_t>(const ScanDims&, const ScanArgs<f16_t>&, hipStream_t);

}  // namespace ckhip
