// scan.h -- sizes, arguments and device code shared by the two directions of
// the selective scan (scan.hip: entry points and single-token step;
// scan_forward.hip, scan_backward.hip: the kernels over windows).
//
//   dt_t = softplus(delta_t + bias)      a_t = exp(dt_t A)
//   h_t  = a_t h_{t-1} + dt_t B_t u_t    y_t = C_t . h_t + D u_t    out = y silu(z)
//
// Layout.  A wave owns 16 channels and walks the steps in tiles of K: lane
// (c, q) = (lane % 16, lane / 16) holds states 16 m + R q + r (r < R, m < M) of
// channel c; R = 4, but 2 for up to 8 states (2048 steps x 8 x 2048 channels x 8
// states: 193 + 343 us against 212 + 495 with half of each lane's states empty).  The per-channel work of a step (loads, softplus, gate, store) is
// done once, by the lane (c, q) with t % 4 = q, and the channel's other lanes
// read its dt and dt u from LDS, four steps an access.  What bounds the kernels
// is the vector ALU: exponentials take 8.5 cycles a wave, plain fp32
// operations 2.7 to 4, exchanges and selects 4.4.  (The outer product dt u x B
// as fp32 matrix instructions was slower: they keep the vector ALU waiting,
// 36 cycles for 4 products a lane.)
//
// Waves.  A SIMD issues to several waves better than to one, so where rows give
// it only one, a workgroup works on TW tiles at once, 4 waves each: every wave
// finds what its tile makes of a zero state, the waves fold these through LDS
// into the state each tile starts from, and every wave goes over its tile from
// there with the decays it holds in registers.
//
// Still fewer rows leave most of the chip idle, and the window is then cut into
// chunks that run side by side: a first launch finds what each chunk makes of a zero
// state (and the sum of its dt, from which its decay exp(A sum dt) follows), and the
// main launch starts each chunk from what those before it make of the window's first
// state.  It folds them itself where they are few, or finds them joined by a small
// launch between the two.  The backward does the same with its adjoint from
// the other end.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "ck.h"
#include "ck_internal.h"
#include "sequence.h"

namespace ckhip {

constexpr int kScanChan = 64;                 // channels per workgroup
constexpr int kScanThreads = 4 * kScanChan;   // threads per time tile (4 waves)
// Time tiles a workgroup works on at once where it works on several: what the
// registers allow (forward 126 of 128 at 16 waves, backward 216 of 256 at 8).
constexpr int kScanFwdTW = 4, kScanBwdTW = 2;
constexpr int64_t kScanMaxN = 64;

// Steps per tile for NP padded states: a lane of the backward holds a_t and
// h_{t-1} of a whole tile in registers (K NP / 2 values).
constexpr int scan_tile(int NP) { return NP <= 16 ? 8 : 4; }
// States are padded to NP = 8, 16, 32 or 64, in blocks of scan_lane states on
// each of a wave's 4 rows of lanes.
constexpr int scan_lane(int NP) { return NP < 16 ? NP / 4 : 4; }
constexpr int scan_blocks(int NP) { return NP < 16 ? 1 : NP / 16; }

// Sizes that both directions share.
struct ScanDims {
  int64_t T, B, D, N, G;
  int NP, K;        // padded states, steps per tile
  int64_t Dg, P;    // channels per group, workgroups per group
  int64_t tiles;    // tiles of the window
  int64_t chunks, chunk_steps;  // chunks of the window (steps: a multiple of K)
  bool waves;       // several time tiles a workgroup (one chunk only)
  bool fold;        // each chunk folds those before it; no launch joins them
};

template <typename E>
struct ScanArgs {
  Seq<const E> u, delta, b, c, z;
  const float *a, *d, *delta_bias, *state0;
  const int32_t* lengths;
  int T, B, D, N, G, Dg, P;
  int chunks, chunk_steps;
  int softplus;
  // [chunks][B][D][NP]: what a chunk makes of a zero state (adjoint), then, joined,
  // the state (adjoint) it starts from; and the sum of its dt, [chunks][B][D]
  float *edge, *dtsum;
  int fold;  // whether each chunk sees to that itself
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
  Seq<E> gb, gc;
  float *ga, *gd, *gbias;
};

template <typename E>
void scan_launch_forward(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream);
template <typename E>
void scan_launch_backward(const ScanDims& d, const ScanArgs<E>& a, hipStream_t stream);

// What a wave computes: 16 of channels [g Dg + blk 64, ...) of row b over the
// steps [t0, t1) of its chunk, of which the row's text covers those up to te.
struct Place {
  int b, g, blk, chunk;
  int t0, t1, te, len;
  int tw;       // the wave's tile among the workgroup's
  int c, q;     // lane: channel of the wave, and its row of lanes
  int wc;       // channel of the workgroup
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
  i /= s.G;
  p.b = i % s.B;
  p.chunk = i / s.B;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  p.tw = wave >> 2;
  p.c = threadIdx.x & 15;
  p.q = (threadIdx.x & 63) >> 4;
  p.wc = (wave & 3) * 16 + p.c;
  const int dg = p.blk * kScanChan + p.wc;
  p.active = dg < s.Dg;
  p.d = p.g * s.Dg + min(dg, s.Dg - 1);
  p.len = s.T;
  if (s.lengths) p.len = min(max(s.lengths[p.b], 0), s.T);
  p.t0 = p.chunk * s.chunk_steps;
  p.t1 = min(p.t0 + s.chunk_steps, s.T);
  p.te = min(p.t1, p.len);
  return p;
}

// Walks one tensor's rows tile by tile: a uniform pointer to the tile's first
// step and the lane's 32-bit byte offset of its own first step in it.
template <typename E>
struct Walk {
  const char* tile;
  uint32_t off;
  uint32_t step;  // bytes between steps

  __device__ __forceinline__ Walk(const Seq<E>& s, int t, int b, int lane_step, int channel)
      : tile(reinterpret_cast<const char*>(s.row(t, b))),
        off((uint32_t)(lane_step * (uint32_t)s.st + (uint32_t)channel) * (uint32_t)sizeof(E)),
        step((uint32_t)s.st * (uint32_t)sizeof(E)) {}
  __device__ __forceinline__ void advance(int steps) { tile += (int64_t)steps * (int64_t)step; }
  // The lane's elements of a tile of 4 KQ steps whose last with text is `last`;
  // past it, that step's.  (A uniform branch: selects of the offsets instead
  // cost a tenth of the forward's vector ALU time.)
  template <int KQ>
  __device__ __forceinline__ void load(std::remove_const_t<E> (&v)[KQ], int q, int last) const {
    if (last >= 4 * KQ - 1) {
#pragma unroll
      for (int i = 0; i < KQ; ++i)
        v[i] = *reinterpret_cast<const E*>(tile + (off + (uint32_t)(4 * i) * step));
    } else {
      const uint32_t most = off + (uint32_t)(last - q) * step;
#pragma unroll
      for (int i = 0; i < KQ; ++i)
        v[i] = *reinterpret_cast<const E*>(tile + min(off + (uint32_t)(4 * i) * step, most));
    }
  }
  __device__ __forceinline__ E* at(int ahead) const {
    using X = std::remove_const_t<E>;
    return reinterpret_cast<X*>(const_cast<char*>(tile) + (off + (uint32_t)ahead * step));
  }
};

using f32x4 = float __attribute__((ext_vector_type(4)));
using f32x2 = float __attribute__((ext_vector_type(2)));

// The lane's states: States<NP>[M], block m holding states 16 m + R q + r.
template <int NP>
using States = std::conditional_t<scan_lane(NP) == 4, f32x4, f32x2>;

template <int NP>
__device__ __forceinline__ void load_rows(States<NP> (&v)[scan_blocks(NP)], const float* p, int q) {
#pragma unroll
  for (int m = 0; m < scan_blocks(NP); ++m)
    v[m] = *reinterpret_cast<const States<NP>*>(p + 16 * m + scan_lane(NP) * q);
}
template <int NP>
__device__ __forceinline__ void store_rows(float* p, const States<NP> (&v)[scan_blocks(NP)],
                                           int q) {
#pragma unroll
  for (int m = 0; m < scan_blocks(NP); ++m)
    *reinterpret_cast<States<NP>*>(p + 16 * m + scan_lane(NP) * q) = v[m];
}
// From and to [rows][N] arrays of the caller (N need not be padded); 0 if absent.
template <int NP>
__device__ __forceinline__ void load_states(States<NP> (&v)[scan_blocks(NP)], const float* s,
                                            int64_t row, int q, int N) {
#pragma unroll
  for (int m = 0; m < scan_blocks(NP); ++m)
#pragma unroll
    for (int r = 0; r < scan_lane(NP); ++r) {
      const int n = 16 * m + scan_lane(NP) * q + r;
      v[m][r] = s && n < N ? s[row * N + n] : 0.0f;
    }
}
// A rate of the decays as the kernels hold it: an infinite one (a state that
// forgets everything) counts as the largest here, whose product with log2 e is
// finite, so that steps past the text, with dt = 0, have the decay 1 and not
// exp(0 inf).  (From dt = 1e-36 on the decay of such a state is 0 all the same.)
__device__ __forceinline__ float scan_rate(float a) {
  constexpr float kMax = 2e38f;
  return fabsf(a) > kMax ? copysignf(kMax, a) : a;
}
template <int NP>
__device__ __forceinline__ void load_rates(States<NP> (&v)[scan_blocks(NP)], const float* A, int d,
                                           int q, int N) {
  load_states<NP>(v, A, d, q, N);
#pragma unroll
  for (int m = 0; m < scan_blocks(NP); ++m)
#pragma unroll
    for (int r = 0; r < scan_lane(NP); ++r) v[m][r] = scan_rate(v[m][r]);
}
template <int NP>
__device__ __forceinline__ void store_states(const States<NP> (&v)[scan_blocks(NP)], float* s,
                                             int64_t row, int q, int N) {
#pragma unroll
  for (int m = 0; m < scan_blocks(NP); ++m)
#pragma unroll
    for (int r = 0; r < scan_lane(NP); ++r) {
      const int n = 16 * m + scan_lane(NP) * q + r;
      if (n < N) s[row * N + n] = v[m][r];
    }
}

template <typename V>
__device__ __forceinline__ V exp2_v(V x) {
  V y;
#pragma unroll
  for (int r = 0; r < (int)(sizeof(V) / 4); ++r) y[r] = exp2_hw(x[r]);
  return y;
}
template <typename V>
__device__ __forceinline__ V fma_v(V a, V b, V c) {
  V y;
#pragma unroll
  for (int r = 0; r < (int)(sizeof(V) / 4); ++r) y[r] = fmaf(a[r], b[r], c[r]);
  return y;
}

// sum of a[r] b[r] added to c, one operation a state
template <typename V>
__device__ __forceinline__ float dot_add(V a, V b, float c) {
#pragma unroll
  for (int r = 0; r < (int)(sizeof(V) / 4); ++r) c = fmaf(a[r], b[r], c);
  return c;
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
// Row q of the lanes gets v[q] summed over the four rows (a channel's states).
__device__ __forceinline__ float rows_reduce4(const float (&v)[4]) {
  return swap16_add(swap32_add(v[0], v[2]), swap32_add(v[1], v[3]));
}
__device__ __forceinline__ float rows_sum(float x) {
  return swap16_add(swap32_add(x, x), swap32_add(x, x));
}

// Orders a wave's LDS accesses through which its lanes exchange values.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave's exchange of one value a step and channel: lane (c, q) puts its steps
// 4 i + q, all rows read four steps at once.  12 floats a channel keep the 16
// channels' reads on different banks.
struct StepsLds {
  static constexpr int kStride = 12, kFloats = 16 * kStride;
  static __device__ __forceinline__ void put(float* p, int c, int q, int i, float v) {
    p[c * kStride + 4 * i + q] = v;
  }
  static __device__ __forceinline__ f32x4 get(const float* p, int c, int i) {
    return *reinterpret_cast<const f32x4*>(p + c * kStride + 4 * i);
  }
};

// The workgroup's B and C over its KT steps as fp32 rows [KT][NP] in LDS, 0 past
// the text's end or N.  A thread moves one value of B or of C (NP < 64; with 8 half
// of them move none), or one of each: loaded a tile ahead, stored behind the tile before.
template <typename E, int NP, int TW>
struct TileBC {
  static constexpr int KT = scan_tile(NP) * TW, kRows = KT * NP;
  static constexpr int kThreads = kScanThreads * TW;
  static constexpr bool kBoth = kRows == kThreads;
  static_assert(kBoth || 2 * kRows <= kThreads, "each thread has its share");

  const char *b, *c;   // the tiles' first step (uniform)
  uint32_t bo, co;     // the thread's byte offsets from it
  uint32_t bstep, cstep;
  int ts, e;           // its step of the tiles, its place in LDS
  bool mine, is_c, spare;
  E vb, vc;

  __device__ __forceinline__ TileBC(const ScanArgs<E>& s, const Place& p, int t) {
    const int tid = threadIdx.x;
    // (uniform: a wave moves values of B or of C)
    is_c = !kBoth && __builtin_amdgcn_readfirstlane(tid) >= kRows;
    spare = !kBoth && __builtin_amdgcn_readfirstlane(tid) >= 2 * kRows;
    e = kBoth ? tid : tid % kRows;
    ts = e / NP;
    const int n = e % NP;
    mine = n < s.N;
    const uint32_t at = (uint32_t)(p.g * s.N + min(n, s.N - 1)) * (uint32_t)sizeof(E);
    const Seq<const E>& first = is_c ? s.c : s.b;
    bstep = (uint32_t)first.st * (uint32_t)sizeof(E);
    cstep = (uint32_t)s.c.st * (uint32_t)sizeof(E);
    b = reinterpret_cast<const char*>(first.row(t, p.b));
    c = reinterpret_cast<const char*>(s.c.row(t, p.b));
    bo = (uint32_t)ts * bstep + at;
    co = (uint32_t)ts * cstep + at;
    vb = vc = (E)0.0f;
  }
  __device__ __forceinline__ void advance(int steps) {
    b += (int64_t)steps * (int64_t)bstep;
    if constexpr (kBoth) c += (int64_t)steps * (int64_t)cstep;
  }
  // last: the last step of the text, relative to the tiles' first
  __device__ __forceinline__ void load(int last) {
    if (NP < 16 && spare) return;
    if (last >= KT - 1) {
      vb = *reinterpret_cast<const E*>(b + bo);
      if constexpr (kBoth) vc = *reinterpret_cast<const E*>(c + co);
    } else {
      vb = vc = (E)0.0f;
      if (ts <= last) {
        vb = *reinterpret_cast<const E*>(b + bo);
        if constexpr (kBoth) vc = *reinterpret_cast<const E*>(c + co);
      }
    }
  }
  // rows: [2][KT][NP], B then C
  __device__ __forceinline__ void store(float* rows) const {
    if (NP < 16 && spare) return;
    rows[(is_c ? kRows : 0) + e] = mine ? (float)vb : 0.0f;
    if constexpr (kBoth) rows[kRows + e] = mine ? (float)vc : 0.0f;
  }
};

template <typename E>
__device__ __forceinline__ void zero_steps(const Seq<E>& s, const Place& p) {
  if (!p.active) return;
  for (int t = max(p.t0, p.len) + p.q; t < p.t1; t += 4) s.row(t, p.b)[p.d] = (E)0.0f;
}

// Decays over many steps at once.  Where a state can grow (A > 0, or negative steps
// without softplus) such a decay may pass fp32's range although the state behind it
// does not: a zero state stays zero however many steps it is kept for.  So it is
// applied as its square root, twice, each at most 2^127: within range for every
// normal state that stays in range itself.
// (Only there: applied to all, roots cost a window's backward 3 % and prompts of many
// chunks and few rows a tenth, 1150 steps x 2 x 109 channels 18.5 -> 20.3 us.)
constexpr float kMaxRoot = 0x1p127f;
// Whether states of the wave can grow: the same for all waves of its channels.
template <int NP>
__device__ __forceinline__ bool scan_grows(const States<NP> (&a)[scan_blocks(NP)], int softplus) {
  bool up = !softplus;
#pragma unroll
  for (int m = 0; m < scan_blocks(NP); ++m)
#pragma unroll
    for (int r = 0; r < scan_lane(NP); ++r) up = up || a[m][r] > 0.0f;
  return __builtin_amdgcn_ballot_w64(up) != 0;
}
// A tile's decay as fold_tiles takes it: its root (not bounded yet) where a state can
// grow, else the decay itself.
template <typename V>
__device__ __forceinline__ V tile_decay(float dt, V a2, bool grows) {
  return exp2_v((grows ? 0.5f * dt : dt) * a2);
}

// Folds what TW tiles make of a zero state (made) and their decays into the
// state the wave's tile starts from; next: the state behind the last of them.
// FORWARD runs up from `start`, else down.  ROOTS: the decays are roots.
template <int NP, int TW, bool FORWARD, bool ROOTS>
__device__ __forceinline__ void fold_tiles_by(States<NP> (&start)[scan_blocks(NP)],
                                              States<NP> (&next)[scan_blocks(NP)],
                                              const float* made, const float* decay,
                                              const Place& p) {
  constexpr int M = scan_blocks(NP);
  States<NP> cur[M];
#pragma unroll
  for (int m = 0; m < M; ++m) cur[m] = start[m];
#pragma unroll
  for (int i = 0; i < TW; ++i) {
    const int w = FORWARD ? i : TW - 1 - i;
    States<NP> mw[M], ew[M];
    load_rows<NP>(mw, made + (w * kScanChan + p.wc) * NP, p.q);
    load_rows<NP>(ew, decay + (w * kScanChan + p.wc) * NP, p.q);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (w == p.tw) start[m] = cur[m];
      if constexpr (ROOTS) {
#pragma unroll
        for (int r = 0; r < scan_lane(NP); ++r) ew[m][r] = fminf(ew[m][r], kMaxRoot);
        cur[m] = fma_v(ew[m], ew[m] * cur[m], mw[m]);
      } else {
        cur[m] = fma_v(ew[m], cur[m], mw[m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m) next[m] = cur[m];
}
template <int NP, int TW, bool FORWARD>
__device__ __forceinline__ void fold_tiles(States<NP> (&start)[scan_blocks(NP)],
                                           States<NP> (&next)[scan_blocks(NP)], const float* made,
                                           const float* decay, const Place& p, bool grows) {
  if (grows)
    fold_tiles_by<NP, TW, FORWARD, true>(start, next, made, decay, p);
  else
    fold_tiles_by<NP, TW, FORWARD, false>(start, next, made, decay, p);
}

// The root of a decay, or the decay itself where no state of the wave can grow, and
// a state kept by it.
template <bool ROOTS>
__device__ __forceinline__ float chunk_decay(float log2_decay) {
  return ROOTS ? fminf(exp2_hw(0.5f * log2_decay), kMaxRoot) : exp2_hw(log2_decay);
}
template <bool ROOTS>
__device__ __forceinline__ float decay_add(float decay, float h, float made) {
  return fmaf(decay, ROOTS ? decay * h : h, made);
}

// The state a chunk starts from, or (not FORWARD) the adjoint: the window's first,
// in h, folded with what the chunks walked before this one make of zero.  The
// same sums as scan_join's, in the same order.
template <int NP, bool FORWARD, bool ROOTS, typename E>
__device__ __forceinline__ void fold_chunks_by(States<NP> (&h)[scan_blocks(NP)],
                                               const States<NP> (&a2)[scan_blocks(NP)],
                                               const ScanArgs<E>& s, const Place& p, int64_t row) {
  constexpr int M = scan_blocks(NP), kAhead = 8 / M;
  const int64_t rows = (int64_t)s.B * s.D;
  const int count = FORWARD ? p.chunk : s.chunks - 1 - p.chunk;
  for (int k0 = 0; k0 < count; k0 += kAhead) {
    States<NP> made[kAhead][M];
    float dt[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = min(k0 + j, count - 1);
      const int64_t at = (FORWARD ? k : s.chunks - 1 - k) * rows + row;
      load_rows<NP>(made[j], s.edge + at * NP, p.q);
      dt[j] = s.dtsum[at];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k0 + j < count) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int r = 0; r < scan_lane(NP); ++r)
            h[m][r] = decay_add<ROOTS>(chunk_decay<ROOTS>(dt[j] * a2[m][r]), h[m][r],
                                       made[j][m][r]);
      }
  }
}

template <int NP, bool FORWARD, typename E>
__device__ __forceinline__ void fold_chunks(States<NP> (&h)[scan_blocks(NP)],
                                            const States<NP> (&a2)[scan_blocks(NP)],
                                            const ScanArgs<E>& s, const Place& p, int64_t row) {
  if (scan_grows<NP>(a2, s.softplus))
    fold_chunks_by<NP, FORWARD, true>(h, a2, s, p, row);
  else
    fold_chunks_by<NP, FORWARD, false>(h, a2, s, p, row);
}

// Joins the chunks: edge[c] from "made of a zero state" to "starts from".
// FORWARD walks up from state0, else down from the state's gradient.
template <bool FORWARD, bool ROOTS>
__device__ __forceinline__ void scan_join_by(float* edge, const float* dtsum, float a2, float cur,
                                             int64_t row, int64_t i, int64_t rows, int NP,
                                             int chunks) {
  // in the order of the walk; the chunk that no other follows has no summary
  auto at = [&](int k) { return (int64_t)(FORWARD ? k : chunks - 1 - k) * rows; };
  for (int k0 = 0; k0 < chunks; k0 += 8) {
    float made[8], dt[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t from = at(min(k0 + j, max(chunks - 2, 0)));
      made[j] = edge[from * NP + i];
      dt[j] = dtsum[from + row];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k0 + j < chunks) {
        edge[at(k0 + j) * NP + i] = cur;
        cur = decay_add<ROOTS>(chunk_decay<ROOTS>(a2 * dt[j]), cur, made[j]);
      }
  }
}
template <bool FORWARD>
__global__ __launch_bounds__(256) void scan_join(float* edge, const float* dtsum, const float* A,
                                                 const float* first, int64_t rows, int D, int N,
                                                 int NP, int chunks, int softplus) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * NP) return;
  const int n = (int)(i % NP);
  const int64_t row = i / NP;
  const float a2 = n < N ? kLog2e * scan_rate(A[row % D * N + n]) : 0.0f;
  const float cur = first && n < N ? first[row * N + n] : 0.0f;
  if (__builtin_amdgcn_ballot_w64(!softplus || a2 > 0.0f) != 0)
    scan_join_by<FORWARD, true>(edge, dtsum, a2, cur, row, i, rows, NP, chunks);
  else
    scan_join_by<FORWARD, false>(edge, dtsum, a2, cur, row, i, rows, NP, chunks);
}

}  // namespace ckhip
