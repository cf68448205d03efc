// scan.h -- sizes, arguments and device code shared by the two directions of
// the selective scan (scan.hip: entry points and single-token step;
// scan_forward.hip, scan_backward.hip: the kernels over windows).
//
//   dt_t = softplus(delta_t + bias)      a_t = exp(dt_t A)
//   h_t  = a_t h_{t-1} + dt_t B_t u_t    y_t = C_t . h_t + D u_t    out = y silu(z)
//
// Work split.  Four adjacent lanes (a quad) own one channel, each of them NL
// of its N states, and walk the steps in tiles of K.  The per-channel work of
// a step (loads, softplus, gate, store) is done by one lane of the quad: lane
// q takes step 4i + q of a tile and the quad reads dt and dt u of the others
// through DPP, so that work is not repeated four times.
//
// Few rows leave most of the chip idle, so the window is then cut into chunks
// that run side by side: a first launch finds what each chunk makes of a zero
// state (and the sum of its dt, from which its decay exp(A sum dt) follows), a
// small one joins these to every chunk's entering state, and the main launch
// starts each chunk from it.  The backward does the same with its adjoint
// from the other end.
#pragma once

#include <hip/hip_runtime.h>

#include "ck.h"
#include "ck_internal.h"
#include "sequence.h"

namespace ckhip {

constexpr int kScanThreads = 256;             // 4 waves
constexpr int kScanChan = kScanThreads / 4;   // channels per workgroup
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
  int64_t chunks, chunk_steps;  // chunks of the window (steps: a multiple of K)
};

template <typename E>
struct ScanArgs {
  Seq<const E> u, delta, b, c, z;
  const float *a, *d, *delta_bias, *state0;
  const int32_t* lengths;
  int T, B, D, N, G, Dg, P;
  int chunks, chunk_steps;
  int softplus;
  // [chunks][B][D][NP]: what a chunk makes of a zero state (adjoint), then
  // the state (adjoint) it starts from; and the sum of its dt, [chunks][B][D]
  float *edge, *dtsum;
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

// What a workgroup computes: channels [g Dg + blk 64, ...) of row b over the
// steps [t0, t1) of its chunk, of which the row's text covers those up to te.
struct Place {
  int b, g, blk, chunk;
  int t0, t1, te, len;
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
  i /= s.G;
  p.b = i % s.B;
  p.chunk = i / s.B;
  p.q = threadIdx.x & 3;
  const int dg = p.blk * kScanChan + (int)(threadIdx.x >> 2);
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
  // element `ahead` steps after the lane's, or of step `last` of the tile if
  // that comes first
  __device__ __forceinline__ E load(int ahead, uint32_t limit) const {
    return *reinterpret_cast<const E*>(tile + min(off + (uint32_t)ahead * step, limit));
  }
  __device__ __forceinline__ E* at(int ahead) const {
    using M = std::remove_const_t<E>;
    return reinterpret_cast<M*>(const_cast<char*>(tile) + (off + (uint32_t)ahead * step));
  }
};

template <int NL>
using StatesV = float __attribute__((ext_vector_type(NL)));

template <int NL>
__device__ __forceinline__ void load_vec(float (&v)[NL], const float* p) {
  const StatesV<NL> w = *reinterpret_cast<const StatesV<NL>*>(p);
#pragma unroll
  for (int k = 0; k < NL; ++k) v[k] = w[k];
}
template <int NL>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[NL]) {
  StatesV<NL> w;
#pragma unroll
  for (int k = 0; k < NL; ++k) w[k] = v[k];
  *reinterpret_cast<StatesV<NL>*>(p) = w;
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

// One thread's share of a tile's B and C (fp32 [K][NP] in LDS, 0 past the
// text's end or N): step threadIdx.x / NP, state threadIdx.x % NP.
template <typename E, int K, int NP>
struct TileBC {
  Walk<const E> b, c;
  bool mine;
  int ts;
  E vb, vc;
  bool in;

  __device__ __forceinline__ TileBC(const ScanArgs<E>& s, const Place& p, int t)
      : b(s.b, t, p.b, (int)threadIdx.x / NP,
          p.g * s.N + min((int)threadIdx.x % NP, s.N - 1)),
        c(s.c, t, p.b, (int)threadIdx.x / NP,
          p.g * s.N + min((int)threadIdx.x % NP, s.N - 1)),
        mine((int)threadIdx.x < K * NP && (int)threadIdx.x % NP < s.N),
        ts((int)threadIdx.x / NP) {}
  // last: the last step of the text, relative to the tile
  __device__ __forceinline__ void load(const ScanArgs<E>&, int last) {
    in = mine && ts <= last;
    if (in) {
      vb = *b.at(0);
      vc = *c.at(0);
    }
  }
  __device__ __forceinline__ void advance(int steps) {
    b.advance(steps);
    c.advance(steps);
  }
  __device__ __forceinline__ void store(float* sb, float* sc) const {
    if ((int)threadIdx.x >= K * NP) return;
    sb[threadIdx.x] = in ? (float)vb : 0.0f;
    sc[threadIdx.x] = in ? (float)vc : 0.0f;
  }
};

// Offset of step `last` of a tile, for Walk::load.
template <typename W>
__device__ __forceinline__ uint32_t walk_limit(const W& w, int q, int last) {
  // the lane's own offset is q steps into the tile
  return last >= scan_tile(1) ? 0xFFFFFFFFu : w.off + (uint32_t)(last - q) * w.step;
}

template <typename E>
__device__ __forceinline__ void zero_steps(const Seq<E>& s, const Place& p) {
  if (!p.active) return;
  for (int t = max(p.t0, p.len) + p.q; t < p.t1; t += 4) s.row(t, p.b)[p.d] = (E)0.0f;
}

// Joins the chunks: edge[c] from "made of a zero state" to "starts from".
// FORWARD walks up from state0, else down from the state's gradient.
template <bool FORWARD>
__global__ __launch_bounds__(256) void scan_join(float* edge, const float* dtsum, const float* A,
                                                 const float* first, int64_t rows, int D, int N,
                                                 int NP, int chunks) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * NP) return;
  const int n = (int)(i % NP);
  const int64_t row = i / NP;
  const float a2 = n < N ? kLog2e * A[row % D * N + n] : 0.0f;
  float cur = first && n < N ? first[row * N + n] : 0.0f;
  for (int k = 0; k < chunks; ++k) {
    const int c = FORWARD ? k : chunks - 1 - k;
    const int64_t at = (int64_t)c * rows;
    // the chunk that no other follows has no summary
    const bool more = k + 1 < chunks;
    const float made = more ? edge[at * NP + i] : 0.0f, dt = more ? dtsum[at + row] : 0.0f;
    edge[at * NP + i] = cur;
    cur = fmaf(exp2_hw(a2 * dt), cur, made);
  }
}

}  // namespace ckhip
