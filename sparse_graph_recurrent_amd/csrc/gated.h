// gated.h -- layout, tiles and gates of the gated scan (gated_forward.hip,
// gated_backward.hip, gated.hip).
//
//   a_t = s(f_t + fb),  q_t = 1 - a_t,  g_t = s(i_t + ib) or q_t
//   h_t = a_t h_{t-1} + g_t x_t,   y_t = h_t or h_t z_t s(z_t)        s(v) = 1 / (1 + exp(-v))
//
// A slot, half a wave, owns kGateStep steps of a group of channels that fills a
// 128-byte line (4 bytes a lane); the 2 W slots of a workgroup of W waves lie one
// behind the other in time and together make a window.  Each slot runs through its
// steps from a state of zero, which gives the pair (product of a, state) of its
// steps; the pairs are folded through LDS into the state before each slot, and the
// slot runs through its steps again, in registers, from there.  So every element is
// read once, whatever the number of waves over the time axis.
//
// Where rows and channels have too few groups for the chip, the steps are cut into
// chunks of workgroups of their own, and a launch before sums up every chunk but the
// one that nothing follows.
#pragma once

#include <hip/hip_runtime.h>

#include "ck.h"
#include "ck_internal.h"
#include "sequence.h"

namespace ckhip {

constexpr int kGateStep = 8;      // steps of a slot, and of a saved state
constexpr int kGateLanes = 32;    // lanes of a slot
constexpr int kGateMaxWaves = 16; // of a workgroup
// (a step's bytes, 4 an element and fewer, in 32 bits: see Rows)
constexpr int64_t kGateMaxStrideT = (int64_t(1) << 30) - 1;

// How a call is spread over the chip.
struct GatePlan {
  int v;        // channels a lane
  int waves;    // of a workgroup
  int groups;   // of channels, in a row
  int chunks;   // of a row's steps
  int chunk;    // steps of a chunk, a multiple of a window's unless there is one
};

template <typename E>
struct GateArgs {
  Seq<const E> x, f, i, z, go;
  Seq<E> out, gx, gf, gi, gz;
  const float *f_bias, *i_bias, *state0, *gstate;
  float *state, *gstate0;
  float* saved;       // [ceil(T / kGateStep)][B][D]: the state before each tile
  float* sums;        // [chunks - 1][B][D][2]: product of a and state (or adjoint) of a chunk
  float* part;        // [B][chunks][2][D]: sums of gf and gi
  const int32_t* lengths;
  int T, B, D, groups, chunks, chunk;
};

// The logistic function of v and of -v: `small` is that of -|v|, `big` that of |v|;
// each has its own relative error ((4 + 1.3 |v|) 2^-24 for the small one), so that a
// gate that is almost open keeps what is missing from it.
struct Gate {
  float small, big;
};
__device__ __forceinline__ Gate gate_hw(float v) {
  const float e = exp2_hw(-kLog2e * fabsf(v));
  const float r = rcp_hw(1.0f + e);
  return Gate{e * r, r};
}

// A step's decay: -q where a >= 1/2 and a where it is below (the sign bit tells), so
// that states neither leak by the rounding of an a next to 1 nor keep what an a next
// to 0 should have taken.
struct Decay {
  float m;
  __device__ __forceinline__ float times(float h, float u) const {  // a h + u
    const float kept = __builtin_bit_cast(
        float, __builtin_bit_cast(int, h) & (__builtin_bit_cast(int, m) >> 31));
    return kept + fmaf(m, h, u);
  }
};
constexpr float kKeep = -0.0f;  // Decay of a step that changes nothing

// The forget gate at v: the decay, q, and a.
struct Forget {
  Decay decay;
  float q, a;
};
__device__ __forceinline__ Forget forget_hw(float v) {
  const Gate g = gate_hw(v);
  const bool open = v >= 0.0f;
  return Forget{Decay{open ? -g.small : g.small}, open ? g.small : g.big,
                open ? g.big : g.small};
}

// kGateStep rows of one tensor at a slot's channels.
template <typename E, int V>
struct GateTile {
  Pack<E, V> v[kGateStep];

  // Rows t .. of which the first n exist for this lane (n <= 0: none).  A lane whose
  // channels pass the row's end has them begin earlier (`c` is the first it loads).
  __device__ __forceinline__ void load(const Seq<const E>& s, int64_t t, int64_t b, int64_t c,
                                       int n) {
    const Rows<const E> rows(s, t, b, c);
    if (__all(n >= kGateStep)) {
#pragma unroll
      for (int k = 0; k < kGateStep; ++k) v[k] = pack_load<true, E, V>(rows.at(k), V);
    } else {
#pragma unroll
      for (int k = 0; k < kGateStep; ++k) {
        v[k] = Pack<E, V>{};
        if (k < n) v[k] = pack_load<true, E, V>(rows.at(k), V);
      }
    }
  }
};

// Where a thread stands: its slot, its channels and its row.
template <int V>
struct GateSpot {
  int wave, waves, lane, upper;  // upper: the wave's second slot
  int group, chunk, b, len;      // len: steps of the row that hold text
  int64_t c;                     // first channel loaded
  int own;                       // the lane's own channels are c + own .. c + V - 1
  bool live;                     // it has any

  template <typename A>
  __device__ __forceinline__ bool at(const A& s, int64_t id, int chunks) {
    group = (int)(id % s.groups);
    const int64_t r = id / s.groups;
    b = (int)(r % s.B);
    chunk = (int)(r / s.B);
    if (chunk >= chunks) return false;
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    waves = (int)blockDim.x >> 6;
    lane = (int)threadIdx.x & (kGateLanes - 1);
    upper = ((int)threadIdx.x >> 5) & 1;
    const int64_t want = ((int64_t)group * kGateLanes + lane) * V;
    live = want < s.D;
    c = min(want, (int64_t)s.D - V);
    own = (int)min(want - c, (int64_t)V);
    len = s.lengths ? max(0, min(s.lengths[b], s.T)) : s.T;
    return true;
  }
};

// The lane's own channels of a packed result, to one row.
template <typename E, int V>
__device__ __forceinline__ void gate_store(E* p, const float (&y)[V], bool live, int own) {
  if (!live) return;
  if (own == 0) return pack_store<true, E, V>(p, y, V);
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (j >= own) p[j] = (E)y[j];
}

// The pair (product of a, state) of some steps.
template <int V>
struct alignas(8 * V) GatePair {
  float p[V], h[V];
};

// Folds the pairs of a workgroup's slots.  Forward in time (REVERSE: backward):
// `carry` is the state before the window and becomes the one behind it; returns the
// state before the thread's slot.  The buffer takes turns, so that one barrier a
// window is enough.
template <bool REVERSE, int V>
__device__ __forceinline__ void gate_fold(GatePair<V> (*lds)[kGateLanes], const GateSpot<V>& at,
                                          const GatePair<V>& mine, float (&carry)[V],
                                          float (&in)[V]) {
  GatePair<V> other, both;
  const bool second = REVERSE ? !at.upper : at.upper;  // behind the wave's other slot
#pragma unroll
  for (int j = 0; j < V; ++j) {
    other.p[j] = __shfl_xor(mine.p[j], 32);
    other.h[j] = __shfl_xor(mine.h[j], 32);
    both.p[j] = mine.p[j] * other.p[j];
    both.h[j] = second ? fmaf(mine.p[j], other.h[j], mine.h[j])
                       : fmaf(other.p[j], mine.h[j], other.h[j]);
  }
  if (!at.upper) lds[at.wave][at.lane] = both;
  __syncthreads();
  float h[V];
#pragma unroll
  for (int j = 0; j < V; ++j) h[j] = carry[j];
#pragma unroll 4
  for (int k = 0; k < at.waves; ++k) {
    const int w = REVERSE ? at.waves - 1 - k : k;
    const GatePair<V> one = lds[w][at.lane];
    if (w == at.wave) {
#pragma unroll
      for (int j = 0; j < V; ++j) in[j] = second ? fmaf(other.p[j], h[j], other.h[j]) : h[j];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = fmaf(one.p[j], h[j], one.h[j]);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) carry[j] = h[j];
}

template <typename E>
ck_status gate_run_forward(const GateArgs<E>& a, const GatePlan& p, hipStream_t stream);
// g_f, g_i: gradients of the biases, or NULL.
template <typename E>
ck_status gate_run_backward(const GateArgs<E>& a, const GatePlan& p, float* g_f, float* g_i,
                            hipStream_t stream);

}  // namespace ckhip
