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
constexpr int kGateFwdWaves = 8, kGateBwdWaves = 8;  // of a workgroup, at most
// Offsets from a window's first step are 32-bit bytes; a window of a single wave (16
// steps) reaches this far.
constexpr int64_t kGateMaxStrideT = (int64_t(1) << 26) - 1;

// How a call is spread over the chip.
struct GatePlan {
  int v;        // channels a lane
  int waves;    // of a workgroup
  int groups;   // of channels, in a row
  int chunks;   // of a row's steps
  int chunk;    // steps of a chunk, a multiple of a slot's unless there is one
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

// A gate s(v), held as the smaller of s(v) and s(-v) with its own relative error
// ((4 + 1.3 |v|) 2^-24), so that a gate that is almost open keeps what is missing from
// it.  Its sign bit is set where the gate is open (v > 0): `m` is what is missing.
struct Gate {
  float m;
  __device__ __forceinline__ bool open() const { return __builtin_bit_cast(int, m) < 0; }
  __device__ __forceinline__ float value() const { return open() ? 1.0f + m : m; }
  __device__ __forceinline__ float rest() const { return open() ? -m : 1.0f - m; }  // s(-v)
  __device__ __forceinline__ float slope() const { return fabsf(m) * (1.0f - fabsf(m)); }
  // 1 where the gate is open, else 0.
  __device__ __forceinline__ float keep() const {
    return __builtin_bit_cast(float, (__builtin_bit_cast(int, m) >> 31) & 0x3F800000);
  }
  // value() h + u: an open gate takes from h what it does not let through, so that
  // states neither leak by the rounding of a decay next to 1 nor keep what one next to
  // 0 should have taken.
  __device__ __forceinline__ float times(float h, float u) const {
    return fmaf(keep(), h, fmaf(m, h, u));
  }
};
constexpr Gate kGateKeep = {-0.0f};  // the decay of a step that changes nothing
// The gate at -nv.
__device__ __forceinline__ Gate gate_hw(float nv) {
  const float e = exp2_hw(-kLog2e * fabsf(nv));
  return Gate{__builtin_copysignf(e * rcp_hw(1.0f + e), nv)};
}

// The rows of one tensor from a window's first step on: an address that the whole
// wave shares and 32-bit offsets.
template <typename E>
struct GateRows {
  using Raw = std::remove_const_t<E>;
  char* base;
  uint32_t step;  // bytes
  __device__ __forceinline__ GateRows(const Seq<E>& s, int64_t t, int64_t b, int64_t c)
      : base(reinterpret_cast<char*>(const_cast<Raw*>(s.row(t, b) + c))),
        step((uint32_t)s.st * (uint32_t)sizeof(E)) {}
  __device__ __forceinline__ E* at(uint32_t offset) const {
    return reinterpret_cast<E*>(base + offset);
  }
  // The next step, as the wave's address.
  __device__ __forceinline__ void next() { base += step; }
};
// An offset that the compiler computes where it is used: one that it carries through a
// loop it carries as a 64-bit address a lane, for each of a tile's rows.
__device__ __forceinline__ uint32_t gate_offset(uint32_t o) {
  asm volatile("" : "+v"(o));
  return o;
}

// Where a thread stands: its slot, its channels and its row.  Lanes whose channels pass
// the row's end have them begin earlier: some channels are worked on in two lanes, which
// come to the same bits and store them both.
template <int V>
struct GateSpot {
  int wave, waves, lane, upper;  // upper: the wave's second slot
  int group, chunk, b, len;      // len: steps of the row that hold text
  int64_t c, c0;                 // first channel loaded, and of the workgroup's
  int cl;                        // c - c0

  template <typename A>
  __device__ __forceinline__ bool at(const A& s, int64_t id, int chunks) {
    // (groups, rows and chunks together are below 2^31: rows times channels below 2^36)
    const uint32_t r = (uint32_t)id / (uint32_t)s.groups;
    group = (int)((uint32_t)id - r * (uint32_t)s.groups);
    chunk = (int)(r / (uint32_t)s.B);
    b = (int)(r - (uint32_t)chunk * (uint32_t)s.B);
    if (chunk >= chunks) return false;
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    waves = (int)blockDim.x >> 6;
    lane = (int)threadIdx.x & (kGateLanes - 1);
    upper = ((int)threadIdx.x >> 5) & 1;
    const int64_t want = ((int64_t)group * kGateLanes + lane) * V;
    c = min(want, (int64_t)s.D - V);
    c0 = min((int64_t)group * kGateLanes * V, (int64_t)s.D - V);
    cl = (int)(c - c0);
    len = s.lengths ? max(0, min(s.lengths[b], s.T)) : s.T;
    return true;
  }
};

template <int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) GateWord {
  uint32_t bits;
};

// kGateStep rows of one tensor at a slot's channels.  Steps behind a row's text load
// its last step instead: a load without branches can stay in flight over the work on
// the tile before.
template <typename E, int V>
struct GateTile {
  static_assert(sizeof(E) * V <= 4, "a lane's channels are held as one register's bits");
  uint32_t v[kGateStep];

  // Channel j of step k.
  __device__ __forceinline__ float get(int k, int j) const {
    if constexpr (std::is_same_v<E, float>) return __builtin_bit_cast(float, v[k]);
    else if constexpr (std::is_same_v<E, bf16_t>)
      return __builtin_bit_cast(float, j ? v[k] & 0xFFFF0000u : v[k] << 16);
    else return (float)__builtin_bit_cast(E, (uint16_t)(j ? v[k] >> 16 : v[k]));
  }

  // Steps from + k of the window that begins at step t, the last of them `last` (>= 0).
  // ALL: they all come before it.
  template <bool ALL>
  __device__ __forceinline__ void load(const Seq<const E>& s, const GateSpot<V>& at, int t,
                                       int from, int last) {
    GateRows<const E> rows(s, t, at.b, at.c0);
    uint32_t o = gate_offset((uint32_t)(ALL ? from : min(from, last)) * rows.step +
                             (uint32_t)at.cl * (uint32_t)sizeof(E));
#pragma unroll
    for (int k = 0; k < kGateStep; ++k) {
      if constexpr (sizeof(E) * V == 4)
        v[k] = reinterpret_cast<const GateWord<alignof(E)>*>(rows.at(o))->bits;
      else
        v[k] = *reinterpret_cast<const uint16_t*>(rows.at(o));
      if constexpr (ALL) rows.next();
      else o += from + k < last ? rows.step : 0;
    }
  }
};

// The pair (product of a, state) of some steps.
template <int V>
struct alignas(8 * V) GatePair {
  float p[V], h[V];
};

// Where the slots of a workgroup meet.  Both take turns, so that one barrier a window
// is enough.
template <int V, int WAVES>
struct GateMeet {
  GatePair<V> pair[2][WAVES][kGateLanes];   // of each wave
  GatePair<V> carry[2][kGateLanes];         // h: the state before a window; p: see gate_fold
};

// Folds the pairs of a workgroup's slots.  Forward in time (REVERSE: backward).
// Returns the state before the thread's slot; the wave that comes last leaves the state
// behind the window as the next one's carry, and with it the product of all decays so
// far.  (The first carry is written before the first window.)
template <bool REVERSE, int V, int WAVES>
__device__ __forceinline__ void gate_fold(GateMeet<V, WAVES>& meet, int turn, const GateSpot<V>& at,
                                          const GatePair<V>& mine, float (&in)[V]) {
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
  if (!at.upper) meet.pair[turn][at.wave][at.lane] = both;
  __syncthreads();
  GatePair<V> c = meet.carry[turn][at.lane];
  const int rank = REVERSE ? at.waves - 1 - at.wave : at.wave;
#pragma unroll 4
  for (int k = 0; k < rank; ++k) {
    const GatePair<V> one = meet.pair[turn][REVERSE ? at.waves - 1 - k : k][at.lane];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      c.h[j] = fmaf(one.p[j], c.h[j], one.h[j]);
      c.p[j] *= one.p[j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) in[j] = second ? fmaf(other.p[j], c.h[j], other.h[j]) : c.h[j];
  if (rank == at.waves - 1 && !at.upper) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      c.h[j] = fmaf(both.p[j], c.h[j], both.h[j]);
      c.p[j] *= both.p[j];
    }
    meet.carry[turn ^ 1][at.lane] = c;
  }
}

// Leaves a chunk's pair to the launch that follows.
template <int V, typename A>
__device__ __forceinline__ void gate_sum_store(const A& s, const GateSpot<V>& at,
                                               const GatePair<V>& pair) {
  float* to = s.sums + ((int64_t)at.chunk * s.B * s.D + (int64_t)at.b * s.D + at.c) * 2;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    to[2 * j] = pair.p[j];
    to[2 * j + 1] = pair.h[j];
  }
}

template <typename E>
ck_status gate_run_forward(const GateArgs<E>& a, const GatePlan& p, hipStream_t stream);
// g_f, g_i: gradients of the biases, or NULL.
template <typename E>
ck_status gate_run_backward(const GateArgs<E>& a, const GatePlan& p, float* g_f, float* g_i,
                            hipStream_t stream);

}  // namespace ckhip
