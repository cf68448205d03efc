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
// A workgroup goes through all windows of its columns (a group of a row's channels).
// Where there are too few columns for the chip, every window has a workgroup of its own
// instead (gate_chain): it leaves its pair where the others see it, and takes the state
// before it from the pairs of the windows before, so that elements are still read once.
//
// HBM bounds long calls: three tensors are read and one is written for each 30 or so
// operations an element.  Measured (bf16): 2048 steps x 8 x 2048 with an output gate
// forward 84 us (4.2 TB/s), backward 123 (5.1 TB/s); a prompt of 16384 x 1 x 2048 82 us
// (4.1 TB/s; as a first pass over chunks and a second from their states, which reads
// twice, 117).  Short calls are bound by latency: 777 x 5 x 1001, fp16, of uneven rows,
// takes 12 and 21 us of its 42 in the two kernels, 2.2 TB/s.
#pragma once

#include <hip/hip_runtime.h>

#include "ck.h"
#include "ck_internal.h"
#include "sequence.h"

namespace ckhip {

constexpr int kGateStep = 8;      // steps of a slot, and of a saved state
constexpr int kGateLanes = 32;    // lanes of a slot
constexpr int kGateWaves = 8;     // of a workgroup, at most
// Offsets from a window's first step are 32-bit bytes; a window of a single wave (16
// steps) reaches this far.
constexpr int64_t kGateMaxStrideT = (int64_t(1) << 26) - 1;

// How a call is spread over the chip.
struct GatePlan {
  int v;        // channels a lane
  int waves;    // of a workgroup
  int groups;   // of channels, in a row
  int windows;  // that are workgroups of their own (1: a workgroup loops over all)
};

template <typename E>
struct GateArgs {
  Seq<const E> x, f, i, z, go;
  Seq<E> out, gx, gf, gi, gz;
  const float *f_bias, *i_bias, *state0, *gstate;
  float *state, *gstate0;
  float* saved;       // [ceil(T / kGateStep)][B][D]: the state before each tile
  float* part;        // [windows][B][2][D]: sums of gf and gi
  uint32_t* ticket;   // of a chain (gate_number), as are the words below
  uint64_t *pairs, *states;
  const int32_t* lengths;
  int T, B, D, groups, windows;
  int split;          // some column does not begin on a cache line
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
  int group, b, len;             // len: steps of the row that hold text
  int64_t c, c0;                 // first channel loaded, and of the workgroup's
  int cl;                        // c - c0

  // Column `id`.  (Groups times rows are below 2^31: rows times channels below 2^36.)
  template <typename A>
  __device__ __forceinline__ void at(const A& s, uint32_t id) {
    b = (int)(id / (uint32_t)s.groups);
    group = (int)(id - (uint32_t)b * (uint32_t)s.groups);
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    waves = (int)blockDim.x >> 6;
    lane = (int)threadIdx.x & (kGateLanes - 1);
    upper = ((int)threadIdx.x >> 5) & 1;
    const int64_t want = ((int64_t)group * kGateLanes + lane) * V;
    c = min(want, (int64_t)s.D - V);
    c0 = min((int64_t)group * kGateLanes * V, (int64_t)s.D - V);
    cl = (int)(c - c0);
    len = s.lengths ? max(0, min(s.lengths[b], s.T)) : s.T;
  }
};

// The column of the a-th of n workgroups that start together.  Where columns do not begin
// on cache lines (`split`), neighbours in a row are put on one XCD (workgroups are dealt
// to them in turn), so that the lines which two of them touch come to one cache: 2048
// steps x 8 x 2047, bf16, forward + backward 319 -> 232 us.  Where they do, columns dealt
// in turn are the better (x 2048: 223 us against 232).
__device__ __forceinline__ uint32_t gate_column(uint32_t a, uint32_t n, int split) {
  if (!split) return a;
  const uint32_t xcd = a % kResXcds, each = n / kResXcds, more = n % kResXcds;
  return xcd * each + min(xcd, more) + a / kResXcds;
}

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
  GatePair<V> pair[2][WAVES][kGateLanes];  // of each wave
  float carry[2][kGateLanes][V];           // the state before a window
};

// The pair of a wave's two slots, of the pair of the thread's; `other`: the wave's other
// slot's.
template <bool REVERSE, int V>
__device__ __forceinline__ GatePair<V> gate_both(const GateSpot<V>& at, const GatePair<V>& mine,
                                                 GatePair<V>& other) {
  GatePair<V> both;
  const bool second = REVERSE ? !at.upper : at.upper;  // behind the wave's other slot
#pragma unroll
  for (int j = 0; j < V; ++j) {
    other.p[j] = __shfl_xor(mine.p[j], 32);
    other.h[j] = __shfl_xor(mine.h[j], 32);
    both.p[j] = mine.p[j] * other.p[j];
    both.h[j] = second ? fmaf(mine.p[j], other.h[j], mine.h[j])
                       : fmaf(other.p[j], mine.h[j], other.h[j]);
  }
  return both;
}

// h: the state before a window; becomes that before the thread's slot.  Returns the
// state behind the wave's steps.
template <bool REVERSE, int V>
__device__ __forceinline__ GatePair<V> gate_through(const GatePair<V> (*pair)[kGateLanes],
                                                    const GateSpot<V>& at,
                                                    const GatePair<V>& both,
                                                    const GatePair<V>& other, float (&h)[V]) {
  const int rank = REVERSE ? at.waves - 1 - at.wave : at.wave;
#pragma unroll 4
  for (int k = 0; k < rank; ++k) {
    const GatePair<V> one = pair[REVERSE ? at.waves - 1 - k : k][at.lane];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = fmaf(one.p[j], h[j], one.h[j]);
  }
  GatePair<V> behind;
  const bool second = REVERSE ? !at.upper : at.upper;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    behind.h[j] = fmaf(both.p[j], h[j], both.h[j]);
    if (second) h[j] = fmaf(other.p[j], h[j], other.h[j]);
  }
  return behind;
}

// Folds the pairs of a workgroup's slots.  Forward in time (REVERSE: backward).
// Returns the state before the thread's slot; the wave that comes last leaves the state
// behind the window as the next one's carry.  (The first carry is written before the
// first window.)
template <bool REVERSE, int V, int WAVES>
__device__ __forceinline__ void gate_fold(GateMeet<V, WAVES>& meet, int turn, const GateSpot<V>& at,
                                          const GatePair<V>& mine, float (&in)[V]) {
  GatePair<V> other;
  const GatePair<V> both = gate_both<REVERSE>(at, mine, other);
  if (!at.upper) meet.pair[turn][at.wave][at.lane] = both;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < V; ++j) in[j] = meet.carry[turn][at.lane][j];
  const GatePair<V> behind = gate_through<REVERSE>(meet.pair[turn], at, both, other, in);
  if ((REVERSE ? at.wave == 0 : at.wave == at.waves - 1) && !at.upper) {
#pragma unroll
    for (int j = 0; j < V; ++j) meet.carry[turn ^ 1][at.lane][j] = behind.h[j];
  }
}

// Windows that are workgroups of their own.  Those of a column take their numbers by the
// column's ticket, in the order in which states pass (by time; in the backward against
// it): a workgroup waits only for such of its column with a lower number, which run
// already, so that every wait ends whatever else the chip runs and in whatever order
// workgroups start.  (One ticket for all columns: its additions, one after the other
// where the chip's parts meet, took longer than the work.)  Window number n
//   - leaves the pair of its steps, which needs no other window;
//   - takes the state before windows kGateRun (n / kGateRun) ..., and the pairs of those
//     between that one and itself;
//   - leaves the state behind it where the next run of windows begins.
// What is left is one 64-bit word a channel, complete in itself, written and read past
// the caches that are not common to the chip, so that no order of other accesses
// matters: a pair's product, never negative, and state; a state with a zero.  Before
// the launch all words hold kGateAbsent.  Runs have a fixed length: results do not go by
// who came first.  A wait of kGatePolls polls (seconds) gives up and goes on with NaN.
constexpr int kGateRun = 8;  // a wave each waits for one of the others, and for the state
constexpr uint64_t kGateAbsent = ~0ull;
constexpr int kGatePolls = 1 << 22;
constexpr int kGateTicket = 32;  // words between two columns' tickets: a cache line each

__device__ __forceinline__ void gate_leave(uint64_t* to, float p, float h) {
  const uint64_t w = (uint64_t)(__builtin_bit_cast(uint32_t, p) & 0x7FFFFFFFu) << 32 |
                     __builtin_bit_cast(uint32_t, h);
  __hip_atomic_store(to, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The words of a lane's channels; each lane of the wave waits for all of them.
template <int V>
__device__ __forceinline__ GatePair<V> gate_await(uint64_t* from) {
  uint64_t w[V];
  bool there = false;
  for (int poll = 0; poll < kGatePolls && !there; ++poll) {
    if (poll) __builtin_amdgcn_s_sleep(1);
    bool mine = true;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[j] = __hip_atomic_load(from + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      mine = mine && w[j] != kGateAbsent;
    }
    there = __all(mine);
  }
  GatePair<V> r;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    r.p[j] = __builtin_bit_cast(float, (uint32_t)(w[j] >> 32));
    r.h[j] = there ? __builtin_bit_cast(float, (uint32_t)w[j]) : __builtin_nanf("");
  }
  return r;
}

template <int V>
struct GateChain {
  GatePair<V> pair[kGateWaves][kGateLanes];    // of the workgroup's waves
  GatePair<V> before[kGateRun][kGateLanes];    // of windows, and the run's state (the last)
  uint32_t ticket;
};

// The workgroup's column (false: it has none), and the number it takes there.
template <int V, typename A>
__device__ __forceinline__ bool gate_number(GateChain<V>& chain, const A& s, GateSpot<V>& at,
                                            int* number) {
  const int64_t id = seq_block();
  const uint32_t cols = (uint32_t)s.groups * (uint32_t)s.B;
  if (id >= (int64_t)cols * s.windows) return false;
  // (a column's windows on all XCDs: 93 us a prompt of 16384 x 1 x 2048 bf16, 105 on one)
  const uint32_t col = gate_column(((uint32_t)id + (uint32_t)id / cols) % cols, cols, s.split);
  if (threadIdx.x == 0)
    chain.ticket = __hip_atomic_fetch_add(s.ticket + (int64_t)col * kGateTicket, 1u,
                                          __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  at.at(s, col);
  __syncthreads();
  *number = (int)__builtin_amdgcn_readfirstlane(chain.ticket);
  return true;
}

// As gate_fold, for window `n` of a chain whose first state is `first`.  `last`: nothing
// comes behind it.  Returns the state behind the window where the thread's wave ends it.
template <bool REVERSE, int V, typename A>
__device__ __forceinline__ GatePair<V> gate_chain(GateChain<V>& chain, const A& s,
                                                  const GateSpot<V>& at, int n, bool last,
                                                  const float* first, const GatePair<V>& mine,
                                                  float (&in)[V]) {
  const int64_t cols = (int64_t)s.B * s.D, col = (int64_t)at.b * s.D + at.c;
  GatePair<V> other;
  const GatePair<V> both = gate_both<REVERSE>(at, mine, other);
  if (!at.upper) chain.pair[at.wave][at.lane] = both;
  __syncthreads();
  const int run = n / kGateRun, place = n % kGateRun;
  if (at.wave == 0 && !last && place != kGateRun - 1) {
    GatePair<V> all = chain.pair[REVERSE ? at.waves - 1 : 0][at.lane];
    for (int k = 1; k < at.waves; ++k) {
      const GatePair<V> one = chain.pair[REVERSE ? at.waves - 1 - k : k][at.lane];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        all.p[j] *= one.p[j];
        all.h[j] = fmaf(one.p[j], all.h[j], one.h[j]);
      }
    }
    if (!at.upper)
#pragma unroll
      for (int j = 0; j < V; ++j) gate_leave(s.pairs + n * cols + col + j, all.p[j], all.h[j]);
  }
  if (at.wave < place || at.wave == kGateRun - 1) {
    GatePair<V> got;
    if (at.wave < place) {
      got = gate_await<V>(s.pairs + (int64_t)(run * kGateRun + at.wave) * cols + col);
    } else if (run > 0) {
      got = gate_await<V>(s.states + (int64_t)(run - 1) * cols + col);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) got.h[j] = first ? first[col + j] : 0.0f;
    }
    if (!at.upper) chain.before[at.wave][at.lane] = got;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < V; ++j) in[j] = chain.before[kGateRun - 1][at.lane].h[j];
  for (int k = 0; k < place; ++k) {
    const GatePair<V> one = chain.before[k][at.lane];
#pragma unroll
    for (int j = 0; j < V; ++j) in[j] = fmaf(one.p[j], in[j], one.h[j]);
  }
  const GatePair<V> behind = gate_through<REVERSE>(chain.pair, at, both, other, in);
  if ((REVERSE ? at.wave == 0 : at.wave == at.waves - 1) && !at.upper && !last &&
      place == kGateRun - 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) gate_leave(s.states + run * cols + col + j, 0.0f, behind.h[j]);
  }
  return behind;
}

template <typename E>
ck_status gate_run_forward(const GateArgs<E>& a, const GatePlan& p, hipStream_t stream);
// g_f, g_i: gradients of the biases, or NULL.
template <typename E>
ck_status gate_run_backward(const GateArgs<E>& a, const GatePlan& p, float* g_f, float* g_i,
                            hipStream_t stream);

}  // namespace ckhip
