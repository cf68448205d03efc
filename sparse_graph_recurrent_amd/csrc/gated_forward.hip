// gated_forward.hip -- forward of the gated scan (gated.h has the formulas and
// the layout).
#include "gated.h"

namespace ckhip {
namespace {

// A window's inputs, for a slot.
template <typename E, int V, bool I>
struct GateInputs {
  GateTile<E, V> x, f, i;
  template <bool ALL>
  __device__ __forceinline__ void load(const GateArgs<E>& s, const GateSpot<V>& at, int t, int slot,
                                       int last) {
    f.template load<ALL>(s.f, at, t, slot, last);
    if constexpr (I) i.template load<ALL>(s.i, at, t, slot, last);
    x.template load<ALL>(s.x, at, t, slot, last);
  }
};

// The biases of a lane's channels (the forget gate's with its sign turned).
template <int V>
struct GateBias {
  float f[V], i[V];
  template <typename A>
  __device__ __forceinline__ GateBias(const A& s, const GateSpot<V>& at, bool own) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f[j] = s.f_bias ? -s.f_bias[at.c + j] : 0.0f;
      i[j] = own && s.i_bias ? s.i_bias[at.c + j] : 0.0f;
    }
  }
};

// A slot's way through its steps: from a state of zero, and then from the one before it.
template <typename E, int V, bool I, bool Z>
struct GateForward {
  Gate a[kGateStep][V];
  float u[kGateStep][V];

  // WHOLE: all steps hold text, else the first n.
  template <bool WHOLE>
  __device__ __forceinline__ GatePair<V> enter(const GateInputs<E, V, I>& in,
                                               const GateBias<V>& bias, int n) {
    GatePair<V> mine;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      mine.p[j] = 1.0f;
      mine.h[j] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kGateStep; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        Gate g = gate_hw(bias.f[j] - in.f.get(k, j));
        float take;
        if constexpr (I) take = sigmoid_hw(in.i.get(k, j) + bias.i[j]);
        else take = g.rest();
        take *= in.x.get(k, j);
        a[k][j] = g;
        u[k][j] = take;
        // (no step at all: one that keeps all of an infinite state makes a NaN of it)
        if (!WHOLE && k >= n) continue;
        mine.h[j] = g.times(mine.h[j], take);
        mine.p[j] = g.times(mine.p[j], 0.0f);
      }
    return mine;
  }

  // t: the window's first step, t1 the end of the steps that are there; h: the state
  // before the slot.
  template <bool WHOLE>
  __device__ __forceinline__ void leave(const GateArgs<E>& s, const GateSpot<V>& at, int t, int slot,
                                        int t1, int n, const GateTile<E, V>& z, float (&h)[V]) {
    if (s.saved && (WHOLE || n > 0))
      pack_store<true, float, V>(s.saved + ((int64_t)((t + slot) / kGateStep) * s.B * s.D +
                                            (int64_t)at.b * s.D + at.c), h, V);
    GateRows<E> out(s.out, t, at.b, at.c0);
    const uint32_t o =
        gate_offset((uint32_t)slot * out.step + (uint32_t)at.cl * (uint32_t)sizeof(E));
#pragma unroll
    for (int k = 0; k < kGateStep; ++k, out.next()) {
      float y[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (WHOLE || k < n) h[j] = a[k][j].times(h[j], u[k][j]);
        y[j] = h[j];
        if constexpr (Z) {
          const float v = z.get(k, j);
          y[j] *= v * sigmoid_hw(v);
        }
        if (!WHOLE && k >= n) y[j] = 0.0f;
      }
      if (WHOLE || t + slot + k < t1) pack_store<true, E, V>(out.at(o), y, V);
    }
  }
};

// Zeros behind the text: the steps [t, t1), a window at a time.
template <typename E, int V>
__device__ __forceinline__ void gate_blank(const GateArgs<E>& s, const GateSpot<V>& at, int t,
                                           int t1, int slot, int window) {
  for (; t < t1; t += window) {
    GateRows<E> out(s.out, t, at.b, at.c0);
    const float none[V] = {};
    const uint32_t o = (uint32_t)slot * out.step + (uint32_t)at.cl * (uint32_t)sizeof(E);
#pragma unroll 1
    for (int k = 0; k < kGateStep && t + slot + k < t1; ++k, out.next())
      pack_store<true, E, V>(out.at(o), none, V);
  }
}

// All windows of a column.  256 columns of 2048 steps, bf16, with an output gate: 84 us
// (4.2 TB/s).  16 waves a workgroup spill (113 us).
template <typename E, int V, bool I, bool Z>
__global__ __launch_bounds__(64 * kGateWaves) void gate_fwd(const GateArgs<E> s) {
  __shared__ GateMeet<V, kGateWaves> meet;
  GateSpot<V> at;
  const int64_t id = seq_block(), cols = (int64_t)s.groups * s.B;
  if (id >= cols) return;
  at.at(s, gate_column((uint32_t)id, (uint32_t)cols, s.split));
  const int window = 2 * at.waves * kGateStep, steps = at.len;
  const int slot = (2 * at.wave + at.upper) * kGateStep;  // its first step in a window
  // A window's inputs are asked for two windows ahead, so that requests are under way
  // at all times: into one of two sets of registers, when what that held has been used.
  GateInputs<E, V, I> even, odd;
  int t = 0;
  if (t < steps) even.template load<false>(s, at, t, slot, steps - 1 - t);
  if (t + window < steps) odd.template load<false>(s, at, t + window, slot, steps - 1 - t - window);
  const int64_t col = (int64_t)at.b * s.D + at.c;
  const GateBias<V> bias(s, at, I);
  if (threadIdx.x < kGateLanes)
#pragma unroll
    for (int j = 0; j < V; ++j) meet.carry[0][at.lane][j] = s.state0 ? s.state0[col + j] : 0.0f;
  int turn = 0;
  // One window.  WHOLE: every slot's steps hold text, and so do those of the window after
  // the next, which is asked for.  (Any choice between ways to ask would have registers
  // copied, and so waited for, where the ways meet.)
  auto work = [&](auto whole, GateInputs<E, V, I>& now) {
    constexpr bool WHOLE = decltype(whole)::value;
    GateTile<E, V> z;
    if constexpr (Z) z.template load<WHOLE>(s.z, at, t, slot, steps - 1 - t);
    const int n = steps - t - slot;  // the slot's steps that hold text
    GateForward<E, V, I, Z> way;
    const GatePair<V> mine = way.template enter<WHOLE>(now, bias, n);
    if constexpr (WHOLE) now.template load<true>(s, at, t + 2 * window, slot, 0);
    float h[V];
    gate_fold<false>(meet, turn, at, mine, h);
    way.template leave<WHOLE>(s, at, t, slot, s.T, n, z, h);
    t += window;
    turn ^= 1;
  };
  while (t + 4 * window <= steps) {
    work(std::true_type(), even);
    work(std::true_type(), odd);
  }
  while (t < steps) {
    work(std::false_type(), even);
    even = odd;
    if (t + window < steps)
      odd.template load<false>(s, at, t + window, slot, steps - 1 - t - window);
  }
  gate_blank<E, V>(s, at, t, s.T, slot, window);
  __syncthreads();
  if (threadIdx.x < kGateLanes && s.state)
    pack_store<true, float, V>(s.state + col, meet.carry[turn][at.lane], V);
}

// A window of a column a workgroup.  32 columns of 16384 steps, bf16: 80 to 86
// us (4.1 TB/s): a workgroup's loads are covered by the other workgroup of its CU alone.
// Registers for 6 or 8 waves a SIMD spill (142 and 180 us against 93 then).
template <typename E, int V, bool I, bool Z>
__global__ __launch_bounds__(64 * kGateWaves) void gate_fwd_chain(const GateArgs<E> s) {
  __shared__ GateChain<V> chain;
  GateSpot<V> at;
  int number;
  if (!gate_number(chain, s, at, &number)) return;
  const int window = 2 * at.waves * kGateStep, t = number * window;
  const int slot = (2 * at.wave + at.upper) * kGateStep;
  const int t1 = min(t + window, s.T);
  const int64_t col = (int64_t)at.b * s.D + at.c;
  if (t >= at.len) {  // behind the text; a row without any hands its state on
    gate_blank<E, V>(s, at, t, t1, slot, window);
    if (t == 0 && s.state && threadIdx.x < kGateLanes)
#pragma unroll
      for (int j = 0; j < V; ++j) s.state[col + j] = s.state0 ? s.state0[col + j] : 0.0f;
    return;
  }
  const bool last = t + window >= at.len;
  const GateBias<V> bias(s, at, I);
  auto work = [&](auto whole) {  // whether every slot's steps hold text
    constexpr bool WHOLE = decltype(whole)::value;
    const int n = at.len - t - slot;
    GateInputs<E, V, I> in;
    GateTile<E, V> z;
    in.template load<WHOLE>(s, at, t, slot, at.len - 1 - t);
    GateForward<E, V, I, Z> way;
    float h[V];
    const GatePair<V> mine = way.template enter<WHOLE>(in, bias, n);
    // (asked for where registers are free again; on its way while the others are awaited)
    if constexpr (Z) z.template load<WHOLE>(s.z, at, t, slot, at.len - 1 - t);
    const GatePair<V> behind = gate_chain<false>(chain, s, at, number, last, s.state0, mine, h);
    if (last && s.state && at.wave == at.waves - 1 && !at.upper)
      pack_store<true, float, V>(s.state + col, behind.h, V);
    way.template leave<WHOLE>(s, at, t, slot, t1, n, z, h);
  };
  if (t + window <= at.len) work(std::true_type());
  else work(std::false_type());
}

template <typename E, int V, bool I, bool Z>
void gate_start(const GateArgs<E>& a, const GatePlan& p, hipStream_t stream) {
  const dim3 grid = seq_grid((int64_t)p.groups * a.B * p.windows);
  if (p.windows > 1) gate_fwd_chain<E, V, I, Z><<<grid, 64 * p.waves, 0, stream>>>(a);
  else gate_fwd<E, V, I, Z><<<grid, 64 * p.waves, 0, stream>>>(a);
}

template <typename E, int V>
ck_status gate_launch(const GateArgs<E>& a, const GatePlan& p, hipStream_t stream) {
  if (a.i.p && a.z.p) gate_start<E, V, true, true>(a, p, stream);
  else if (a.i.p) gate_start<E, V, true, false>(a, p, stream);
  else if (a.z.p) gate_start<E, V, false, true>(a, p, stream);
  else gate_start<E, V, false, false>(a, p, stream);
  CK_HIP_TRY(hipGetLastError());
  return CK_OK;
}

}  // namespace

template <typename E>
ck_status gate_run_forward(const GateArgs<E>& a, const GatePlan& p, hipStream_t stream) {
  if constexpr (sizeof(E) == 2)
    if (p.v == 2) return gate_launch<E, 2>(a, p, stream);
  return gate_launch<E, 1>(a, p, stream);
}
template ck_status gate_run_forward(const GateArgs<float>&, const GatePlan&, hipStream_t);
template ck_status gate_run_forward(const GateArgs<bf16_t>&, const GatePlan&, hipStream_t);
template ck_status gate_run_forward(const GateArgs<f16_t>&, const GatePlan&, hipStream_t);

}  // namespace ckhip
