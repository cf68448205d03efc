// gated_forward.hip -- forward of the gated scan (gated.h has the formulas and
// the layout).
#include "gated.h"

namespace ckhip {
namespace {

// SUM: the pairs of all chunks but the last, for the launch that follows.
template <typename E, int V, bool I, bool Z, bool SUM>
__global__ __launch_bounds__(64 * kGateFwdWaves) void gate_fwd(const GateArgs<E> s) {
  __shared__ GateMeet<V, kGateFwdWaves> meet;
  GateSpot<V> at;
  if (!at.at(s, seq_block(), SUM ? s.chunks - 1 : s.chunks)) return;
  const int t0 = at.chunk * s.chunk, t1 = min(t0 + s.chunk, s.T);
  const int window = 2 * at.waves * kGateStep;
  const int slot = (2 * at.wave + at.upper) * kGateStep;  // its first step in a window
  const int steps = min(at.len, t1);
  // A window's inputs are asked for two windows ahead, so that requests are under way
  // at all times: into one of two sets of registers, when what that held has been used.
  struct Inputs {
    GateTile<E, V> x, f, i;
  } even, odd;
  auto fetch = [&](auto all, Inputs& in, int t) {
    constexpr bool ALL = decltype(all)::value;
    const int last = steps - 1 - t;
    in.f.template load<ALL>(s.f, at, t, slot, last);
    if constexpr (I) in.i.template load<ALL>(s.i, at, t, slot, last);
    in.x.template load<ALL>(s.x, at, t, slot, last);
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  int t = t0;
  if (t < steps) fetch(no, even, t);
  if (t + window < steps) fetch(no, odd, t + window);
  const int64_t col = (int64_t)at.b * s.D + at.c;
  float fb[V], ib[V];  // (of the forget gate with its sign turned)
#pragma unroll
  for (int j = 0; j < V; ++j) {
    fb[j] = s.f_bias ? -s.f_bias[at.c + j] : 0.0f;
    ib[j] = I && s.i_bias ? s.i_bias[at.c + j] : 0.0f;
  }
  if (threadIdx.x < kGateLanes) {
    GatePair<V> c;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      c.p[j] = 1.0f;
      c.h[j] = !SUM && s.state0 ? s.state0[col + j] : 0.0f;
    }
    if constexpr (!SUM)
      for (int k = 0; k < at.chunk; ++k) {
        const float* p = s.sums + ((int64_t)k * s.B * s.D + col) * 2;
#pragma unroll
        for (int j = 0; j < V; ++j) c.h[j] = fmaf(p[2 * j], c.h[j], p[2 * j + 1]);
      }
    meet.carry[0][at.lane] = c;
  }
  int turn = 0;
  // One window.  WHOLE: every slot's steps hold text, and so do those of the window after
  // the next, which is asked for.  (Any choice between ways to ask would have registers
  // copied, and so waited for, where the ways meet.)
  auto work = [&](auto whole, Inputs& now) {
    constexpr bool WHOLE = decltype(whole)::value;
    GateTile<E, V> z;
    if constexpr (Z) z.template load<WHOLE>(s.z, at, t, slot, steps - 1 - t);
    const int n = steps - t - slot;  // the slot's steps that hold text
    Gate a[kGateStep][V];
    float u[kGateStep][V], h[V];
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
        Gate g = gate_hw(fb[j] - now.f.get(k, j));
        float take;
        if constexpr (I) take = sigmoid_hw(now.i.get(k, j) + ib[j]);
        else take = g.rest();
        take *= now.x.get(k, j);
        if (!WHOLE && k >= n) g = kGateKeep, take = 0.0f;
        a[k][j] = g;
        u[k][j] = take;
        mine.h[j] = g.times(mine.h[j], take);
        mine.p[j] = g.times(mine.p[j], 0.0f);
        if (j == V - 1) __builtin_amdgcn_sched_barrier(0);
      }
    if constexpr (WHOLE) fetch(yes, now, t + 2 * window);
    gate_fold<false>(meet, turn, at, mine, h);
    t += window;
    turn ^= 1;
    if constexpr (SUM) return;
    const int first = t - window;
    if (s.saved && (WHOLE || n > 0))
      pack_store<true, float, V>(
          s.saved + ((int64_t)((first + slot) / kGateStep) * s.B * s.D + col), h, V);
    GateRows<E> out(s.out, first, at.b, at.c0);
    const uint32_t o =
        gate_offset((uint32_t)slot * out.step + (uint32_t)at.cl * (uint32_t)sizeof(E));
#pragma unroll
    for (int k = 0; k < kGateStep; ++k, out.next()) {
      float y[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[j] = a[k][j].times(h[j], u[k][j]);
        y[j] = h[j];
        if constexpr (Z) {
          const float v = z.get(k, j);
          y[j] *= v * sigmoid_hw(v);
        }
        if (!WHOLE && k >= n) y[j] = 0.0f;
      }
      if (WHOLE || first + slot + k < t1) pack_store<true, E, V>(out.at(o), y, V);
    }
  };
  while (t + 4 * window <= steps) {
    work(yes, even);
    work(yes, odd);
  }
  while (t < steps) {
    work(no, even);
    even = odd;
    if (t + window < steps) fetch(no, odd, t + window);
  }
  if constexpr (!SUM)
    for (; t < t1; t += window) {  // behind the text
      GateRows<E> out(s.out, t, at.b, at.c0);
      const float none[V] = {};
      const uint32_t o = (uint32_t)slot * out.step + (uint32_t)at.cl * (uint32_t)sizeof(E);
#pragma unroll 1
      for (int k = 0; k < kGateStep && t + slot + k < t1; ++k, out.next())
        pack_store<true, E, V>(out.at(o), none, V);
    }
  __syncthreads();
  if (threadIdx.x >= kGateLanes) return;
  const GatePair<V> c = meet.carry[turn][at.lane];
  if constexpr (SUM) gate_sum_store<V>(s, at, c);
  else if (s.state && at.chunk == s.chunks - 1)
    pack_store<true, float, V>(s.state + col, c.h, V);
}

template <typename E, int V>
ck_status gate_launch(const GateArgs<E>& a, const GatePlan& p, hipStream_t stream) {
  const int threads = 64 * p.waves;
  const int64_t cols = (int64_t)p.groups * a.B;
  if (p.chunks > 1) {
    const dim3 grid = seq_grid(cols * (p.chunks - 1));
    if (a.i.p) gate_fwd<E, V, true, false, true><<<grid, threads, 0, stream>>>(a);
    else gate_fwd<E, V, false, false, true><<<grid, threads, 0, stream>>>(a);
  }
  const dim3 grid = seq_grid(cols * p.chunks);
  if (a.i.p && a.z.p) gate_fwd<E, V, true, true, false><<<grid, threads, 0, stream>>>(a);
  else if (a.i.p) gate_fwd<E, V, true, false, false><<<grid, threads, 0, stream>>>(a);
  else if (a.z.p) gate_fwd<E, V, false, true, false><<<grid, threads, 0, stream>>>(a);
  else gate_fwd<E, V, false, false, false><<<grid, threads, 0, stream>>>(a);
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
