// gated_forward.hip -- forward of the gated scan (gated.h has the formulas and
// the layout).
#include "gated.h"

namespace ckhip {
namespace {

// A tile's decays and inputs, from its loaded rows; steps past `n` change nothing.
template <typename E, int V, bool I>
__device__ __forceinline__ void gate_inputs(const GateTile<E, V>& x, const GateTile<E, V>& f,
                                            const GateTile<E, V>& i, const float (&fb)[V],
                                            const float (&ib)[V], int n, Decay (&a)[kGateStep][V],
                                            float (&u)[kGateStep][V]) {
#pragma unroll
  for (int k = 0; k < kGateStep; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Forget g = forget_hw((float)f.v[k].v[j] + fb[j]);
      float take = g.q;
      if constexpr (I) take = sigmoid_hw((float)i.v[k].v[j] + ib[j]);
      a[k][j] = k < n ? g.decay : Decay{kKeep};
      u[k][j] = k < n ? take * (float)x.v[k].v[j] : 0.0f;
    }
}

template <int V>
__device__ __forceinline__ GatePair<V> gate_pair(const Decay (&a)[kGateStep][V],
                                                 const float (&u)[kGateStep][V]) {
  GatePair<V> r;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    r.p[j] = 1.0f;
    r.h[j] = 0.0f;
#pragma unroll
    for (int k = 0; k < kGateStep; ++k) {
      r.h[j] = a[k][j].times(r.h[j], u[k][j]);
      r.p[j] = a[k][j].times(r.p[j], 0.0f);
    }
  }
  return r;
}

template <int V>
__device__ __forceinline__ void gate_bias(const float* bias, int64_t c, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = bias ? bias[c + j] : 0.0f;
}

template <typename E, int V, bool I, bool Z>
__global__ __launch_bounds__(64 * kGateMaxWaves) void gate_fwd(const GateArgs<E> s) {
  __shared__ GatePair<V> lds[2][kGateMaxWaves][kGateLanes];
  GateSpot<V> at;
  if (!at.at(s, seq_block(), s.chunks)) return;
  const int t0 = at.chunk * s.chunk, t1 = min(t0 + s.chunk, s.T);
  const int window = 2 * at.waves * kGateStep;
  float fb[V], ib[V], carry[V];
  gate_bias<V>(s.f_bias, at.c, fb);
  gate_bias<V>(I ? s.i_bias : nullptr, at.c, ib);
  const int64_t col = (int64_t)at.b * s.D + at.c;
  gate_bias<V>(s.state0, col, carry);
  for (int k = 0; k < at.chunk; ++k) {
    const float* p = s.sums + ((int64_t)k * s.B * s.D + col) * 2;
#pragma unroll
    for (int j = 0; j < V; ++j) carry[j] = fmaf(p[2 * j], carry[j], p[2 * j + 1]);
  }
  int turn = 0;
  for (int t = t0; t < t1; t += window, turn ^= 1) {
    const int first = t + (2 * at.wave + at.upper) * kGateStep;
    const int n = at.len - first;  // the slot's steps that hold text
    if (t < at.len) {
      GateTile<E, V> x, f, i, z;
      x.load(s.x, first, at.b, at.c, n);
      f.load(s.f, first, at.b, at.c, n);
      if constexpr (I) i.load(s.i, first, at.b, at.c, n);
      if constexpr (Z) z.load(s.z, first, at.b, at.c, n);
      Decay a[kGateStep][V];
      float u[kGateStep][V], h[V];
      gate_inputs<E, V, I>(x, f, i, fb, ib, n, a, u);
      gate_fold<false, V>(lds[turn], at, gate_pair<V>(a, u), carry, h);
      if (s.saved && n > 0)
        gate_store<float, V>(s.saved + ((int64_t)(first / kGateStep) * s.B * s.D + col), h, at.live,
                             at.own);
      const Rows<E> out(s.out, first, at.b, at.c);
#pragma unroll
      for (int k = 0; k < kGateStep; ++k) {
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          h[j] = a[k][j].times(h[j], u[k][j]);
          y[j] = h[j];
          if constexpr (Z) {
            const float v = (float)z.v[k].v[j];
            y[j] *= v * sigmoid_hw(v);
          }
          if (k >= n) y[j] = 0.0f;
        }
        if (first + k < t1) gate_store<E, V>(out.at(k), y, at.live, at.own);
      }
    } else {
      const Rows<E> out(s.out, first, at.b, at.c);
      const float none[V] = {};
      for (int k = 0; k < kGateStep && first + k < t1; ++k)
        gate_store<E, V>(out.at(k), none, at.live, at.own);
    }
  }
  if (s.state && at.chunk == s.chunks - 1 && threadIdx.x < kGateLanes)
    gate_store<float, V>(s.state + col, carry, at.live, at.own);
}

// The pairs of all chunks but the last.  A slot takes a run of steps of its own.
template <typename E, int V, bool I>
__global__ __launch_bounds__(64 * kGateMaxWaves) void gate_sum(const GateArgs<E> s) {
  __shared__ GatePair<V> lds[kGateMaxWaves][kGateLanes];
  GateSpot<V> at;
  if (!at.at(s, seq_block(), s.chunks - 1)) return;
  const int run = s.chunk / (2 * at.waves);  // a multiple of a tile's steps
  const int t0 = at.chunk * s.chunk + (2 * at.wave + at.upper) * run;
  float fb[V], ib[V];
  gate_bias<V>(s.f_bias, at.c, fb);
  gate_bias<V>(I ? s.i_bias : nullptr, at.c, ib);
  GatePair<V> all;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    all.p[j] = 1.0f;
    all.h[j] = 0.0f;
  }
  for (int t = t0; t < t0 + run && t < at.len; t += kGateStep) {
    const int n = at.len - t;
    GateTile<E, V> x, f, i;
    x.load(s.x, t, at.b, at.c, n);
    f.load(s.f, t, at.b, at.c, n);
    if constexpr (I) i.load(s.i, t, at.b, at.c, n);
    Decay a[kGateStep][V];
    float u[kGateStep][V];
    gate_inputs<E, V, I>(x, f, i, fb, ib, n, a, u);
#pragma unroll
    for (int k = 0; k < kGateStep; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        all.h[j] = a[k][j].times(all.h[j], u[k][j]);
        all.p[j] = a[k][j].times(all.p[j], 0.0f);
      }
  }
  // (from a state of zero, and from one of one without inputs)
  float h[V] = {}, in[V];
  gate_fold<false, V>(lds, at, all, h, in);
  float p[V];
#pragma unroll
  for (int j = 0; j < V; ++j) p[j] = 1.0f;
  for (int w = 0; w < at.waves; ++w)
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] *= lds[w][at.lane].p[j];
  if (threadIdx.x < kGateLanes && at.live) {
    float* to = s.sums + ((int64_t)at.chunk * s.B * s.D + (int64_t)at.b * s.D + at.c) * 2;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j >= at.own) {
        to[2 * j] = p[j];
        to[2 * j + 1] = h[j];
      }
  }
}

template <typename E, int V>
ck_status gate_launch(const GateArgs<E>& a, const GatePlan& p, hipStream_t stream) {
  const int threads = 64 * p.waves;
  const int64_t cols = (int64_t)p.groups * a.B;
  if (p.chunks > 1) {
    const dim3 grid = seq_grid(cols * (p.chunks - 1));
    if (a.i.p) gate_sum<E, V, true><<<grid, threads, 0, stream>>>(a);
    else gate_sum<E, V, false><<<grid, threads, 0, stream>>>(a);
  }
  const dim3 grid = seq_grid(cols * p.chunks);
  if (a.i.p && a.z.p) gate_fwd<E, V, true, true><<<grid, threads, 0, stream>>>(a);
  else if (a.i.p) gate_fwd<E, V, true, false><<<grid, threads, 0, stream>>>(a);
  else if (a.z.p) gate_fwd<E, V, false, true><<<grid, threads, 0, stream>>>(a);
  else gate_fwd<E, V, false, false><<<grid, threads, 0, stream>>>(a);
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
