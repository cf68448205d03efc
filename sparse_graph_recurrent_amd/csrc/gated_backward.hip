// gated_backward.hip -- backward of the gated scan (gated.h has the forward's
// formulas and the layout).
//
//   Y_t = dL/dy_t  or  dL/dy_t z_t s(z_t)
//   H_t = Y_t + a_{t+1} H_{t+1}       H_{T-1} = Y_{T-1} + dL/dstate,   dL/dstate0 = a_0 H_0
//   gx = g H,   gf = H (h_{t-1} - x_t [tied]) a q,   gi = H x g (1 - g)
//   gz = dL/dy h s(z) (1 + z (1 - s(z)))
//
// A slot computes its states again from the one that the forward left at its first
// step, and folds backwards in time as the forward does forwards.
#include "gated.h"

namespace ckhip {
namespace {

constexpr int kGateBwdWaves = 8;

// silu(z) and its derivative.
struct Silu {
  float value, slope;
};
__device__ __forceinline__ Silu silu_hw(float z) {
  const float s = sigmoid_hw(z);
  return Silu{z * s, s * fmaf(z, 1.0f - s, 1.0f)};
}

template <typename E, int V, bool I, bool Z>
__global__ __launch_bounds__(64 * kGateBwdWaves) void gate_bwd(const GateArgs<E> s) {
  __shared__ GatePair<V> lds[2][kGateBwdWaves][kGateLanes];
  __shared__ float bias[2 * kGateBwdWaves][2 * V][kGateLanes];
  GateSpot<V> at;
  if (!at.at(s, seq_block(), s.chunks)) return;
  const int t0 = at.chunk * s.chunk, t1 = min(t0 + s.chunk, s.T);
  const int window = 2 * at.waves * kGateStep;
  float fb[V], ib[V], carry[V], sum_f[V] = {}, sum_i[V] = {};
  const int64_t col = (int64_t)at.b * s.D + at.c;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    fb[j] = s.f_bias ? s.f_bias[at.c + j] : 0.0f;
    ib[j] = I && s.i_bias ? s.i_bias[at.c + j] : 0.0f;
    carry[j] = s.gstate ? s.gstate[col + j] : 0.0f;
  }
  for (int k = s.chunks - 1; k > at.chunk; --k) {
    const float* p = s.sums + ((int64_t)(k - 1) * s.B * s.D + col) * 2;
#pragma unroll
    for (int j = 0; j < V; ++j) carry[j] = fmaf(p[2 * j], carry[j], p[2 * j + 1]);
  }
  int turn = 0;
  const int windows = (t1 - t0 + window - 1) / window;
  for (int w = windows - 1; w >= 0; --w) {
    const int t = t0 + w * window;
    const int first = t + (2 * at.wave + at.upper) * kGateStep;
    const Rows<E> gx(s.gx, first, at.b, at.c), gf(s.gf, first, at.b, at.c),
        gi(s.gi, first, at.b, at.c), gz(s.gz, first, at.b, at.c);
    if (t >= at.len) {
      const float none[V] = {};
      for (int k = 0; k < kGateStep && first + k < t1; ++k) {
        gate_store<E, V>(gx.at(k), none, at.live, at.own);
        gate_store<E, V>(gf.at(k), none, at.live, at.own);
        if constexpr (I) gate_store<E, V>(gi.at(k), none, at.live, at.own);
        if constexpr (Z) gate_store<E, V>(gz.at(k), none, at.live, at.own);
      }
      continue;
    }
    const int n = at.len - first;
    GateTile<E, V> x, f, i, z, go;
    x.load(s.x, first, at.b, at.c, n);
    f.load(s.f, first, at.b, at.c, n);
    if constexpr (I) i.load(s.i, first, at.b, at.c, n);
    if constexpr (Z) z.load(s.z, first, at.b, at.c, n);
    go.load(s.go, first, at.b, at.c, n);
    float h[V] = {};
    if (n > 0) {
      const float* p = s.saved + ((int64_t)(first / kGateStep) * s.B * s.D + col);
#pragma unroll
      for (int j = 0; j < V; ++j) h[j] = p[j];
    }
    Decay a[kGateStep][V];
    float before[kGateStep][V], y[kGateStep][V], dz[kGateStep][V];
    GatePair<V> mine;
#pragma unroll
    for (int k = 0; k < kGateStep; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const Forget g = forget_hw((float)f.v[k].v[j] + fb[j]);
        float take = g.q;
        if constexpr (I) take = sigmoid_hw((float)i.v[k].v[j] + ib[j]);
        a[k][j] = k < n ? g.decay : Decay{kKeep};
        before[k][j] = h[j];
        h[j] = a[k][j].times(h[j], k < n ? take * (float)x.v[k].v[j] : 0.0f);
        y[k][j] = k < n ? (float)go.v[k].v[j] : 0.0f;
        if constexpr (Z) {
          const Silu v = silu_hw((float)z.v[k].v[j]);
          dz[k][j] = k < n ? y[k][j] * h[j] * v.slope : 0.0f;
          y[k][j] = k < n ? y[k][j] * v.value : 0.0f;
        }
      }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      mine.p[j] = 1.0f;
      mine.h[j] = 0.0f;
#pragma unroll
      for (int k = kGateStep - 1; k >= 0; --k) {
        mine.h[j] = a[k][j].times(mine.h[j] + y[k][j], 0.0f);
        mine.p[j] = a[k][j].times(mine.p[j], 0.0f);
      }
    }
    float c[V];
    gate_fold<true, V>(lds[turn], at, mine, carry, c);
    turn ^= 1;
#pragma unroll
    for (int k = kGateStep - 1; k >= 0; --k) {
      float vx[V], vf[V], vi[V], vz[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float gh = y[k][j] + c[j], xv = (float)x.v[k].v[j];
        const Forget g = forget_hw((float)f.v[k].v[j] + fb[j]);
        const bool runs = k < n;
        float take = g.q, from = before[k][j];
        if constexpr (I) {
          const float v = (float)i.v[k].v[j] + ib[j];
          const Gate in = gate_hw(v);
          take = v >= 0.0f ? in.big : in.small;
          vi[j] = runs ? gh * xv * (in.big * in.small) : 0.0f;
          sum_i[j] += vi[j];
        } else {
          from -= xv;
        }
        vx[j] = runs ? take * gh : 0.0f;
        vf[j] = runs ? gh * from * (g.a * g.q) : 0.0f;
        sum_f[j] += vf[j];
        if constexpr (Z) vz[j] = dz[k][j];
        c[j] = a[k][j].times(gh, 0.0f);
      }
      if (first + k < t1) {
        gate_store<E, V>(gx.at(k), vx, at.live, at.own);
        gate_store<E, V>(gf.at(k), vf, at.live, at.own);
        if constexpr (I) gate_store<E, V>(gi.at(k), vi, at.live, at.own);
        if constexpr (Z) gate_store<E, V>(gz.at(k), vz, at.live, at.own);
      }
    }
  }
  if (s.gstate0 && at.chunk == 0 && threadIdx.x < kGateLanes)
    gate_store<float, V>(s.gstate0 + col, carry, at.live, at.own);
  if (!s.part) return;
  // the slots' sums, one channel and gate a thread
  const int slot = 2 * at.wave + at.upper;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    bias[slot][j][at.lane] = sum_f[j];
    bias[slot][V + j][at.lane] = sum_i[j];
  }
  __syncthreads();
  float* part = s.part + ((int64_t)at.chunk * s.B + at.b) * 2 * s.D;
  for (int o = threadIdx.x; o < 2 * V * kGateLanes; o += blockDim.x) {
    const int lane = o % kGateLanes, j = o / kGateLanes % V, gate = o / kGateLanes / V;
    float sum = 0.0f;
    for (int k = 0; k < 2 * at.waves; ++k) sum += bias[k][gate * V + j][lane];
    // (a lane's channels begin earlier where they pass the row's end)
    const int64_t want = ((int64_t)at.group * kGateLanes + lane) * V;
    const int64_t ch = min(want, (int64_t)s.D - V) + j;
    if (want < s.D && ch >= want) part[(int64_t)gate * s.D + ch] = sum;
  }
}

// The pairs (product of a, adjoint) of all chunks but the first.
template <typename E, int V, bool Z>
__global__ __launch_bounds__(64 * kGateBwdWaves) void gate_bsum(const GateArgs<E> s) {
  __shared__ GatePair<V> lds[kGateBwdWaves][kGateLanes];
  GateSpot<V> at;
  if (!at.at(s, seq_block(), s.chunks - 1)) return;
  const int run = s.chunk / (2 * at.waves);  // a multiple of a tile's steps
  const int t0 = (at.chunk + 1) * s.chunk + (2 * at.wave + at.upper) * run;
  float fb[V];
  GatePair<V> all;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    fb[j] = s.f_bias ? s.f_bias[at.c + j] : 0.0f;
    all.p[j] = 1.0f;
    all.h[j] = 0.0f;
  }
  for (int t = t0 + run - kGateStep; t >= t0; t -= kGateStep) {
    const int n = at.len - t;
    if (n <= 0) continue;
    GateTile<E, V> f, z, go;
    f.load(s.f, t, at.b, at.c, n);
    if constexpr (Z) z.load(s.z, t, at.b, at.c, n);
    go.load(s.go, t, at.b, at.c, n);
#pragma unroll
    for (int k = kGateStep - 1; k >= 0; --k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        Decay a = forget_hw((float)f.v[k].v[j] + fb[j]).decay;
        float y = (float)go.v[k].v[j];
        if constexpr (Z) y *= silu_hw((float)z.v[k].v[j]).value;
        if (k >= n) a = Decay{kKeep}, y = 0.0f;
        all.h[j] = a.times(all.h[j] + y, 0.0f);
        all.p[j] = a.times(all.p[j], 0.0f);
      }
  }
  float h[V] = {}, in[V], p[V];
  gate_fold<true, V>(lds, at, all, h, in);
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

// g_f_bias and g_i_bias: the workgroups' sums, in their order.  A wave an output's 64
// channels would have long walks: kBiasRows threads share them.
constexpr int kBiasCols = 32, kBiasRows = 8;
__global__ __launch_bounds__(kBiasCols * kBiasRows) void gate_bias_sum(
    const float* part, int D, int64_t rows, float* g_f, float* g_i) {
  __shared__ float lds[kBiasRows][kBiasCols];
  const int x = threadIdx.x % kBiasCols, y = threadIdx.x / kBiasCols;
  const int64_t o = seq_block() * kBiasCols + x;
  float sum = 0.0f;
  if (o < 2 * (int64_t)D)
    for (int64_t r = y; r < rows; r += kBiasRows) sum += part[r * 2 * D + o];
  lds[y][x] = sum;
  __syncthreads();
  if (y != 0 || o >= 2 * (int64_t)D) return;
  for (int k = 1; k < kBiasRows; ++k) sum += lds[k][x];
  float* to = o < D ? g_f : g_i;
  if (to) to[o < D ? o : o - D] = sum;
}

template <typename E, int V>
ck_status gate_launch(const GateArgs<E>& a, const GatePlan& p, float* g_f, float* g_i,
                      hipStream_t stream) {
  const int threads = 64 * p.waves;
  const int64_t cols = (int64_t)p.groups * a.B;
  if (p.chunks > 1) {
    const dim3 grid = seq_grid(cols * (p.chunks - 1));
    if (a.z.p) gate_bsum<E, V, true><<<grid, threads, 0, stream>>>(a);
    else gate_bsum<E, V, false><<<grid, threads, 0, stream>>>(a);
  }
  const dim3 grid = seq_grid(cols * p.chunks);
  if (a.i.p && a.z.p) gate_bwd<E, V, true, true><<<grid, threads, 0, stream>>>(a);
  else if (a.i.p) gate_bwd<E, V, true, false><<<grid, threads, 0, stream>>>(a);
  else if (a.z.p) gate_bwd<E, V, false, true><<<grid, threads, 0, stream>>>(a);
  else gate_bwd<E, V, false, false><<<grid, threads, 0, stream>>>(a);
  if (a.part)
    gate_bias_sum<<<seq_grid((2 * (int64_t)a.D + kBiasCols - 1) / kBiasCols), kBiasCols * kBiasRows,
                    0, stream>>>(a.part, a.D, (int64_t)a.B * p.chunks, g_f, g_i);
  CK_HIP_TRY(hipGetLastError());
  return CK_OK;
}

}  // namespace

template <typename E>
ck_status gate_run_backward(const GateArgs<E>& a, const GatePlan& p, float* g_f, float* g_i,
                            hipStream_t stream) {
  if constexpr (sizeof(E) == 2)
    if (p.v == 2) return gate_launch<E, 2>(a, p, g_f, g_i, stream);
  return gate_launch<E, 1>(a, p, g_f, g_i, stream);
}
template ck_status gate_run_backward(const GateArgs<float>&, const GatePlan&, float*, float*,
                                     hipStream_t);
template ck_status gate_run_backward(const GateArgs<bf16_t>&, const GatePlan&, float*, float*,
                                     hipStream_t);
template ck_status gate_run_backward(const GateArgs<f16_t>&, const GatePlan&, float*, float*,
                                     hipStream_t);

}  // namespace ckhip
