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

// silu(z) and its derivative.
struct Silu {
  float value, slope;
};
__device__ __forceinline__ Silu silu_hw(float z) {
  const float s = sigmoid_hw(z);
  return Silu{z * s, s * fmaf(z, 1.0f - s, 1.0f)};
}

// SUM: the pairs (product of a, adjoint) of all chunks but the first, for the launch
// that follows.
template <typename E, int V, bool I, bool Z, bool SUM>
__global__ __launch_bounds__(64 * kGateBwdWaves) void gate_bwd(const GateArgs<E> s) {
  __shared__ GateMeet<V, kGateBwdWaves> meet;
  __shared__ float bias[SUM ? 1 : 2 * kGateBwdWaves][2 * V][kGateLanes];
  GateSpot<V> at;
  if (!at.at(s, seq_block(), SUM ? s.chunks - 1 : s.chunks)) return;
  const int t0 = (at.chunk + (SUM ? 1 : 0)) * s.chunk, t1 = min(t0 + s.chunk, s.T);
  const int window = 2 * at.waves * kGateStep;
  const int slot = (2 * at.wave + at.upper) * kGateStep;  // its first step in a window
  const int steps = min(at.len, t1);
  const int64_t col = (int64_t)at.b * s.D + at.c;
  GateTile<E, V> x, f, i, z, go, nx, nf, ni, nz, ngo;
  float nbefore[V] = {};
  auto fetch = [&](auto all, int t) {
    constexpr bool ALL = decltype(all)::value;
    const int last = steps - 1 - t;
    nf.template load<ALL>(s.f, at, t, slot, last);
    if constexpr (!SUM) {
      if constexpr (I) ni.template load<ALL>(s.i, at, t, slot, last);
      nx.template load<ALL>(s.x, at, t, slot, last);
      const float* p =
          s.saved + ((int64_t)((t + (ALL ? slot : min(slot, last))) / kGateStep) * s.B * s.D + col);
#pragma unroll
      for (int j = 0; j < V; ++j) nbefore[j] = p[j];
    }
    if constexpr (Z) nz.template load<ALL>(s.z, at, t, slot, last);
    ngo.template load<ALL>(s.go, at, t, slot, last);
  };
  int t = t0 + (t1 - t0 - 1) / window * window;  // windows from the last to the first
  for (; t >= t0 && t >= steps; t -= window) {   // behind the text
    if constexpr (SUM) continue;
    GateRows<E> gx(s.gx, t, at.b, at.c0), gf(s.gf, t, at.b, at.c0), gi(s.gi, t, at.b, at.c0),
        gz(s.gz, t, at.b, at.c0);
    const float none[V] = {};
    const uint32_t own = (uint32_t)at.cl * (uint32_t)sizeof(E);
#pragma unroll 1
    for (int k = slot; k < slot + kGateStep && t + k < t1; ++k) {
      pack_store<true, E, V>(gx.at((uint32_t)k * gx.step + own), none, V);
      pack_store<true, E, V>(gf.at((uint32_t)k * gf.step + own), none, V);
      if constexpr (I) pack_store<true, E, V>(gi.at((uint32_t)k * gi.step + own), none, V);
      if constexpr (Z) pack_store<true, E, V>(gz.at((uint32_t)k * gz.step + own), none, V);
    }
  }
  if (t >= t0) fetch(std::false_type(), t);
  float fb[V], ib[V], sum_f[V] = {}, sum_i[V] = {};  // (the biases with their sign turned)
#pragma unroll
  for (int j = 0; j < V; ++j) {
    fb[j] = s.f_bias ? -s.f_bias[at.c + j] : 0.0f;
    ib[j] = I && s.i_bias ? -s.i_bias[at.c + j] : 0.0f;
  }
  if (threadIdx.x < kGateLanes) {
    GatePair<V> c;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      c.p[j] = 1.0f;
      c.h[j] = !SUM && s.gstate ? s.gstate[col + j] : 0.0f;
    }
    if constexpr (!SUM)
      for (int k = s.chunks - 1; k > at.chunk; --k) {
        const float* p = s.sums + ((int64_t)(k - 1) * s.B * s.D + col) * 2;
#pragma unroll
        for (int j = 0; j < V; ++j) c.h[j] = fmaf(p[2 * j], c.h[j], p[2 * j + 1]);
      }
    meet.carry[0][at.lane] = c;
  }
  int turn = 0;
  // WHOLE: every slot's steps hold text.  NEXT: another window
  // follows (full of text), and is on its way while this one is worked on.
  auto work = [&](auto whole, auto next) {
    constexpr bool WHOLE = decltype(whole)::value;
    x = nx, f = nf, i = ni, z = nz, go = ngo;
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = nbefore[j];
    if constexpr (decltype(next)::value) fetch(std::true_type(), t - window);
    const int n = steps - t - slot;  // the slot's steps that hold text
    Gate a[kGateStep][V], in[kGateStep][V];
    float before[kGateStep][V], y[kGateStep][V], c[V];
    GatePair<V> mine;
    GateRows<E> gz(s.gz, t, at.b, at.c0);
    const uint32_t own = (uint32_t)at.cl * (uint32_t)sizeof(E);
    const uint32_t oz = gate_offset((uint32_t)slot * gz.step + own);
#pragma unroll
    for (int k = 0; k < kGateStep; ++k, gz.next()) {
      float vz[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        Gate g = gate_hw(fb[j] - f.get(k, j));
        if (!WHOLE && k >= n) g = kGateKeep;
        a[k][j] = g;
        if constexpr (!SUM) {
          float take = g.rest();
          if constexpr (I) {
            in[k][j] = gate_hw(ib[j] - i.get(k, j));
            take = in[k][j].value();
          }
          take *= x.get(k, j);
          if (!WHOLE && k >= n) take = 0.0f;
          before[k][j] = h[j];
          h[j] = g.times(h[j], take);
        }
        float v = go.get(k, j);
        if constexpr (Z) {
          const Silu gate = silu_hw(z.get(k, j));
          if constexpr (!SUM) vz[j] = !WHOLE && k >= n ? 0.0f : v * h[j] * gate.slope;
          v *= gate.value;
        }
        y[k][j] = !WHOLE && k >= n ? 0.0f : v;
      }
      if constexpr (Z && !SUM)
        if (WHOLE || t + slot + k < t1) pack_store<true, E, V>(gz.at(oz), vz, V);
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
    gate_fold<true>(meet, turn, at, mine, c);
    if constexpr (SUM) return;
    const GateRows<E> gx(s.gx, t, at.b, at.c0), gf(s.gf, t, at.b, at.c0), gi(s.gi, t, at.b, at.c0);
    const uint32_t ox = gate_offset((uint32_t)slot * gx.step + own),
                   of = gate_offset((uint32_t)slot * gf.step + own),
                   oi = I ? gate_offset((uint32_t)slot * gi.step + own) : 0;
#pragma unroll
    for (int k = kGateStep - 1; k >= 0; --k) {
      float vx[V], vf[V], vi[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float gh = y[k][j] + c[j], xv = x.get(k, j);
        const bool runs = WHOLE || k < n;
        float take, from = before[k][j];
        if constexpr (I) {
          take = in[k][j].value();
          vi[j] = runs ? gh * xv * in[k][j].slope() : 0.0f;
          sum_i[j] += vi[j];
        } else {
          take = a[k][j].rest();
          from -= xv;
        }
        vx[j] = runs ? take * gh : 0.0f;
        vf[j] = runs ? gh * from * a[k][j].slope() : 0.0f;
        sum_f[j] += vf[j];
        c[j] = a[k][j].times(gh, 0.0f);
      }
      if (WHOLE || t + slot + k < t1) {
        const auto row = [&](const GateRows<E>& r, uint32_t o) {
          return reinterpret_cast<E*>((r.base + (uint64_t)k * r.step) + o);
        };
        pack_store<true, E, V>(row(gx, ox), vx, V);
        pack_store<true, E, V>(row(gf, of), vf, V);
        if constexpr (I) pack_store<true, E, V>(row(gi, oi), vi, V);
      }
    }
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  // (only the first window, the row's last, can be short of text)
  if (t > t0 && t + window > steps) {
    work(no, yes);
    t -= window;
    turn ^= 1;
  }
  for (; t > t0; t -= window, turn ^= 1) work(yes, yes);
  if (t == t0) {
    if (t + window <= steps) work(yes, no);
    else work(no, no);
    turn ^= 1;
  }
  if constexpr (!SUM)
    if (s.part) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        bias[slot / kGateStep][j][at.lane] = sum_f[j];
        bias[slot / kGateStep][V + j][at.lane] = sum_i[j];
      }
    }
  __syncthreads();
  if (threadIdx.x < kGateLanes) {
    const GatePair<V> c = meet.carry[turn][at.lane];
    if constexpr (SUM) gate_sum_store<V>(s, at, c);
    else if (s.gstate0 && at.chunk == 0) pack_store<true, float, V>(s.gstate0 + col, c.h, V);
  }
  if constexpr (SUM) return;
  if (!s.part) return;
  // the slots' sums, one channel and gate a thread
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
    if (a.z.p) gate_bwd<E, V, false, true, true><<<grid, threads, 0, stream>>>(a);
    else gate_bwd<E, V, false, false, true><<<grid, threads, 0, stream>>>(a);
  }
  const dim3 grid = seq_grid(cols * p.chunks);
  if (a.i.p && a.z.p) gate_bwd<E, V, true, true, false><<<grid, threads, 0, stream>>>(a);
  else if (a.i.p) gate_bwd<E, V, true, false, false><<<grid, threads, 0, stream>>>(a);
  else if (a.z.p) gate_bwd<E, V, false, true, false><<<grid, threads, 0, stream>>>(a);
  else gate_bwd<E, V, false, false, false><<<grid, threads, 0, stream>>>(a);
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
