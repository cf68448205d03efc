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

// What a slot reads of a window.
template <typename E, int V, bool I, bool Z>
struct GateInputs {
  GateTile<E, V> x, f, i, z, go;
  float before[V];
  template <bool ALL>
  __device__ __forceinline__ void load(const GateArgs<E>& s, const GateSpot<V>& at, int t, int slot,
                                       int last) {
    f.template load<ALL>(s.f, at, t, slot, last);
    if constexpr (I) i.template load<ALL>(s.i, at, t, slot, last);
    x.template load<ALL>(s.x, at, t, slot, last);
    const float* p = s.saved + ((int64_t)((t + (ALL ? slot : min(slot, last))) / kGateStep) * s.B *
                                    s.D + (int64_t)at.b * s.D + at.c);
#pragma unroll
    for (int j = 0; j < V; ++j) before[j] = p[j];
    if constexpr (Z) z.template load<ALL>(s.z, at, t, slot, last);
    go.template load<ALL>(s.go, at, t, slot, last);
  }
};

// What the bias gradients of a thread's channels add up to: within a window in fp32,
// from window to window in 64 bits (a long row's sum would swallow its steps' parts one
// by one), which wait in LDS meanwhile.
template <int V>
using GateSums = double[2 * kGateWaves][2 * V][kGateLanes];

// The biases of a lane's channels, their sign turned.
template <int V>
struct GateBias {
  float f[V], i[V];
  template <typename A>
  __device__ __forceinline__ GateBias(const A& s, const GateSpot<V>& at, bool own) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f[j] = s.f_bias ? -s.f_bias[at.c + j] : 0.0f;
      i[j] = own && s.i_bias ? -s.i_bias[at.c + j] : 0.0f;
    }
  }
};

// A slot's way back through its steps: from an adjoint of zero, and then from the one
// behind it.  WHOLE: all steps hold text, else the first n.
template <typename E, int V, bool I, bool Z>
struct GateBackward {
  Gate a[kGateStep][V], own[kGateStep][V];
  float before[kGateStep][V], y[kGateStep][V];

  template <bool WHOLE>
  __device__ __forceinline__ GatePair<V> enter(const GateArgs<E>& s, const GateSpot<V>& at, int t,
                                               int slot, int t1, int n,
                                               const GateInputs<E, V, I, Z>& in,
                                               const GateBias<V>& bias) {
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = in.before[j];
    GateRows<E> gz(s.gz, t, at.b, at.c0);
    const uint32_t oz =
        gate_offset((uint32_t)slot * gz.step + (uint32_t)at.cl * (uint32_t)sizeof(E));
#pragma unroll
    for (int k = 0; k < kGateStep; ++k, gz.next()) {
      float vz[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        Gate g = gate_hw(bias.f[j] - in.f.get(k, j));
        if (!WHOLE && k >= n) g = kGateKeep;
        a[k][j] = g;
        float take = g.rest();
        if constexpr (I) {
          own[k][j] = gate_hw(bias.i[j] - in.i.get(k, j));
          take = own[k][j].value();
        }
        take *= in.x.get(k, j);
        if (!WHOLE && k >= n) take = 0.0f;
        before[k][j] = h[j];
        h[j] = g.times(h[j], take);
        float v = in.go.get(k, j);
        if constexpr (Z) {
          const Silu gate = silu_hw(in.z.get(k, j));
          vz[j] = !WHOLE && k >= n ? 0.0f : v * h[j] * gate.slope;
          v *= gate.value;
        }
        y[k][j] = !WHOLE && k >= n ? 0.0f : v;
      }
      if constexpr (Z)
        if (WHOLE || t + slot + k < t1) pack_store<true, E, V>(gz.at(oz), vz, V);
    }
    GatePair<V> mine;
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
    return mine;
  }

  // c: a H of the step behind the slot.  ONE: the workgroup's only window.
  template <bool WHOLE, bool ONE>
  __device__ __forceinline__ void leave(const GateArgs<E>& s, const GateSpot<V>& at, int t, int slot,
                                        int t1, int n, const GateTile<E, V>& x, GateSums<V>& sums,
                                        float (&c)[V]) {
    float sum_f[V] = {}, sum_i[V] = {};
    const GateRows<E> gx(s.gx, t, at.b, at.c0), gf(s.gf, t, at.b, at.c0), gi(s.gi, t, at.b, at.c0);
    const uint32_t lane = (uint32_t)at.cl * (uint32_t)sizeof(E);
    const uint32_t ox = gate_offset((uint32_t)slot * gx.step + lane),
                   of = gate_offset((uint32_t)slot * gf.step + lane),
                   oi = I ? gate_offset((uint32_t)slot * gi.step + lane) : 0;
#pragma unroll
    for (int k = kGateStep - 1; k >= 0; --k) {
      float vx[V], vf[V], vi[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float gh = y[k][j] + c[j], xv = x.get(k, j);
        const bool runs = WHOLE || k < n;
        float take, from = before[k][j];
        if constexpr (I) {
          take = own[k][j].value();
          vi[j] = runs ? gh * xv * own[k][j].slope() : 0.0f;
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
    if (!s.part) return;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      double &f = sums[2 * at.wave + at.upper][j][at.lane],
             &i = sums[2 * at.wave + at.upper][V + j][at.lane];
      f = (ONE ? 0.0 : f) + (double)sum_f[j];
      if (I || ONE) i = (ONE ? 0.0 : i) + (double)sum_i[j];
    }
  }
};

// Zeros in a window behind the text.
template <typename E, int V, bool I, bool Z>
__device__ __forceinline__ void gate_blank(const GateArgs<E>& s, const GateSpot<V>& at, int t,
                                           int slot, int t1) {
  const GateRows<E> gx(s.gx, t, at.b, at.c0), gf(s.gf, t, at.b, at.c0), gi(s.gi, t, at.b, at.c0),
      gz(s.gz, t, at.b, at.c0);
  const float none[V] = {};
  const uint32_t lane = (uint32_t)at.cl * (uint32_t)sizeof(E);
#pragma unroll 1
  for (uint32_t k = slot; k < (uint32_t)slot + kGateStep && t + (int)k < t1; ++k) {
    pack_store<true, E, V>(gx.at(k * gx.step + lane), none, V);
    pack_store<true, E, V>(gf.at(k * gf.step + lane), none, V);
    if constexpr (I) pack_store<true, E, V>(gi.at(k * gi.step + lane), none, V);
    if constexpr (Z) pack_store<true, E, V>(gz.at(k * gz.step + lane), none, V);
  }
}

// (a thread clears and adds to its own sums alone, until gate_part)
template <int V>
__device__ __forceinline__ void gate_clear_sums(GateSums<V>& sums, const GateSpot<V>& at) {
#pragma unroll
  for (int j = 0; j < 2 * V; ++j) sums[2 * at.wave + at.upper][j][at.lane] = 0.0;
}

// A workgroup's part of the bias gradients: its slots' sums in their order, one channel
// and gate a thread.  (All threads call it.)  It is rounded to fp32, as what comes of the
// parts is: both by half a step of theirs, however many steps and rows there are.
template <int V, typename A>
__device__ __forceinline__ void gate_part(const A& s, const GateSpot<V>& at,
                                          const GateSums<V>& sums, int64_t row) {
  __syncthreads();
  float* part = s.part + row * 2 * s.D;
  for (int o = threadIdx.x; o < 2 * V * kGateLanes; o += blockDim.x) {
    const int lane = o % kGateLanes, j = o / kGateLanes % V, gate = o / kGateLanes / V;
    double sum = 0.0;
    for (int k = 0; k < 2 * at.waves; ++k) sum += sums[k][gate * V + j][lane];
    // (a lane's channels begin earlier where they pass the row's end)
    const int64_t want = ((int64_t)at.group * kGateLanes + lane) * V;
    const int64_t ch = min(want, (int64_t)s.D - V) + j;
    if (want < s.D && ch >= want) part[(int64_t)gate * s.D + ch] = (float)sum;
  }
}

// All windows of a column, from the last to the first.  256 columns of 2048 steps, bf16,
// with an output gate: 123 us (5.1 TB/s).
template <typename E, int V, bool I, bool Z>
__global__ __launch_bounds__(64 * kGateWaves) void gate_bwd(const GateArgs<E> s) {
  __shared__ GateMeet<V, kGateWaves> meet;
  __shared__ GateSums<V> sums;
  GateSpot<V> at;
  const int64_t id = seq_block(), cols = (int64_t)s.groups * s.B;
  if (id >= cols) return;
  at.at(s, gate_column((uint32_t)id, (uint32_t)cols, s.split));
  const int window = 2 * at.waves * kGateStep, steps = at.len;
  const int slot = (2 * at.wave + at.upper) * kGateStep;  // its first step in a window
  const int64_t col = (int64_t)at.b * s.D + at.c;
  int t = s.T > 0 ? (s.T - 1) / window * window : -window;
  for (; t >= 0 && t >= steps; t -= window) gate_blank<E, V, I, Z>(s, at, t, slot, s.T);
  GateInputs<E, V, I, Z> in, next;
  if (t >= 0) next.template load<false>(s, at, t, slot, steps - 1 - t);
  const GateBias<V> bias(s, at, I);
  if (s.part) gate_clear_sums<V>(sums, at);
  if (threadIdx.x < kGateLanes)
#pragma unroll
    for (int j = 0; j < V; ++j) meet.carry[0][at.lane][j] = s.gstate ? s.gstate[col + j] : 0.0f;
  int turn = 0;
  // WHOLE: every slot's steps hold text.  NEXT: another window follows (full of text), and
  // is on its way while this one is worked on.
  auto work = [&](auto whole, auto follows) {
    constexpr bool WHOLE = decltype(whole)::value;
    in = next;
    if constexpr (decltype(follows)::value)
      next.template load<true>(s, at, t - window, slot, 0);
    const int n = steps - t - slot;  // the slot's steps that hold text
    GateBackward<E, V, I, Z> way;
    float c[V];
    const GatePair<V> mine = way.template enter<WHOLE>(s, at, t, slot, s.T, n, in, bias);
    gate_fold<true>(meet, turn, at, mine, c);
    way.template leave<WHOLE, false>(s, at, t, slot, s.T, n, in.x, sums, c);
    t -= window;
    turn ^= 1;
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  // (only the first window, the row's last, can be short of text)
  if (t > 0 && t + window > steps) work(no, yes);
  while (t > 0) work(yes, yes);
  if (t == 0) {
    if (window <= steps) work(yes, no);
    else work(no, no);
  }
  __syncthreads();
  if (threadIdx.x < kGateLanes && s.gstate0)
    pack_store<true, float, V>(s.gstate0 + col, meet.carry[turn][at.lane], V);
  if (s.part) gate_part<V>(s, at, sums, at.b);
}

// A window of a column a workgroup.  Two run on a CU where a thread has 128 registers:
// with fp32 (81 to 110), and with 16-bit types without gates of their own, which are held
// there (127; 2048 steps of 64 columns: 30.5 us, and 34.6 with the 129 they would take).
// With such gates (148 to 190) one does: held to 128 it spills, 94 -> 139 us.  80 columns
// of 777 steps, fp16: 21 us.
template <typename E, int V, bool I, bool Z>
__global__ __launch_bounds__(64 * kGateWaves, V == 2 && !I && !Z ? 4 : 2) void gate_bwd_chain(const GateArgs<E> s) {
  __shared__ GateChain<V> chain;
  __shared__ GateSums<V> sums;
  GateSpot<V> at;
  int behind;  // windows behind this one
  if (!gate_number(chain, s, at, &behind)) return;
  const int index = s.windows - 1 - behind;
  const int window = 2 * at.waves * kGateStep, t = index * window, t1 = min(t + window, s.T);
  const int slot = (2 * at.wave + at.upper) * kGateStep;
  const int64_t col = (int64_t)at.b * s.D + at.c;
  const GateBias<V> bias(s, at, I);
  if (t >= at.len) {  // behind the text; a row without any hands its adjoint on
    gate_blank<E, V, I, Z>(s, at, t, slot, t1);
    if (s.part) gate_clear_sums<V>(sums, at);
    if (t == 0 && s.gstate0 && threadIdx.x < kGateLanes)
#pragma unroll
      for (int j = 0; j < V; ++j) s.gstate0[col + j] = s.gstate ? s.gstate[col + j] : 0.0f;
  } else {
    auto work = [&](auto whole) {  // whether every slot's steps hold text
      constexpr bool WHOLE = decltype(whole)::value;
      const int n = at.len - t - slot;
      GateInputs<E, V, I, Z> in;
      in.template load<WHOLE>(s, at, t, slot, at.len - 1 - t);
      GateBackward<E, V, I, Z> way;
      float c[V];
      const GatePair<V> mine = way.template enter<WHOLE>(s, at, t, slot, t1, n, in, bias);
      const int number = (at.len - 1) / window - index;
      const GatePair<V> before =
          gate_chain<true>(chain, s, at, number, index == 0, s.gstate, mine, c);
      if (index == 0 && s.gstate0 && at.wave == 0 && !at.upper)
        pack_store<true, float, V>(s.gstate0 + col, before.h, V);
      way.template leave<WHOLE, true>(s, at, t, slot, t1, n, in.x, sums, c);
    };
    if (t + window <= at.len) work(std::true_type());
    else work(std::false_type());
  }
  if (s.part) gate_part<V>(s, at, sums, (int64_t)index * s.B + at.b);
}

// g_f_bias and g_i_bias: the workgroups' sums, in their order.  A wave an output's 64
// channels would have long walks: kBiasRows threads share them (4.7 us for 8 rows of
// 2 x 2048 channels: latency).
constexpr int kBiasCols = 32, kBiasRows = 8;
__global__ __launch_bounds__(kBiasCols * kBiasRows) void gate_bias_sum(
    const float* part, int D, int64_t rows, float* g_f, float* g_i) {
  __shared__ double lds[kBiasRows][kBiasCols];
  const int x = threadIdx.x % kBiasCols, y = threadIdx.x / kBiasCols;
  const int64_t o = seq_block() * kBiasCols + x;
  double sum = 0.0;
  if (o < 2 * (int64_t)D)
#pragma unroll 4
    for (int64_t r = y; r < rows; r += kBiasRows) sum += (double)part[r * 2 * D + o];
  lds[y][x] = sum;
  __syncthreads();
  if (y != 0 || o >= 2 * (int64_t)D) return;
  for (int k = 1; k < kBiasRows; ++k) sum += lds[k][x];
  float* to = o < D ? g_f : g_i;
  if (to) to[o < D ? o : o - D] = (float)sum;
}

template <typename E, int V, bool I, bool Z>
void gate_start(const GateArgs<E>& a, const GatePlan& p, hipStream_t stream) {
  const dim3 grid = seq_grid((int64_t)p.groups * a.B * p.windows);
  if (p.windows > 1) gate_bwd_chain<E, V, I, Z><<<grid, 64 * p.waves, 0, stream>>>(a);
  else gate_bwd<E, V, I, Z><<<grid, 64 * p.waves, 0, stream>>>(a);
}

template <typename E, int V>
ck_status gate_launch(const GateArgs<E>& a, const GatePlan& p, float* g_f, float* g_i,
                      hipStream_t stream) {
  if (a.i.p && a.z.p) gate_start<E, V, true, true>(a, p, stream);
  else if (a.i.p) gate_start<E, V, true, false>(a, p, stream);
  else if (a.z.p) gate_start<E, V, false, true>(a, p, stream);
  else gate_start<E, V, false, false>(a, p, stream);
  if (a.part)
    gate_bias_sum<<<seq_grid((2 * (int64_t)a.D + kBiasCols - 1) / kBiasCols), kBiasCols * kBiasRows,
                    0, stream>>>(a.part, a.D, (int64_t)a.B * p.windows, g_f, g_i);
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
