// conv.hip -- short causal convolution: forward, backward and single-token
// step.
//
//   p_t = bias + sum_k w_k x_{t - (W-1) + k},   y_t = p_t or p_t sigmoid(p_t)
//
// HBM bounds all three (2 W + 4 operations an element against 4 to 8 bytes):
// a thread owns four adjacent channels and walks a run of steps with the last
// W - 1 inputs in registers, so that within a run every input is read once; a
// run reads W - 1 steps before it again (and after it, in the backward).  The
// next four rows are in flight while four are worked on.  Measured, W = 4, bf16,
// silu: 2048 steps x 8 rows x 2048 channels forward 28 us (5.1 TB/s, what a copy
// reaches), backward 48 to 55 us (4.0 to 4.5 TB/s, three waves a SIMD) and 5 us for
// its sums, 82 for the pass; ragged prompts of 1023 x 16 x 1025 fp16 channels (rows
// at odd addresses) 16.8 us, 3.6 TB/s; 256 tokens of 2048 channels 4.6 us, mostly
// the launch.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ck.h"
#include "ck_internal.h"
#include "sequence.h"

namespace ckhip {
namespace {

constexpr int64_t kConvMaxW = 8;
constexpr int kConvThreads = 256;
constexpr int kConvRun = 16;     // steps per thread, forward
constexpr int kConvAhead = 4;    // rows in flight: loaded while the ones before are worked on
// and backward, whose run reads 2 (W - 1) steps more: the shortest with which all
// workgroups run at once, as many a CU as registers allow (1000 x 32 x 500 bf16, all
// of a training pass: 53 us in 672 workgroups of runs of 24; 58 in 1008 of 16).  Runs
// of 8 where even those would fit: 1816 x 14 x 152 bf16 32 us against 30.
constexpr int kConvRunBwdMax = 48, kConvRunBwdMin = 16;
constexpr int64_t kConvCus = 256;
constexpr int kConvV = 4;        // channels per thread
// (a step's bytes, 4 an element and fewer, in 32 bits: see Rows)
constexpr int64_t kConvMaxStrideT = (int64_t(1) << 30) - 1;

template <typename E>
struct ConvArgs {
  Seq<const E> x, gy;
  Seq<E> y, gx;
  const float *weight, *bias;
  const E *state0, *gstate;
  E *state, *gstate0;
  const int32_t* lengths;
  float* part;   // backward: [parts][W + 1][D]
  int T, B, D;
  int nv;        // channel groups of kConvV
  int vx;        // of them per workgroup (at most 64)
  int pairs;     // (row, run) pairs per workgroup: 256 / vx
  int runs;      // runs of the window
  int run;       // steps of a run (a multiple of kConvAhead)
  int silu;
};

struct ConvPlace {
  int b, run, c, len;
  int n;        // channels of this group (fewer than kConvV only if D is)
  int again;    // of them, those that the group before has too
  bool active;
};

// Workgroup: vx channel groups times `pairs` (row, run) pairs.  A last group that
// would be short begins earlier and writes what its neighbour writes: with code of
// its own, element by element, it made its whole wave wait (256 steps x 24 x 498
// channels, bf16: forward 14 us against 8, backward 36 against 15).
template <typename E>
__device__ __forceinline__ ConvPlace conv_place(const ConvArgs<E>& s) {
  ConvPlace p;
  const int vblocks = (s.nv + s.vx - 1) / s.vx;
  const int vi = (int)(blockIdx.x % vblocks) * s.vx + (int)threadIdx.x % s.vx;
  const int ty = (int)threadIdx.x / s.vx;
  const int64_t br = (int64_t)(blockIdx.x / vblocks) * s.pairs + ty;
  p.active = vi < s.nv && ty < s.pairs && br < (int64_t)s.B * s.runs;
  p.c = max(min(vi * kConvV, s.D - kConvV), 0);
  p.n = s.D - p.c;
  p.again = vi * kConvV - p.c;
  p.run = (int)(br % s.runs);
  p.b = (int)min(br / s.runs, (int64_t)s.B - 1);
  p.len = s.T;
  if (s.lengths) p.len = min(max(s.lengths[p.b], 0), s.T);
  return p;
}

constexpr int V = kConvV;

template <bool FULL, int W>
__device__ __forceinline__ void conv_weights(float (&w)[W][V], float (&bias)[V],
                                             const float* weight, const float* b, int c, int n) {
  const Pack<float, V * W> wp =
      pack_load<FULL, float, V * W>(weight + (int64_t)c * W, n * W);
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = wp.v[i * W + k];
  Pack<float, V> bp = {};
  if (b) bp = pack_load<FULL, float, V>(b + c, n);
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = bp.v[i];
}

// Input at step t, which may lie before the window (state0) but not at or
// past the row's length.
template <bool FULL, int W, typename E>
__device__ __forceinline__ void conv_input(float (&x)[V], const ConvArgs<E>& s,
                                           const ConvPlace& p, int t) {
  Pack<E, V> v = {};
  if (t >= 0)
    v = pack_load<FULL, E, V>(s.x.row(t, p.b) + p.c, p.n);
  else if (s.state0)
    v = pack_load<FULL, E, V>(s.state0 + ((int64_t)(t + W - 1) * s.B + p.b) * s.D + p.c, p.n);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = (float)v.v[i];
}

// Rows rel .. rel + kConvAhead - 1 of a run, those past `last` replaced by it.
template <bool FULL, typename E>
__device__ __forceinline__ void conv_rows(Pack<E, V> (&r)[kConvAhead], const Rows<const E>& rows,
                                          int rel, int last, int n) {
#pragma unroll
  for (int i = 0; i < kConvAhead; ++i)
    r[i] = pack_load<FULL, E, V>(rows.at(min(rel + i, last)), n);
}

template <bool FULL, int W, typename E>
__device__ __forceinline__ void conv_fwd_run(const ConvArgs<E>& s, const ConvPlace& p) {
  const int t0 = p.run * kConvRun, t1 = min(t0 + kConvRun, s.T);
  const int te = min(t1, p.len), n = te - t0;
  Rows<E> ry(s.y, t0, p.b, p.c);
  if (n > 0) {
    float w[W][V], bias[V];
    Pack<E, V> now[kConvAhead], next[kConvAhead];
    const Rows<const E> rx(s.x, t0, p.b, p.c);
    conv_rows<FULL>(now, rx, 0, n - 1, p.n);
    conv_weights<FULL, W>(w, bias, s.weight, s.bias, p.c, p.n);
    float x[W][V];  // steps t - W + 1 .. t
#pragma unroll
    for (int k = 0; k < W - 1; ++k) conv_input<FULL, W>(x[k], s, p, t0 - (W - 1) + k);
    for (int t = 0; t < n; t += kConvAhead) {
      if (t + kConvAhead < n) conv_rows<FULL>(next, rx, t + kConvAhead, n - 1, p.n);
#pragma unroll
      for (int j = 0; j < kConvAhead; ++j) {
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          x[W - 1][i] = (float)now[j].v[i];
          float a = bias[i];
#pragma unroll
          for (int k = 0; k < W; ++k) a = fmaf(w[k][i], x[k][i], a);
          y[i] = s.silu ? a * sigmoid_hw(a) : a;
#pragma unroll
          for (int k = 0; k + 1 < W; ++k) x[k][i] = x[k + 1][i];
        }
        if (t + j < n) pack_store<FULL, E, V>(ry.at(t + j), y, p.n);
      }
#pragma unroll
      for (int j = 0; j < kConvAhead; ++j) now[j] = next[j];
    }
  }
  const float zero[V] = {};
  for (int t = max(n, 0); t < t1 - t0; ++t) pack_store<FULL, E, V>(ry.at(t), zero, p.n);
  if (s.state && p.run == max(p.len - 1, 0) / kConvRun) {
    for (int k = 0; k < W - 1; ++k) {
      float x[V];
      conv_input<FULL, W>(x, s, p, p.len - (W - 1) + k);
      pack_store<FULL, E, V>(s.state + ((int64_t)k * s.B + p.b) * s.D + p.c, x, p.n);
    }
  }
}

template <typename E, int W>
__global__ __launch_bounds__(kConvThreads) void conv_fwd(const ConvArgs<E> s) {
  const ConvPlace p = conv_place(s);
  if (!p.active) return;
  if (p.n >= V)
    conv_fwd_run<true, W>(s, p);
  else
    conv_fwd_run<false, W>(s, p);
}

template <bool FULL, int W, typename E>
__device__ __forceinline__ void conv_bwd_run(float (&gw)[W + 1][V], const ConvArgs<E>& s,
                                             const ConvPlace& p) {
  // steps are counted from the run's first; step t completes the gradient of
  // the input W - 1 steps earlier, so the run goes on for W - 1 steps behind
  // its own, and run 0 starts with the gradients of state0
  const int t0 = p.run * s.run, t1 = min(s.run, s.T - t0);
  const int len = p.len - t0, last = min(len, t1 + W - 1) - 1;
  const Rows<const E> rx(s.x, t0, p.b, p.c), rg(s.gy, t0, p.b, p.c);
  Rows<E> ro(s.gx, t0, p.b, p.c);
  float w[W][V], bias[V], x[W][V], ga[W][V];  // ga: dL/dp of steps t - W + 1 .. t
  Pack<E, V> xn[kConvAhead] = {}, gn[kConvAhead] = {};
  if (last >= 0) {
    conv_rows<FULL>(xn, rx, 0, last, p.n);
    conv_rows<FULL>(gn, rg, 0, last, p.n);
  }
  conv_weights<FULL, W>(w, bias, s.weight, s.bias, p.c, p.n);
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) ga[k][i] = x[k][i] = 0.0f;
  if (last >= 0) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) conv_input<FULL, W>(x[k], s, p, t0 - (W - 1) + k);
  }
  // OWN: the weights' gradients of these steps are this run's
  auto steps = [&](auto own, int tb) {
    constexpr bool OWN = decltype(own)::value;
    Pack<E, V> xp[kConvAhead] = {}, gp[kConvAhead] = {};
    if (tb + kConvAhead <= last) {
      conv_rows<FULL>(xp, rx, tb + kConvAhead, last, p.n);
      conv_rows<FULL>(gp, rg, tb + kConvAhead, last, p.n);
    }
#pragma unroll
    for (int j = 0; j < kConvAhead; ++j) {
      const int t = tb + j;
      // Past the text (as a run's own steps past its end are) dL/dp is 0 whatever the
      // loads, of its last row, make of it; and nothing is added to the weights'
      // gradients, since 0 times an infinite input of the window would be.
      const bool in = t <= last;
      float gx[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[W - 1][i] = (float)xn[j].v[i];
        float g = (float)gn[j].v[i];
        if (s.silu) {
          float a = bias[i];
#pragma unroll
          for (int k = 0; k < W; ++k) a = fmaf(w[k][i], x[k][i], a);
          const float sg = sigmoid_hw(a);
          g *= sg * fmaf(a, 1.0f - sg, 1.0f);
        }
        ga[W - 1][i] = in ? g : 0.0f;
        if (OWN && in) {
#pragma unroll
          for (int k = 0; k < W; ++k) gw[k][i] = fmaf(ga[W - 1][i], x[k][i], gw[k][i]);
          gw[W][i] += ga[W - 1][i];
        }
        gx[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) gx[i] = fmaf(w[k][i], ga[W - 1 - k][i], gx[i]);
#pragma unroll
        for (int k = 0; k + 1 < W; ++k) {
          x[k][i] = x[k + 1][i];
          ga[k][i] = ga[k + 1][i];
        }
      }
      const int ti = t - (W - 1);       // the input whose gradient is complete
      const int slot = ti - len + W - 1;  // its row in the final state
      if (s.gstate && slot >= 0 && slot < W - 1 && t < t1 + W - 1) {
        const Pack<E, V> gs =
            pack_load<FULL, E, V>(s.gstate + ((int64_t)slot * s.B + p.b) * s.D + p.c, p.n);
#pragma unroll
        for (int i = 0; i < V; ++i) gx[i] += (float)gs.v[i];
      }
      if (ti >= 0 && ti < t1) {
        if (ti >= len) {
#pragma unroll
          for (int i = 0; i < V; ++i) gx[i] = 0.0f;
        }
        pack_store<FULL, E, V>(ro.at(ti), gx, p.n);
      } else if (ti + t0 < 0 && t < t1 + W - 1 && s.gstate0) {
        pack_store<FULL, E, V>(s.gstate0 + ((int64_t)t * s.B + p.b) * s.D + p.c, gx, p.n);
      }
    }
#pragma unroll
    for (int j = 0; j < kConvAhead; ++j) {
      xn[j] = xp[j];
      gn[j] = gp[j];
    }
  };
  for (int t = 0; t < t1; t += kConvAhead) steps(std::true_type(), t);
  // (behind a shorter run, the window's last, no text follows)
  const int tail = (t1 + kConvAhead - 1) / kConvAhead * kConvAhead;
#pragma unroll
  for (int t = 0; t < W - 1; t += kConvAhead) steps(std::false_type(), tail + t);
}

// (as many waves a SIMD as conv_dims_backward counts on)
template <typename E, int W>
__global__ __launch_bounds__(kConvThreads, W <= 4 ? 3 : 2) void conv_bwd(const ConvArgs<E> s) {
  __shared__ float red[kConvThreads * V];  // [pairs of the workgroup][vx * V]
  const ConvPlace p = conv_place(s);
  float gw[W + 1][V];
#pragma unroll
  for (int k = 0; k <= W; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) gw[k][i] = 0.0f;
  if (p.active) {
    if (p.n >= V)
      conv_bwd_run<true, W>(gw, s, p);
    else
      conv_bwd_run<false, W>(gw, s, p);
  }
  // the workgroup's (row, run) pairs, summed in order, one tap at a time
  const int n = s.vx * V;
  const int vi = (int)threadIdx.x % s.vx, ty = (int)threadIdx.x / s.vx;
  const int vblocks = (s.nv + s.vx - 1) / s.vx;
  const int c0 = (int)(blockIdx.x % vblocks) * n;
  float* part = s.part + (int64_t)(blockIdx.x / vblocks) * (W + 1) * s.D + c0;
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i >= p.again) red[ty * n + vi * V + i - p.again] = gw[k][i];
    __syncthreads();
    for (int e = threadIdx.x; e < n && c0 + e < s.D; e += kConvThreads) {
      float sum = 0.0f;
      for (int r = 0; r < s.pairs; ++r) sum += red[r * n + e];
      part[(int64_t)k * s.D + e] = sum;
    }
  }
}

// Gradients of the weights and the bias: the workgroups' sums in a fixed
// order.  A workgroup takes 32 sums, eight threads each one a stretch of the
// parts.
template <int W>
__global__ __launch_bounds__(256) void conv_sum(const float* part, int D, int64_t parts,
                                                float* gw, float* gbias) {
  __shared__ float red[8][32];
  const int64_t n = (int64_t)D * (W + 1), i = seq_block() * 32 + (threadIdx.x & 31);
  const int y = threadIdx.x >> 5;
  const int64_t each = (parts + 7) / 8, r0 = each * y, r1 = min(r0 + each, parts);
  float sum = 0.0f;
  if (i < n) {
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) sum += part[r * n + i];
  }
  red[y][threadIdx.x & 31] = sum;
  __syncthreads();
  if (y != 0 || i >= n) return;
  sum = 0.0f;
  for (int j = 0; j < 8; ++j) sum += red[j][threadIdx.x];
  const int k = (int)(i / D), d = (int)(i % D);
  if (k < W)
    gw[(int64_t)d * W + k] = sum;
  else if (gbias)
    gbias[d] = sum;
}

template <bool FULL, int W, typename E>
__device__ __forceinline__ void conv_one_row(const ConvArgs<E>& s, const ConvPlace& p) {
  float w[W][V], bias[V], x[W][V], y[V];
#pragma unroll
  for (int k = 0; k < W; ++k) conv_input<FULL, W>(x[k], s, p, k - (W - 1));
  conv_weights<FULL, W>(w, bias, s.weight, s.bias, p.c, p.n);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float a = bias[i];
#pragma unroll
    for (int k = 0; k < W; ++k) a = fmaf(w[k][i], x[k][i], a);
    y[i] = s.silu ? a * sigmoid_hw(a) : a;
  }
  pack_store<FULL, E, V>(s.y.row(0, p.b) + p.c, y, p.n);
#pragma unroll
  for (int k = 0; k + 1 < W; ++k)
    pack_store<FULL, E, V>(s.state + ((int64_t)k * s.B + p.b) * s.D + p.c, x[k + 1], p.n);
}

template <typename E, int W>
__global__ __launch_bounds__(kConvThreads) void conv_one(const ConvArgs<E> s) {
  const int64_t i0 = seq_block() * kConvThreads + threadIdx.x;
  if (i0 >= (int64_t)s.B * s.nv) return;
  ConvPlace p = {};
  p.b = (int)(i0 / s.nv);
  p.c = (int)(i0 % s.nv) * V;
  p.n = s.D - p.c;
  if (p.n >= V)
    conv_one_row<true, W>(s, p);
  else
    conv_one_row<false, W>(s, p);
}

struct ConvDims {
  int nv, vx, pairs, run, runs;
  int64_t vblocks, pblocks;  // workgroups over the channels, over the (row, run) pairs
};
ConvDims conv_dims(const ck_conv_shape& s, int run) {
  ConvDims d;
  d.nv = (int)((s.D + kConvV - 1) / kConvV);
  // (as many groups in each workgroup as in the others: of 256 threads 228 have
  // work at 152 channels, 152 if a row took 64)
  d.vblocks = (d.nv + 63) / 64;
  d.vx = (int)((d.nv + d.vblocks - 1) / d.vblocks);
  d.pairs = kConvThreads / d.vx;
  d.run = run;
  d.runs = (int)std::max<int64_t>((s.T + run - 1) / run, 1);
  d.pblocks = (s.B * d.runs + d.pairs - 1) / d.pairs;
  return d;
}

ck_status conv_check_shape(const ck_conv_shape* s) {
  if (!s) {
    set_error("shape is NULL");
    return CK_ERR_NULL_ARG;
  }
  const ck_status rc = seq_check_shape(s->T, s->B, s->D, s->dtype);
  if (rc != CK_OK) return rc;
  if (s->W < 1 || s->W > kConvMaxW) {
    set_error("W must be in [1, 8] (got %lld)", (long long)s->W);
    return CK_ERR_BAD_SIZE;
  }
  // (the backward's runs are no shorter)
  const ConvDims d = conv_dims(*s, kConvRun);
  if (d.pblocks >= kSeqMaxThreads / kConvThreads / d.vblocks) {
    set_error("T=%lld, B=%lld or D=%lld is too large", (long long)s->T, (long long)s->B,
              (long long)s->D);
    return CK_ERR_TOO_LARGE;
  }
  return CK_OK;
}

ck_status conv_check_state(const void* p, const ck_conv_shape& s, bool optional, const char* what) {
  if (s.W == 1) return CK_OK;  // a state of no elements
  return seq_check(ck_seq{const_cast<void*>(p), 0, 0}, s.dtype, optional, what);
}

ck_status conv_check_out(const ck_conv_shape& s, const ck_seq& q, bool optional,
                         const char* what) {
  return seq_check_out(q, s.T, s.B, s.D, s.dtype, optional, what, kConvMaxStrideT);
}

ConvDims conv_dims_backward(const ck_conv_shape& s) {
  const int64_t round = kConvCus * (s.W <= 4 ? 3 : 2);
  ConvDims d = conv_dims(s, kConvRunBwdMax);
  for (int run = kConvRunBwdMax; run >= kConvRunBwdMin; run -= kConvAhead) {
    const ConvDims shorter = conv_dims(s, run);
    if (shorter.vblocks * shorter.pblocks > round) break;
    d = shorter;
  }
  return d;
}

template <typename E>
ConvArgs<E> conv_args(const ck_conv_shape& s, const ck_seq& x, const float* weight,
                      const float* bias, const void* state0, const int32_t* lengths) {
  ConvArgs<E> a = {};
  a.x = seq_of<const E>(x);
  a.weight = weight;
  a.bias = bias;
  a.state0 = s.W > 1 ? static_cast<const E*>(state0) : nullptr;
  a.lengths = lengths;
  a.T = (int)s.T; a.B = (int)s.B; a.D = (int)s.D;
  a.silu = s.silu;
  return a;
}

template <typename F>
void conv_by_width(int W, F&& fn) {
  switch (W) {
    case 1: fn(std::integral_constant<int, 1>()); break;
    case 2: fn(std::integral_constant<int, 2>()); break;
    case 3: fn(std::integral_constant<int, 3>()); break;
    case 4: fn(std::integral_constant<int, 4>()); break;
    case 5: fn(std::integral_constant<int, 5>()); break;
    case 6: fn(std::integral_constant<int, 6>()); break;
    case 7: fn(std::integral_constant<int, 7>()); break;
    default: fn(std::integral_constant<int, 8>()); break;
  }
}

}  // namespace
}  // namespace ckhip

using namespace ckhip;

extern "C" ck_status ck_conv_sizes(const ck_conv_shape* shape, size_t* workspace_bytes) {
  clear_error();
  const ck_status rc = conv_check_shape(shape);
  if (rc != CK_OK) return rc;
  const size_t need =
      (size_t)conv_dims_backward(*shape).pblocks * shape->D * (shape->W + 1) * 4;
  if (workspace_bytes) *workspace_bytes = need;
  return CK_OK;
}

extern "C" ck_status ck_conv_forward(const ck_conv_shape* shape, ck_seq x, const float* weight,
                                     const float* bias, const void* state0,
                                     const int32_t* lengths, ck_seq y, void* state,
                                     hipStream_t stream) {
  clear_error();
  ck_status rc = conv_check_shape(shape);
  if (rc != CK_OK) return rc;
  const bool none = shape->T == 0;
  if (!weight) {
    set_error("weight is NULL");
    return CK_ERR_NULL_ARG;
  }
  rc = seq_check(x, shape->dtype, none, "x", kConvMaxStrideT);
  if (rc == CK_OK) rc = conv_check_out(*shape, y, none, "y");
  if (rc == CK_OK) rc = conv_check_state(state0, *shape, true, "state0");
  if (rc == CK_OK) rc = conv_check_state(state, *shape, true, "state");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    conv_by_width((int)shape->W, [&](auto w) {
      constexpr int W = decltype(w)::value;
      const ConvDims d = conv_dims(*shape, kConvRun);
      ConvArgs<E> a = conv_args<E>(*shape, x, weight, bias, state0, lengths);
      a.y = seq_of<E>(y);
      a.state = W > 1 ? static_cast<E*>(state) : nullptr;
      a.nv = d.nv; a.vx = d.vx; a.pairs = d.pairs; a.run = d.run; a.runs = d.runs;
      conv_fwd<E, W><<<(unsigned)(d.vblocks * d.pblocks), kConvThreads, 0, stream>>>(a);
    });
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}

extern "C" ck_status ck_conv_backward(const ck_conv_shape* shape, ck_seq x, const float* weight,
                                      const float* bias, const void* state0,
                                      const int32_t* lengths, ck_seq grad_y,
                                      const void* grad_state, ck_seq grad_x, float* grad_weight,
                                      float* grad_bias, void* grad_state0, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  ck_status rc = conv_check_shape(shape);
  if (rc != CK_OK) return rc;
  const bool none = shape->T == 0;
  if (!weight || !grad_weight) {
    set_error("weight or its gradient is NULL");
    return CK_ERR_NULL_ARG;
  }
  rc = seq_check(x, shape->dtype, none, "x", kConvMaxStrideT);
  if (rc == CK_OK) rc = seq_check(grad_y, shape->dtype, none, "grad_y", kConvMaxStrideT);
  if (rc == CK_OK) rc = conv_check_out(*shape, grad_x, none, "grad_x");
  if (rc == CK_OK) rc = conv_check_state(state0, *shape, true, "state0");
  if (rc == CK_OK) rc = conv_check_state(grad_state, *shape, true, "grad_state");
  if (rc == CK_OK) rc = conv_check_state(grad_state0, *shape, true, "grad_state0");
  if (rc != CK_OK) return rc;
  size_t need = 0;
  rc = ck_conv_sizes(shape, &need);
  if (rc == CK_OK) rc = seq_check_ws(workspace, workspace_bytes, need);
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    conv_by_width((int)shape->W, [&](auto w) {
      constexpr int W = decltype(w)::value;
      const ConvDims d = conv_dims_backward(*shape);
      ConvArgs<E> a = conv_args<E>(*shape, x, weight, bias, state0, lengths);
      a.gy = seq_of<const E>(grad_y);
      a.gx = seq_of<E>(grad_x);
      a.gstate = W > 1 ? static_cast<const E*>(grad_state) : nullptr;
      a.gstate0 = W > 1 ? static_cast<E*>(grad_state0) : nullptr;
      a.part = static_cast<float*>(workspace);
      a.nv = d.nv; a.vx = d.vx; a.pairs = d.pairs; a.run = d.run; a.runs = d.runs;
      conv_bwd<E, W><<<(unsigned)(d.vblocks * d.pblocks), kConvThreads, 0, stream>>>(a);
      conv_sum<W><<<seq_grid((shape->D * (W + 1) + 31) / 32), 256, 0, stream>>>(
          a.part, a.D, d.pblocks, grad_weight, grad_bias);
    });
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}

extern "C" ck_status ck_conv_step(const ck_conv_shape* shape, ck_seq x, const float* weight,
                                  const float* bias, const void* state0, ck_seq y, void* state,
                                  hipStream_t stream) {
  clear_error();
  ck_status rc = conv_check_shape(shape);
  if (rc != CK_OK) return rc;
  if (shape->T != 1) {
    set_error("a step takes T = 1 (got %lld)", (long long)shape->T);
    return CK_ERR_BAD_SIZE;
  }
  if (!weight) {
    set_error("weight is NULL");
    return CK_ERR_NULL_ARG;
  }
  rc = seq_check(x, shape->dtype, false, "x", kConvMaxStrideT);
  if (rc == CK_OK) rc = conv_check_out(*shape, y, false, "y");
  if (rc == CK_OK) rc = conv_check_state(state0, *shape, true, "state0");
  if (rc == CK_OK) rc = conv_check_state(state, *shape, false, "state");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    conv_by_width((int)shape->W, [&](auto w) {
      constexpr int W = decltype(w)::value;
      ConvArgs<E> a = conv_args<E>(*shape, x, weight, bias, state0, nullptr);
      a.y = seq_of<E>(y);
      a.state = W > 1 ? static_cast<E*>(state) : nullptr;
      a.nv = (int)((shape->D + kConvV - 1) / kConvV);
      const int64_t n = shape->B * a.nv;
      conv_one<E, W><<<seq_grid((n + kConvThreads - 1) / kConvThreads), kConvThreads, 0,
                       stream>>>(a);
    });
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}
