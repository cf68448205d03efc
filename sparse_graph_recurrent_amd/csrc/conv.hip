// conv.hip -- short causal convolution: forward, backward and single-token
// step.
//
//   p_t = bias + sum_k w_k x_{t - (W-1) + k},   y_t = p_t or p_t sigmoid(p_t)
//
// HBM bounds all three (2 W + 4 operations an element against 4 to 8 bytes):
// a thread owns V adjacent channels (16 bytes) and walks a run of steps with
// the last W - 1 inputs in registers, so that within a run every input is
// read once; a run reads W - 1 steps before it again (and after it, in the
// backward).
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
constexpr int kConvRunBwd = 32;  // and backward, whose run reads 2 (W - 1) steps more

template <typename E>
struct ConvArgs {
  Seq<const E> x, gy;
  Seq<E> y, gx;
  const float *weight, *bias;
  const E *state0, *gstate;
  E *state, *gstate0;
  const int32_t* lengths;
  float* part;   // backward: [parts][D][W + 1]
  int T, B, D;
  int nv;        // channel groups of V
  int vx;        // of them per workgroup (a power of two at most 64)
  int runs;      // runs of the window
  int silu;
};

struct ConvPlace {
  int b, run, c, len;
  bool active;
};

// Workgroup: vx channel groups times 256 / vx (row, run) pairs.
template <int V, typename E>
__device__ __forceinline__ ConvPlace conv_place(const ConvArgs<E>& s) {
  ConvPlace p;
  const int vblocks = (s.nv + s.vx - 1) / s.vx;
  const int vi = (int)(blockIdx.x % vblocks) * s.vx + ((int)threadIdx.x & (s.vx - 1));
  const int64_t br = (int64_t)(blockIdx.x / vblocks) * (kConvThreads / s.vx) +
                     (int)threadIdx.x / s.vx;
  p.active = vi < s.nv && br < (int64_t)s.B * s.runs;
  p.c = vi * V;
  p.run = (int)(br % s.runs);
  p.b = (int)min(br / s.runs, (int64_t)s.B - 1);
  p.len = s.T;
  if (s.lengths) p.len = min(max(s.lengths[p.b], 0), s.T);
  return p;
}

template <int V, int W>
__device__ __forceinline__ void conv_weights(float (&w)[W][V], float (&bias)[V],
                                             const float* weight, const float* b, int c) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = weight[(int64_t)(c + i) * W + k];
    bias[i] = b ? b[c + i] : 0.0f;
  }
}

// Input at step t, which may lie before the window (state0) but not at or
// past the row's length.
template <int V, int W, typename E>
__device__ __forceinline__ void conv_input(float (&x)[V], const ConvArgs<E>& s, int b, int c,
                                           int t) {
  if (t >= 0) {
    pack_load<E, V>(x, s.x.row(t, b) + c);
  } else if (s.state0) {
    pack_load<E, V>(x, s.state0 + ((int64_t)(t + W - 1) * s.B + b) * s.D + c);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = 0.0f;
  }
}

template <typename E, int V, int W>
__global__ __launch_bounds__(kConvThreads) void conv_fwd(const ConvArgs<E> s) {
  const ConvPlace p = conv_place<V>(s);
  if (!p.active) return;
  const int t0 = p.run * kConvRun, t1 = min(t0 + kConvRun, s.T);
  const int te = min(t1, p.len);
  float w[W][V], bias[V];
  conv_weights<V, W>(w, bias, s.weight, s.bias, p.c);
  if (t0 < te) {
    float x[W][V];  // steps t - W + 1 .. t
#pragma unroll
    for (int k = 0; k < W - 1; ++k) conv_input<V, W>(x[k], s, p.b, p.c, t0 - (W - 1) + k);
#pragma unroll 4
    for (int t = t0; t < te; ++t) {
      pack_load<E, V>(x[W - 1], s.x.row(t, p.b) + p.c);
      float y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float a = bias[i];
#pragma unroll
        for (int k = 0; k < W; ++k) a = fmaf(w[k][i], x[k][i], a);
        y[i] = s.silu ? a * sigmoid_hw(a) : a;
#pragma unroll
        for (int k = 0; k + 1 < W; ++k) x[k][i] = x[k + 1][i];
      }
      pack_store<E, V>(s.y.row(t, p.b) + p.c, y);
    }
  }
  const float zero[V] = {};
  for (int t = max(t0, te); t < t1; ++t) pack_store<E, V>(s.y.row(t, p.b) + p.c, zero);
  if (s.state && p.run == max(p.len - 1, 0) / kConvRun) {
    for (int k = 0; k < W - 1; ++k) {
      float x[V];
      conv_input<V, W>(x, s, p.b, p.c, p.len - (W - 1) + k);
      pack_store<E, V>(s.state + ((int64_t)k * s.B + p.b) * s.D + p.c, x);
    }
  }
}

template <typename E, int V, int W>
__global__ __launch_bounds__(kConvThreads) void conv_bwd(const ConvArgs<E> s) {
  __shared__ float red[kConvThreads * V];  // [pairs of the workgroup][vx * V]
  const ConvPlace p = conv_place<V>(s);
  float gw[W + 1][V];
#pragma unroll
  for (int k = 0; k <= W; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) gw[k][i] = 0.0f;
  if (p.active) {
    const int t0 = p.run * kConvRunBwd, t1 = min(t0 + kConvRunBwd, s.T);
    float w[W][V], bias[V], x[W][V], ga[W][V];  // ga: dL/dp of steps t - W + 1 .. t
    conv_weights<V, W>(w, bias, s.weight, s.bias, p.c);
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) ga[k][i] = 0.0f;
    if (t0 < p.len) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) conv_input<V, W>(x[k], s, p.b, p.c, t0 - (W - 1) + k);
    }
    // step t completes the gradient of the input W - 1 steps earlier; run 0
    // starts with those of state0
#pragma unroll 2
    for (int t = t0; t < t1 + W - 1; ++t) {
      if (t < p.len) {
        float g[V];
        pack_load<E, V>(x[W - 1], s.x.row(t, p.b) + p.c);
        pack_load<E, V>(g, s.gy.row(t, p.b) + p.c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (s.silu) {
            float a = bias[i];
#pragma unroll
            for (int k = 0; k < W; ++k) a = fmaf(w[k][i], x[k][i], a);
            const float sg = sigmoid_hw(a);
            g[i] *= sg * fmaf(a, 1.0f - sg, 1.0f);
          }
          ga[W - 1][i] = g[i];
          if (t < t1) {
#pragma unroll
            for (int k = 0; k < W; ++k) gw[k][i] = fmaf(g[i], x[k][i], gw[k][i]);
            gw[W][i] += g[i];
          }
#pragma unroll
          for (int k = 0; k + 1 < W; ++k) x[k][i] = x[k + 1][i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) ga[W - 1][i] = 0.0f;
      }
      const int ti = t - (W - 1);  // the input whose gradient is complete
      float gx[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        gx[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) gx[i] = fmaf(w[k][i], ga[W - 1 - k][i], gx[i]);
#pragma unroll
        for (int k = 0; k + 1 < W; ++k) ga[k][i] = ga[k + 1][i];
      }
      const int slot = ti - p.len + W - 1;  // its row in the final state
      if (s.gstate && slot >= 0 && slot < W - 1) {
        float gs[V];
        pack_load<E, V>(gs, s.gstate + ((int64_t)slot * s.B + p.b) * s.D + p.c);
#pragma unroll
        for (int i = 0; i < V; ++i) gx[i] += gs[i];
      }
      if (ti >= t0) {
        if (ti >= p.len) {
#pragma unroll
          for (int i = 0; i < V; ++i) gx[i] = 0.0f;
        }
        pack_store<E, V>(s.gx.row(ti, p.b) + p.c, gx);
      } else if (ti < 0 && s.gstate0) {
        pack_store<E, V>(s.gstate0 + ((int64_t)t * s.B + p.b) * s.D + p.c, gx);
      }
    }
  }
  // the workgroup's (row, run) pairs, summed in order, one tap at a time
  const int n = s.vx * V, pairs = kConvThreads / s.vx;
  const int vi = (int)threadIdx.x & (s.vx - 1), ty = (int)threadIdx.x / s.vx;
  const int vblocks = (s.nv + s.vx - 1) / s.vx;
  const int c0 = (int)(blockIdx.x % vblocks) * n;
  float* part = s.part + ((int64_t)(blockIdx.x / vblocks) * s.D + c0) * (W + 1);
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) red[ty * n + vi * V + i] = gw[k][i];
    __syncthreads();
    for (int e = threadIdx.x; e < n && c0 + e < s.D; e += kConvThreads) {
      float sum = 0.0f;
      for (int r = 0; r < pairs; ++r) sum += red[r * n + e];
      part[(int64_t)e * (W + 1) + k] = sum;
    }
  }
}

// Gradients of the weights and the bias: the workgroups' sums, in order.
template <int W>
__global__ __launch_bounds__(256) void conv_sum(const float* part, int64_t D, int64_t parts,
                                                float* gw, float* gbias) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= D * (W + 1)) return;
  const int k = (int)(i % (W + 1));
  float sum = 0.0f;
  for (int64_t r = 0; r < parts; ++r) sum += part[r * D * (W + 1) + i];
  if (k < W)
    gw[i / (W + 1) * W + k] = sum;
  else if (gbias)
    gbias[i / (W + 1)] = sum;
}

template <typename E, int V, int W>
__global__ __launch_bounds__(kConvThreads) void conv_one(const ConvArgs<E> s) {
  const int64_t i0 = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  if (i0 >= (int64_t)s.B * s.nv) return;
  const int b = (int)(i0 / s.nv), c = (int)(i0 % s.nv) * V;
  float w[W][V], bias[V], x[W][V], y[V];
  conv_weights<V, W>(w, bias, s.weight, s.bias, c);
#pragma unroll
  for (int k = 0; k < W; ++k) conv_input<V, W>(x[k], s, b, c, k - (W - 1));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float a = bias[i];
#pragma unroll
    for (int k = 0; k < W; ++k) a = fmaf(w[k][i], x[k][i], a);
    y[i] = s.silu ? a * sigmoid_hw(a) : a;
  }
  pack_store<E, V>(s.y.row(0, b) + c, y);
#pragma unroll
  for (int k = 0; k + 1 < W; ++k)
    pack_store<E, V>(s.state + ((int64_t)k * s.B + b) * s.D + c, x[k + 1]);
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
  // workgroups of one launch (a thread of the scalar path takes one channel)
  const int64_t pairs = s->B * (s->T / kConvRun + 1), nv = s->D;
  if ((pairs / 4 + 1) > INT_MAX / (nv / 32 + 1)) {
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

struct ConvDims {
  int nv, vx, runs;
  int64_t vblocks, pblocks;  // workgroups over the channels, over the (row, run) pairs
};
ConvDims conv_dims(const ck_conv_shape& s, int V, int run) {
  ConvDims d;
  d.nv = (int)(s.D / V);
  d.vx = 1;
  while (d.vx < 64 && d.vx < d.nv) d.vx *= 2;
  d.runs = (int)std::max<int64_t>((s.T + run - 1) / run, 1);
  d.vblocks = (d.nv + d.vx - 1) / d.vx;
  const int pairs = kConvThreads / d.vx;
  d.pblocks = (s.B * d.runs + pairs - 1) / pairs;
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

// fn(V, W) as constants: V the elements of 16 bytes when all rows of the
// call's tensors can be read so, else 1.
template <typename E, typename F>
void conv_by_kind(const ck_conv_shape& s, std::initializer_list<ck_seq> seqs,
                  std::initializer_list<const void*> states, F&& fn) {
  constexpr int V = 16 / sizeof(E);
  bool vec = s.D % V == 0;
  for (const ck_seq& q : seqs) vec = vec && seq_vec_ok<E, V>(q);
  for (const void* p : states) vec = vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  conv_by_width((int)s.W, [&](auto w) {
    if (vec)
      fn(std::integral_constant<int, V>(), w);
    else
      fn(std::integral_constant<int, 1>(), w);
  });
}

}  // namespace
}  // namespace ckhip

using namespace ckhip;

extern "C" ck_status ck_conv_sizes(const ck_conv_shape* shape, size_t* workspace_bytes) {
  clear_error();
  const ck_status rc = conv_check_shape(shape);
  if (rc != CK_OK) return rc;
  // enough for either path (the scalar path's workgroups take at most as many pairs)
  size_t need = 0;
  for (int V : {1, (int)(16 / seq_elem_bytes(shape->dtype))})
    if (shape->D % V == 0)
      need = std::max(need, (size_t)conv_dims(*shape, V, kConvRunBwd).pblocks * shape->D *
                                (shape->W + 1) * 4);
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
  rc = seq_check(x, shape->dtype, none, "x");
  if (rc == CK_OK) rc = seq_check(y, shape->dtype, none, "y");
  if (rc == CK_OK) rc = conv_check_state(state0, *shape, true, "state0");
  if (rc == CK_OK) rc = conv_check_state(state, *shape, true, "state");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    conv_by_kind<E>(*shape, {x, y}, {state0, state}, [&](auto v, auto w) {
      constexpr int V = decltype(v)::value, W = decltype(w)::value;
      const ConvDims d = conv_dims(*shape, V, kConvRun);
      ConvArgs<E> a = conv_args<E>(*shape, x, weight, bias, state0, lengths);
      a.y = seq_of<E>(y);
      a.state = W > 1 ? static_cast<E*>(state) : nullptr;
      a.nv = d.nv; a.vx = d.vx; a.runs = d.runs;
      conv_fwd<E, V, W><<<(unsigned)(d.vblocks * d.pblocks), kConvThreads, 0, stream>>>(a);
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
  rc = seq_check(x, shape->dtype, none, "x");
  if (rc == CK_OK) rc = seq_check(grad_y, shape->dtype, none, "grad_y");
  if (rc == CK_OK) rc = seq_check(grad_x, shape->dtype, none, "grad_x");
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
    conv_by_kind<E>(*shape, {x, grad_y, grad_x}, {state0, grad_state, grad_state0},
                    [&](auto v, auto w) {
      constexpr int V = decltype(v)::value, W = decltype(w)::value;
      const ConvDims d = conv_dims(*shape, V, kConvRunBwd);
      ConvArgs<E> a = conv_args<E>(*shape, x, weight, bias, state0, lengths);
      a.gy = seq_of<const E>(grad_y);
      a.gx = seq_of<E>(grad_x);
      a.gstate = W > 1 ? static_cast<const E*>(grad_state) : nullptr;
      a.gstate0 = W > 1 ? static_cast<E*>(grad_state0) : nullptr;
      a.part = static_cast<float*>(workspace);
      a.nv = d.nv; a.vx = d.vx; a.runs = d.runs;
      conv_bwd<E, V, W><<<(unsigned)(d.vblocks * d.pblocks), kConvThreads, 0, stream>>>(a);
      conv_sum<W><<<(unsigned)((shape->D * (W + 1) + 255) / 256), 256, 0, stream>>>(
          a.part, shape->D, d.pblocks, grad_weight, grad_bias);
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
  rc = seq_check(x, shape->dtype, false, "x");
  if (rc == CK_OK) rc = seq_check(y, shape->dtype, false, "y");
  if (rc == CK_OK) rc = conv_check_state(state0, *shape, true, "state0");
  if (rc == CK_OK) rc = conv_check_state(state, *shape, false, "state");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    conv_by_kind<E>(*shape, {x, y}, {state0, state}, [&](auto v, auto w) {
      constexpr int V = decltype(v)::value, W = decltype(w)::value;
      ConvArgs<E> a = conv_args<E>(*shape, x, weight, bias, state0, nullptr);
      a.y = seq_of<E>(y);
      a.state = W > 1 ? static_cast<E*>(state) : nullptr;
      a.nv = (int)(shape->D / V);
      const int64_t n = shape->B * a.nv;
      conv_one<E, V, W><<<(unsigned)((n + kConvThreads - 1) / kConvThreads), kConvThreads, 0,
                          stream>>>(a);
    });
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}
