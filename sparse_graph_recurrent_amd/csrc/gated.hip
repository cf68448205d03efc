// gated.hip -- entry points of the gated scan (gated.h has its formulas and its
// layout), the rule that spreads a call over the chip, and the single-token step.
#include "gated.h"

#include <algorithm>
#include <initializer_list>

namespace ckhip {
namespace {

constexpr int64_t kGateCus = 256;

ck_status gate_check_shape(const ck_gated_shape* s) {
  if (!s) {
    set_error("shape is NULL");
    return CK_ERR_NULL_ARG;
  }
  return seq_check_shape(s->T, s->B, s->D, s->dtype);
}

GatePlan gate_plan(const ck_gated_shape& s, int most_waves) {
  GatePlan p;
  p.v = s.dtype == CK_F32 || s.D < 2 ? 1 : 2;
  const int64_t groups = (s.D + kGateLanes * p.v - 1) / (kGateLanes * p.v);
  p.groups = (int)groups;
  const int64_t cols = groups * s.B;
  // (a launch holds fewer than 2^32 threads along its first dimension)
  if (cols >= kSeqGridX / 4) most_waves = std::min(most_waves, 8);
  const int64_t pairs = (s.T + 2 * kGateStep - 1) / (2 * kGateStep);
  p.waves = (int)std::min<int64_t>(most_waves, std::max<int64_t>(1, pairs));
  const int64_t window = 2 * kGateStep * p.waves;
  int64_t want = std::max<int64_t>(1, kGateCus / cols);
  want = std::max<int64_t>(1, std::min(want, s.T / window));
  const int64_t per = (s.T + want - 1) / want;
  p.chunk = (int)((per + window - 1) / window * window);
  p.chunks = p.chunk ? (int)((s.T + p.chunk - 1) / p.chunk) : 1;
  return p;
}

// Fewer waves where a window's offsets would pass 32 bits (the chunks stay: the
// workspace does not go by strides).
void gate_reach(GatePlan* p, int dtype, std::initializer_list<const ck_seq*> tensors) {
  int64_t step = 1;
  for (const ck_seq* q : tensors)
    if (q->data) step = std::max(step, q->stride_t * (int64_t)seq_elem_bytes(dtype));
  const int64_t steps = (UINT32_MAX - 256) / step + 1;
  p->waves = (int)std::min<int64_t>(p->waves, std::max<int64_t>(1, steps / (2 * kGateStep)));
}

// Workspace: the chunks' pairs, then (backward) the bias gradients' parts.
struct GateWs {
  size_t part, total;
};
GateWs gate_ws(const ck_gated_shape& s, const GatePlan& p, bool backward) {
  const size_t col = (size_t)s.B * s.D * sizeof(float);
  GateWs w;
  w.part = ((size_t)(p.chunks - 1) * 2 * col + 255) & ~size_t(255);
  w.total = w.part + (backward ? (size_t)p.chunks * 2 * col : 0);
  return w;
}

ck_status gate_check_f32(const void* p, const char* what) {
  if (reinterpret_cast<uintptr_t>(p) % sizeof(float) == 0) return CK_OK;
  set_error("%s is not aligned to its element type", what);
  return CK_ERR_BAD_VALUE;
}

ck_status gate_check_out(const ck_gated_shape& s, const ck_seq& q, bool optional,
                         const char* what) {
  return seq_check_out(q, s.T, s.B, s.D, s.dtype, optional, what, kGateMaxStrideT);
}

ck_status gate_check_inputs(const ck_gated_shape* shape, const ck_gated_inputs* in) {
  ck_status rc = gate_check_shape(shape);
  if (rc != CK_OK) return rc;
  if (!in) {
    set_error("inputs are NULL");
    return CK_ERR_NULL_ARG;
  }
  const bool none = shape->T == 0;
  rc = seq_check(in->x, shape->dtype, none, "x", kGateMaxStrideT);
  if (rc == CK_OK) rc = seq_check(in->f, shape->dtype, none, "f", kGateMaxStrideT);
  if (rc == CK_OK) rc = seq_check(in->i, shape->dtype, true, "i", kGateMaxStrideT);
  if (rc == CK_OK) rc = seq_check(in->z, shape->dtype, true, "z", kGateMaxStrideT);
  if (rc == CK_OK) rc = gate_check_f32(in->f_bias, "f_bias");
  if (rc == CK_OK) rc = gate_check_f32(in->i_bias, "i_bias");
  if (rc == CK_OK) rc = gate_check_f32(in->state0, "state0");
  return rc;
}

template <typename E>
GateArgs<E> gate_args(const ck_gated_shape& s, const GatePlan& p, const ck_gated_inputs& in,
                      void* workspace) {
  GateArgs<E> a = {};
  a.x = seq_of<const E>(in.x);
  a.f = seq_of<const E>(in.f);
  a.i = seq_of<const E>(in.i);
  a.z = seq_of<const E>(in.z);
  a.f_bias = in.f_bias;
  a.i_bias = in.i_bias;
  a.state0 = in.state0;
  a.lengths = in.lengths;
  a.sums = static_cast<float*>(workspace);
  a.T = (int)s.T;
  a.B = (int)s.B;
  a.D = (int)s.D;
  a.groups = p.groups;
  a.chunks = p.chunks;
  a.chunk = p.chunk;
  return a;
}

// One token a row: a thread owns V channels.  Bound by the launch.
constexpr int kGateOneThreads = 256;
template <typename E, int V>
__global__ __launch_bounds__(kGateOneThreads) void gate_one(const GateArgs<E> s, int64_t threads) {
  const int64_t id = seq_block() * kGateOneThreads + threadIdx.x;
  if (id >= threads) return;
  const int per = (s.D + V - 1) / V;
  const int64_t b = id / per;
  const int c = (int)(id % per) * V, n = s.D - c;
  auto get = [&](const Seq<const E>& q) {
    return n >= V ? pack_load<true, E, V>(q.row(0, b) + c, V)
                  : pack_load<false, E, V>(q.row(0, b) + c, n);
  };
  const Pack<E, V> x = get(s.x), f = get(s.f);
  Pack<E, V> i = {}, z = {};
  if (s.i.p) i = get(s.i);
  if (s.z.p) z = get(s.z);
  float y[V], h[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    h[j] = y[j] = 0.0f;
    if (j >= n) continue;
    const Gate g = gate_hw((s.f_bias ? -s.f_bias[c + j] : 0.0f) - (float)f.v[j]);
    float take = g.rest();
    if (s.i.p) take = sigmoid_hw((float)i.v[j] + (s.i_bias ? s.i_bias[c + j] : 0.0f));
    const float before = s.state0 ? s.state0[b * s.D + c + j] : 0.0f;
    y[j] = h[j] = g.times(before, take * (float)x.v[j]);
    if (s.z.p) {
      const float v = (float)z.v[j];
      y[j] *= v * sigmoid_hw(v);
    }
  }
  E* out = s.out.row(0, b) + c;
  float* state = s.state + b * s.D + c;
  if (n >= V) {
    pack_store<true, E, V>(out, y, V);
    pack_store<true, float, V>(state, h, V);
  } else {
    pack_store<false, E, V>(out, y, n);
    pack_store<false, float, V>(state, h, n);
  }
}

}  // namespace
}  // namespace ckhip

using namespace ckhip;

extern "C" ck_status ck_gated_sizes(const ck_gated_shape* shape, size_t* saved_bytes,
                                    size_t* forward_bytes, size_t* backward_bytes) {
  clear_error();
  const ck_status rc = gate_check_shape(shape);
  if (rc != CK_OK) return rc;
  const ck_gated_shape& s = *shape;
  if (saved_bytes)
    *saved_bytes = (size_t)((s.T + kGateStep - 1) / kGateStep) * s.B * s.D * sizeof(float);
  if (forward_bytes) *forward_bytes = gate_ws(s, gate_plan(s, kGateFwdWaves), false).total;
  if (backward_bytes) *backward_bytes = gate_ws(s, gate_plan(s, kGateBwdWaves), true).total;
  return CK_OK;
}

extern "C" ck_status ck_gated_forward(const ck_gated_shape* shape, const ck_gated_inputs* in,
                                      ck_seq out, float* state, void* saved, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  ck_status rc = gate_check_inputs(shape, in);
  if (rc == CK_OK) rc = gate_check_out(*shape, out, shape->T == 0, "out");
  if (rc == CK_OK) rc = gate_check_f32(state, "state");
  if (rc != CK_OK) return rc;
  GatePlan p = gate_plan(*shape, kGateFwdWaves);
  gate_reach(&p, shape->dtype, {&in->x, &in->f, &in->i, &in->z, &out});
  rc = seq_check_ws(workspace, workspace_bytes, gate_ws(*shape, p, false).total);
  if (rc == CK_OK && saved) rc = check_aligned(saved, "saved");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    GateArgs<E> a = gate_args<E>(*shape, p, *in, workspace);
    a.out = seq_of<E>(out);
    a.state = state;
    a.saved = static_cast<float*>(saved);
    return gate_run_forward(a, p, stream);
  });
}

extern "C" ck_status ck_gated_backward(const ck_gated_shape* shape, const ck_gated_inputs* in,
                                       const void* saved, ck_seq grad_out, const float* grad_state,
                                       const ck_gated_grads* grads, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  ck_status rc = gate_check_inputs(shape, in);
  if (rc != CK_OK) return rc;
  const bool none = shape->T == 0;
  if (!grads || (!saved && !none)) {
    set_error("grads or saved is NULL");
    return CK_ERR_NULL_ARG;
  }
  rc = seq_check(grad_out, shape->dtype, none, "grad_out", kGateMaxStrideT);
  if (rc == CK_OK) rc = gate_check_out(*shape, grads->x, none, "the gradient of x");
  if (rc == CK_OK) rc = gate_check_out(*shape, grads->f, none, "the gradient of f");
  if (rc == CK_OK) rc = gate_check_out(*shape, grads->i, none || !in->i.data, "the gradient of i");
  if (rc == CK_OK) rc = gate_check_out(*shape, grads->z, none || !in->z.data, "the gradient of z");
  if (rc == CK_OK) rc = gate_check_f32(grad_state, "grad_state");
  if (rc == CK_OK) rc = gate_check_f32(grads->f_bias, "the gradient of f_bias");
  if (rc == CK_OK) rc = gate_check_f32(grads->i_bias, "the gradient of i_bias");
  if (rc == CK_OK) rc = gate_check_f32(grads->state0, "the gradient of state0");
  if (rc == CK_OK && saved) rc = check_aligned(saved, "saved");
  if (rc != CK_OK) return rc;
  GatePlan p = gate_plan(*shape, kGateBwdWaves);
  gate_reach(&p, shape->dtype, {&in->x, &in->f, &in->i, &in->z, &grad_out, &grads->x, &grads->f,
                                &grads->i, &grads->z});
  const GateWs ws = gate_ws(*shape, p, true);
  rc = seq_check_ws(workspace, workspace_bytes, ws.total);
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    GateArgs<E> a = gate_args<E>(*shape, p, *in, workspace);
    a.saved = static_cast<float*>(const_cast<void*>(saved));
    a.go = seq_of<const E>(grad_out);
    a.gstate = grad_state;
    a.gx = seq_of<E>(grads->x);
    a.gf = seq_of<E>(grads->f);
    a.gi = seq_of<E>(grads->i);
    a.gz = seq_of<E>(grads->z);
    a.gstate0 = grads->state0;
    if (grads->f_bias || grads->i_bias)
      a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.part);
    return gate_run_backward(a, p, grads->f_bias, grads->i_bias, stream);
  });
}

extern "C" ck_status ck_gated_step(const ck_gated_shape* shape, const ck_gated_inputs* in,
                                   ck_seq out, float* state, hipStream_t stream) {
  clear_error();
  ck_status rc = gate_check_shape(shape);
  if (rc != CK_OK) return rc;
  if (shape->T != 1) {
    set_error("a step takes T = 1 (got %lld)", (long long)shape->T);
    return CK_ERR_BAD_SIZE;
  }
  rc = gate_check_inputs(shape, in);
  if (rc == CK_OK) rc = gate_check_out(*shape, out, false, "out");
  if (rc != CK_OK) return rc;
  if (!state || in->lengths) {
    set_error(state ? "a step takes no lengths" : "state is NULL");
    return state ? CK_ERR_BAD_VALUE : CK_ERR_NULL_ARG;
  }
  rc = gate_check_f32(state, "state");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    constexpr int V = sizeof(E) == 2 ? 2 : 1;
    GateArgs<E> a = gate_args<E>(*shape, GatePlan{}, *in, nullptr);
    a.out = seq_of<E>(out);
    a.state = state;
    const int64_t threads = shape->B * ((shape->D + V - 1) / V);
    gate_one<E, V><<<seq_grid((threads + kGateOneThreads - 1) / kGateOneThreads), kGateOneThreads,
                     0, stream>>>(a, threads);
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}
