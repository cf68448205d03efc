// gated.hip -- entry points of the gated scan (gated.h has its formulas and its
// layout), the rule that spreads a call over the chip, and the single-token step.
#include "gated.h"

#include <algorithm>
#include <initializer_list>

#include "overlap.h"

namespace ckhip {
namespace {

// A workgroup of the loop over windows fills a CU, so that columns are worked on in
// rounds of one a CU; a chain has a workgroup a window, whatever the columns.  Loop / chain,
// us, with both gates (2048 steps of so many columns, and 256 of them):
//
//                          32          128          256          288          512
//   bf16 forward        48 / 17      51 / 42      80 / 83     132 / 95     159 / 156
//        backward       83 / 30     111 / 96     141 / 180    232 / 202    279 / 342
//   fp32 forward        31 / 14      37 / 32      72 / 66     117 / 76     147 / 128
//        backward       55 / 22      89 / 64     134 / 129    201 / 148    257 / 247
//   256 steps, bf16   10 / 9.4      11 / 10      13 / 14      23 / 19      27 / 23
//        backward       17 / 14      20 / 17      23 / 30      35 / 36      40 / 51
//
// So the forward loops where its columns are one full round, the backward where no round in
// four is lost.  The rule is that of 16-bit types with gates of their own, of whose chain
// one workgroup runs on a CU backward and two forward.  fp32 has two or more in both
// directions, and would gain up to 9 % from the chain at 256 columns (512 backward: 4 %).
// Where it is taken at a loss: without gates of their own a chain of two to eight windows
// pays more for its words than it gains (fp32, 256 steps of 32 columns 7.1 / 10.0 us, and
// 6.3 / 8.7 looped; 1024 of 128 backward 26, and 22).
constexpr int64_t kGateCus = 256;
constexpr int64_t kGateColumns = 4096;  // of a chain, at most: each has a ticket

ck_status gate_check_shape(const ck_gated_shape* s) {
  if (!s) {
    set_error("shape is NULL");
    return CK_ERR_NULL_ARG;
  }
  return seq_check_shape(s->T, s->B, s->D, s->dtype);
}

// How a call with these step strides (bytes; 0: any) is spread over the chip.
GatePlan gate_plan(const ck_gated_shape& s, int64_t step, bool backward) {
  GatePlan p;
  p.v = s.dtype == CK_F32 || s.D < 2 ? 1 : 2;
  const int64_t groups = (s.D + kGateLanes * p.v - 1) / (kGateLanes * p.v);
  p.groups = (int)groups;
  const int64_t cols = groups * s.B;
  const int64_t pairs = (s.T + 2 * kGateStep - 1) / (2 * kGateStep);
  // a window's offsets are 32 bits
  const int64_t reach = step ? ((UINT32_MAX - 256) / step + 1) / (2 * kGateStep) : kGateWaves;
  p.waves = (int)std::max<int64_t>(1, std::min({(int64_t)kGateWaves, pairs, reach}));
  p.windows = 1;
  const int64_t windows = (pairs + kGateWaves - 1) / kGateWaves;
  const int64_t rounds = (cols + kGateCus - 1) / kGateCus;
  const bool full = backward ? 4 * cols >= 3 * kGateCus * rounds
                             : rounds == 1 && 20 * cols >= 19 * kGateCus;
  if (!full && cols <= kGateColumns && windows > 1 && p.waves == kGateWaves &&
      windows * cols < INT_MAX)
    p.windows = (int)windows;
  return p;
}

using GateTensors = std::initializer_list<const ck_seq*>;
int64_t gate_step(int dtype, GateTensors tensors) {
  int64_t step = 1;
  for (const ck_seq* q : tensors)
    if (q->data) step = std::max(step, q->stride_t * (int64_t)seq_elem_bytes(dtype));
  return step;
}

// Whether columns of the tensors begin off cache lines.
int gate_split(const ck_gated_shape& s, GateTensors tensors) {
  const uint64_t e = seq_elem_bytes(s.dtype);
  uint64_t bits = s.D * e;
  for (const ck_seq* q : tensors)
    if (q->data)
      bits |= reinterpret_cast<uintptr_t>(q->data) | (q->stride_t * e) | (q->stride_b * e);
  return bits % 128 != 0;
}

// Workspace: a chain's tickets and words, then (backward) the bias gradients' parts.  (It
// does not go by strides: long ones leave the chain's share unused.)
struct GateWs {
  size_t pairs, states, part, total;
};
GateWs gate_ws(const ck_gated_shape& s, bool backward) {
  const GatePlan p = gate_plan(s, 0, backward);
  const int64_t windows = p.windows;
  const int64_t col = s.B * s.D, runs = windows / kGateRun;
  GateWs w;
  w.pairs = windows > 1 ? (size_t)p.groups * s.B * kGateTicket * sizeof(uint32_t) : 0;
  w.pairs = (w.pairs + 255) & ~size_t(255);
  w.states = w.pairs + (windows > 1 ? (size_t)windows * col * sizeof(uint64_t) : 0);
  w.part = (w.states + (windows > 1 ? (size_t)runs * col * sizeof(uint64_t) : 0) + 255) &
           ~size_t(255);
  w.total = w.part + (backward ? (size_t)windows * 2 * col * sizeof(float) : 0);
  return w;
}

// The states that a forward leaves, in bytes.
size_t gate_saved(const ck_gated_shape& s) {
  return (size_t)((s.T + kGateStep - 1) / kGateStep) * s.B * s.D * sizeof(float);
}

ck_status gate_check_f32(const void* p, const char* what) {
  if (reinterpret_cast<uintptr_t>(p) % sizeof(float) == 0) return CK_OK;
  set_error("%s is not aligned to its element type", what);
  return CK_ERR_BAD_VALUE;
}

// The tensors of a call, for which of them may not share memory.
class GateSpans {
 public:
  explicit GateSpans(const ck_gated_shape& s) : s_(s), e_((int64_t)seq_elem_bytes(s.dtype)) {}
  void seq(const char* name, const ck_seq& q, bool written = false) {
    // (strides up to 2^60 elements: nothing lies further apart, their bytes stay in 64 bits)
    add(name, q.data, s_.T, s_.T > 1 ? std::min(q.stride_t, kFar) * e_ : 0, s_.B,
        s_.B > 1 ? std::min(q.stride_b, kFar) * e_ : 0, s_.D * e_, written);
  }
  void state(const char* name, const float* p, bool written = false) {
    bytes(name, p, (size_t)(s_.B * s_.D) * sizeof(float), written);
  }
  void bias(const char* name, const float* p, bool written = false) {
    bytes(name, p, (size_t)s_.D * sizeof(float), written);
  }
  void bytes(const char* name, const void* p, size_t n, bool written) {
    add(name, p, 1, 0, 1, 0, (int64_t)n, written);
  }
  // What a call reads of its inputs (a backward does not read state0).
  void inputs(const ck_gated_inputs& in, bool backward = false) {
    seq("x", in.x), seq("f", in.f), seq("i", in.i), seq("z", in.z);
    bias("f_bias", in.f_bias);
    if (in.i.data) bias("i_bias", in.i_bias);
    if (!backward) state("state0", in.state0);
    bytes("lengths", in.lengths, (size_t)s_.B * sizeof(int32_t), false);
  }
  // in_place: what is written may be an input itself (the same elements).
  ck_status check(bool in_place = false) const {
    for (int k = 0; k < n_; ++k) {
      const Span& w = v_[k];
      if (!w.written) continue;
      for (int o = 0; o < n_; ++o) {
        const Span& r = v_[o];
        if (w.end <= r.at || r.end <= w.at || o == k || (r.written && o < k)) continue;
        if (!pieces_meet(pieces(w), pieces(r)) || (in_place && !r.written && same(w, r))) continue;
        set_error("%s must not lie over %s", w.name, r.name);
        return CK_ERR_BAD_VALUE;
      }
    }
    return CK_OK;
  }

 private:
  struct Span {  // (as Pieces)
    uintptr_t at, end;
    int64_t n0, s0, n1, s1, bytes;
    const char* name;
    bool written;
  };
  static constexpr int64_t kFar = int64_t(1) << 60;
  static Pieces pieces(const Span& p) {
    Pieces q;
    q.at = p.at, q.n0 = p.n0, q.s0 = p.s0, q.n1 = p.n1, q.s1 = p.s1, q.bytes = p.bytes;
    return q;
  }
  static bool same(const Span& a, const Span& b) {
    return a.at == b.at && a.n0 == b.n0 && a.s0 == b.s0 && a.n1 == b.n1 && a.s1 == b.s1 &&
           a.bytes == b.bytes;
  }
  void add(const char* name, const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1,
           int64_t bytes, bool written) {
    if (!p || n0 <= 0 || bytes <= 0) return;
    Span& q = v_[n_++];
    q = Span{reinterpret_cast<uintptr_t>(p), 0, n0, s0, n1, s1, bytes, name, written};
    const __int128 end = pieces(q).end();
    q.end = end > (__int128)UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)end;
  }
  const ck_gated_shape& s_;
  int64_t e_;
  int n_ = 0;
  Span v_[20];
};

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
                      void* workspace, const GateWs& ws) {
  GateArgs<E> a = {};
  a.x = seq_of<const E>(in.x);
  a.f = seq_of<const E>(in.f);
  a.i = seq_of<const E>(in.i);
  a.z = seq_of<const E>(in.z);
  a.f_bias = in.f_bias;
  a.i_bias = in.i_bias;
  a.state0 = in.state0;
  a.lengths = in.lengths;
  if (p.windows > 1) {
    char* at = static_cast<char*>(workspace);
    a.ticket = reinterpret_cast<uint32_t*>(at);
    a.pairs = reinterpret_cast<uint64_t*>(at + ws.pairs);
    a.states = reinterpret_cast<uint64_t*>(at + ws.states);
  }
  a.T = (int)s.T;
  a.B = (int)s.B;
  a.D = (int)s.D;
  a.groups = p.groups;
  a.windows = p.windows;
  return a;
}

// The tickets and words of a chain, before its launch: all of `bytes` from `base` on,
// zeros up to `tickets`.  (A kernel: a graph's own memory sets have come out wrong when
// replayed.)
constexpr int kGateClearThreads = 256;
__global__ __launch_bounds__(kGateClearThreads) void gate_clear(char* base, int64_t tickets,
                                                                int64_t bytes) {
  const int64_t at = ((int64_t)blockIdx.x * kGateClearThreads + threadIdx.x) * 16;
  const uint32_t w = at < tickets ? 0u : ~0u;
  if (at + 16 <= bytes) *reinterpret_cast<uint4*>(base + at) = make_uint4(w, w, w, w);
  else if (at < bytes) *reinterpret_cast<uint2*>(base + at) = make_uint2(w, w);
}
template <typename E>
void gate_prepare(const GateArgs<E>& a, const GateWs& ws, hipStream_t stream) {
  static_assert(kGateAbsent == ~0ull);
  if (!a.ticket) return;
  const int64_t bytes = ws.states + a.windows / kGateRun * (int64_t)a.B * a.D * sizeof(uint64_t);
  const int64_t each = kGateClearThreads * 16;
  gate_clear<<<(unsigned)((bytes + each - 1) / each), kGateClearThreads, 0, stream>>>(
      reinterpret_cast<char*>(a.ticket), ws.pairs, bytes);
}

// One token a row: a thread owns V channels.  Bound by the launch (2.7 us for 1 x 256).
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
  if (saved_bytes) *saved_bytes = gate_saved(s);
  if (forward_bytes) *forward_bytes = gate_ws(s, false).total;
  if (backward_bytes) *backward_bytes = gate_ws(s, true).total;
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
  const GateTensors tensors = {&in->x, &in->f, &in->i, &in->z, &out};
  const GatePlan p = gate_plan(*shape, gate_step(shape->dtype, tensors), false);
  const GateWs ws = gate_ws(*shape, false);
  rc = seq_check_ws(workspace, workspace_bytes, ws.total);
  if (rc == CK_OK && saved) rc = check_aligned(saved, "saved");
  if (rc != CK_OK) return rc;
  // (windows that wait for one another read the inputs while others have written; groups
  // of channels that do not fill one share a channel)
  GateSpans spans(*shape);
  spans.seq("out", out, true);
  spans.state("state", state, true);
  spans.bytes("saved", saved, gate_saved(*shape), true);
  spans.bytes("the workspace", workspace, ws.total, true);
  spans.inputs(*in);
  rc = spans.check();
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    GateArgs<E> a = gate_args<E>(*shape, p, *in, workspace, ws);
    a.out = seq_of<E>(out);
    a.state = state;
    a.saved = static_cast<float*>(saved);
    a.split = gate_split(*shape, tensors);
    gate_prepare(a, ws, stream);
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
  const GateTensors tensors = {&in->x, &in->f, &in->i, &in->z, &grad_out,
                               &grads->x, &grads->f, &grads->i, &grads->z};
  const GatePlan p = gate_plan(*shape, gate_step(shape->dtype, tensors), true);
  const GateWs ws = gate_ws(*shape, true);
  rc = seq_check_ws(workspace, workspace_bytes, ws.total);
  if (rc != CK_OK) return rc;
  GateSpans spans(*shape);
  spans.seq("the gradient of x", grads->x, true);
  spans.seq("the gradient of f", grads->f, true);
  if (in->i.data) spans.seq("the gradient of i", grads->i, true);
  if (in->z.data) spans.seq("the gradient of z", grads->z, true);
  spans.bias("the gradient of f_bias", grads->f_bias, true);
  spans.bias("the gradient of i_bias", grads->i_bias, true);
  spans.state("the gradient of state0", grads->state0, true);
  spans.bytes("the workspace", workspace, ws.total, true);
  spans.bytes("saved", saved, gate_saved(*shape), false);
  spans.seq("grad_out", grad_out);
  spans.state("grad_state", grad_state);
  spans.inputs(*in, true);
  rc = spans.check();
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    GateArgs<E> a = gate_args<E>(*shape, p, *in, workspace, ws);
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
    a.split = gate_split(*shape, tensors);
    gate_prepare(a, ws, stream);
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
  GateSpans spans(*shape);  // (a thread reads its channels' inputs before it writes them)
  spans.seq("out", out, true);
  spans.state("state", state, true);
  spans.inputs(*in);
  rc = spans.check(true);
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    constexpr int V = sizeof(E) == 2 ? 2 : 1;
    GateArgs<E> a = gate_args<E>(*shape, GatePlan{}, *in, nullptr, GateWs{});
    a.out = seq_of<E>(out);
    a.state = state;
    const int64_t threads = shape->B * ((shape->D + V - 1) / V);
    gate_one<E, V><<<seq_grid((threads + kGateOneThreads - 1) / kGateOneThreads), kGateOneThreads,
                     0, stream>>>(a, threads);
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}
