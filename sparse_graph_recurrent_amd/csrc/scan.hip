// scan.hip -- entry points of the selective scan and its single-token step;
// scan_forward.hip and scan_backward.hip hold the kernels over windows.
#include "scan.h"

#include <algorithm>
#include <type_traits>

namespace ckhip {
namespace {

ScanDims scan_dims(const ck_scan_shape& s) {
  ScanDims d;
  d.T = s.T; d.B = s.B; d.D = s.D; d.N = s.N; d.G = s.G;
  d.NL = s.N <= 4 ? 1 : s.N <= 8 ? 2 : s.N <= 16 ? 4 : s.N <= 32 ? 8 : 16;
  d.NP = 4 * d.NL;
  d.K = scan_tile(d.NL);
  d.Dg = s.D / s.G;
  d.P = (d.Dg + kScanChan - 1) / kScanChan;
  d.tiles = (s.T + d.K - 1) / d.K;
  d.chunks = 1;
  d.chunk_steps = std::max<int64_t>(d.tiles, 1) * d.K;
  return d;
}

// Cuts the window into at most `want` chunks of whole tiles.
void scan_cut(ScanDims* d, int64_t want) {
  const int64_t per = std::max<int64_t>((d->tiles + want - 1) / std::max<int64_t>(want, 1), 1);
  d->chunk_steps = per * d->K;
  d->chunks = std::max<int64_t>((d->tiles + per - 1) / per, 1);
}

// Workgroups below which the window is cut, and the shortest chunk.
constexpr int64_t kScanFwdGroups = 512, kScanBwdGroups = 512, kScanMinChunk = 64;

ScanDims scan_dims(const ck_scan_shape& s, bool backward) {
  ScanDims d = scan_dims(s);
  const int64_t wgs = d.P * d.G * d.B, goal = backward ? kScanBwdGroups : kScanFwdGroups;
  if (wgs * 2 <= goal)
    scan_cut(&d, std::min(goal / wgs, std::max<int64_t>(s.T / kScanMinChunk, 1)));
  return d;
}

template <typename E, int NL>
__global__ __launch_bounds__(kScanThreads) void scan_one(const ScanArgs<E> s) {
  const Place p = scan_place(s);
  if (!p.active) return;  // whole quads
  const int64_t row = (int64_t)p.b * s.D + p.d;
  float a[NL], h[NL];
  load_a<NL>(a, s.a, p.d, p.q, s.N);
  load_state<NL>(h, s.state0, row, p.q, s.N);
  const float raw = (float)s.delta.row(0, p.b)[p.d] + (s.delta_bias ? s.delta_bias[p.d] : 0.0f);
  const float dt = s.softplus ? softplus_hw(raw) : raw;
  const float u = (float)s.u.row(0, p.b)[p.d], x = dt * u;
  const E *pb = s.b.row(0, p.b) + (int64_t)p.g * s.N, *pc = s.c.row(0, p.b) + (int64_t)p.g * s.N;
  float y = 0.0f;
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    const int n = p.q * NL + k;
    if (n < s.N) {
      h[k] = fmaf(exp2_hw(dt * (kLog2e * a[k])), h[k], x * (float)pb[n]);
      y = fmaf((float)pc[n], h[k], y);
    }
  }
  y = quad_sum(y);
  if (s.d) y = fmaf(s.d[p.d], u, y);
  if (s.z.p) {
    const float zf = (float)s.z.row(0, p.b)[p.d];
    y *= zf * sigmoid_hw(zf);
  }
  if (p.q == 0) s.out.row(0, p.b)[p.d] = (E)y;
  store_state<NL>(h, s.state, row, p.q, s.N);
}

// Workspace byte offsets of a call.
struct ScanWs {
  size_t edge, dtsum, part_bc, part_a, total;
};
ScanWs scan_ws(const ScanDims& d, bool backward) {
  size_t at = 0;
  auto take = [&](int64_t floats) {
    const size_t here = at;
    at += ((size_t)floats * 4 + 255) & ~size_t(255);
    return here;
  };
  const int64_t edges = d.chunks > 1 ? d.chunks * d.B * d.D : 0;
  ScanWs w;
  w.edge = take(edges * d.NP);
  w.dtsum = take(edges);
  w.part_bc = take(backward ? d.P * d.T * d.B * d.G * 2 * d.NP : 0);
  w.part_a = take(backward ? d.chunks * d.B * d.D * (d.NP + 2) : 0);
  w.total = at;
  return w;
}
size_t scan_saved(const ScanDims& d) { return (size_t)(d.tiles * d.B * d.D) * d.NP * 4; }

ck_status scan_check_shape(const ck_scan_shape* s) {
  if (!s) {
    set_error("shape is NULL");
    return CK_ERR_NULL_ARG;
  }
  const ck_status rc = seq_check_shape(s->T, s->B, s->D, s->dtype);
  if (rc != CK_OK) return rc;
  if (s->N < 1 || s->N > kScanMaxN || s->G < 1 || s->G > s->D || s->D % s->G != 0) {
    set_error("N must be in [1, 64] and G must divide D (N=%lld G=%lld D=%lld)", (long long)s->N,
              (long long)s->G, (long long)s->D);
    return CK_ERR_BAD_SIZE;
  }
  const ScanDims d = scan_dims(*s);
  if (d.P * d.G * d.B >= INT_MAX || d.D * d.NP >= INT_MAX ||
      (d.T > 0 && d.B * d.G * d.NP >= (int64_t(1) << 36) / d.T)) {
    set_error("B=%lld, D=%lld or T=%lld is too large", (long long)d.B, (long long)d.D,
              (long long)d.T);
    return CK_ERR_TOO_LARGE;
  }
  return CK_OK;
}

ck_status scan_check_inputs(const ck_scan_shape& s, const ck_scan_inputs* in) {
  if (!in || !in->a) {
    set_error("inputs or A is NULL");
    return CK_ERR_NULL_ARG;
  }
  const bool none = s.T == 0;
  ck_status rc = seq_check(in->u, s.dtype, none, "u");
  if (rc == CK_OK) rc = seq_check(in->delta, s.dtype, none, "delta");
  if (rc == CK_OK) rc = seq_check(in->b, s.dtype, none, "B");
  if (rc == CK_OK) rc = seq_check(in->c, s.dtype, none, "C");
  if (rc == CK_OK) rc = seq_check(in->z, s.dtype, true, "z");
  return rc;
}

template <typename E>
ScanArgs<E> scan_args(const ck_scan_shape& s, const ScanDims& d, const ck_scan_inputs& in,
                      void* workspace, const ScanWs& ws) {
  ScanArgs<E> a = {};
  auto part = [&](size_t at) {
    return workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + at) : nullptr;
  };
  a.edge = part(ws.edge);
  a.dtsum = part(ws.dtsum);
  a.part_bc = part(ws.part_bc);
  a.part_a = part(ws.part_a);
  a.u = seq_of<const E>(in.u);
  a.delta = seq_of<const E>(in.delta);
  a.b = seq_of<const E>(in.b);
  a.c = seq_of<const E>(in.c);
  a.z = seq_of<const E>(in.z);
  a.a = in.a;
  a.d = in.d;
  a.delta_bias = in.delta_bias;
  a.state0 = in.state0;
  a.lengths = in.lengths;
  a.T = (int)d.T; a.B = (int)d.B; a.D = (int)d.D; a.N = (int)d.N; a.G = (int)d.G;
  a.Dg = (int)d.Dg; a.P = (int)d.P;
  a.chunks = (int)d.chunks; a.chunk_steps = (int)d.chunk_steps;
  a.softplus = s.delta_softplus;
  return a;
}

template <typename F>
void scan_by_states(int NL, F&& fn) {
  switch (NL) {
    case 1: fn(std::integral_constant<int, 1>()); break;
    case 2: fn(std::integral_constant<int, 2>()); break;
    case 4: fn(std::integral_constant<int, 4>()); break;
    case 8: fn(std::integral_constant<int, 8>()); break;
    default: fn(std::integral_constant<int, 16>()); break;
  }
}

}  // namespace
}  // namespace ckhip

using namespace ckhip;

extern "C" ck_status ck_scan_sizes(const ck_scan_shape* shape, size_t* saved_bytes,
                                   size_t* forward_bytes, size_t* backward_bytes) {
  clear_error();
  const ck_status rc = scan_check_shape(shape);
  if (rc != CK_OK) return rc;
  const ScanDims d = scan_dims(*shape);
  if (saved_bytes) *saved_bytes = scan_saved(d);
  if (forward_bytes) *forward_bytes = scan_ws(scan_dims(*shape, false), false).total;
  if (backward_bytes) *backward_bytes = scan_ws(scan_dims(*shape, true), true).total;
  return CK_OK;
}

extern "C" ck_status ck_scan_forward(const ck_scan_shape* shape, const ck_scan_inputs* in,
                                     ck_seq out, float* state, void* saved, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  ck_status rc = scan_check_shape(shape);
  if (rc == CK_OK) rc = scan_check_inputs(*shape, in);
  if (rc == CK_OK) rc = seq_check(out, shape->dtype, shape->T == 0, "out");
  if (rc != CK_OK) return rc;
  const ScanDims d = scan_dims(*shape, false);
  const ScanWs ws = scan_ws(d, false);
  rc = seq_check_ws(workspace, workspace_bytes, ws.total);
  if (rc == CK_OK && saved) rc = check_aligned(saved, "saved");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    ScanArgs<E> a = scan_args<E>(*shape, d, *in, workspace, ws);
    a.out = seq_of<E>(out);
    a.state = state;
    a.saved = static_cast<float*>(saved);
    scan_launch_forward(d, a, stream);
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}

extern "C" ck_status ck_scan_backward(const ck_scan_shape* shape, const ck_scan_inputs* in,
                                      const void* saved, ck_seq grad_out, const float* grad_state,
                                      const ck_scan_grads* grads, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  ck_status rc = scan_check_shape(shape);
  if (rc == CK_OK) rc = scan_check_inputs(*shape, in);
  if (rc != CK_OK) return rc;
  const bool none = shape->T == 0;
  if (!grads || !grads->a || (!saved && !none)) {
    set_error("grads, the gradient of A or saved is NULL");
    return CK_ERR_NULL_ARG;
  }
  rc = seq_check(grad_out, shape->dtype, none, "grad_out");
  if (rc == CK_OK) rc = seq_check(grads->u, shape->dtype, none, "the gradient of u");
  if (rc == CK_OK) rc = seq_check(grads->delta, shape->dtype, none, "the gradient of delta");
  if (rc == CK_OK) rc = seq_check(grads->b, shape->dtype, none, "the gradient of B");
  if (rc == CK_OK) rc = seq_check(grads->c, shape->dtype, none, "the gradient of C");
  if (rc == CK_OK)
    rc = seq_check(grads->z, shape->dtype, none || !in->z.data, "the gradient of z");
  if (rc != CK_OK) return rc;
  const ScanDims d = scan_dims(*shape, true);
  const ScanWs ws = scan_ws(d, true);
  rc = seq_check_ws(workspace, workspace_bytes, ws.total);
  if (rc == CK_OK && saved) rc = check_aligned(saved, "saved");
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    ScanArgs<E> a = scan_args<E>(*shape, d, *in, workspace, ws);
    a.saved = static_cast<float*>(const_cast<void*>(saved));
    a.go = seq_of<const E>(grad_out);
    a.gstate = grad_state;
    a.gu = seq_of<E>(grads->u);
    a.gdelta = seq_of<E>(grads->delta);
    a.gz = seq_of<E>(grads->z);
    a.gstate0 = grads->state0;
    a.gb = seq_of<E>(grads->b);
    a.gc = seq_of<E>(grads->c);
    a.ga = grads->a;
    a.gd = grads->d;
    a.gbias = grads->delta_bias;
    scan_launch_backward(d, a, stream);
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}

extern "C" ck_status ck_scan_step(const ck_scan_shape* shape, const ck_scan_inputs* in, ck_seq out,
                                  float* state, hipStream_t stream) {
  clear_error();
  ck_status rc = scan_check_shape(shape);
  if (rc != CK_OK) return rc;
  if (shape->T != 1) {
    set_error("a step takes T = 1 (got %lld)", (long long)shape->T);
    return CK_ERR_BAD_SIZE;
  }
  rc = scan_check_inputs(*shape, in);
  if (rc == CK_OK) rc = seq_check(out, shape->dtype, false, "out");
  if (rc != CK_OK) return rc;
  if (!state || in->lengths) {
    set_error(state ? "a step takes no lengths" : "state is NULL");
    return state ? CK_ERR_BAD_VALUE : CK_ERR_NULL_ARG;
  }
  const ScanDims d = scan_dims(*shape);
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    ScanArgs<E> a = scan_args<E>(*shape, d, *in, nullptr, ScanWs{});
    a.out = seq_of<E>(out);
    a.state = state;
    scan_by_states(d.NL, [&](auto nl) {
      scan_one<E, decltype(nl)::value>
          <<<(unsigned)(d.P * d.G * d.B), kScanThreads, 0, stream>>>(a);
    });
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}
