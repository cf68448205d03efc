// scan.hip -- entry points of the selective scan and its single-token step;
// scan_forward.hip and scan_backward.hip hold the kernels over windows.
#include "scan.h"

#include <algorithm>
#include <type_traits>

namespace ckhip {
namespace {

ScanDims scan_sizes(const ck_scan_shape& s) {
  ScanDims d;
  d.T = s.T; d.B = s.B; d.D = s.D; d.N = s.N; d.G = s.G;
  d.NP = s.N <= 8 ? 8 : s.N <= 16 ? 16 : s.N <= 32 ? 32 : 64;
  d.K = scan_tile(d.NP);
  d.Dg = s.D / s.G;
  d.P = (d.Dg + kScanChan - 1) / kScanChan;
  d.tiles = (s.T + d.K - 1) / d.K;
  d.waves = d.fold = false;
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

// How a window is spread over the chip, by the workgroups that its rows and
// channels give (forward + backward of 2048 channels in bf16, 1024 steps, us; passes
// below 50 us in a graph, since the host bounds them one by one):
//   - from kScanFewGroups on, each walks the window alone (384: 618 against 711
//     with several tiles each; 512: 635 against 768 cut);
//   - a workgroup a CU, nearly (256): several tiles each (366 against 409 cut;
//     but 192 workgroups: 355 against 331, and from 257 on some CU would have two);
//   - fewer: cut to about kScanGoalGroups (128: 243 against 353 with several tiles
//     each; uncut 439).  The second pass over the steps costs 0.7 of a forward's
//     and 0.25 of a backward's main launch.
// Chunks of fewer than kScanLongChunk steps pay more for their ends than they
// spread (512 steps x 16 x 512: 126 against 138 in chunks of 32), unless the chip
// is far from full: then what counts is that the workgroups that fit at once
// (kScanRound of them backward) take the window in one round of shorter chunks
// (332 steps x 3 x 64 channels: 37 against 62; 657 x 17 x 128: 70 against 87;
// 14803 x 2 x 131: 187 against 197 in a round and a half).
// Rows of unequal lengths leave CUs idle unless cut, and are cut finer.  Windows
// too short to cut take several tiles each: up to 127 steps (100 steps x 50 x 256:
// 57 against 61), but where at most half of the CUs have a workgroup up to 64.
// There a launch less in each direction counts, and it depends on the caller: 64
// steps x 8 x 256 take 40 against 44 called one by one, which the host bounds, but
// 36 against 29 in a graph (x 32 x 256: 39 against 43, and 39 against 38).  Beyond,
// with a third round of tiles, cutting costs the host little or nothing and saves
// the graph more (72 steps x 8 x 256: 42 against 44, and 42 against 33; 88 steps x
// 32 x 256: 48 against 44, and 49 against 44).
// Workgroups that run at once, or read few chunks (half of `chunks` each, 4 KB of
// what another XCD wrote), fold the chunks before their own (256 steps x 8 x 256:
// 39 against 44 joined by a launch; 200 x 30 x 640: 120 against 124; but 2048 x 4 x
// 1024 in 32 chunks: 233 against 224, and 1023 x 16 x 1024 ragged, forward alone,
// in 8: 91 against 86).
constexpr int64_t kScanFewGroups = 384, kScanCus = 256, kScanGoalGroups = 2048, kScanRound = 512;
constexpr int64_t kScanMinChunk = 16, kScanLongChunk = 64, kScanShort = 65;  // steps
constexpr int64_t kScanFold = 8192;  // chunks times workgroups

ScanDims scan_dims(const ck_scan_shape& s, bool ragged) {
  ScanDims d = scan_sizes(s);
  const int64_t wgs = d.P * d.G * d.B;
  const bool is_short = s.T < (2 * wgs <= kScanCus ? kScanShort : 2 * kScanLongChunk);
  if (d.NP <= 16 && wgs <= kScanCus && (is_short || (!ragged && wgs > kScanCus * 13 / 16))) {
    d.waves = true;
  } else if (wgs < kScanFewGroups && !is_short) {
    // chunks are joined one after the other, eight in about a step's time of a
    // lone wave: no more of them than about a chunk has steps
    int64_t most = 64;
    while (most * most < s.T) most *= 2;
    int64_t want = std::min({kScanGoalGroups / wgs, s.T / kScanLongChunk, most});
    const int64_t fine =
        std::min({kScanRound * (ragged ? 2 : 1) / wgs, s.T / kScanMinChunk, most});
    if (want * wgs < 2 * kScanRound && 2 * fine >= want) want = fine;
    scan_cut(&d, want);
    const int64_t all = wgs * d.chunks;
    d.fold = d.chunks > 1 && (all <= kScanRound || all * d.chunks <= kScanFold);
  }
  return d;
}

// One token.  A quad of lanes takes a channel, each lane NL adjacent states, so
// that the states (which are all but a few bytes of what the step reads and
// writes, and bound it) move in 16-byte accesses.  256 tokens of 2048 channels x
// 16 states: 15.6 us, 4.6 TB/s; one token of 256 channels: 2.7 us, the launch.
constexpr int kOneThreads = 256;

template <bool FULL, int NL, typename E>
__device__ __forceinline__ void scan_one_row(const ScanArgs<E>& s, int b, int d, int q) {
  const int64_t row = (int64_t)b * s.D + d;
  const int n0 = q * NL, left = s.N - n0;
  const Pack<float, NL> a = pack_load<FULL, float, NL>(s.a + (int64_t)d * s.N + n0, left);
  Pack<float, NL> h = {};
  if (s.state0) h = pack_load<FULL, float, NL>(s.state0 + row * s.N + n0, left);
  const int64_t at = (int64_t)(d / s.Dg) * s.N + n0;
  const Pack<E, NL> bb = pack_load<FULL, E, NL>(s.b.row(0, b) + at, left);
  const Pack<E, NL> cc = pack_load<FULL, E, NL>(s.c.row(0, b) + at, left);
  const float raw = (float)s.delta.row(0, b)[d] + (s.delta_bias ? s.delta_bias[d] : 0.0f);
  const float dt = s.softplus ? softplus_hw(raw).value : raw;
  const float u = (float)s.u.row(0, b)[d], x = dt * u;
  float y = 0.0f, hn[NL];
#pragma unroll
  for (int k = 0; k < NL; ++k) {
    hn[k] = fmaf(exp2_hw(dt * (kLog2e * scan_rate(a.v[k]))), h.v[k], x * (float)bb.v[k]);
    y += FULL || k < left ? (float)cc.v[k] * hn[k] : 0.0f;
  }
  y = quad_sum(y);
  if (s.d) y = fmaf(s.d[d], u, y);
  if (s.z.p) {
    const float zf = (float)s.z.row(0, b)[d];
    y *= zf * sigmoid_hw(zf);
  }
  if (q == 0) s.out.row(0, b)[d] = (E)y;
  pack_store<FULL, float, NL>(s.state + row * s.N + n0, hn, left);
}

template <typename E, int NL>
__global__ __launch_bounds__(kOneThreads) void scan_one(const ScanArgs<E> s) {
  const int64_t i = seq_block() * (kOneThreads / 4) + (threadIdx.x >> 2);
  if (i >= (int64_t)s.B * s.D) return;  // whole quads
  const int b = (int)(i / s.D), d = (int)(i % s.D), q = threadIdx.x & 3;
  if (s.N == 4 * NL)
    scan_one_row<true, NL>(s, b, d, q);
  else
    scan_one_row<false, NL>(s, b, d, q);
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
  w.part_a = take(backward ? (d.waves ? kScanBwdTW : d.chunks) * d.B * d.D * (d.NP + 2) : 0);
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
  const ScanDims d = scan_sizes(*s);
  if (d.P * d.G * d.B >= kSeqMaxThreads / kScanThreads || d.D * d.NP >= INT_MAX ||
      d.G * d.N > (int64_t(1) << 28) ||  // (byte offsets in a step of B or C: 32 bits)
      (d.T > 0 && d.B * d.G * d.NP >= (int64_t(1) << 36) / d.T)) {
    set_error("B=%lld, D=%lld or T=%lld is too large", (long long)d.B, (long long)d.D,
              (long long)d.T);
    return CK_ERR_TOO_LARGE;
  }
  return CK_OK;
}

// The largest step stride of a tensor of `row` elements a step: offsets from a
// tile's first step are 32-bit bytes.  Where a workgroup works on several tiles they
// reach over 32 steps, else over one tile.
int64_t scan_max_stride(const ck_scan_shape& s, const ScanDims& d, int64_t row) {
  if (d.waves) return (int64_t(1) << 24) - 1;
  return (UINT32_MAX / (int64_t)seq_elem_bytes(s.dtype) - row) / (d.K - 1);
}

ck_status scan_check_out(const ck_scan_shape& s, const ScanDims& d, const ck_seq& q, bool optional,
                         const char* what) {
  return seq_check_out(q, s.T, s.B, s.D, s.dtype, optional, what, scan_max_stride(s, d, s.D));
}

// Sizes and inputs of a call; d: how it is spread over the chip.
ck_status scan_check_inputs(const ck_scan_shape* shape, const ck_scan_inputs* in, ScanDims* d) {
  ck_status rc = scan_check_shape(shape);
  if (rc != CK_OK) return rc;
  if (!in || !in->a) {
    set_error("inputs or A is NULL");
    return CK_ERR_NULL_ARG;
  }
  const ck_scan_shape& s = *shape;
  *d = scan_dims(s, in->lengths != nullptr);
  const bool none = s.T == 0;
  const int64_t most = scan_max_stride(s, *d, s.D), most_bc = scan_max_stride(s, *d, s.G * s.N);
  rc = seq_check(in->u, s.dtype, none, "u", most);
  if (rc == CK_OK) rc = seq_check(in->delta, s.dtype, none, "delta", most);
  if (rc == CK_OK) rc = seq_check(in->b, s.dtype, none, "B", most_bc);
  if (rc == CK_OK) rc = seq_check(in->c, s.dtype, none, "C", most_bc);
  if (rc == CK_OK) rc = seq_check(in->z, s.dtype, true, "z", most);
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
  a.fold = d.fold;
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

template <typename E, int NL>
void scan_launch_one(const ScanArgs<E>& a, hipStream_t stream) {
  const int64_t n = (int64_t)a.B * a.D, per = kOneThreads / 4;
  scan_one<E, NL><<<seq_grid((n + per - 1) / per), kOneThreads, 0, stream>>>(a);
}

}  // namespace
}  // namespace ckhip

using namespace ckhip;

extern "C" ck_status ck_scan_sizes(const ck_scan_shape* shape, size_t* saved_bytes,
                                   size_t* forward_bytes, size_t* backward_bytes) {
  clear_error();
  const ck_status rc = scan_check_shape(shape);
  if (rc != CK_OK) return rc;
  const ScanDims d = scan_sizes(*shape);
  if (saved_bytes) *saved_bytes = scan_saved(d);
  auto most = [&](bool backward) {  // whether lengths will be given or not
    return std::max(scan_ws(scan_dims(*shape, false), backward).total,
                    scan_ws(scan_dims(*shape, true), backward).total);
  };
  if (forward_bytes) *forward_bytes = most(false);
  if (backward_bytes) *backward_bytes = most(true);
  return CK_OK;
}

extern "C" ck_status ck_scan_forward(const ck_scan_shape* shape, const ck_scan_inputs* in,
                                     ck_seq out, float* state, void* saved, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  ScanDims d;
  ck_status rc = scan_check_inputs(shape, in, &d);
  if (rc == CK_OK) rc = scan_check_out(*shape, d, out, shape->T == 0, "out");
  if (rc != CK_OK) return rc;
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
  ScanDims d;
  ck_status rc = scan_check_inputs(shape, in, &d);
  if (rc != CK_OK) return rc;
  const bool none = shape->T == 0;
  if (!grads || !grads->a || (!saved && !none)) {
    set_error("grads, the gradient of A or saved is NULL");
    return CK_ERR_NULL_ARG;
  }
  rc = seq_check(grad_out, shape->dtype, none, "grad_out", scan_max_stride(*shape, d, d.D));
  if (rc == CK_OK) rc = scan_check_out(*shape, d, grads->u, none, "the gradient of u");
  if (rc == CK_OK) rc = scan_check_out(*shape, d, grads->delta, none, "the gradient of delta");
  auto check_bc = [&](const ck_seq& q, const char* what) {
    return seq_check_out(q, d.T, d.B, d.G * d.N, shape->dtype, none, what);
  };
  if (rc == CK_OK) rc = check_bc(grads->b, "the gradient of B");
  if (rc == CK_OK) rc = check_bc(grads->c, "the gradient of C");
  if (rc == CK_OK)
    rc = scan_check_out(*shape, d, grads->z, none || !in->z.data, "the gradient of z");
  if (rc != CK_OK) return rc;
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
  ScanDims d;
  rc = scan_check_inputs(shape, in, &d);
  if (rc == CK_OK) rc = scan_check_out(*shape, d, out, false, "out");
  if (rc != CK_OK) return rc;
  if (!state || in->lengths) {
    set_error(state ? "a step takes no lengths" : "state is NULL");
    return state ? CK_ERR_BAD_VALUE : CK_ERR_NULL_ARG;
  }
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    ScanArgs<E> a = scan_args<E>(*shape, d, *in, nullptr, ScanWs{});
    a.out = seq_of<E>(out);
    a.state = state;
    if (a.N <= 4)
      scan_launch_one<E, 1>(a, stream);
    else if (a.N <= 8)
      scan_launch_one<E, 2>(a, stream);
    else if (a.N <= 16)
      scan_launch_one<E, 4>(a, stream);
    else if (a.N <= 32)
      scan_launch_one<E, 8>(a, stream);
    else
      scan_launch_one<E, 16>(a, stream);
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}
