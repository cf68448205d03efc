// dropout.hip -- dropout whose mask is recomputed from counters.
//
//   out = residual + (r >= q ? x * 65536 / (65536 - q) : 0)
//
// r is 16 bits of Philox4x32-10 (Salmon et al., SC 2011): one evaluation, of
// ten rounds of two 32 x 32 -> 64 bit products, gives eight adjacent channels
// their values, so that at 16-bit tensors (4 bytes an element and more) HBM
// and not the generator bounds the kernel.  16 bits a value make p a multiple
// of 2^-16; the scale uses that multiple, so the mean is kept exactly.
// Measured: 2048 x 8 x 2048 bf16 with a residual 38 us (5.3 TB/s), without
// (backward) 25 to 30 us (4.5 to 5.3 TB/s; ALU 54 and 71 % busy); one mask held over
// 64 steps of 32 x 5000 fp32 states 18 us from memory (4.5 TB/s), 14 us from the
// last-level cache.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "ck.h"
#include "ck_internal.h"
#include "sequence.h"

namespace ckhip {
namespace {

constexpr int kDropThreads = 256;
constexpr int kDropHeld = 4;  // steps a thread gives one held mask to

template <typename E>
struct DropArgs {
  Seq<const E> x, res;
  Seq<E> out;
  const int64_t* counter;
  uint64_t offset;
  uint32_t seed_lo, seed_hi;
  int T, B, D, cols;  // cols: groups of 8 channels
  int runs;           // held masks: runs of kDropHeld steps
  uint32_t q;
  float scale;
};

__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// A thread's N channels from c on.
template <typename E, bool HELD, int N>
__device__ __forceinline__ void drop_rows(const DropArgs<E>& s, const uint32_t (&h)[8], int b,
                                          int run, int c) {
  const int t0 = HELD ? run * kDropHeld : run, t1 = HELD ? min(t0 + kDropHeld, s.T) : run + 1;
#pragma unroll 2
  for (int t = t0; t < t1; ++t) {
    const Pack<E, N> x = pack_load<true, E, N>(s.x.row(t, b) + c, N);
    Pack<E, N> z = {};
    if (s.res.p) z = pack_load<true, E, N>(s.res.row(t, b) + c, N);
    float y[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
      y[k] = (float)z.v[k] + (h[k] >= s.q ? (float)x.v[k] * s.scale : 0.0f);
    pack_store<true, E, N>(s.out.row(t, b) + c, y, N);
  }
}

template <typename E, bool HELD>
__global__ __launch_bounds__(kDropThreads) void drop(const DropArgs<E> s) {
  const int64_t i = seq_block() * kDropThreads + threadIdx.x;
  const int col = (int)(i % s.cols);
  const int64_t r = i / s.cols;
  const int b = (int)(r % s.B), run = (int)(r / s.B);
  if (r >= (int64_t)s.B * (HELD ? s.runs : s.T)) return;
  const uint64_t off = s.offset + (s.counter ? (uint64_t)*s.counter : 0);
  const uint32_t mrow = HELD ? (uint32_t)b : (uint32_t)r;
  const uint4 w = philox((uint32_t)col, mrow, (uint32_t)off, (uint32_t)(off >> 32), s.seed_lo,
                         s.seed_hi);
  const uint32_t h[8] = {w.x & 0xFFFF, w.x >> 16, w.y & 0xFFFF, w.y >> 16,
                         w.z & 0xFFFF, w.z >> 16, w.w & 0xFFFF, w.w >> 16};
  // A row's last group, where it is short, has its wave wait: in few wide accesses
  // (984 x 36 x 383 fp16, held, forward + backward: 28 us, element by element 37).
  const int c = col * 8;
  if (c + 8 <= s.D) return drop_rows<E, HELD, 8>(s, h, b, run, c);
  switch (s.D & 7) {
    case 1: return drop_rows<E, HELD, 1>(s, h, b, run, c);
    case 2: return drop_rows<E, HELD, 2>(s, h, b, run, c);
    case 3: return drop_rows<E, HELD, 3>(s, h, b, run, c);
    case 4: return drop_rows<E, HELD, 4>(s, h, b, run, c);
    case 5: return drop_rows<E, HELD, 5>(s, h, b, run, c);
    case 6: return drop_rows<E, HELD, 6>(s, h, b, run, c);
    default: return drop_rows<E, HELD, 7>(s, h, b, run, c);
  }
}

ck_status drop_run(const ck_dropout_shape* s, const ck_seq& x, const ck_seq& res, const ck_seq& out,
                   hipStream_t stream) {
  if (!s) {
    set_error("shape is NULL");
    return CK_ERR_NULL_ARG;
  }
  ck_status rc = seq_check_shape(s->T, s->B, s->D, s->dtype);
  if (rc != CK_OK) return rc;
  if (!(s->p >= 0.0 && s->p <= 1.0)) {
    set_error("p must be in [0, 1] (got %g)", s->p);
    return CK_ERR_BAD_VALUE;
  }
  const int64_t rows = s->T * s->B, cols = (s->D + 7) / 8;
  if (rows >= (int64_t(1) << 32) || rows * cols / kDropThreads >= INT_MAX - 1) {
    set_error("T=%lld, B=%lld or D=%lld is too large", (long long)s->T, (long long)s->B,
              (long long)s->D);
    return CK_ERR_TOO_LARGE;
  }
  const bool none = s->T == 0;
  rc = seq_check(x, s->dtype, none, "the input");
  if (rc == CK_OK) rc = seq_check(res, s->dtype, true, "residual");
  if (rc == CK_OK) rc = seq_check_out(out, s->T, s->B, s->D, s->dtype, none, "the output");
  if (rc != CK_OK || none) return rc;
  const uint32_t q = (uint32_t)std::floor(65536.0 * s->p + 0.5);
  return seq_dispatch(s->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    DropArgs<E> a = {};
    a.x = seq_of<const E>(x);
    a.res = seq_of<const E>(res);
    a.out = seq_of<E>(out);
    a.counter = s->counter;
    a.offset = s->offset;
    a.seed_lo = (uint32_t)s->seed;
    a.seed_hi = (uint32_t)(s->seed >> 32);
    a.T = (int)s->T; a.B = (int)s->B; a.D = (int)s->D;
    a.cols = (int)cols;
    a.runs = (int)((s->T + kDropHeld - 1) / kDropHeld);
    a.q = q;
    a.scale = q < 65536 ? (float)(65536.0 / (65536.0 - q)) : 0.0f;
    const int64_t n = (s->held ? (int64_t)a.runs * s->B : rows) * cols;
    const dim3 grid = seq_grid((n + kDropThreads - 1) / kDropThreads);
    if (s->held)
      drop<E, true><<<grid, kDropThreads, 0, stream>>>(a);
    else
      drop<E, false><<<grid, kDropThreads, 0, stream>>>(a);
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}

}  // namespace
}  // namespace ckhip

using namespace ckhip;

extern "C" ck_status ck_dropout_forward(const ck_dropout_shape* shape, ck_seq x, ck_seq residual,
                                        ck_seq out, hipStream_t stream) {
  clear_error();
  return drop_run(shape, x, residual, out, stream);
}

extern "C" ck_status ck_dropout_backward(const ck_dropout_shape* shape, ck_seq grad_out,
                                         ck_seq grad_x, hipStream_t stream) {
  clear_error();
  return drop_run(shape, grad_out, ck_seq{nullptr, 0, 0}, grad_x, stream);
}
