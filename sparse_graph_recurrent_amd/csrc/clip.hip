// clip.hip -- the norm of all gradients of a model, and their scaling to a limit.
//
//   n = sqrt(sum over all tensors of g^2),   c = max_norm / n if n > max_norm else 1,   out = c g
//
// HBM bounds both launches: the norm has to be known before anything is scaled, so
// every gradient is read twice and written once.  Squares are summed in 64 bits (a
// conversion and a multiply-add an element; the vector ALU is 10 to 22 % busy): no
// gradient that its type can hold overflows them.  Measured: 14 tensors of 26 M fp32 66 us
// (4.7 TB/s over the three passes; sums 17 us and scaling 35 where the last-level cache
// has what fits it), 60 tensors of 60 M bf16 82 us (4.4 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "ck.h"
#include "ck_internal.h"
#include "sequence.h"

namespace ckhip {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipTable = 96;      // tensors a launch (the table is its argument: at most 4 KB)
constexpr int kClipAccess = 16;     // bytes a thread and access
constexpr int kClipDeep = 8;        // accesses of a thread in a chunk, at most
constexpr int kClipUnit = kClipThreads * kClipAccess;  // bytes of a chunk of one access a thread
// Workgroups of a launch: all run at once (4 waves a SIMD); as many partial sums.  (2048:
// 67.5 and 85 us for 66 and 82.)
constexpr int kClipBlocks = 1024;

struct ClipTable {
  const void* in[kClipTable];
  void* out[kClipTable];
  int64_t n[kClipTable];          // bytes
  int64_t first[kClipTable + 1];  // first chunk of each tensor
  int8_t dtype[kClipTable];
  int count;
  int units;  // of a chunk
};

// A thread's share of a chunk: as many accesses as the chunk has units.
typedef uint32_t ClipWord __attribute__((ext_vector_type(4), aligned(2)));
struct ClipChunk {
  ClipWord v[kClipDeep];

  // Chunk `chunk` of tensor i.  What lies behind the tensor's end counts as 0.
  __device__ __forceinline__ void load(const ClipTable& t, int i, int64_t chunk) {
    const char* p = static_cast<const char*>(t.in[i]);
    const int64_t n = t.n[i], base = chunk * t.units * kClipUnit;
    const int thread = threadIdx.x * kClipAccess;
    if (base + (int64_t)t.units * kClipUnit <= n) {
#pragma unroll
      for (int u = 0; u < kClipDeep; ++u)
        if (u < t.units)
          v[u] = *reinterpret_cast<const ClipWord*>(p + base + u * kClipUnit + thread);
    } else {
#pragma unroll
      for (int u = 0; u < kClipDeep; ++u) {
        v[u] = ClipWord{};
        if (u >= t.units) continue;
        const int64_t at = base + u * kClipUnit + thread;
        if (at + kClipAccess <= n) {
          v[u] = *reinterpret_cast<const ClipWord*>(p + at);
        } else {
#pragma unroll
          for (int k = 0; k < kClipAccess / 2; ++k)  // (elements are 2 or 4 bytes)
            if (at + 2 * k < n)
              v[u][k / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + at + 2 * k)
                             << 16 * (k & 1);
        }
      }
    }
  }
};

// Elements of an access as fp32, and back.
template <typename E>
__device__ __forceinline__ float clip_get(const ClipWord& w, int k) {
  if constexpr (sizeof(E) == 4) return __builtin_bit_cast(float, (uint32_t)w[k]);
  else return (float)__builtin_bit_cast(E, (uint16_t)(w[k / 2] >> 16 * (k & 1)));
}
template <typename E>
constexpr int kClipElems = kClipAccess / (int)sizeof(E);

// Chunks b, b + G, .. of a table, in turn (BACK: from the last).
template <bool BACK>
struct ClipWalk {
  const ClipTable& t;
  int64_t chunks, k;
  int i;
  __device__ __forceinline__ explicit ClipWalk(const ClipTable& table)
      : t(table), chunks(table.first[table.count]), k(blockIdx.x), i(BACK ? table.count - 1 : 0) {
    seek();
  }
  __device__ __forceinline__ bool more() const { return k < chunks; }
  __device__ __forceinline__ void next() {
    k += gridDim.x;
    seek();
  }
  // The chunk within tensor i.
  __device__ __forceinline__ int64_t chunk() const {
    return (BACK ? chunks - 1 - k : k) - t.first[i];
  }
  __device__ __forceinline__ void seek() {
    if (!more()) return;
    if constexpr (BACK) while (chunks - 1 - k < t.first[i]) --i;
    else while (k >= t.first[i + 1]) ++i;
  }
};

__device__ __forceinline__ double clip_block_sum(double x) {
  __shared__ double lds[kClipThreads / 64];
#pragma unroll
  for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int w = 0; w < kClipThreads / 64; ++w) x += lds[w];
  return x;
}

template <typename E>
__device__ __forceinline__ void clip_square(const ClipChunk& c, int units, double& sum) {
#pragma unroll
  for (int u = 0; u < kClipDeep; ++u)
    if (u < units)
#pragma unroll
      for (int k = 0; k < kClipElems<E>; ++k) {
        const double g = (double)clip_get<E>(c.v[u], k);
        sum = fma(g, g, sum);
      }
}

__global__ __launch_bounds__(kClipThreads) void clip_norm(const ClipTable t, double* part) {
  double sum = 0.0;
  for (ClipWalk<false> w(t); w.more(); w.next()) {
    ClipChunk c;
    c.load(t, w.i, w.chunk());
    if (t.dtype[w.i] == CK_F32) clip_square<float>(c, t.units, sum);
    else if (t.dtype[w.i] == CK_BF16) clip_square<bf16_t>(c, t.units, sum);
    else clip_square<f16_t>(c, t.units, sum);
  }
  sum = clip_block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <typename E>
__device__ __forceinline__ void clip_write(const ClipTable& t, int i, int64_t chunk,
                                           const ClipChunk& c, double scale) {
  char* p = static_cast<char*>(t.out[i]);
  const int64_t n = t.n[i], base = chunk * t.units * kClipUnit;
#pragma unroll
  for (int u = 0; u < kClipDeep; ++u) {
    if (u >= t.units) continue;
    const int64_t at = base + u * kClipUnit + (int64_t)threadIdx.x * kClipAccess;
    float y[kClipElems<E>];
#pragma unroll
    for (int k = 0; k < kClipElems<E>; ++k) {
      // (in 64 bits: a factor may lie below the range of fp32 though no gradient does)
      y[k] = (float)((double)clip_get<E>(c.v[u], k) * scale);
    }
    E* to = reinterpret_cast<E*>(p + at);
    if (at + kClipAccess <= n) pack_store<true, E, kClipElems<E>>(to, y, 0);
    else if (at < n) pack_store<false, E, kClipElems<E>>(to, y, (int)((n - at) / (int)sizeof(E)));
  }
}

// A thread's share of the partial sums.
__device__ __forceinline__ double clip_parts(const double* part, int64_t parts) {
  double sum = 0.0;
#pragma unroll 4
  for (int64_t k = threadIdx.x; k < parts; k += kClipThreads) sum += part[k];
  return sum;
}

// The sum of the partial sums of several launches, left as the first of them.  (Each of as
// many scaling launches would have all its workgroups add all of them up: work by the
// square of the number of tensors.)
__global__ __launch_bounds__(kClipThreads) void clip_fold(double* part, int64_t parts) {
  const double sum = clip_block_sum(clip_parts(part, parts));  // (read before it is written)
  if (threadIdx.x == 0) part[0] = sum;
}

// Every workgroup adds the partial sums, in one order, for itself.  `same`: every
// output of the table is its gradient, so that nothing is to do where nothing is
// scaled.  Chunks are taken last first: the last are what the sums' launch left in
// the last-level cache.
__global__ __launch_bounds__(kClipThreads) void clip_scale(const ClipTable t, const double* part,
                                                           int parts, double max_norm, int same,
                                                           float* norm) {
  const double n = sqrt(clip_block_sum(clip_parts(part, parts)));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  // a norm that is not finite scales nothing: there is no direction to keep
  const bool scales = n > max_norm && (float)n < __builtin_inff();
  if (!scales && same) return;
  const double c = scales ? max_norm / n : 1.0;
  for (ClipWalk<true> w(t); w.more(); w.next()) {
    if (!t.out[w.i]) continue;
    ClipChunk x;
    x.load(t, w.i, w.chunk());
    if (t.dtype[w.i] == CK_F32) clip_write<float>(t, w.i, w.chunk(), x, c);
    else if (t.dtype[w.i] == CK_BF16) clip_write<bf16_t>(t, w.i, w.chunk(), x, c);
    else clip_write<f16_t>(t, w.i, w.chunk(), x, c);
  }
}

// most: the bytes of all gradients.
ck_status clip_check(const ck_clip_tensor* tensors, int64_t count, int64_t* most) {
  *most = 0;
  if (count < 0) {
    set_error("bad count %lld", (long long)count);
    return CK_ERR_BAD_SIZE;
  }
  if (count > (int64_t(1) << 20)) {
    set_error("count=%lld is too large", (long long)count);
    return CK_ERR_TOO_LARGE;
  }
  if (count > 0 && !tensors) {
    set_error("tensors are NULL");
    return CK_ERR_NULL_ARG;
  }
  for (int64_t i = 0; i < count; ++i) {
    const ck_clip_tensor& t = tensors[i];
    if (t.n < 0) {
      set_error("tensor %lld has %lld elements", (long long)i, (long long)t.n);
      return CK_ERR_BAD_SIZE;
    }
    if (t.n > (int64_t(1) << 44)) {
      set_error("tensor %lld is too large", (long long)i);
      return CK_ERR_TOO_LARGE;
    }
    if (t.dtype != CK_F32 && t.dtype != CK_BF16 && t.dtype != CK_F16) {
      set_error("unknown element type %d", t.dtype);
      return CK_ERR_BAD_VALUE;
    }
    if (t.n > 0 && !t.grad) {
      set_error("tensor %lld is NULL", (long long)i);
      return CK_ERR_NULL_ARG;
    }
    const size_t e = seq_elem_bytes(t.dtype);
    if (reinterpret_cast<uintptr_t>(t.grad) % e || reinterpret_cast<uintptr_t>(t.out) % e) {
      set_error("tensor %lld is not aligned to its element type", (long long)i);
      return CK_ERR_BAD_VALUE;
    }
    *most += t.n * (int64_t)e;
    if (*most > (int64_t(1) << 60)) {
      set_error("the tensors are too large");
      return CK_ERR_TOO_LARGE;
    }
  }
  return CK_OK;
}

// Whether what is written lies over something else that is written, or that is read
// as another tensor.
bool clip_overlaps(const ck_clip_tensor* tensors, int64_t count, const float* norm) {
  struct Range {
    uintptr_t from, to;
    bool written;
  };
  std::vector<Range> ranges;
  ranges.reserve(2 * count + 1);
  const uintptr_t n = reinterpret_cast<uintptr_t>(norm);
  ranges.push_back({n, n + sizeof(float), true});
  for (int64_t i = 0; i < count; ++i) {
    const ck_clip_tensor& t = tensors[i];
    const size_t bytes = (size_t)t.n * seq_elem_bytes(t.dtype);
    const uintptr_t g = reinterpret_cast<uintptr_t>(t.grad), o = reinterpret_cast<uintptr_t>(t.out);
    if (!bytes) continue;
    if (o) ranges.push_back({o, o + bytes, true});
    if (o != g) ranges.push_back({g, g + bytes, false});
  }
  std::sort(ranges.begin(), ranges.end(),
            [](const Range& a, const Range& b) { return a.from < b.from; });
  uintptr_t any = 0, written = 0;  // the furthest ends so far
  for (const Range& r : ranges) {
    if (r.from < (r.written ? any : written)) return true;
    any = std::max(any, r.to);
    if (r.written) written = std::max(written, r.to);
  }
  return false;
}

size_t clip_workspace(int64_t count) {
  const int64_t launches = std::max<int64_t>(1, (count + kClipTable - 1) / kClipTable);
  return (size_t)launches * kClipBlocks * sizeof(double);
}

// The table of the tensors [i, ..) that a launch takes; the first that it does not.
int64_t clip_fill(const ck_clip_tensor* tensors, int64_t count, int64_t i, int units,
                  ClipTable* t, bool* same) {
  t->count = 0;
  t->units = units;
  t->first[0] = 0;
  *same = true;
  for (; i < count && t->count < kClipTable; ++i) {
    const ck_clip_tensor& x = tensors[i];
    if (x.n == 0) continue;
    const int k = t->count++;
    t->in[k] = x.grad;
    t->out[k] = x.out;
    t->n[k] = x.n * (int64_t)seq_elem_bytes(x.dtype);
    t->dtype[k] = (int8_t)x.dtype;
    const int64_t unit = (int64_t)units * kClipUnit;
    t->first[k + 1] = t->first[k] + (t->n[k] + unit - 1) / unit;
    if (x.out && x.out != x.grad) *same = false;
  }
  return i;
}

}  // namespace
}  // namespace ckhip

using namespace ckhip;

extern "C" ck_status ck_clip_sizes(int64_t count, size_t* workspace_bytes) {
  clear_error();
  if (count < 0) {
    set_error("bad count %lld", (long long)count);
    return CK_ERR_BAD_SIZE;
  }
  if (workspace_bytes) *workspace_bytes = clip_workspace(count);
  return CK_OK;
}

extern "C" ck_status ck_clip_grad_norm(const ck_clip_tensor* tensors, int64_t count,
                                       double max_norm, float* norm, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  int64_t total = 0;
  ck_status rc = clip_check(tensors, count, &total);
  if (rc != CK_OK) return rc;
  if (!(max_norm >= 0.0)) {
    set_error("max_norm must not be negative (got %g)", max_norm);
    return CK_ERR_BAD_VALUE;
  }
  if (!norm) {
    set_error("norm is NULL");
    return CK_ERR_NULL_ARG;
  }
  if (reinterpret_cast<uintptr_t>(norm) % sizeof(float)) {
    set_error("norm is not aligned to its element type");
    return CK_ERR_BAD_VALUE;
  }
  rc = seq_check_ws(workspace, workspace_bytes, clip_workspace(count));
  if (rc != CK_OK) return rc;
  try {
    if (clip_overlaps(tensors, count, norm)) {
      set_error("a tensor that is written lies over another one");
      return CK_ERR_BAD_VALUE;
    }
  } catch (const std::bad_alloc&) {
    set_error("out of host memory");
    return CK_ERR_NOMEM;
  }
  // chunks long enough to keep loads in flight, short enough to reach all CUs
  int units = kClipDeep;
  while (units > 1 && total / ((int64_t)units * kClipUnit) < kClipBlocks) units >>= 1;
  double* part = static_cast<double*>(workspace);
  ClipTable t;
  bool same;
  int parts = 0, launches = 0;
  int64_t i = 0;
  do {
    i = clip_fill(tensors, count, i, units, &t, &same);
    const int blocks =
        (int)std::min<int64_t>(kClipBlocks, std::max<int64_t>(1, t.first[t.count]));
    clip_norm<<<blocks, kClipThreads, 0, stream>>>(t, part + parts);
    parts += blocks;
    ++launches;
  } while (i < count);
  if (launches > 1) {
    clip_fold<<<1, kClipThreads, 0, stream>>>(part, parts);
    parts = 1;
  }
  i = 0;
  float* to = norm;
  do {
    i = clip_fill(tensors, count, i, units, &t, &same);
    bool writes = false;
    for (int k = 0; k < t.count; ++k) writes = writes || t.out[k];
    if (!writes && !to) continue;
    const int64_t chunks = writes ? t.first[t.count] : 1;
    const int blocks = (int)std::min<int64_t>(kClipBlocks, std::max<int64_t>(1, chunks));
    clip_scale<<<blocks, kClipThreads, 0, stream>>>(t, part, parts, writes ? max_norm : INFINITY,
                                                    same ? 1 : 0, to);
    to = nullptr;
  } while (i < count);
  CK_HIP_TRY(hipGetLastError());
  return CK_OK;
}
