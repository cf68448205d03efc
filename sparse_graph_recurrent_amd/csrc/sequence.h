// sequence.h -- element types, argument checks and lane exchanges shared by
// the sequence operators (convolution, selective scan, dropout).
#pragma once

#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "ck.h"
#include "ck_internal.h"

namespace ckhip {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

inline size_t seq_elem_bytes(int dtype) { return dtype == CK_F32 ? 4 : 2; }

// Calls fn with a null pointer of the element type of `dtype` (checked before).
template <typename F>
ck_status seq_dispatch(int dtype, F&& fn) {
  switch (dtype) {
    case CK_F32: return fn((float*)nullptr);
    case CK_BF16: return fn((bf16_t*)nullptr);
    default: return fn((f16_t*)nullptr);
  }
}

// T >= 0 steps (an empty window is allowed), B and D positive, and every
// count the kernels hold in 32 bits below 2^31, with room for the ends of tiles,
// runs and workgroups that lie past T or D.
inline ck_status seq_check_shape(int64_t T, int64_t B, int64_t D, int dtype) {
  if (T < 0 || B <= 0 || D <= 0) {
    set_error("bad sizes: T=%lld B=%lld D=%lld", (long long)T, (long long)B, (long long)D);
    return CK_ERR_BAD_SIZE;
  }
  constexpr int64_t most = INT_MAX - 1024;
  if (T > most || B > most || D > most || B * D >= (int64_t(1) << 36) ||
      (T > 0 && B * D > (int64_t(1) << 46) / T)) {
    set_error("T=%lld, B=%lld or D=%lld is too large", (long long)T, (long long)B, (long long)D);
    return CK_ERR_TOO_LARGE;
  }
  if (dtype != CK_F32 && dtype != CK_BF16 && dtype != CK_F16) {
    set_error("unknown element type %d", dtype);
    return CK_ERR_BAD_VALUE;
  }
  return CK_OK;
}

// A [T, B, ...] tensor: present unless optional, aligned to its elements, with
// strides in range (a zero stride broadcasts an input; max_stride_t: what a
// kernel's 32-bit offsets from a 64-bit row address reach).
inline ck_status seq_check(const ck_seq& s, int dtype, bool optional, const char* what,
                           int64_t max_stride_t = INT64_MAX) {
  if (!s.data) {
    if (optional) return CK_OK;
    set_error("%s is NULL", what);
    return CK_ERR_NULL_ARG;
  }
  if (reinterpret_cast<uintptr_t>(s.data) % seq_elem_bytes(dtype) != 0) {
    set_error("%s is not aligned to its element type", what);
    return CK_ERR_BAD_VALUE;
  }
  if (s.stride_t < 0 || s.stride_t > max_stride_t || s.stride_b < 0) {
    set_error("%s has strides (%lld, %lld); they must be in [0, %lld] and not negative", what,
              (long long)s.stride_t, (long long)s.stride_b, (long long)max_stride_t);
    return CK_ERR_BAD_VALUE;
  }
  return CK_OK;
}

// An output: rows of `row` elements that would be written over one another (a zero
// stride, as a broadcast tensor has) are refused.
inline ck_status seq_check_out(const ck_seq& s, int64_t T, int64_t B, int64_t row, int dtype,
                               bool optional, const char* what,
                               int64_t max_stride_t = INT64_MAX) {
  const ck_status rc = seq_check(s, dtype, optional, what, max_stride_t);
  if (rc != CK_OK || !s.data) return rc;
  if (T > 0 && ((T > 1 && s.stride_t < row) || (B > 1 && s.stride_b < row))) {
    set_error("%s has strides (%lld, %lld): its rows of %lld elements overlap", what,
              (long long)s.stride_t, (long long)s.stride_b, (long long)row);
    return CK_ERR_BAD_VALUE;
  }
  return CK_OK;
}

// A launch holds fewer than 2^32 threads along a dimension of its grid.
constexpr int64_t kSeqMaxThreads = int64_t(1) << 32;
// Workgroups whose kernel takes its number from seq_block(), and leaves when there is
// nothing for it, go on in the grid's second dimension.
constexpr int64_t kSeqGridX = int64_t(1) << 22;
inline dim3 seq_grid(int64_t workgroups) {
  if (workgroups <= kSeqGridX) return dim3((unsigned)workgroups);
  return dim3((unsigned)kSeqGridX, (unsigned)((workgroups + kSeqGridX - 1) / kSeqGridX));
}
__device__ __forceinline__ int64_t seq_block() {
  return (int64_t)blockIdx.y * kSeqGridX + blockIdx.x;
}

inline ck_status seq_check_ws(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return CK_OK;
  if (!workspace) {
    set_error("workspace is NULL");
    return CK_ERR_NULL_ARG;
  }
  const ck_status rc = check_aligned(workspace, "workspace");
  if (rc != CK_OK) return rc;
  if (bytes < need) {
    set_error("workspace of %zu bytes is below the %zu required", bytes, need);
    return CK_ERR_WORKSPACE;
  }
  return CK_OK;
}

// Typed view of a ck_seq inside a kernel.
template <typename E>
struct Seq {
  E* p;
  int64_t st, sb;
  __device__ __forceinline__ E* row(int64_t t, int64_t b) const { return p + t * st + b * sb; }
};
template <typename E>
Seq<E> seq_of(const ck_seq& s) {
  return Seq<E>{static_cast<E*>(s.data), s.stride_t, s.stride_b};
}

// V adjacent elements as one load or store of up to 16 bytes an access.  The
// type asks for no more than the element's own alignment: global memory takes
// wide accesses at any address (rows of odd length start anywhere), at full
// rate where they are aligned.
template <typename E, int V>
struct __attribute__((packed, aligned(alignof(E)))) Pack {
  E v[V];
};
// FULL: all V elements are there; else the first n, 0 beyond.
template <bool FULL, typename E, int V>
__device__ __forceinline__ Pack<E, V> pack_load(const E* p, int n) {
  if constexpr (FULL) return *reinterpret_cast<const Pack<E, V>*>(p);
  Pack<E, V> w;
#pragma unroll
  for (int i = 0; i < V; ++i) w.v[i] = i < n ? p[i] : (E)0.0f;
  return w;
}
template <bool FULL, typename E, int V>
__device__ __forceinline__ void pack_store(E* p, const float (&x)[V], int n) {
  Pack<E, V> w;
#pragma unroll
  for (int i = 0; i < V; ++i) w.v[i] = (E)x[i];
  if constexpr (FULL) {
    *reinterpret_cast<Pack<E, V>*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = w.v[i];
  }
}
// The rows of one tensor from step t on at a thread's channels: one 32 x 32 +
// 64 bit multiply-add an address.
template <typename E>
struct Rows {
  const char* base;
  uint32_t step;
  __device__ __forceinline__ Rows(const Seq<E>& s, int64_t t, int64_t b, int64_t c)
      : base(reinterpret_cast<const char*>(s.row(t, b) + c)),
        step((uint32_t)s.st * (uint32_t)sizeof(E)) {}
  __device__ __forceinline__ E* at(int rel) const {
    using M = std::remove_const_t<E>;
    return reinterpret_cast<M*>(const_cast<char*>(base) + (uint64_t)(uint32_t)rel * step);
  }
};

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + exp(-x)): the exponential's overflow for x below -88 makes the
// reciprocal an exact 0.  Hardware exponential and reciprocal, and the rounding of
// the exponent: relative error up to about (4 + 1.3 |x|) 2^-24 for x < 0, which is
// 2^-17 where the value is about to vanish, and 4 2^-24 for x > 0.
__device__ __forceinline__ float sigmoid_hw(float x) {
  return rcp_hw(1.0f + exp2_hw(-kLog2e * x));
}

// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp(-|x|), and its derivative
// 1 / (1 + exp(-x)).  The part of e that the sum w = 1 + e rounds away is added
// back, to first order and without its factor 1 / w (which changes it by less
// than 2^-24 of the result): for very negative x both go over into exp(x), with
// sigmoid_hw's relative error.
struct Softplus {
  float value, slope;
};
__device__ __forceinline__ Softplus softplus_hw(float x) {
  const float e = exp2_hw(-kLog2e * fabsf(x));
  const float w = 1.0f + e, r = rcp_hw(w);
  const float l = fmaf(kLn2, __builtin_amdgcn_logf(w), e - (w - 1.0f));
  return Softplus{fmaxf(x, 0.0f) + l, x < 0.0f ? e * r : r};
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float quad_xor1(float x) { return dpp<0xB1>(x); }
__device__ __forceinline__ float quad_xor2(float x) { return dpp<0x4E>(x); }
__device__ __forceinline__ float quad_sum(float x) {
  x += quad_xor1(x);
  return x + quad_xor2(x);
}
}  // namespace ckhip
