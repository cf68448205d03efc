// beam.hip -- beam search's selection over beams and vocabulary, and the
// reordering of the states that the beams carry.
//
//   score(k, v) = s_k + x_kv - log sum_w exp x_kw
//   the K best (k, v) of a text, by score descending, then k V + v ascending
//
// HBM bounds the selection: every logit is read once and kept in registers.  A wave
// takes kBeamSpan adjacent logits of a row (so few rows still fill the chip) and
// leaves their maximum, their sum of exponentials and their K best in order; a
// workgroup a text joins these row by row and then takes K times the best head of
// the K rows' lists.
//
// The K best of a wave: the K-th largest of its lanes' maxima is a limit that at
// least K logits reach and few more (fewer than K lanes lie above it).  Those above it
// are ranked by counting, those at it follow in the order of the vocabulary.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>

#include "ck.h"
#include "ck_internal.h"
#include "sequence.h"

namespace ckhip {
namespace {

constexpr int kBeamMaxK = 32;
constexpr int kBeamV = 8;        // logits a lane and access
constexpr int kBeamPacks = 8;    // accesses of a wave
constexpr int kBeamSpan = 64 * kBeamV * kBeamPacks;
constexpr int kBeamWaves = 4;    // of a workgroup that reads logits
constexpr int kBeamJoinWaves = 16;

// A logit and its place as one number that orders by value, then by the lower place;
// 0: none.
__device__ __forceinline__ uint32_t beam_order(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);  // (-0 is 0)
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float beam_value(uint32_t o) {
  return __builtin_bit_cast(float, o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t beam_key(float x, uint32_t v) {
  return (uint64_t)beam_order(x) << 32 | (uint32_t)~v;
}
__device__ __forceinline__ uint32_t beam_place(uint64_t key) { return ~(uint32_t)key; }

// Lanes of `mask` below this one.
__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int m = 32; m; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
  return x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
  return x;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t x) {
#pragma unroll
  for (int m = 32; m; m >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)x, m);
    x = o > x ? o : x;
  }
  return x;
}

template <typename E>
struct BeamArgs {
  Seq<const E> x;  // row (text, beam)
  const float* scores;
  const uint8_t* finished;
  float2* sums;      // [B K][parts]: maximum and sum of exponentials
  uint64_t* best;    // [B K][parts][K] keys in order
  float* out_scores;
  int64_t *parents, *tokens;
  uint8_t* out_finished;
  int64_t eos;       // -1: none
  int B, K, V, parts;
};

// Whether a row's logits are not looked at: it goes on with the end token alone, or
// nothing that follows from it has a score.
template <typename E>
__device__ __forceinline__ bool beam_skips(const BeamArgs<E>& s, int64_t row) {
  const float score = s.scores[row];
  return (s.finished && s.finished[row]) || !(score > -__builtin_inff());
}

template <typename E>
__global__ __launch_bounds__(64 * kBeamWaves) void beam_part(const BeamArgs<E> s, int64_t waves) {
  extern __shared__ uint64_t beam_lds[];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int64_t id = seq_block() * (blockDim.x >> 6) + wave;
  if (id >= waves) return;
  const int64_t row = id / s.parts;
  const int part = (int)(id % s.parts);
  if (beam_skips(s, row)) return;
  const int K = s.K;
  // Above the limit lie at most K - 1 lanes' logits; at it, K count.
  const int room = (K - 1) * kBeamV * kBeamPacks;
  uint64_t* above = beam_lds + (int64_t)wave * (room + K);
  uint64_t* level = above + room;

  const E* p = s.x.row(row / K, row % K);
  const int64_t base = (int64_t)part * kBeamSpan;
  float x[kBeamPacks][kBeamV];
#pragma unroll
  for (int j = 0; j < kBeamPacks; ++j) {
    const int64_t v = base + j * 64 * kBeamV + lane * kBeamV;
    Pack<E, kBeamV> w;
    if (v + kBeamV <= s.V) {
      w = pack_load<true, E, kBeamV>(p + v, kBeamV);
    } else {
#pragma unroll
      for (int k = 0; k < kBeamV; ++k) {
        w.v[k] = (E)-__builtin_inff();
        if (v + k < s.V) w.v[k] = p[v + k];
      }
    }
#pragma unroll
    for (int k = 0; k < kBeamV; ++k) x[j][k] = (float)w.v[k];
  }
  float top[kBeamPacks], best, most, sum;
  auto look = [&](float zero) {  // maxima and the sum
    best = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < kBeamPacks; ++j) {
      top[j] = x[j][0];
#pragma unroll
      for (int k = 1; k < kBeamV; ++k) top[j] = fmaxf(top[j], x[j][k]);
      best = fmaxf(best, top[j]);
    }
    most = wave_max(best);
    const float m = most == -__builtin_inff() ? zero : most;
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kBeamPacks; ++j)
#pragma unroll
      for (int k = 0; k < kBeamV; ++k) sum += exp2_hw((x[j][k] - m) * kLog2e);
    sum = wave_sum(sum);
  };
  look(-__builtin_inff());
  if (!(sum < __builtin_inff())) {
    // A NaN, +inf, or no logit above -inf makes the sum a NaN.  (None of the others
    // does: each term is at most 1.)  A NaN counts as -inf, +inf as the largest
    // finite value.
#pragma unroll
    for (int j = 0; j < kBeamPacks; ++j)
#pragma unroll
      for (int k = 0; k < kBeamV; ++k)
        x[j][k] = x[j][k] != x[j][k] ? -__builtin_inff() : fminf(x[j][k], FLT_MAX);
    look(0.0f);
  }
  if (lane == 0) s.sums[row * s.parts + part] = make_float2(most, sum);

  // The K-th largest of the lanes' maxima (a lane without logits: the lowest).
  const int64_t there = s.V - base;  // logits from here on
  const uint32_t mine = lane * kBeamV < there ? beam_order(best) : 0;
  uint32_t limit = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t more = limit | 1u << bit;
    if (__popcll(__ballot(mine >= more)) >= K) limit = more;
  }
  // Fewer than K lanes with logits: every logit counts.
  const bool every = limit == 0;
  const float border = every ? -__builtin_inff() : beam_value(limit);
  int n = 0, at_border = 0;
#pragma unroll
  for (int j = 0; j < kBeamPacks; ++j) {
    const int64_t first = j * 64 * kBeamV + lane * kBeamV;
    const bool some = first < there && top[j] >= border;
    if (!__ballot(some)) continue;
    uint64_t hit[kBeamV];
#pragma unroll
    for (int k = 0; k < kBeamV; ++k) {
      const bool over = first + k < there && x[j][k] > border;
      const uint64_t mask = __ballot(over);
      if (over) above[n + lanes_below(mask)] = beam_key(x[j][k], (uint32_t)(base + first + k));
      n += __popcll(mask);
      hit[k] = __ballot(first + k < there && x[j][k] == border);
    }
    int before = at_border;  // of the pack's logits at the border, lanes below and own ones before
#pragma unroll
    for (int k = 0; k < kBeamV; ++k) before += lanes_below(hit[k]);
#pragma unroll
    for (int k = 0; k < kBeamV; ++k) {
      at_border += __popcll(hit[k]);
      if (hit[k] >> lane & 1) {
        if (before < K) level[before] = beam_key(x[j][k], (uint32_t)(base + first + k));
        ++before;
      }
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  uint64_t* out = s.best + (row * s.parts + part) * K;
  for (int i = lane; i < n; i += 64) {
    const uint64_t key = above[i];
    int rank = 0;
    for (int o = 0; o < n; ++o) rank += above[o] > key;
    if (rank < K) out[rank] = key;
  }
  for (int i = lane; i < K - n; i += 64) out[n + i] = i < at_border ? level[i] : 0;
}

// Takes the K best of `n` keys, no two alike but 0, in order: of the lane's, K times
// the best of the wave.  Written to list[0 .. K).
constexpr int kBeamHold = 8;  // keys a lane holds at a time
__device__ __forceinline__ void beam_take(const uint64_t* keys, int64_t n, int K, int lane,
                                          uint64_t* list) {
  uint64_t kept = 0;  // lane i: the i-th best so far
  for (int64_t base = 0; base < n; base += 64 * kBeamHold) {
    uint64_t hold[kBeamHold], next = 0;
#pragma unroll
    for (int e = 0; e < kBeamHold; ++e) {
      const int64_t i = base + e * 64 + lane;
      hold[e] = i < n ? keys[i] : 0;
    }
    for (int k = 0; k < K; ++k) {
      uint64_t best = kept;
#pragma unroll
      for (int e = 0; e < kBeamHold; ++e) best = hold[e] > best ? hold[e] : best;
      best = wave_max(best);
      if (lane == k) next = best;
      if (best == 0) continue;
      if (kept == best) kept = 0;
#pragma unroll
      for (int e = 0; e < kBeamHold; ++e) hold[e] = hold[e] == best ? 0 : hold[e];
    }
    kept = next;
  }
  if (lane < K) list[lane] = kept;
}

template <typename E>
__global__ __launch_bounds__(64 * kBeamJoinWaves) void beam_join(const BeamArgs<E> s) {
  __shared__ uint64_t list[kBeamMaxK][kBeamMaxK];
  // a row's maximum, and the logarithm of its sum relative to that (their sum would
  // lose the one in the other where logits are large)
  __shared__ double tops[kBeamMaxK], logs[kBeamMaxK];
  const int64_t text = seq_block();
  if (text >= s.B) return;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = (int)blockDim.x >> 6, lane = threadIdx.x & 63, K = s.K;
  for (int k = wave; k < K; k += waves) {
    const int64_t row = text * K + k;
    if (beam_skips(s, row)) {
      // (the end token first, if there is one to go on with, then the others: no score)
      if (lane < K) {
        const bool ends = s.finished && s.finished[row] && s.scores[row] > -__builtin_inff();
        const int64_t eos = ends ? s.eos : s.V;
        const int64_t v = ends && lane == 0 ? eos : lane - (ends && lane <= eos ? 1 : 0);
        const float x = ends && lane == 0 ? 0.0f : -__builtin_inff();
        list[k][lane] = lane < s.V ? beam_key(x, (uint32_t)v) : 0;
      }
      if (lane == 0) tops[k] = logs[k] = 0.0;
      continue;
    }
    const float2* sums = s.sums + row * s.parts;
    float most = -__builtin_inff();
    for (int p = lane; p < s.parts; p += 64) most = fmaxf(most, sums[p].x);
    most = wave_max(most);
    double sum = 0.0;
    if (most > -__builtin_inff())
      for (int p = lane; p < s.parts; p += 64)
        if (sums[p].x > -__builtin_inff())
          sum += (double)sums[p].y * exp((double)sums[p].x - (double)most);
#pragma unroll
    for (int m = 32; m; m >>= 1) sum += __shfl_xor(sum, m);
    if (lane == 0) {
      tops[k] = (double)most;
      logs[k] = sum > 0.0 ? log(sum) : 0.0;
    }
    beam_take(s.best + row * s.parts * K, (int64_t)s.parts * K, K, lane, list[k]);
  }
  __syncthreads();
  if (wave != 0) return;
  // Lane k goes through row k's list; scores are compared in 64 bits.
  int taken = 0;
  const double from = lane < K ? (double)s.scores[text * K + lane] : 0.0;
  const bool done = lane < K && s.finished && s.finished[text * K + lane];
  auto head = [&]() -> uint64_t {  // ordered score; 0: the list is at its end
    const uint64_t key = lane < K && taken < K ? list[lane][taken] : 0;
    if (key == 0) return 0;
    const float x = beam_value((uint32_t)(key >> 32));
    double score = from + (((double)x - tops[lane]) - logs[lane]);
    if (!(x > -__builtin_inff()) || !(score > -__builtin_inf())) score = -__builtin_inf();
    const uint64_t u = __builtin_bit_cast(uint64_t, score + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
  };
  uint64_t mine = head();
  for (int r = 0; r < K; ++r) {
    const uint64_t best = wave_max(mine);
    if (lane == __ffsll((unsigned long long)__ballot(mine == best)) - 1) {
      const uint64_t u = best ^ ((uint64_t)((int64_t)~best >> 63) | 0x8000000000000000ull);
      const int64_t o = text * K + r, v = beam_place(list[lane][taken]);
      s.out_scores[o] = (float)__builtin_bit_cast(double, u);
      s.parents[o] = lane;
      s.tokens[o] = v;
      if (s.out_finished) s.out_finished[o] = done || v == s.eos;
      ++taken;
      mine = head();
    }
  }
}

// ------------------------------------------------------------------ reordering

constexpr int kMoveThreads = 256;
constexpr int kMoveTable = 32;  // states a launch

struct MoveState {
  const char* in;
  char* out;
  int64_t in_row, in_seg, out_row, out_seg;  // bytes
  int64_t bytes;                             // adjacent ones of a segment
  int64_t packs;                             // of a segment
  int64_t items;                             // packs of a row
  int64_t first;                             // first workgroup
  int64_t blocks;                            // workgroups a text
};
struct MoveTable {
  MoveState s[kMoveTable];
  const int64_t* parents;
  int64_t first;  // one behind the last workgroup
  int count, K, B;
};

template <int N>
struct __attribute__((packed, aligned(1))) Bytes {
  uint8_t v[N];
};

// One pack of all of a text's rows: every row is read before any is written, so that
// a state may be reordered in place.
template <int N, int KM>
__device__ __forceinline__ void move_pack(const MoveState& s, const int64_t* parents, int K,
                                          const char* in, char* out) {
  Bytes<N> v[KM];
#pragma unroll
  for (int k = 0; k < KM; ++k)
    if (k < K) {
      const int64_t from = min(max(parents[k], (int64_t)0), (int64_t)K - 1);
      v[k] = *reinterpret_cast<const Bytes<N>*>(in + from * s.in_row);
    }
#pragma unroll
  for (int k = 0; k < KM; ++k)
    if (k < K) *reinterpret_cast<Bytes<N>*>(out + k * s.out_row) = v[k];
}

template <int N, int KM>
__global__ __launch_bounds__(kMoveThreads) void move_rows(const MoveTable t) {
  const int64_t block = seq_block();
  if (block >= t.first) return;
  int i = 0;
  while (i + 1 < t.count && t.s[i + 1].first <= block) ++i;
  const MoveState& s = t.s[i];
  const int64_t text = (block - s.first) / s.blocks;
  const int64_t item = (block - s.first) % s.blocks * kMoveThreads + threadIdx.x;
  if (item >= s.items) return;
  const int64_t seg = item / s.packs, at = item % s.packs * N;
  const int64_t* parents = t.parents + text * t.K;
  const char* in = s.in + text * t.K * s.in_row + seg * s.in_seg + at;
  char* out = s.out + text * t.K * s.out_row + seg * s.out_seg + at;
  const int left = (int)min(s.bytes - at, (int64_t)N);
  if (left == N) return move_pack<N, KM>(s, parents, t.K, in, out);
  int o = 0;
  if constexpr (N > 8)
    if (left & 8) move_pack<8, KM>(s, parents, t.K, in, out), o = 8;
  if constexpr (N > 4)
    if (left & 4) move_pack<4, KM>(s, parents, t.K, in + o, out + o), o += 4;
  if (left & 2) move_pack<2, KM>(s, parents, t.K, in + o, out + o), o += 2;
  if (left & 1) move_pack<1, KM>(s, parents, t.K, in + o, out + o);
}

ck_status beam_check_shape(const ck_beam_shape* s) {
  if (!s) {
    set_error("shape is NULL");
    return CK_ERR_NULL_ARG;
  }
  if (s->B <= 0 || s->K <= 0 || s->V <= 0 || s->K > kBeamMaxK) {
    set_error("bad sizes: B=%lld K=%lld V=%lld (K at most %d)", (long long)s->B, (long long)s->K,
              (long long)s->V, kBeamMaxK);
    return CK_ERR_BAD_SIZE;
  }
  if (s->V > INT_MAX - 2 * kBeamSpan || s->B > (int64_t(1) << 30) ||
      s->B * s->K > (int64_t(1) << 40) / s->V) {
    set_error("B=%lld, K=%lld or V=%lld is too large", (long long)s->B, (long long)s->K,
              (long long)s->V);
    return CK_ERR_TOO_LARGE;
  }
  if (s->dtype != CK_F32 && s->dtype != CK_BF16 && s->dtype != CK_F16) {
    set_error("unknown element type %d", s->dtype);
    return CK_ERR_BAD_VALUE;
  }
  if (s->eos < -1 || s->eos >= s->V) {
    set_error("eos must be -1 or below V (got %lld)", (long long)s->eos);
    return CK_ERR_BAD_VALUE;
  }
  return CK_OK;
}

struct BeamWs {
  int parts;
  size_t best, total;
};
BeamWs beam_ws(const ck_beam_shape& s) {
  BeamWs w;
  w.parts = (int)((s.V + kBeamSpan - 1) / kBeamSpan);
  const size_t rows = (size_t)(s.B * s.K) * w.parts;
  w.best = (rows * sizeof(float2) + 255) & ~size_t(255);
  w.total = w.best + rows * s.K * sizeof(uint64_t);
  return w;
}

ck_status beam_check_out(const void* p, size_t align, const char* what) {
  if (!p) {
    set_error("%s is NULL", what);
    return CK_ERR_NULL_ARG;
  }
  if (reinterpret_cast<uintptr_t>(p) % align) {
    set_error("%s is not aligned to its element type", what);
    return CK_ERR_BAD_VALUE;
  }
  return CK_OK;
}

// Rows or segments of a state lie over one another.
bool move_overlaps(int64_t rows, int64_t row, int64_t segs, int64_t seg, int64_t bytes) {
  if (rows > 1 && segs > 1) {
    if (row < bytes || seg < bytes) return true;
    return row < seg ? (seg - bytes) / (rows - 1) < row : (row - bytes) / (segs - 1) < seg;
  }
  return rows > 1 ? row < bytes : segs > 1 && seg < bytes;
}

template <int N, int KM>
void move_launch(MoveTable& t, hipStream_t stream) {
  t.first = 0;
  for (int i = 0; i < t.count; ++i) {
    MoveState& s = t.s[i];
    s.packs = (s.bytes + N - 1) / N;
    s.items *= s.packs;
    s.blocks = (s.items + kMoveThreads - 1) / kMoveThreads;
    s.first = t.first;
    t.first += s.blocks * t.B;
  }
  move_rows<N, KM><<<seq_grid(t.first), kMoveThreads, 0, stream>>>(t);
}

}  // namespace
}  // namespace ckhip

using namespace ckhip;

extern "C" ck_status ck_beam_sizes(const ck_beam_shape* shape, size_t* workspace_bytes) {
  clear_error();
  const ck_status rc = beam_check_shape(shape);
  if (rc != CK_OK) return rc;
  if (workspace_bytes) *workspace_bytes = beam_ws(*shape).total;
  return CK_OK;
}

extern "C" ck_status ck_beam_select(const ck_beam_shape* shape, ck_seq logits, const float* scores,
                                    const uint8_t* finished, float* out_scores, int64_t* parents,
                                    int64_t* tokens, uint8_t* out_finished, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  ck_status rc = beam_check_shape(shape);
  if (rc != CK_OK) return rc;
  rc = seq_check(logits, shape->dtype, false, "logits");
  if (rc == CK_OK) rc = beam_check_out(scores, 4, "scores");
  if (rc == CK_OK) rc = beam_check_out(out_scores, 4, "out_scores");
  if (rc == CK_OK) rc = beam_check_out(parents, 8, "parents");
  if (rc == CK_OK) rc = beam_check_out(tokens, 8, "tokens");
  if (rc != CK_OK) return rc;
  if (finished && shape->eos < 0) {
    set_error("finished beams go on with an end token: eos is missing");
    return CK_ERR_BAD_VALUE;
  }
  const BeamWs ws = beam_ws(*shape);
  rc = seq_check_ws(workspace, workspace_bytes, ws.total);
  if (rc != CK_OK) return rc;
  return seq_dispatch(shape->dtype, [&](auto* e) -> ck_status {
    using E = std::remove_pointer_t<decltype(e)>;
    BeamArgs<E> a = {};
    a.x = seq_of<const E>(logits);
    a.scores = scores;
    a.finished = finished;
    a.sums = static_cast<float2*>(workspace);
    a.best = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + ws.best);
    a.out_scores = out_scores;
    a.parents = parents;
    a.tokens = tokens;
    a.out_finished = out_finished;
    a.eos = shape->eos;
    a.B = (int)shape->B;
    a.K = (int)shape->K;
    a.V = (int)shape->V;
    a.parts = ws.parts;
    const int64_t waves = shape->B * shape->K * ws.parts;
    const int per = shape->K > 16 ? kBeamWaves / 2 : kBeamWaves;  // (32 KB of LDS at most)
    const size_t lds =
        (size_t)per * sizeof(uint64_t) * ((shape->K - 1) * kBeamV * kBeamPacks + shape->K);
    beam_part<E><<<seq_grid((waves + per - 1) / per), 64 * per, lds, stream>>>(a, waves);
    // (a launch holds fewer than 2^32 threads along its first dimension)
    const int64_t join = shape->B < kSeqGridX / 2 ? kBeamJoinWaves : kBeamWaves;
    beam_join<E><<<seq_grid(shape->B), 64 * (int)std::min(shape->K, join), 0, stream>>>(a);
    CK_HIP_TRY(hipGetLastError());
    return CK_OK;
  });
}

extern "C" ck_status ck_beam_reorder(const ck_beam_state* states, int64_t count,
                                     const int64_t* parents, int64_t B, int64_t K,
                                     hipStream_t stream) {
  clear_error();
  if (count < 0 || B <= 0 || K <= 0 || K > kBeamMaxK) {
    set_error("bad sizes: count=%lld B=%lld K=%lld (K at most %d)", (long long)count, (long long)B,
              (long long)K, kBeamMaxK);
    return CK_ERR_BAD_SIZE;
  }
  if (B > (int64_t(1) << 30) || count > 4096) {
    set_error("B=%lld or count=%lld is too large", (long long)B, (long long)count);
    return CK_ERR_TOO_LARGE;
  }
  if ((count > 0 && !states) || !parents) {
    set_error("states or parents are NULL");
    return CK_ERR_NULL_ARG;
  }
  if (reinterpret_cast<uintptr_t>(parents) % 8) {
    set_error("parents are not aligned to their element type");
    return CK_ERR_BAD_VALUE;
  }
  const int64_t most = int64_t(1) << 44;
  for (int64_t i = 0; i < count; ++i) {
    const ck_beam_state& s = states[i];
    if (s.segments < 0 || s.bytes < 0) {
      set_error("state %lld: bad sizes", (long long)i);
      return CK_ERR_BAD_SIZE;
    }
    if (s.segments == 0 || s.bytes == 0) continue;
    if (s.segments > most / s.bytes || s.segments * s.bytes > most / B) {
      set_error("state %lld is too large", (long long)i);
      return CK_ERR_TOO_LARGE;
    }
    if (!s.in || !s.out) {
      set_error("state %lld is NULL", (long long)i);
      return CK_ERR_NULL_ARG;
    }
    if (s.in_row < 0 || s.in_segment < 0 || s.out_row < 0 || s.out_segment < 0 ||
        move_overlaps(B * K, s.out_row, s.segments, s.out_segment, s.bytes)) {
      set_error("state %lld: strides are negative, or rows of the output overlap", (long long)i);
      return CK_ERR_BAD_VALUE;
    }
    if (s.in == s.out && ((B * K > 1 && s.in_row != s.out_row) ||
                          (s.segments > 1 && s.in_segment != s.out_segment))) {
      set_error("state %lld: its output is the state itself with other strides", (long long)i);
      return CK_ERR_BAD_VALUE;
    }
    for (int64_t o = 0; o < i; ++o)
      if (states[o].segments && states[o].bytes &&
          (states[o].out == s.out || states[o].in == s.out || states[o].out == s.in)) {
        set_error("states %lld and %lld share memory that is written", (long long)o, (long long)i);
        return CK_ERR_BAD_VALUE;
      }
  }
  MoveTable t = {};
  t.parents = parents;
  t.K = (int)K;
  t.B = (int)B;
  for (int64_t i = 0; i < count;) {
    t.count = 0;
    for (; i < count && t.count < kMoveTable; ++i) {
      const ck_beam_state& s = states[i];
      if (s.segments == 0 || s.bytes == 0) continue;
      MoveState& m = t.s[t.count++];
      m.in = static_cast<const char*>(s.in);
      m.out = static_cast<char*>(s.out);
      m.in_row = s.in_row;
      m.in_seg = s.in_segment;
      m.out_row = s.out_row;
      m.out_seg = s.out_segment;
      m.bytes = s.bytes;
      m.items = s.segments;
    }
    if (t.count == 0) break;
    // as many bytes a thread holds for every width: 8 rows of 16, 16 of 8, 32 of 4
    if (K <= 8) move_launch<16, 8>(t, stream);
    else if (K <= 16) move_launch<8, 16>(t, stream);
    else move_launch<4, 32>(t, stream);
    CK_HIP_TRY(hipGetLastError());
  }
  return CK_OK;
}
