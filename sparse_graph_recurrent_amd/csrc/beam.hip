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
// the K rows' lists.  64 texts x 8 beams x 50021 logits, bf16, some beams
// finished: 16.4 us (43 MB of logits, 2.6 TB/s: a wave's loads, 8 us at a copy's rate, then its
// sums and its search, and nothing follows that would cover them) and 7.6 for the join
// (latency: 8 rows' 104 keys, then 8 rounds).  Parts of 2048 logits: the same.
// Rows of one part each are looked at and joined by one workgroup.
//
// The K best of a wave: the K-th largest of its lanes' maxima is a limit that at
// least K logits reach and few more (fewer than K lanes lie above it).  Those above it
// are ranked by counting, those at it follow in the order of the vocabulary.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <new>
#include <vector>

#include "beam_lds.h"
#include "ck.h"
#include "ck_internal.h"
#include "overlap.h"
#include "sequence.h"

namespace ckhip {
namespace {

constexpr int kBeamSpan = 64 * kBeamV * kBeamPacks;
constexpr int kBeamWaves = 4;    // of a workgroup that reads logits
constexpr int kBeamJoinWaves = 16;
constexpr size_t kBeamWholeLds = 48 << 10;  // of a workgroup that does all of a text, at most

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
// Lane i takes what a lane before it has (CTRL: a DPP control; ROWS: which rows of 16
// lanes do), or `none` where there is no such lane.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t lane_before(uint32_t x, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, CTRL, ROWS, 0xF, false);
}
// fn over all lanes, by the vector ALU alone (an exchange through LDS takes longer than
// all six steps here): rows of 16 lanes, then rows to rows; lane 63 has it all.
template <typename F>
__device__ __forceinline__ uint32_t wave_all(uint32_t x, uint32_t none, F&& fn) {
  x = fn(x, lane_before<0x111>(x, none));
  x = fn(x, lane_before<0x112>(x, none));
  x = fn(x, lane_before<0x114>(x, none));
  x = fn(x, lane_before<0x118>(x, none));
  x = fn(x, lane_before<0x142, 0xA>(x, none));
  x = fn(x, lane_before<0x143, 0xC>(x, none));
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float value(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ float wave_max(float x) {
  return value(wave_all(bits(x), bits(-__builtin_inff()), [](uint32_t a, uint32_t b) {
    return bits(fmaxf(value(a), value(b)));
  }));
}
__device__ __forceinline__ float wave_sum(float x) {
  return value(wave_all(bits(x), 0u,
                        [](uint32_t a, uint32_t b) { return bits(value(a) + value(b)); }));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  return wave_all(x, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint64_t wave_max(uint64_t x) {
  const uint32_t high = wave_max((uint32_t)(x >> 32));
  return (uint64_t)high << 32 | wave_max((uint32_t)(x >> 32) == high ? (uint32_t)x : 0u);
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
  const uint8_t done = s.finished ? s.finished[row] : 0;
  return (done != 0) | !(score > -__builtin_inff());  // (both loads set out together)
}

// A lane's logits, as they came: 16-bit ones in half the registers, so that all waves of
// a call find room at once.
typedef uint32_t BeamWords __attribute__((ext_vector_type(4), aligned(2)));
template <typename E>
struct BeamLogits {
  static constexpr int kParts = kBeamV * (int)sizeof(E) / 16;
  BeamWords w[kBeamPacks][kParts];

  // A wave's logits from p on, the first `there` of them, at this lane's places; -inf
  // behind them.  (One branch for all: loads stay in flight together.)
  __device__ __forceinline__ void load(const E* p, int there) {
    if (there == kBeamSpan) {
#pragma unroll
      for (int j = 0; j < kBeamPacks; ++j)
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          w[j][i] = reinterpret_cast<const BeamWords*>(p + j * 64 * kBeamV)[i];
    } else {
      const uint32_t none = sizeof(E) == 4 ? 0xFF800000u
                            : std::is_same_v<E, bf16_t> ? 0xFF80FF80u : 0xFC00FC00u;
      const int left = there - ((int)threadIdx.x & 63) * kBeamV;
#pragma unroll
      for (int j = 0; j < kBeamPacks; ++j) {
        BeamWords t[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) t[i] = BeamWords{none, none, none, none};
        const E* at = p + j * 64 * kBeamV;
        const int n = left - j * 64 * kBeamV;
        if (n >= kBeamV) {
#pragma unroll
          for (int i = 0; i < kParts; ++i) t[i] = reinterpret_cast<const BeamWords*>(at)[i];
        } else {
#pragma unroll
          for (int k = 0; k < kBeamV; ++k)
            if (k < n) put(t, k, at[k]);
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) w[j][i] = t[i];
      }
    }
    anew();
  }
  static __device__ __forceinline__ void put(BeamWords (&t)[kParts], int k, E x) {
    if constexpr (sizeof(E) == 4) {
      t[k / 4][k % 4] = bits((float)x);
    } else {
      const uint32_t was = t[0][k / 2], u = __builtin_bit_cast(uint16_t, x);
      t[0][k / 2] = k & 1 ? (was & 0xFFFFu) | u << 16 : (was & 0xFFFF0000u) | u;
    }
  }
  __device__ __forceinline__ float get(int j, int k) const {
    if constexpr (sizeof(E) == 4) return value(w[j][k / 4][k % 4]);
    else if constexpr (std::is_same_v<E, bf16_t>)
      return value(k & 1 ? w[j][0][k / 2] & 0xFFFF0000u : w[j][0][k / 2] << 16);
    else return (float)__builtin_bit_cast(E, (uint16_t)(w[j][0][k / 2] >> 16 * (k & 1)));
  }
  // A NaN counts as -inf, +inf as the largest finite value.
  __device__ __forceinline__ float sane(int j, int k) const {
    const float x = get(j, k);
    return x != x ? -__builtin_inff() : fminf(x, FLT_MAX);
  }
  // Has the compiler convert again what follows, rather than keep it.
  __device__ __forceinline__ void anew() {
#pragma unroll
    for (int j = 0; j < kBeamPacks; ++j)
#pragma unroll
      for (int i = 0; i < kParts; ++i) asm("" : "+v"(w[j][i]));
  }
};

// A wave's part of a row.
template <typename E>
__device__ __forceinline__ void beam_look(const BeamArgs<E>& s, uint32_t row, int part, char* lds) {
  if (beam_skips(s, row)) return;
  const int K = s.K, lane = threadIdx.x & 63;
  const BeamLds room(K);
  float* hits = reinterpret_cast<float*>(lds);                       // [packs][kBeamV]
  uint64_t* above = reinterpret_cast<uint64_t*>(lds + room.above_at);
  uint64_t* level = reinterpret_cast<uint64_t*>(lds + room.level_at);  // [K]
  int* places = reinterpret_cast<int*>(lds + room.places_at);        // [packs]

  const uint32_t text = row / (uint32_t)K;
  const E* p = s.x.row(text, row - text * (uint32_t)K);
  const int64_t base = (int64_t)part * kBeamSpan;
  const int there = (int)min((int64_t)kBeamSpan, s.V - base);  // logits of this part
  BeamLogits<E> x;
  x.load(p + base + lane * kBeamV, there);
  float top[kBeamPacks], best, most, sum;
  auto look = [&](auto careful) {  // maxima and the sum
    constexpr bool CAREFUL = decltype(careful)::value;
    const auto get = [&](int j, int k) { return CAREFUL ? x.sane(j, k) : x.get(j, k); };
    best = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < kBeamPacks; ++j) {
      top[j] = get(j, 0);
#pragma unroll
      for (int k = 1; k < kBeamV; ++k) top[j] = fmaxf(top[j], get(j, k));
      best = fmaxf(best, top[j]);
    }
    most = wave_max(best);
    x.anew();
    const float m = CAREFUL && most == -__builtin_inff() ? 0.0f : most, shift = m * kLog2e;
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kBeamPacks; ++j)
#pragma unroll
      for (int k = 0; k < kBeamV; ++k)
        sum += exp2_hw(CAREFUL ? (get(j, k) - m) * kLog2e : fmaf(get(j, k), kLog2e, -shift));
    sum = wave_sum(sum);
    // (what `shift` was rounded by is the same in every term)
    if constexpr (!CAREFUL) sum *= exp2_hw(-fmaf(m, kLog2e, -shift));
  };
  look(std::false_type());
  // A NaN, +inf, no logit above -inf, or a maximum that times log2(e) is beyond range
  // makes the sum a NaN or infinite.  (None of the others does: each term is about 1 at
  // most.)
  const bool odd = !(sum < __builtin_inff());
  x.anew();
  if (odd) {
    look(std::true_type());
    x.anew();
  }
  if (lane == 0) s.sums[(int64_t)row * s.parts + part] = make_float2(most, sum);

  // The K-th largest of the lanes' maxima (a lane without logits: the lowest), bit by
  // bit.  16-bit logits as fp32 have the lowest bits 0, or, ordered, of negative ones 1.
  constexpr int kFree = std::is_same_v<E, float> ? 0 : std::is_same_v<E, bf16_t> ? 16 : 13;
  const uint32_t mine = lane * kBeamV < there ? beam_order(best) : 0;
  const int lowest = odd ? 0 : kFree;
  uint32_t limit = 0;
  auto decide = [&](int bit) {
    const uint32_t more = limit | 1u << bit;
    if (__popcll(__ballot(mine >= more)) >= K) limit = more;
  };
#pragma unroll
  for (int bit = 31; bit >= kFree; --bit) decide(bit);
#pragma unroll 1
  for (int bit = kFree - 1; bit >= lowest; --bit) decide(bit);
  // Fewer than K lanes with logits: every logit counts.
  const bool every = limit == 0;
  if (!(limit >> 31)) limit |= (1u << lowest) - 1;
  const float border = every ? -__builtin_inff() : beam_value(limit);
  // The accesses with a logit above the limit, and the first K of those with one at it
  // (in which every logit that can count lies), in the order of the vocabulary.
  int packs = 0, ties = 0;
#pragma unroll
  for (int j = 0; j < kBeamPacks; ++j) {
    const int first = j * 64 * kBeamV + lane * kBeamV;
    const bool over = top[j] > border, at = top[j] == border && first < there;
    const uint64_t at_mask = __ballot(at);
    if (!(at_mask | __ballot(over))) continue;
    const bool take = over || (at && ties + lanes_below(at_mask) < K);
    const uint64_t mask = __ballot(take);
    if (take) {
      const int o = packs + lanes_below(mask);
      places[o] = first;
#pragma unroll
      for (int k = 0; k < kBeamV; k += 4)
        *reinterpret_cast<float4*>(hits + o * kBeamV + k) =
            make_float4(x.sane(j, k), x.sane(j, k + 1), x.sane(j, k + 2), x.sane(j, k + 3));
    }
    packs += __popcll(mask);
    ties += __popcll(at_mask);
  }
  auto settle = [] {  // a wave's own writes to LDS, before its reads by other lanes
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  settle();
  int n = 0, at_border = 0;
  for (int e = lane; e - lane < packs * kBeamV; e += 64) {
    const bool is = e < packs * kBeamV;
    const float v = is ? hits[e] : 0.0f;
    const int place = is ? places[e / kBeamV] + e % kBeamV : there;
    const bool over = place < there && v > border, at = place < there && v == border;
    const uint64_t over_mask = __ballot(over), at_mask = __ballot(at);
    const uint64_t key = beam_key(v, (uint32_t)(base + place));
    if (over) above[n + lanes_below(over_mask)] = key;
    if (at && at_border + lanes_below(at_mask) < K) level[at_border + lanes_below(at_mask)] = key;
    n += __popcll(over_mask);
    at_border += __popcll(at_mask);
  }
  settle();
  uint64_t* out = s.best + ((int64_t)row * s.parts + part) * K;
  for (int i = lane; i < n; i += 64) {
    const uint64_t key = above[i];
    int rank = 0;
    for (int o = 0; o < n; ++o) rank += above[o] > key;
    if (rank < K) out[rank] = key;
  }
  for (int i = lane; i < K - n; i += 64) out[n + i] = i < at_border ? level[i] : 0;
}

extern __shared__ __attribute__((aligned(16))) char beam_lds[];

template <typename E>
__global__ __launch_bounds__(64 * kBeamWaves) void beam_part(const BeamArgs<E> s, int64_t waves) {
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t id = seq_block() * (blockDim.x >> 6) + wave;
  if (id >= waves) return;
  const uint32_t row = (uint32_t)id / (uint32_t)s.parts;  // (waves are below 2^31)
  beam_look(s, row, (int)((uint32_t)id - row * (uint32_t)s.parts),
            beam_lds + wave * BeamLds(s.K).bytes);
}

// Takes the K best of `n` keys, no two alike but 0, in order: of the lane's, K times
// the best of the wave.  Written to list[0 .. K).  `hold`: the first HOLD keys of the
// lane, loaded.
template <int HOLD>
struct BeamHold {
  uint64_t key[HOLD];
  __device__ __forceinline__ void load(const uint64_t* keys, int64_t n, int64_t base, int lane) {
#pragma unroll
    for (int e = 0; e < HOLD; ++e) {
      const int64_t i = base + e * 64 + lane;
      key[e] = i < n ? keys[i] : 0;
    }
  }
};
template <int HOLD>
__device__ __forceinline__ void beam_take(BeamHold<HOLD> hold, const uint64_t* keys, int64_t n,
                                          int K, int lane, uint64_t* list) {
  uint64_t kept = 0;  // lane i: the i-th best so far
  for (int64_t base = 0;;) {
    uint64_t next = 0;
    for (int k = 0; k < K; ++k) {
      uint64_t best = kept;
#pragma unroll
      for (int e = 0; e < HOLD; ++e) best = hold.key[e] > best ? hold.key[e] : best;
      best = wave_max(best);
      if (best == 0) break;
      if (lane == k) next = best;
      if (kept == best) kept = 0;
#pragma unroll
      for (int e = 0; e < HOLD; ++e) hold.key[e] = hold.key[e] == best ? 0 : hold.key[e];
    }
    kept = next;
    base += 64 * HOLD;
    if (base >= n) break;
    hold.load(keys, n, base, lane);
  }
  if (lane < K) list[lane] = kept;
}

// Joins a text's rows.  (All waves of the workgroup call it.)
template <typename E>
__device__ __forceinline__ void beam_merge(const BeamArgs<E>& s, int64_t text) {
  __shared__ uint64_t list[kBeamMaxK][kBeamMaxK];
  // a row's maximum, and the logarithm of its sum relative to that (their sum would
  // lose the one in the other where logits are large)
  __shared__ double tops[kBeamMaxK], logs[kBeamMaxK];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = (int)blockDim.x >> 6, lane = threadIdx.x & 63, K = s.K;
  const int64_t keys = (int64_t)s.parts * K;
  for (int k = wave; k < K; k += waves) {
    const int64_t row = text * K + k;
    // (what a row that is skipped left there is not used: all loads set out together)
    const uint64_t* from = s.best + row * keys;
    BeamHold<2> hold;
    hold.load(from, keys, 0, lane);
    const float2* sums = s.sums + row * s.parts;
    const float2 one = lane < s.parts ? sums[lane] : make_float2(-__builtin_inff(), 0.0f);
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
    float most = one.x;
    for (int p = lane + 64; p < s.parts; p += 64) most = fmaxf(most, sums[p].x);
    most = wave_max(most);
    double sum = 0.0;
    if (most > -__builtin_inff()) {
      if (one.x > -__builtin_inff()) sum = (double)one.y * exp((double)one.x - (double)most);
      for (int p = lane + 64; p < s.parts; p += 64)
        if (sums[p].x > -__builtin_inff())
          sum += (double)sums[p].y * exp((double)sums[p].x - (double)most);
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) sum += __shfl_xor(sum, m);
    if (lane == 0) {
      tops[k] = (double)most;
      logs[k] = sum > 0.0 ? log(sum) : 0.0;
    }
    if (s.parts == 1) {  // (in order already)
      if (lane < K) list[k][lane] = hold.key[0];
    } else if (keys <= 128) {
      beam_take(hold, from, keys, K, lane, list[k]);
    } else {
      BeamHold<8> more;
      more.load(from, keys, 0, lane);
      beam_take(more, from, keys, K, lane, list[k]);
    }
  }
  __syncthreads();
  if (wave != 0) return;
  // Scores are compared in 64 bits, ordered as numbers; 0: the list is at its end.
  // (Scores are read before any is written: the outputs may be they.)
  const auto score_of = [&](int k, double from, uint64_t key) -> uint64_t {
    if (key == 0) return 0;
    const float x = beam_value((uint32_t)(key >> 32));
    double score = from + (((double)x - tops[k]) - logs[k]);
    if (!(x > -__builtin_inff()) || !(score > -__builtin_inf())) score = -__builtin_inf();
    const uint64_t u = __builtin_bit_cast(uint64_t, score + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
  };
  const auto write = [&](int r, int k, uint64_t key, uint64_t order, bool done) {
    const uint64_t u = order ^ ((uint64_t)((int64_t)~order >> 63) | 0x8000000000000000ull);
    const int64_t o = text * K + r, v = beam_place(key);
    s.out_scores[o] = (float)__builtin_bit_cast(double, u);
    s.parents[o] = k;
    s.tokens[o] = v;
    if (s.out_finished) s.out_finished[o] = done || v == s.eos;
  };
  const auto ends = [&](int k) { return s.finished && s.finished[text * K + k]; };
  // A continuation a lane, its place by how many come before it: 0.4 us faster than one
  // after the other with 4 beams, 0.6 slower with 8.
  if (K <= 4) {
    const int k = min(lane / K, K - 1);
    const uint64_t key = lane < K * K ? list[k][lane % K] : 0;
    const uint64_t mine = score_of(k, (double)s.scores[text * K + k], key);
    const bool done = ends(k);
    int rank = 0;
    for (int o = 0; o < K * K; ++o) {
      const uint64_t other =
          (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(mine >> 32), o) << 32 |
          (uint32_t)__builtin_amdgcn_readlane((int)mine, o);
      rank += other > mine || (other == mine && o < lane);
    }
    if (mine && rank < K) write(rank, k, key, mine, done);
    return;
  }
  // Lane k goes through row k's list.
  int taken = 0;
  const bool done = lane < K && ends(lane);
  const double from = lane < K ? (double)s.scores[text * K + lane] : 0.0;
  const auto head = [&] { return lane < K && taken < K ? list[lane][taken] : 0; };
  uint64_t key = head(), mine = score_of(lane, from, key);
  const auto next = [&] {
    ++taken;
    key = head();
    mine = score_of(lane, from, key);
  };
  for (int r = 0; r < K; ++r) {
    const uint64_t best = wave_max(mine);
    if (lane == __ffsll((unsigned long long)__ballot(mine == best)) - 1) {
      write(r, lane, key, best, done);
      next();
    }
  }
}

template <typename E>
__global__ __launch_bounds__(64 * kBeamJoinWaves) void beam_join(const BeamArgs<E> s) {
  const int64_t text = seq_block();
  if (text < s.B) beam_merge(s, text);
}

// Both for a text, where its rows are a wave each: with 4 beams of 28 logits 8.9 us
// against 10.5 in two launches, of 4096 (bf16) 8.0 against 9.7, 1024 texts of those 13.6
// against 16.5.  (Rows of several waves: 1024 x 4 x 16384 49 us against 35.)
template <typename E>
__global__ __launch_bounds__(64 * kBeamJoinWaves) void beam_whole(const BeamArgs<E> s) {
  const int64_t text = seq_block();
  if (text >= s.B) return;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  beam_look(s, (uint32_t)text * s.K + (uint32_t)(wave / s.parts), wave % s.parts,
            beam_lds + wave * BeamLds(s.K).bytes);
  __syncthreads();
  beam_merge(s, text);
}

// ------------------------------------------------------------------ reordering

constexpr int kMoveThreads = 256;
constexpr int kMoveTable = 32;  // states a launch

struct MoveState {
  const char* in;
  char* out;
  int64_t in_row, in_seg, out_row, out_seg;  // bytes
  int64_t bytes;                             // adjacent ones of a segment
  int64_t first;                             // first workgroup
  int64_t blocks;                            // workgroups a text
  uint32_t packs, segs;                      // of a segment; of a row
};
struct MoveTable {
  MoveState s[kMoveTable];
  const int64_t* parents;
  int64_t first;  // one behind the last workgroup
  int count, B;
};

// N bytes at any address as one access.
template <int N> struct MoveBytes;
template <> struct MoveBytes<16> {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(1)));
};
template <> struct MoveBytes<8> {
  typedef uint32_t type __attribute__((ext_vector_type(2), aligned(1)));
};
template <> struct MoveBytes<4> { typedef uint32_t type __attribute__((aligned(1))); };
template <> struct MoveBytes<2> { typedef uint16_t type __attribute__((aligned(1))); };
template <> struct MoveBytes<1> { typedef uint8_t type; };

// HBM bounds it: 64 x 8 beams of 172 KB each, four states: 31 us (5.7 TB/s; parents that
// are taken twice come from a cache), 22 where the last-level cache has them.
// One pack of all of a text's rows: every row is read before any is written, so that
// a state may be reordered in place.  parent: lane k's is row k's.
template <int N, int K>
__device__ __forceinline__ void move_pack(const MoveState& s, int parent, const char* in,
                                          char* out) {
  using T = typename MoveBytes<N>::type;
  T v[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
    v[k] = *reinterpret_cast<const T*>(in + __builtin_amdgcn_readlane(parent, k) * s.in_row);
#pragma unroll
  for (int k = 0; k < K; ++k) *reinterpret_cast<T*>(out + k * s.out_row) = v[k];
}

// K beams a text: known to the compiler, so that the rows of a pack stay in registers.
template <int N, int K>
__global__ __launch_bounds__(kMoveThreads) void move_rows(const MoveTable t) {
  const int64_t block = seq_block();
  if (block >= t.first) return;
  int i = 0;
  while (i + 1 < t.count && t.s[i + 1].first <= block) ++i;
  const MoveState& s = t.s[i];
  // (both fit 32 bits: workgroups of a state, and packs of a row)
  const uint32_t of = (uint32_t)(block - s.first), blocks = (uint32_t)s.blocks;
  const uint32_t text = of / blocks, item = of % blocks * kMoveThreads + threadIdx.x;
  const int lane = threadIdx.x & 63;
  int parent = 0;
  if (lane < K)
    parent = (int)min(max(t.parents[(int64_t)text * K + lane], (int64_t)0), (int64_t)K - 1);
  const uint32_t seg = item / s.packs;
  const int64_t at = (int64_t)(item - seg * s.packs) * N;
  if (seg >= s.segs) return;
  const char* in = s.in + (int64_t)text * K * s.in_row + (int64_t)seg * s.in_seg + at;
  char* out = s.out + (int64_t)text * K * s.out_row + (int64_t)seg * s.out_seg + at;
  const int left = (int)min(s.bytes - at, (int64_t)N);
  if (left == N) return move_pack<N, K>(s, parent, in, out);
  int o = 0;  // a row's last bytes
#pragma unroll 1
  for (; o + 4 <= left; o += 4) move_pack<4, K>(s, parent, in + o, out + o);
#pragma unroll 1
  for (; o < left; ++o) move_pack<1, K>(s, parent, in + o, out + o);
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
  if (s->B * s->K * ((s->V + kBeamSpan - 1) / kBeamSpan) >= INT_MAX) {
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

// What is written must not lie over anything else of a call, but new scores and ends over
// the old ones.
ck_status beam_check_apart(const ck_beam_shape& s, const ck_seq& logits, const float* scores,
                           const uint8_t* finished, const float* out_scores,
                           const int64_t* parents, const int64_t* tokens,
                           const uint8_t* out_finished, const void* workspace, size_t ws_bytes) {
  struct Span {
    const char* name;
    uintptr_t at;
    size_t bytes;
  };
  const size_t n = (size_t)(s.B * s.K);
  const auto span = [](const char* name, const void* p, size_t bytes) {
    return Span{name, reinterpret_cast<uintptr_t>(p), p ? bytes : 0};
  };
  const Span v[] = {span("out_scores", out_scores, 4 * n), span("parents", parents, 8 * n),
                    span("tokens", tokens, 8 * n), span("out_finished", out_finished, n),
                    span("the workspace", workspace, ws_bytes), span("scores", scores, 4 * n),
                    span("finished", finished, n)};
  constexpr int kWritten = 5, kAll = 7;
  const int64_t e = (int64_t)seq_elem_bytes(s.dtype);
  Pieces x = range_of(logits.data, (size_t)(s.V * e));
  const int64_t far = int64_t(1) << 60;  // (nothing lies further apart)
  x.n0 = s.B, x.s0 = s.B > 1 ? std::min(logits.stride_t, far) * e : 0;
  x.n1 = s.K, x.s1 = s.K > 1 ? std::min(logits.stride_b, far) * e : 0;
  const __int128 end = x.end();
  for (int k = 0; k < kWritten; ++k) {
    const Span& w = v[k];
    if (!w.bytes) continue;
    const char* over = nullptr;
    for (int o = k + 1; o < kAll; ++o)
      if (w.at < v[o].at + v[o].bytes && v[o].at < w.at + w.bytes &&
          !(w.at == v[o].at && ((k == 0 && o == 5) || (k == 3 && o == 6))))
        over = v[o].name;
    if (w.at < end && x.at < w.at + w.bytes &&
        pieces_meet(x, range_of(reinterpret_cast<const void*>(w.at), w.bytes)))
      over = "logits";
    if (over) {
      set_error("%s must not lie over %s", w.name, over);
      return CK_ERR_BAD_VALUE;
    }
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

// What is written must not lie over anything else of a call, but a state's output over
// the state itself.  Tensors are looked at in the order of their addresses, so that only
// those are compared whose ranges cross: of many states, slices of one tensor, which lie
// side by side in its rows.
ck_status move_check_apart(const ck_beam_state* states, int64_t count, const int64_t* parents,
                           int64_t rows) {
  struct Span {
    Slice at;
    int64_t state;  // -1: the parents
    int written;    // 0 or 1
    int pieces;     // which
  };
  std::vector<Span> v;
  std::vector<Pieces> pieces;
  v.reserve(2 * count + 1), pieces.reserve(2 * count + 1);
  const auto add = [&](const Pieces& p, int64_t state, int written) {
    v.push_back(Span{slice_of(p), state, written, (int)pieces.size()});
    pieces.push_back(p);
  };
  add(range_of(parents, (size_t)rows * sizeof(int64_t)), -1, 0);
  for (int64_t i = 0; i < count; ++i) {
    const ck_beam_state& s = states[i];
    if (s.segments == 0 || s.bytes == 0) continue;
    Pieces p = range_of(s.out, (size_t)s.bytes);
    p.n0 = rows, p.s0 = s.out_row, p.n1 = s.segments, p.s1 = s.out_segment;
    add(p, i, 1);
    if (s.in == s.out) continue;
    p.at = reinterpret_cast<uintptr_t>(s.in), p.s0 = s.in_row, p.s1 = s.in_segment;
    add(p, i, 0);
  }
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.at.at < b.at.at; });
  for (size_t i = 0; i < v.size(); ++i)
    for (size_t o = i + 1; o < v.size() && v[o].at.at < v[i].at.end; ++o) {
      const Span &a = v[i], &b = v[o];
      if (side_by_side(a.at, b.at) || !(a.written | b.written) ||
          !pieces_meet(pieces[a.pieces], pieces[b.pieces]))
        continue;
      const int64_t first = std::min(a.state, b.state), last = std::max(a.state, b.state);
      if (first < 0) set_error("state %lld: its output lies over the parents", (long long)last);
      else if (first == last) set_error("state %lld: its output lies over it", (long long)last);
      else
        set_error("states %lld and %lld share memory that is written", (long long)first,
                  (long long)last);
      return CK_ERR_BAD_VALUE;
    }
  return CK_OK;
}

template <int K>
void move_launch(MoveTable& t, hipStream_t stream) {
  // a thread holds at most 128 bytes: packs of 16, of 8 or of 4 for more rows
  constexpr int N = K <= 8 ? 16 : K <= 16 ? 8 : 4;
  t.first = 0;
  for (int i = 0; i < t.count; ++i) {
    MoveState& s = t.s[i];
    s.packs = (uint32_t)((s.bytes + N - 1) / N);
    s.blocks = ((int64_t)s.packs * s.segs + kMoveThreads - 1) / kMoveThreads;
    s.first = t.first;
    t.first += s.blocks * t.B;
  }
  move_rows<N, K><<<seq_grid(t.first), kMoveThreads, 0, stream>>>(t);
}
template <int K>
void move_by_beams(int64_t k, MoveTable& t, hipStream_t stream) {
  if (k == K) return move_launch<K>(t, stream);
  if constexpr (K > 1) move_by_beams<K - 1>(k, t, stream);
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
  if (rc == CK_OK)
    rc = beam_check_apart(*shape, logits, scores, finished, out_scores, parents, tokens,
                          out_finished, workspace, ws.total);
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
    const int64_t each = shape->K * ws.parts, waves = shape->B * each;
    const size_t one = BeamLds((int)shape->K).bytes;
    if (ws.parts == 1 && each <= kBeamJoinWaves && each * one <= kBeamWholeLds &&
        shape->B < kSeqGridX / 4) {
      beam_whole<E><<<seq_grid(shape->B), 64 * (int)each, each * one, stream>>>(a);
      CK_HIP_TRY(hipGetLastError());
      return CK_OK;
    }
    // (at most 52.4 KB of LDS: 32 beams; 50.8 with 16)
    const int per = shape->K > 16 ? kBeamWaves / 2 : kBeamWaves;
    beam_part<E><<<seq_grid((waves + per - 1) / per), 64 * per, per * one, stream>>>(a, waves);
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
  const int64_t most = int64_t(1) << 39;  // bytes of a beam of all texts; of a row below 2^32
  for (int64_t i = 0; i < count; ++i) {
    const ck_beam_state& s = states[i];
    if (s.segments < 0 || s.bytes < 0) {
      set_error("state %lld: bad sizes", (long long)i);
      return CK_ERR_BAD_SIZE;
    }
    if (s.segments == 0 || s.bytes == 0) continue;
    if (s.segments > (int64_t)UINT32_MAX / s.bytes || s.segments * s.bytes > most / B) {
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
  }
  try {
    const ck_status rc = move_check_apart(states, count, parents, B * K);
    if (rc != CK_OK) return rc;
  } catch (const std::bad_alloc&) {
    set_error("out of host memory");
    return CK_ERR_NOMEM;
  }
  MoveTable t = {};
  t.parents = parents;
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
      m.segs = (uint32_t)s.segments;
    }
    if (t.count == 0) break;
    move_by_beams<kBeamMaxK>(K, t, stream);
    CK_HIP_TRY(hipGetLastError());
  }
  return CK_OK;
}
