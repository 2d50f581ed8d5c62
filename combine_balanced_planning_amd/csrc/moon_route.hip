// moon_route.hip — top-k routing with per-expert counts and a balance loss,
// and its gradient.
//
// For a token with logits x over E experts: scores s = softmax(x) or
// 1/(1+e^-x), selection key = x (or s + bias with a selection bias), the K
// largest keys in descending order, the lowest id among equal keys, weights
// w_k = scale * s[id_k] (/ sum over k).  With p = s / sum(s), P[e] = sum over a
// rank's valid tokens of p[e], C[e] = their routes to e and n their number,
//   loss = coef * E / (K n^2) * sum_e C[e] P[e]
// (C is a count and carries no gradient).  The gradient with G = dL/ds is
//   softmax: dx = s (G + b - sum_j s_j (G_j + b_j)),
//   sigmoid: dx = s (1 - s) (G + (b - sum_j p_j b_j) / sum(s)),
// b[e] = dloss * coef * E / (K n^2) * C[e], G[id_k] = scale * dw_k, or with
// renormalised weights scale / N * (dw_k - sum_j dw_j s_j / N), N = sum_k s.
//
// One wave per token, lane l holds experts l, l + 64, ...: the logits are
// read once, coalesced, and everything else stays in registers.  The K-th
// largest of the lanes' maxima bounds the K-th largest value from below; bisection
// of its bits with a ballot a round finds it.  The values that reach it, K and a
// few more, are packed into lanes and ranked by comparing all pairs.  All but
// the maxima and the picks are compared as the numbers they are (an integer key
// for every expert takes a third more vector instructions).
// Sums over tokens are kept per wave in registers, then per workgroup in LDS,
// then per workgroup in the workspace, and added in a fixed order at each step,
// so results repeat bit for bit.
#include <algorithm>

#include "moon_rows.h"

namespace moon {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopk = 64;
enum { kSoftmax, kSigmoid, kBiased };

struct RouteArgs {
  const void* logits;
  const float* bias;
  const uint8_t* valid;
  int32_t* topk;
  float* weights;
  int32_t *counts, *tokens;
  float *psum, *loss;
  float* part_p;    // [R][nblk][E]
  int32_t* part_c;  // [R][nblk][E]
  int32_t* part_n;  // [R][nblk]
  int32_t R, S, E, K, nblk;
  int32_t sigmoid, renorm, stats, sums;
  float scale, coef;
};

struct RouteGradArgs {
  const void* logits;
  const uint8_t* valid;
  const int32_t* topk;
  const float* d_weights;
  const int32_t *counts, *tokens;
  const float* d_loss;
  void* d_logits;
  int32_t R, S, E, K;
  int32_t sigmoid, renorm;
  float scale, coef;
};

// A float's bits as an unsigned key of the same order: -0 equal to +0, NaN
// below every number, 0 left over for "no candidate".
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return x != x ? 1u : k;
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// Scores up to a common factor: a score is off by |x - shift| 2^-23 and the
// units of v_exp_f32 and v_rcp_f32.  (The shift is taken off first: its product
// with log2(e) would overflow, or drown the difference, for large logits.)
constexpr float kLog2e = 1.44269504088896341f;
__device__ __forceinline__ float exp_shifted(float x, float shift) {
  return __builtin_amdgcn_exp2f((x - shift) * kLog2e);
}
__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2e));
}

// Keys of a wave that are at least t.
template <int J>
__device__ __forceinline__ int count_at_least(const uint32_t (&key)[J], uint32_t t) {
  int n = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) n += __popcll(__ballot(key[j] >= t));
  return n;
}

// `first` plus the lanes of the ballot below this one.
__device__ __forceinline__ int lanes_before(uint64_t ballot, int first = 0) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(ballot >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)ballot, first));
}

// A key and its expert as one number: larger keys first, then lower ids.
__device__ __forceinline__ uint64_t pick_of(uint32_t key, int id) {
  return (uint64_t)key << 32 | (uint32_t)~id;
}
__device__ __forceinline__ uint32_t pick_key(uint64_t p) { return (uint32_t)(p >> 32); }
__device__ __forceinline__ int pick_id(uint64_t p) { return (int)~(uint32_t)p; }

__device__ __forceinline__ float read_lane(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* base, int64_t i) {
  if (BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[i] << 16);
  return static_cast<const float*>(base)[i];
}

// Takes the largest two-word key out of the wave; returns its expert, or -1
// when no candidate is left.  Among equal keys the lowest id wins: word j holds
// ids j*64 .. j*64 + 63 by lane.
template <int J>
__device__ __forceinline__ int take_largest(uint32_t (&hi)[J], const uint32_t (&lo)[J], int lane) {
  uint32_t m = hi[0];
#pragma unroll
  for (int j = 1; j < J; ++j) m = max(m, hi[j]);
  const uint32_t top = wave_max_u32(m);
  if (top == 0) return -1;
  uint32_t l = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) l = max(l, hi[j] == top ? lo[j] : 0u);
  const uint32_t low = wave_max_u32(l);
  int id = -1;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (id < 0) {
      const uint64_t b = __ballot(hi[j] == top && lo[j] == low);
      if (b != 0) {
        const int win = __builtin_ctzll(b);
        id = j * kLanes + win;
        if (lane == win) hi[j] = 0;
      }
    }
  }
  return id;
}

// Selection by score + bias in 64 bits; lane k returns the k-th id.
template <int J, bool BF16>
__device__ __attribute__((noinline)) int select_wide(const void* logits, int64_t at,
                                                     const float* bias, int E, int K, int lane) {
  uint32_t hi[J], lo[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = j * kLanes + lane;
    hi[j] = lo[j] = 0;
    if (e < E) {
      const float x = load_logit<BF16>(logits, at + e);
      double v = 1.0 / (1.0 + exp(-(double)x)) + (double)bias[e] + 0.0;
      if (x == -INFINITY) v = -INFINITY;
      const uint64_t b = (uint64_t)__double_as_longlong(v);
      const uint64_t k = (b >> 63) != 0 ? ~b : (b | (1ull << 63));
      hi[j] = v != v ? 1u : (uint32_t)(k >> 32);
      lo[j] = v != v ? 0u : (uint32_t)k;
    }
  }
  int mine = 0;
  for (int k = 0; k < K; ++k) {
    const int id = take_largest(hi, lo, lane);
    if (lane == k) mine = id;
  }
  return mine;
}

__device__ __forceinline__ float reciprocal_or_zero(float v) {
  return v > 0.0f ? 1.0f / v : (v == 0.0f ? 0.0f : v);  // NaN stays
}

// Writes a rank's counts, probability sums, valid tokens and loss.  Called by
// a whole workgroup; per(e, &p, &c) gives expert e's sums.
template <class Per>
__device__ __forceinline__ void finish_rank(const RouteArgs& a, int r, int n, float* red,
                                            const Per& per) {
  float part = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float p;
    int32_t c;
    per(e, &p, &c);
    part += p * (float)c;
    if (a.psum != nullptr) a.psum[r * a.E + e] = p;
    // tokens outside the batch count as K routes to expert 0, as their ids say
    if (a.counts != nullptr) a.counts[r * a.E + e] = c + (e == 0 ? a.K * (a.S - n) : 0);
  }
  if (a.tokens != nullptr && threadIdx.x == 0) a.tokens[r] = n;
  if (a.loss != nullptr) {
    const float ws = wave_sum(part);
    __syncthreads();
    if ((threadIdx.x & (kLanes - 1)) == 0) red[threadIdx.x / kLanes] = ws;
    __syncthreads();
    if (threadIdx.x == 0) {
      float sum = 0.0f;
      for (int i = 0; i < (int)blockDim.x / kLanes; ++i) sum += red[i];
      a.loss[r] = n > 0 ? a.coef * (float)a.E / ((float)a.K * (float)n) * (sum / (float)n) : 0.0f;
    }
  }
}

// The kernel's arguments, read again: what only the end of k_route needs would
// else sit in scalar registers through its loop and push others out (147
// against 145 us a training step at R=16, S=8192, E=384, softmax; the biased
// kernel, which spills vector registers, takes 227 and would take 222 without).
__device__ __forceinline__ RouteArgs late_args() {
  const __attribute__((address_space(4))) RouteArgs* p =
      (const __attribute__((address_space(4))) RouteArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  RouteArgs a;
  a.counts = p->counts;
  a.tokens = p->tokens;
  a.psum = p->psum;
  a.loss = p->loss;
  a.part_p = p->part_p;
  a.part_c = p->part_c;
  a.part_n = p->part_n;
  a.S = p->S;
  a.E = p->E;
  a.K = p->K;
  a.nblk = p->nblk;
  a.coef = p->coef;
  return a;
}

// Held to 64 registers for eight waves a SIMD: a token is a chain of dependent
// steps, and more waves hide it.  What selects, whether sums over tokens (or a
// token's sum of scores) are wanted and whether the words are full are template
// arguments: told at run time they cost branches and spilled scalars.
// At R=16, S=8192, E=384, fp32, softmax with sums the kernel takes 64 to 72
// us, the vector unit busy 72 % of the shorter with 221 vector and 159 scalar instructions a
// token; the logits alone take 41 us to read.  With four waves a SIMD a training
// step there takes 158 us against 145, a prefill at R=8, S=4096, E=256 with a
// bias 28.4 against 24.8.  The biased kernels with sums are the exception: they
// need more than 64 registers (15 spilled at E=256, 25 at E=384, 42 at E=512)
// and a training step takes 227 us at E=384 and 54 at E=256, with four waves
// 159 and 49.
template <int J, bool BF16, int Score, bool Sums, bool Whole>
__global__ void __launch_bounds__(kMaxWaves* kLanes) __attribute__((amdgpu_waves_per_eu(8)))
    k_route(RouteArgs a) {
  constexpr bool biased = Score == kBiased, sigmoid = Score != kSoftmax;
  const int E = Whole ? J * kLanes : a.E;  // Whole: the words are full
  extern __shared__ float lds[];  // [waves][64] picks; biased: [waves][64] their scores;
                                  // with stats also [E] counts, [waves] tokens,
                                  // [waves]; with Sums [waves][E] sums
  const int lane = threadIdx.x & (kLanes - 1);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int waves = blockDim.x / kLanes;
  const int r = blockIdx.y, blk = blockIdx.x;
  uint64_t* const picks = reinterpret_cast<uint64_t*>(lds) + w * kLanes;
  float* const scores = lds + 2 * waves * kLanes + w * kLanes;
  int32_t* const red_c = reinterpret_cast<int32_t*>(lds + (biased ? 3 : 2) * waves * kLanes);
  int32_t* const red_n = red_c + E;
  float* const red_l = reinterpret_cast<float*>(red_n + waves);
  float* const red_p = red_l + waves;
  if (a.stats) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) red_c[e] = 0;
    __syncthreads();
  }
  float acc[J], bias[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = j * kLanes + lane;
    acc[j] = 0.0f;
    bias[j] = biased && e < E ? a.bias[e] : 0.0f;
  }
  int32_t n_valid = 0;
  // The next token's logits are on their way while one is worked on.
  const uint32_t step = a.nblk * waves, tokens = a.S;  // a sum of the two fits
  float ahead[J];
  uint32_t ahead_ok = 1;
  const auto fetch = [&](uint32_t t) {
    const int64_t tok = (int64_t)r * a.S + t;
    if (a.valid != nullptr) ahead_ok = a.valid[tok];
    const void* const row = static_cast<const char*>(a.logits) + tok * E * (BF16 ? 2 : 4);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t e = j * kLanes + lane;
      ahead[j] = load_logit<BF16>(row, Whole ? e : min(e, (uint32_t)E - 1));
    }
  };
  const uint32_t begin = blk * waves + w;
  if (begin < tokens) fetch(begin);
  for (uint32_t t = begin; t < tokens; t += step) {
    const int64_t tok = (int64_t)r * a.S + t;
    const int64_t at = tok * E;
    const int ok = __builtin_amdgcn_readfirstlane((int)ahead_ok);
    // v: what is selected by, NaN where there is no expert; s: the scores.
    float s[J], v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      s[j] = ahead[j];
      v[j] = j * kLanes + lane < E ? s[j] : NAN;
    }
    if (t + step < tokens) fetch(t + step);
    if (ok == 0) {
      if (lane < a.K) {
        a.topk[tok * a.K + lane] = 0;
        a.weights[tok * a.K + lane] = 0.0f;
      }
      continue;
    }
    ++n_valid;
    if (sigmoid && (biased || Sums)) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float x = v[j];
        s[j] = logistic(s[j]);
        if (biased) v[j] = x > -INFINITY ? s[j] + bias[j] : x;
      }
    }
    // (made quiet first: the three-way maximum would return a signalling NaN)
    float best = __builtin_canonicalizef(v[0]);
#pragma unroll
    for (int j = 1; j < J; ++j) best = fmaxf(best, __builtin_canonicalizef(v[j]));
    const uint32_t mine = lane < E ? order_key(best) : 0u;
    const uint32_t top = wave_max_u32(mine);
    // At least K of the lanes' maxima are >= lo (min(E, 64) lanes have one),
    // fewer than K are >= hi.
    uint32_t lo = wave_min_u32(mine == 0u ? ~0u : mine), hi = top + 1u;
    float shift = 0.0f, total = 0.0f;
    if (!sigmoid) {
      // Nothing but masked experts or NaN: scores 0 (NaN) with no shift.
      const float m = key_value(top);
      shift = top == 1u || m == -INFINITY ? 0.0f : m;
    }
    if (Sums) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (!sigmoid) s[j] = exp_shifted(s[j], shift);
        if (j * kLanes + lane >= E) s[j] = 0.0f;
        total += s[j];
      }
      total = wave_sum(total);
    }
    // A few maxima too many cost less than the rounds that would tell them.
    const int enough = a.K + (a.K >> 1);
    while (hi - lo > 1u) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const int n = __popcll(__ballot(mine >= mid));
      const bool many = n >= a.K;
      lo = many ? mid : lo;
      // (hi = lo ends it)
      hi = many ? (n <= enough ? mid : hi) : mid;
    }
    // Comparisons of numbers from here: NaN takes no part, so a row that needs
    // one finds fewer than K.
    const float least = key_value(lo);
    uint64_t in[J];
    int first[J], found = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      in[j] = __ballot(v[j] >= least);
      first[j] = found;
      found += __popcll(in[j]);
    }
    const bool plain = found >= a.K && found <= kLanes;
    if (plain) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (v[j] >= least) {
          const int i = lanes_before(in[j], first[j]);
          picks[i] = (uint64_t)__float_as_uint(v[j]) << 32 | (uint32_t)~(j * kLanes + lane);
          if (biased) scores[i] = s[j];
        }
      }
    } else {
      // Too many for the lanes (large K, long runs of equal keys) or NaN: on by
      // all keys, and of those equal at the end the first ones, as many as
      // there is room for.
      uint32_t key[J];
#pragma unroll
      for (int j = 0; j < J; ++j) key[j] = j * kLanes + lane < E ? order_key(v[j]) : 0u;
      hi = top + 1u;
      while (hi - lo > 1u) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (count_at_least(key, mid) >= a.K)
          lo = mid;
        else
          hi = mid;
      }
      found = a.K;
      const int room = a.K - count_at_least(key, lo + 1u);
      int ties = 0, at_pick = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint64_t eq = __ballot(key[j] == lo);
        const bool take = key[j] > lo || (key[j] == lo && lanes_before(eq, ties) < room);
        const uint64_t b = __ballot(take);
        if (take)
          picks[lanes_before(b, at_pick)] =
              (uint64_t)__float_as_uint(v[j]) << 32 | (uint32_t)~(j * kLanes + lane);
        at_pick += __popcll(b);
        ties += __popcll(eq);
      }
    }
    found = __builtin_amdgcn_readfirstlane(found);
    wave_lds_sync();
    uint64_t p = picks[lane];  // whatever was there behind the last
    const float mine_v = __uint_as_float(pick_key(p));
    p = (uint64_t)order_key(mine_v) << 32 | (uint32_t)p;
    picks[lane] = lane < found ? p : 0;  // nothing is ranked behind zeros
    wave_lds_sync();
    int rank = lane < found ? 0 : kLanes;
#pragma unroll 1
    for (int k = 0; k < found; k += 4) {
      uint64_t other[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) other[i] = picks[k + i];
#pragma unroll
      for (int i = 0; i < 4; ++i) rank += other[i] > p ? 1 : 0;
    }
    wave_lds_sync();
    int id = pick_id(p);
    float sel;
    if (biased) {
      // A score in 32 bits plus its bias is off by a few units in the last
      // place, below 5e-7 * max(1, |sum|): neighbours nearer than twice that
      // are told apart in 64 bits.  Only pairs of neighbours need a look, and
      // the largest that was not picked only if nothing between is picked.
      const float near = 1e-6f * fmaxf(1.0f, fabsf(mine_v));
      float* const by_rank = reinterpret_cast<float*>(picks);
      if (rank < found) by_rank[rank] = mine_v;
      wave_lds_sync();
      const float below = by_rank[min(rank, found - 2) + 1];
      sel = scores[lane];
      wave_lds_sync();
      bool close = !plain || (rank < a.K && rank + 1 < found && mine_v - below <= near);
      if (found == a.K) {
        float next = -INFINITY;
#pragma unroll
        for (int j = 0; j < J; ++j) next = fmaxf(next, v[j] < least ? v[j] : -INFINITY);
        const float left = key_value(wave_max_u32(order_key(next)));
        close = close || least - left <= 1e-6f * fmaxf(1.0f, fabsf(least));
      }
      if (__ballot(close) != 0) {
        id = select_wide<J, BF16>(a.logits, at, a.bias, E, a.K, lane);
        rank = lane;
        sel = lane < a.K ? logistic(load_logit<BF16>(a.logits, at + id)) : 0.0f;
      }
      if (rank >= a.K) sel = 0.0f;
    } else {
      sel = rank < a.K ? (sigmoid ? logistic(mine_v) : exp_shifted(mine_v, shift)) : 0.0f;
    }
    // One division for both: by the picks' sum in lane 0, by all scores' in lane 1.
    float out = a.scale, inv = 0.0f;
    if (Sums || a.renorm) {
      const float picked = a.renorm ? wave_sum(sel) : 0.0f;
      const float q = reciprocal_or_zero(lane == 0 ? picked : total);
      inv = read_lane(q, 1);
      out *= a.renorm ? sel * read_lane(q, 0) : sigmoid ? sel : sel * inv;
    } else {
      out *= sel;
    }
    if (rank < a.K) {
      int32_t* const ids = a.topk + tok * a.K;
      float* const weights = a.weights + tok * a.K;
      ids[(uint32_t)rank] = id;
      weights[(uint32_t)rank] = out;
      if (a.stats) atomicAdd(&red_c[id], 1);  // whole numbers: any order
    }
    if (Sums) {
#pragma unroll
      for (int j = 0; j < J; ++j) acc[j] = fmaf(s[j], inv, acc[j]);
    }
  }
  if (!a.stats) return;
  const RouteArgs late = late_args();
  if (Sums) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = j * kLanes + lane;
      if (e < E) red_p[w * E + e] = acc[j];
    }
  }
  if (lane == 0) red_n[w] = n_valid;
  __syncthreads();
  int32_t n = 0;
  for (int i = 0; i < waves; ++i) n += red_n[i];
  const auto per = [&](int e, float* p, int32_t* c) {
    float sum = 0.0f;
    if (Sums)
      for (int i = 0; i < waves; ++i) sum += red_p[i * E + e];
    *p = sum;
    *c = red_c[e];
  };
  if (late.nblk == 1) {
    finish_rank(late, r, n, red_l, per);
    return;
  }
  const int64_t row = (int64_t)r * late.nblk + blk;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float p;
    per(e, &p, &late.part_c[row * E + e]);
    if (Sums) late.part_p[row * E + e] = p;
  }
  if (threadIdx.x == 0) late.part_n[row] = n;
}

// Adds the workgroups' sums of a rank: 1024 threads, as many to an expert as
// there are, each a fixed share of the partial sums.
template <bool Sums>
__global__ void __launch_bounds__(1024) k_route_finish(RouteArgs a, int experts) {
  __shared__ float red[1024 / kLanes];
  __shared__ float part_p[1024];
  __shared__ int32_t part_c[1024];
  __shared__ int32_t tokens;
  const int r = blockIdx.x;
  const int64_t row = (int64_t)r * a.nblk;
  const int e = threadIdx.x % experts, share = threadIdx.x / experts, shares = 1024 / experts;
  if (threadIdx.x == 0) tokens = 0;
  __syncthreads();
  int32_t n = 0;
  for (int i = threadIdx.x; i < a.nblk; i += 1024) n += a.part_n[row + i];
  if (n != 0) atomicAdd(&tokens, n);  // whole numbers: any order
  float sum = 0.0f;
  int32_t cnt = 0;
  if (e < a.E) {
#pragma unroll 16
    for (int i = share; i < a.nblk; i += shares) {
      if (Sums) sum += a.part_p[(row + i) * a.E + e];
      cnt += a.part_c[(row + i) * a.E + e];
    }
  }
  part_p[threadIdx.x] = sum;
  part_c[threadIdx.x] = cnt;
  __syncthreads();
  finish_rank(a, r, tokens, red, [&](int x, float* p, int32_t* c) {
    *p = 0.0f;
    *c = 0;
    for (int i = 0; i < shares; ++i) {
      *p += part_p[i * experts + x];
      *c += part_c[i * experts + x];
    }
  });
}

// HBM bounds it: the logits once and their gradient once, 0.4 GB at R=16,
// S=8192, E=384, fp32 in 75 us (5.4 TB/s).  8192 workgroups at most: with the
// forward before it a step takes 145 us, with 4096 the same within 1 us, with
// 16384, set up too often, 153.
template <int J, bool BF16>
__global__ void __launch_bounds__(256) k_route_grad(RouteGradArgs a, int nblk) {
  __shared__ float lds[4][J * kLanes];  // a wave's experts, by id
  const int lane = threadIdx.x & (kLanes - 1);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int r = blockIdx.y;
  float b[J];
  {
    float base = 0.0f;
    if (a.d_loss != nullptr) {
      const float n = (float)a.tokens[r];
      if (n > 0.0f) base = a.d_loss[r] * (a.coef * (float)a.E / ((float)a.K * n) / n);
    }
    const int32_t pads = a.d_loss != nullptr ? a.K * (a.S - a.tokens[r]) : 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = j * kLanes + lane;
      b[j] = a.d_loss != nullptr && e < a.E
                 ? base * (float)(a.counts[r * a.E + e] - (e == 0 ? pads : 0)) : 0.0f;
    }
  }
  // The next token's logits, ids and weight gradients are on their way while
  // one is worked on.
  const uint32_t step = nblk * 4, tokens = a.S;  // a sum of the two fits
  float ahead[J], ahead_dw = 0.0f;
  int32_t ahead_id = -1;
  uint32_t ahead_ok = 1;
  const auto fetch = [&](uint32_t t) {
    const int64_t tok = (int64_t)r * a.S + t;
    if (a.valid != nullptr) ahead_ok = a.valid[tok];
#pragma unroll
    for (int j = 0; j < J; ++j)
      ahead[j] = load_logit<BF16>(a.logits, tok * a.E + min(j * kLanes + lane, a.E - 1));
    if (a.d_weights != nullptr && lane < a.K) {
      ahead_id = a.topk[tok * a.K + lane];
      ahead_dw = a.d_weights[tok * a.K + lane];
    }
  };
  const uint32_t begin = blockIdx.x * 4 + w;
  if (begin < tokens) fetch(begin);
  for (uint32_t t = begin; t < tokens; t += step) {
    const int64_t at = ((int64_t)r * a.S + t) * a.E;
    const int ok = __builtin_amdgcn_readfirstlane((int)ahead_ok);
    float d[J], x[J];
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] = j * kLanes + lane < a.E ? ahead[j] : -INFINITY;
    const int id = ahead_id;
    const bool picked = id >= 0 && id < a.E;
    const float dw = picked ? ahead_dw : 0.0f;
    if (t + step < tokens) fetch(t + step);
    if (ok == 0) {
#pragma unroll
      for (int j = 0; j < J; ++j) d[j] = 0.0f;
    } else {
      float s[J], shift = 0.0f;
      if (!a.sigmoid) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const uint32_t k = order_key(x[j]);
          m = max(m, j * kLanes + lane < a.E ? k : 0u);
        }
        m = wave_max_u32(m);
        const float top = key_value(m);
        shift = m == 1u || top == -INFINITY ? 0.0f : top;
      }
      float total = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        s[j] = a.sigmoid ? logistic(x[j]) : exp_shifted(x[j], shift);
        total += s[j];
      }
      total = wave_sum(total);
      const float inv = reciprocal_or_zero(total);
      if (a.d_weights != nullptr) {
        // scores by id, then the gradients that go to them
        float* const at_id = lds[w];
#pragma unroll
        for (int j = 0; j < J; ++j) at_id[j * kLanes + lane] = s[j];
        wave_lds_sync();
        const float sel = picked ? at_id[id] : 0.0f;
        wave_lds_sync();
#pragma unroll
        for (int j = 0; j < J; ++j) at_id[j * kLanes + lane] = 0.0f;
        // s * dL/ds from the quotient: sums of small sigmoids have reciprocals
        // near the end of fp32, and a gradient times one would pass it
        float g;
        if (a.renorm) {
          const float share = sel * reciprocal_or_zero(wave_sum(sel));
          g = a.scale * share * (dw - wave_sum(dw * share));
        } else {
          g = a.scale * dw * (a.sigmoid ? sel : sel * inv);
        }
        wave_lds_sync();
        if (picked) atomicAdd(&at_id[id], g);  // a token's ids differ: no order
        wave_lds_sync();
#pragma unroll
        for (int j = 0; j < J; ++j) d[j] = at_id[j * kLanes + lane];
        wave_lds_sync();
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j) d[j] = 0.0f;
      }
      // d is s times the weights' part of dL/ds here; p = s * inv
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        dot = fmaf(s[j] * inv, b[j], dot);
        if (!a.sigmoid) dot += d[j];
      }
      dot = wave_sum(dot);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float sds = fmaf(s[j] * inv, b[j] - dot, d[j]);
        d[j] = a.sigmoid ? sds * logistic(-x[j]) : sds;
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = j * kLanes + lane;
      if (e < a.E) {
        if (BF16)
          static_cast<uint16_t*>(a.d_logits)[at + e] = (uint16_t)pack_bf16(d[j], 0.0f);
        else
          static_cast<float*>(a.d_logits)[at + e] = d[j];
      }
    }
  }
}

// How a call is cut: waves per workgroup and workgroups per rank.  Up to 32
// tokens a rank one workgroup of 16 waves does it all in one launch, at most
// two tokens a wave; beyond that workgroups of 16 waves, two to a compute unit
// (512 in all; 1024 of eight waves take the same within 1 us at R=16, S=8192,
// E=384 and leave twice the partial sums), and a second launch of 4 to 5 us adds
// their partial sums (calls of the binding, R=8, E=256, bf16 with a bias: 32
// tokens 8.4 us in one launch, 48 tokens 10.2 in one and 12 to 13 in two, 64
// tokens 12.8 and 12 to 13).  Without counts, sums or loss there is nothing to
// add and every four tokens get a workgroup.
constexpr int kOneLaunchTokens = 32;

void route_cut(int R, int S, bool stats, int* waves, int* nblk) {
  if (stats && S <= kOneLaunchTokens) {
    *waves = std::min(kMaxWaves, S);
    *nblk = 1;
    return;
  }
  *waves = stats ? kMaxWaves : 4;
  const int want = (int)(((int64_t)S + *waves - 1) / *waves);
  *nblk = std::min(want, stats ? std::max(2, 512 / R) : 65536);
}

size_t route_workspace(int R, int S, int E, bool stats) {
  int waves, nblk;
  route_cut(R, S, stats, &waves, &nblk);
  return nblk == 1 || !stats ? 0 : (size_t)R * nblk * (2 * (size_t)E + 1) * 4;
}

template <int J, bool BF16, int Score, bool Sums>
void launch_route(const RouteArgs& a, int waves, hipStream_t s) {
  const size_t words = (size_t)waves * kLanes * (Score == kBiased ? 3 : 2) + (a.stats ? (size_t)a.E + 2 * waves : 0) +
                       (Sums && a.stats ? (size_t)waves * a.E : 0);
  const dim3 grid(a.nblk, a.R), block(waves * kLanes);
  if (a.E == J * kLanes)
    hipLaunchKernelGGL((k_route<J, BF16, Score, Sums, true>), grid, block, words * 4, s, a);
  else
    hipLaunchKernelGGL((k_route<J, BF16, Score, Sums, false>), grid, block, words * 4, s, a);
}

template <int J, bool BF16, int Score>
void launch_route(const RouteArgs& a, int waves, hipStream_t s) {
  // softmax weights that are not renormalised need the sum of all scores
  if (a.sums || (Score == kSoftmax && !a.renorm))
    launch_route<J, BF16, Score, true>(a, waves, s);
  else
    launch_route<J, BF16, Score, false>(a, waves, s);
}

template <int J, bool BF16>
hipError_t run_route(const RouteArgs& a, int waves, hipStream_t s) {
  if (!a.sigmoid)
    launch_route<J, BF16, kSoftmax>(a, waves, s);
  else if (a.bias == nullptr)
    launch_route<J, BF16, kSigmoid>(a, waves, s);
  else
    launch_route<J, BF16, kBiased>(a, waves, s);
  if (a.stats && a.nblk > 1) {
    int experts = kLanes;  // the power of two that holds E
    while (experts < a.E) experts *= 2;
    if (a.sums)
      hipLaunchKernelGGL(k_route_finish<true>, dim3(a.R), dim3(1024), 0, s, a, experts);
    else
      hipLaunchKernelGGL(k_route_finish<false>, dim3(a.R), dim3(1024), 0, s, a, experts);
  }
  return hipGetLastError();
}

template <int J, bool BF16>
hipError_t run_route_grad(const RouteGradArgs& a, hipStream_t s) {
  const int nblk = std::max(1, std::min((int)(((int64_t)a.S + 3) / 4), 8192 / a.R));
  hipLaunchKernelGGL((k_route_grad<J, BF16>), dim3(nblk, a.R), dim3(256), 0, s, a, nblk);
  return hipGetLastError();
}

// Words of 64 experts per token, rounded to the instantiated counts.
#define MOON_BY_WORDS(J_, FN, BF, ...)                         \
  (J_ <= 1 ? FN<1, BF>(__VA_ARGS__) : J_ <= 2 ? FN<2, BF>(__VA_ARGS__) \
   : J_ <= 3 ? FN<3, BF>(__VA_ARGS__) : J_ <= 4 ? FN<4, BF>(__VA_ARGS__) \
   : J_ <= 6 ? FN<6, BF>(__VA_ARGS__) : FN<8, BF>(__VA_ARGS__))

moon_status check_config(const moon_route_config* c) {
  if (c == nullptr || (c->flags & ~(MOON_ROUTE_SIGMOID | MOON_ROUTE_RENORM)) != 0)
    return MOON_ERR_INVALID_ARG;
  if (c->dtype != MOON_DTYPE_F32 && c->dtype != MOON_DTYPE_BF16) return MOON_ERR_INVALID_ARG;
  if (c->R < 1 || c->S < 1 || c->E < 1 || c->K < 1 || c->K > c->E) return MOON_ERR_INVALID_ARG;
  if (c->R > 32 || c->E > kMaxExperts || c->K > kMaxTopk ||
      (int64_t)c->R * c->S * c->K >= (int64_t)1 << 31)
    return MOON_ERR_UNSUPPORTED;
  return MOON_OK;
}

}  // namespace
}  // namespace moon

extern "C" {

moon_status moon_route_workspace(const moon_route_config* cfg, size_t* bytes) {
  if (bytes == nullptr) return MOON_ERR_INVALID_ARG;
  *bytes = 0;
  const moon_status st = moon::check_config(cfg);
  if (st != MOON_OK) return st;
  *bytes = moon::route_workspace(cfg->R, cfg->S, cfg->E, true);
  return MOON_OK;
}

moon_status moon_route(const moon_route_config* cfg, const void* logits_rse, const float* bias_e,
                       const uint8_t* valid_rs, int32_t* topk_rsk, float* weights_rsk,
                       int32_t* tokens_per_expert_re, int32_t* valid_tokens_r,
                       float* prob_sums_re, float* loss_r, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  using moon::is_aligned;
  const moon_status st = moon::check_config(cfg);
  if (st != MOON_OK) return st;
  if (logits_rse == nullptr || topk_rsk == nullptr || weights_rsk == nullptr)
    return MOON_ERR_INVALID_ARG;
  if (bias_e != nullptr && (cfg->flags & MOON_ROUTE_SIGMOID) == 0) return MOON_ERR_INVALID_ARG;
  if (!is_aligned(logits_rse, cfg->dtype == MOON_DTYPE_F32 ? 4 : 2) || !is_aligned(bias_e, 4) ||
      !is_aligned(topk_rsk, 4) || !is_aligned(weights_rsk, 4) ||
      !is_aligned(tokens_per_expert_re, 4) || !is_aligned(valid_tokens_r, 4) ||
      !is_aligned(prob_sums_re, 4) || !is_aligned(loss_r, 4) || !is_aligned(workspace, 4))
    return MOON_ERR_INVALID_ARG;
  moon::RouteArgs a = {};
  a.logits = logits_rse;
  a.bias = bias_e;
  a.valid = valid_rs;
  a.topk = topk_rsk;
  a.weights = weights_rsk;
  a.counts = tokens_per_expert_re;
  a.tokens = valid_tokens_r;
  a.psum = prob_sums_re;
  a.loss = loss_r;
  a.R = cfg->R;
  a.S = cfg->S;
  a.E = cfg->E;
  a.K = cfg->K;
  a.sigmoid = (cfg->flags & MOON_ROUTE_SIGMOID) != 0;
  a.renorm = (cfg->flags & MOON_ROUTE_RENORM) != 0;
  a.scale = cfg->scale;
  a.coef = cfg->loss_coef;
  a.stats = tokens_per_expert_re != nullptr || valid_tokens_r != nullptr ||
            prob_sums_re != nullptr || loss_r != nullptr;
  a.sums = prob_sums_re != nullptr || loss_r != nullptr;
  int waves;
  moon::route_cut(a.R, a.S, a.stats != 0, &waves, &a.nblk);
  const size_t need = moon::route_workspace(a.R, a.S, a.E, a.stats != 0);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return MOON_ERR_INVALID_ARG;
    const size_t n = (size_t)a.R * a.nblk * a.E;
    a.part_p = static_cast<float*>(workspace);
    a.part_c = reinterpret_cast<int32_t*>(a.part_p + n);
    a.part_n = a.part_c + n;
  }
  const int J = (a.E + moon::kLanes - 1) / moon::kLanes;
  using namespace moon;
  const hipError_t e = cfg->dtype == MOON_DTYPE_BF16
                           ? MOON_BY_WORDS(J, run_route, true, a, waves, stream)
                           : MOON_BY_WORDS(J, run_route, false, a, waves, stream);
  return e == hipSuccess ? MOON_OK : MOON_ERR_HIP;
}

moon_status moon_route_backward(const moon_route_config* cfg, const void* logits_rse,
                                const uint8_t* valid_rs, const int32_t* topk_rsk,
                                const float* d_weights_rsk, const int32_t* tokens_per_expert_re,
                                const int32_t* valid_tokens_r, const float* d_loss_r,
                                void* d_logits_rse, hipStream_t stream) {
  using moon::is_aligned;
  const moon_status st = moon::check_config(cfg);
  if (st != MOON_OK) return st;
  if (logits_rse == nullptr || d_logits_rse == nullptr) return MOON_ERR_INVALID_ARG;
  if (d_weights_rsk != nullptr && topk_rsk == nullptr) return MOON_ERR_INVALID_ARG;
  if (d_loss_r != nullptr && (tokens_per_expert_re == nullptr || valid_tokens_r == nullptr))
    return MOON_ERR_INVALID_ARG;
  const uintptr_t el = cfg->dtype == MOON_DTYPE_F32 ? 4 : 2;
  if (!is_aligned(logits_rse, el) || !is_aligned(d_logits_rse, el) || !is_aligned(topk_rsk, 4) ||
      !is_aligned(d_weights_rsk, 4) || !is_aligned(tokens_per_expert_re, 4) ||
      !is_aligned(valid_tokens_r, 4) || !is_aligned(d_loss_r, 4))
    return MOON_ERR_INVALID_ARG;
  moon::RouteGradArgs a = {};
  a.logits = logits_rse;
  a.valid = valid_rs;
  a.topk = topk_rsk;
  a.d_weights = d_weights_rsk;
  a.counts = tokens_per_expert_re;
  a.tokens = valid_tokens_r;
  a.d_loss = d_loss_r;
  a.d_logits = d_logits_rse;
  a.R = cfg->R;
  a.S = cfg->S;
  a.E = cfg->E;
  a.K = cfg->K;
  a.sigmoid = (cfg->flags & MOON_ROUTE_SIGMOID) != 0;
  a.renorm = (cfg->flags & MOON_ROUTE_RENORM) != 0;
  a.scale = cfg->scale;
  a.coef = cfg->loss_coef;
  const int J = (a.E + moon::kLanes - 1) / moon::kLanes;
  using namespace moon;
  const hipError_t e = cfg->dtype == MOON_DTYPE_BF16
                           ? MOON_BY_WORDS(J, run_route_grad, true, a, stream)
                           : MOON_BY_WORDS(J, run_route_grad, false, a, stream);
  return e == hipSuccess ? MOON_OK : MOON_ERR_HIP;
}

}  // extern "C"
