// moon_rows.h — what the routing and expert operators share: the group layout
// of a plan as kernels walk it, bf16 and microscaling helpers, wave reductions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moon.h"

namespace moon {

constexpr int kLanes = 64;

typedef uint32_t vec4u __attribute__((ext_vector_type(4)));
typedef uint32_t vec2u __attribute__((ext_vector_type(2)));
typedef float vec2f __attribute__((ext_vector_type(2)));
typedef __bf16 vec2bf __attribute__((ext_vector_type(2)));

// A plan's groups.  Only a rank's own experts and its slots can hold rows, so
// a rank has `per` = Eg + B entries: j < Eg is expert u*Eg + j, Eg + i slot i.
struct Groups {
  const int32_t *cu, *zfr, *status;
  int32_t R, E, EB, Eg, B, per, NvS;
  int32_t N;  // routes per rank (its window's capacity where the caller leaves it out)
};

struct Span {
  int32_t begin, real_end, end;  // local rows: routes, then padding
};

// Rows of entry j of rank u, clamped to the window whatever the arrays hold.
__device__ __forceinline__ Span group_span(const Groups& g, int u, int j) {
  const int gi = j < g.Eg ? u * g.Eg + j : g.E + (j - g.Eg);
  const int at = u * g.EB + gi;
  Span s;
  s.begin = gi > 0 ? g.cu[at - 1] : 0;
  s.end = g.cu[at];
  s.real_end = g.zfr[2 * at];
  s.begin = min(max(s.begin, 0), g.NvS);
  s.end = min(max(s.end, s.begin), g.NvS);
  s.real_end = min(max(s.real_end, s.begin), s.end);
  return s;
}

// Which of the rows [r0, r0 + n), n <= 64, of rank u hold routes (real) and
// which are padding.  Called by a whole workgroup; LDS words m[2].
__device__ __forceinline__ void row_masks(const Groups& g, int u, int r0, int n,
                                          unsigned long long* m, unsigned long long* real,
                                          unsigned long long* pad) {
  if (threadIdx.x < 2) m[threadIdx.x] = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < g.per; j += blockDim.x) {
    const Span s = group_span(g, u, j);
    if (s.end <= r0 || s.begin >= r0 + n) continue;
    for (int k = 0; k < 2; ++k) {
      const int a = max(k == 0 ? s.begin : s.real_end, r0) - r0;
      const int b = min(k == 0 ? s.real_end : s.end, r0 + n) - r0;
      if (a < b) atomicOr(&m[k], (b - a == 64 ? ~0ull : ((1ull << (b - a)) - 1ull)) << a);
    }
  }
  __syncthreads();
  *real = m[0];
  *pad = m[1];
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A word as two bf16 values (by value: a bit cast of a vector's element takes
// its first element).
__device__ __forceinline__ vec2bf as_bf16x2(uint32_t w) { return __builtin_bit_cast(vec2bf, w); }

// Two floats to packed bf16, nearest even, NaN kept.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  vec2bf v;
  v.x = (__bf16)a;
  v.y = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

// e^x with the argument's rounding carried along: the product x*log2(e) is
// taken in two pieces, so the relative error stays at about two units in the
// last place for all x (exp2 of the rounded product alone loses |x| of them).
// +-infinity and NaN keep their meaning.
__device__ __forceinline__ float exp_f32(float x) {
  const float t = x * 1.44269504088896341f;
  const float lo = fmaf(x, 1.44269504088896341f, -t) + x * 1.925963033500e-8f;
  const float y = __builtin_amdgcn_exp2f(t);
  const float z = fmaf(y, lo * 0.693147180559945f, y);
  return fabsf(t) < 128.0f ? z : y;
}

// 1 / (1 + e^-x).
__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x));
}

template <int Ctrl, int Rows>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t ident, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)ident, (int)v, Ctrl, Rows, 0xF, false);
}

// Largest value of the wave (in every lane's register as a scalar).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_u32<0x111, 0xF>(0, v));
  v = max(v, dpp_u32<0x112, 0xF>(0, v));
  v = max(v, dpp_u32<0x114, 0xF>(0, v));
  v = max(v, dpp_u32<0x118, 0xF>(0, v));
  v = max(v, dpp_u32<0x142, 0xA>(0, v));
  v = max(v, dpp_u32<0x143, 0xC>(0, v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Smallest value of the wave.
__device__ __forceinline__ uint32_t wave_min_u32(uint32_t v) { return ~wave_max_u32(~v); }

template <int Ctrl, int Rows>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(dpp_u32<Ctrl, Rows>(0u, __float_as_uint(v)));
}

// Sum over the wave, the same order of additions every time.
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);
  v = dpp_add<0x143, 0xC>(v);
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Largest of the four lanes of a quad (quad_perm swaps).
__device__ __forceinline__ uint32_t quad_max_u32(uint32_t v) {
  v = max(v, dpp_u32<0xB1, 0xF>(0, v));
  return max(v, dpp_u32<0x4E, 0xF>(0, v));
}

// One byte of each quad of a 16-lane row as a word, in every lane of the row.
__device__ __forceinline__ uint32_t quad_bytes(uint32_t b) {
  uint32_t v = b << (8 * ((threadIdx.x >> 2) & 3));
  v |= dpp_u32<0x124, 0xF>(0, v);  // row_ror:4
  return v | dpp_u32<0x128, 0xF>(0, v);  // row_ror:8
}

// Orders LDS accesses of one wave's lanes among each other (the hardware runs
// them in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---- host side ----

// Checks the part of a plan's arrays that the operators read and describes
// its groups.
inline moon_status make_groups(const moon_plan_arrays* p, Groups* g) {
  if (p == nullptr || p->cu_seqlens == nullptr || p->zero_fill_ranges == nullptr ||
      p->status == nullptr || ((uintptr_t)p->cu_seqlens & 3) != 0 ||
      ((uintptr_t)p->zero_fill_ranges & 3) != 0 || ((uintptr_t)p->status & 3) != 0)
    return MOON_ERR_INVALID_ARG;
  if (p->R < 1 || p->E < 1 || p->B < 1 || p->NvS < 1) return MOON_ERR_INVALID_ARG;
  if (p->E % p->R != 0) return MOON_ERR_TOPOLOGY;
  if (p->R > 32 || p->E > 512 || (int64_t)p->R * p->B > 8192 || p->NvS > 1 << 29 ||
      (int64_t)p->R * p->NvS >= (int64_t)1 << 31)
    return MOON_ERR_UNSUPPORTED;
  g->cu = p->cu_seqlens;
  g->zfr = p->zero_fill_ranges;
  g->status = p->status;
  g->R = p->R;
  g->E = p->E;
  g->B = p->B;
  g->EB = p->E + p->B;
  g->Eg = p->E / p->R;
  g->per = g->Eg + p->B;
  g->NvS = p->NvS;
  g->N = p->N > 0 && p->N < p->NvS ? p->N : p->NvS;
  return MOON_OK;
}

inline bool is_aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace moon
