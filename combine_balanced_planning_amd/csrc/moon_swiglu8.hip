// moon_swiglu8.hip — the experts' gated activation with its inputs kept in 8
// bits, and its gradient from them.
//
// For every row of the window that holds a route, gate g and up u (F values
// each, gate first) and row weight w (1 without weights):
//   forward   h = w * g / (1 + e^-g) * u
//   backward  dg = w dh u s(g) (1 + g (1 - s(g))),  du = w dh g s(g),
//             dw = sum over F of dh g s(g) u,       s(g) = 1/(1+e^-g),
// the backward with g and u as the 8-bit values kept by the forward: 32
// neighbouring values share a scale 2^(c-127), the smallest power of two under
// which the largest of them is at most 448, and are rounded to nearest even
// e4m3 (relative error 2^-4 at most, no saturation).  That is half of bf16's
// bytes plus 1/32.  A block that holds an infinity or a NaN keeps the scale
// byte 255 and reads back as NaN.  Sums and products are fp32; h, dg and du are
// rounded once, to bf16.
//
// HBM bounds both directions: 8 bytes per value pair forward (4 read, 2
// written as h, 2 kept) and 8 backward.  A lane takes eight neighbouring gate
// values and the eight up values beside them, four lanes share a scale.
#include <algorithm>

#include "moon_rows.h"

namespace moon {
namespace {

struct SwigluArgs {
  const void* x;          // gate_up (forward) or dh (backward)
  const float* w;
  void* y;                // h (forward) or d_gate_up (backward)
  uint8_t *saved, *scales;
  float* dw;
  int32_t F, per_wg, lanes;
};

// Eight bf16 values to e4m3 under the scale of their block of 32 (a quad).
__device__ __forceinline__ vec2u to_e4m3(vec4u v, uint32_t* scale_byte) {
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo = max(lo, v[i] & 0x7FFFu);
    hi = max(hi, v[i] & 0x7FFF0000u);
  }
  const uint32_t m = quad_max_u32(max(lo << 16, hi));
  const uint32_t e = m >> 23;
  // amax = 1.f * 2^(e-127): 448 = 1.75 * 2^8 holds it under 2^(e-135), or
  // under twice that when 1.f is beyond 1.75
  const uint32_t up = (m & 0x7FFFFFu) > 0x600000u ? 7u : 8u;
  const uint32_t c = e == 255u ? 255u : (e > up ? e - up : 0u);
  *scale_byte = c;
  vec2u out = {0u, 0u};
  if (c == 255u) return out;
  const float scale = __uint_as_float(c == 0u ? 0x00400000u : c << 23);
  typedef short vec2s __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    vec2s p = {0, 0};
    p = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(p, as_bf16x2(v[2 * i]), scale, false);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(p, as_bf16x2(v[2 * i + 1]), scale, true);
    out[i] = __builtin_bit_cast(uint32_t, p);
  }
  return out;
}

__device__ __forceinline__ void from_e4m3(vec2u v, uint32_t scale_byte, float (&f)[8]) {
  const float scale = __uint_as_float(
      scale_byte == 255u ? 0x7FC00000u : scale_byte == 0u ? 0x00400000u : scale_byte << 23);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const vec2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], false);
    const vec2f b = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], true);
    f[4 * i] = a.x * scale;
    f[4 * i + 1] = a.y * scale;
    f[4 * i + 2] = b.x * scale;
    f[4 * i + 3] = b.y * scale;
  }
}

__device__ __forceinline__ void unpack(vec4u v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
}

__device__ __forceinline__ vec4u pack(const float (&f)[8]) {
  const vec4u o = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                   pack_bf16(f[6], f[7])};
  return o;
}

__global__ void __launch_bounds__(256) k_swiglu_save8(SwigluArgs a, Groups g) {
  __shared__ unsigned long long m[2];
  if (g.status[0] != 0) return;
  const int u = blockIdx.y, r0 = blockIdx.x * a.per_wg, n = min(a.per_wg, g.NvS - r0);
  unsigned long long real, pad;
  row_masks(g, u, r0, n, m, &real, &pad);
  const int lane = threadIdx.x & (a.lanes - 1), vecs = a.F / 8;
  for (int i = threadIdx.x / a.lanes; i < n; i += 256 / a.lanes) {
    const int64_t row = (int64_t)u * g.NvS + r0 + i;
    vec4u* h = static_cast<vec4u*>(a.y) + row * vecs;
    if ((real >> i) & 1ull) {
      const vec4u* x = static_cast<const vec4u*>(a.x) + row * 2 * vecs;
      vec2u* saved = reinterpret_cast<vec2u*>(a.saved) + row * 2 * vecs;
      uint8_t* scales = a.scales + row * (a.F / 16);
      const float w = a.w != nullptr ? a.w[row] : 1.0f;
      for (int c = lane; c < vecs; c += a.lanes) {
        const vec4u gv = x[c], uv = x[vecs + c];
        uint32_t gs, us;
        saved[c] = to_e4m3(gv, &gs);
        saved[vecs + c] = to_e4m3(uv, &us);
        if ((c & 3) == 0) {
          scales[c / 4] = (uint8_t)gs;
          scales[a.F / 32 + c / 4] = (uint8_t)us;
        }
        float gf[8], uf[8];
        unpack(gv, gf);
        unpack(uv, uf);
#pragma unroll
        for (int k = 0; k < 8; ++k) gf[k] = w * (gf[k] * sigmoid_f32(gf[k]) * uf[k]);
        h[c] = pack(gf);
      }
    } else if ((pad >> i) & 1ull) {
      const vec4u zero = {0u, 0u, 0u, 0u};
      for (int c = lane; c < vecs; c += a.lanes) h[c] = zero;
    }
  }
}

__global__ void __launch_bounds__(256) k_swiglu_grad8(SwigluArgs a, Groups g) {
  __shared__ unsigned long long m[2];
  if (g.status[0] != 0) return;
  const int u = blockIdx.y, r0 = blockIdx.x * a.per_wg, n = min(a.per_wg, g.NvS - r0);
  unsigned long long real, pad;
  row_masks(g, u, r0, n, m, &real, &pad);
  const int lane = threadIdx.x & (a.lanes - 1), vecs = a.F / 8;
  for (int i = threadIdx.x / a.lanes; i < n; i += 256 / a.lanes) {
    const int64_t row = (int64_t)u * g.NvS + r0 + i;
    vec4u* dx = static_cast<vec4u*>(a.y) + row * 2 * vecs;
    if ((real >> i) & 1ull) {
      const vec4u* dhp = static_cast<const vec4u*>(a.x) + row * vecs;
      const vec2u* saved = reinterpret_cast<const vec2u*>(a.saved) + row * 2 * vecs;
      const uint8_t* scales = a.scales + row * (a.F / 16);
      const float w = a.w != nullptr ? a.w[row] : 1.0f;
      float sum = 0.0f;
      for (int c = lane; c < vecs; c += a.lanes) {
        float dh[8], gf[8], uf[8];
        unpack(dhp[c], dh);
        from_e4m3(saved[c], scales[c / 4], gf);
        from_e4m3(saved[vecs + c], scales[a.F / 32 + c / 4], uf);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float s = sigmoid_f32(gf[k]), act = gf[k] * s;
          sum += dh[k] * act * uf[k];
          const float d = w * dh[k];
          gf[k] = d * uf[k] * (s * (1.0f + gf[k] * (1.0f - s)));
          uf[k] = d * act;
        }
        dx[c] = pack(gf);
        dx[vecs + c] = pack(uf);
      }
      if (a.dw != nullptr) {
        for (int k = 1; k < a.lanes; k *= 2) sum += __shfl_xor(sum, k);
        if (lane == 0) a.dw[row] = sum;
      }
    } else if ((pad >> i) & 1ull) {
      const vec4u zero = {0u, 0u, 0u, 0u};
      for (int c = lane; c < 2 * vecs; c += a.lanes) dx[c] = zero;
      if (a.dw != nullptr && lane == 0) a.dw[row] = 0.0f;
    }
  }
}

moon_status check(SwigluArgs* a, const moon_plan_arrays* plan, Groups* g) {
  const moon_status st = make_groups(plan, g);
  if (st != MOON_OK) return st;
  if (a->x == nullptr || a->y == nullptr || a->saved == nullptr || a->scales == nullptr ||
      !is_aligned(a->x, 16) || !is_aligned(a->y, 16) || !is_aligned(a->saved, 16) ||
      !is_aligned(a->w, 4) || !is_aligned(a->dw, 4) || a->F < 32 || a->F % 32 != 0)
    return MOON_ERR_INVALID_ARG;
  if (a->F > 65536) return MOON_ERR_UNSUPPORTED;
  a->lanes = kLanes;
  while (a->lanes > 4 && a->lanes / 2 >= a->F / 8) a->lanes /= 2;
  const int64_t rows = (int64_t)g->R * g->NvS;
  a->per_wg = (int)std::max<int64_t>(1, std::min<int64_t>(64, rows / 16384));
  a->per_wg = std::max(a->per_wg, std::min(64, 256 / a->lanes));
  return MOON_OK;
}

}  // namespace
}  // namespace moon

extern "C" {

moon_status moon_swiglu_save8(const moon_plan_arrays* plan, const void* gate_up,
                              const float* row_weights, int32_t F, void* h, uint8_t* saved,
                              uint8_t* saved_scales, hipStream_t stream) {
  moon::SwigluArgs a = {};
  a.x = gate_up;
  a.w = row_weights;
  a.y = h;
  a.saved = saved;
  a.scales = saved_scales;
  a.F = F;
  moon::Groups g;
  const moon_status st = moon::check(&a, plan, &g);
  if (st != MOON_OK) return st;
  const dim3 grid((g.NvS + a.per_wg - 1) / a.per_wg, g.R);
  hipLaunchKernelGGL(moon::k_swiglu_save8, grid, dim3(256), 0, stream, a, g);
  return hipGetLastError() == hipSuccess ? MOON_OK : MOON_ERR_HIP;
}

moon_status moon_swiglu_grad8(const moon_plan_arrays* plan, const void* dh, const uint8_t* saved,
                              const uint8_t* saved_scales, const float* row_weights, int32_t F,
                              void* d_gate_up, float* d_row_weights, hipStream_t stream) {
  moon::SwigluArgs a = {};
  a.x = dh;
  a.w = row_weights;
  a.y = d_gate_up;
  a.saved = const_cast<uint8_t*>(saved);
  a.scales = const_cast<uint8_t*>(saved_scales);
  a.dw = d_row_weights;
  a.F = F;
  moon::Groups g;
  const moon_status st = moon::check(&a, plan, &g);
  if (st != MOON_OK) return st;
  const dim3 grid((g.NvS + a.per_wg - 1) / a.per_wg, g.R);
  hipLaunchKernelGGL(moon::k_swiglu_grad8, grid, dim3(256), 0, stream, a, g);
  return hipGetLastError() == hipSuccess ? MOON_OK : MOON_ERR_HIP;
}

}  // extern "C"
