// moon_mx4.hip — rows to microscaled 4-bit floating point (MXFP4) and back.
//
// 32 neighbouring values of a row share one scale 2^(c - 127), stored as the
// byte c = max(floor(log2(amax)) - 2, -127) + 127, and each value is kept as
// e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and the sign): value / scale rounded to
// nearest, ties to the even code, saturating at 6.  A block that holds an
// infinity or a NaN gets the scale byte 255 (NaN) and reads back as NaN.
// The scale is a power of two and 4-bit values times it are exact in bf16
// and fp32, so the only rounding is the one to e2m1.
//
// Both directions move bytes and little else, so HBM bounds them.  The 4-bit
// side is a quarter of the bytes and what is used next: it is stored and loaded
// as usual, while wide bf16 values stream past the caches (non-temporal), which
// took quantising and reading back from 470 to 394 us at 65536 x 7168 (2.4 GB:
// 6.0 TB/s).  fp32 values go through them: 426 us to 4 bits (5.0 TB/s) and 584
// back (3.6 TB/s) at that size.  A lane takes eight neighbouring values (one
// 16-byte load of bf16, two of fp32, a 4-byte word of codes), four lanes share a
// block, and a row is spread over up to 64 lanes.  With a plan only rows that hold routes are converted,
// padding rows are zeroed and rows behind a rank's last group are not touched.
#include <algorithm>

#include "moon_rows.h"

namespace moon {
namespace {

struct Mx4Args {
  const void* x;    // values read (quantise) or null
  void* y;          // values written (dequantise) or null
  uint8_t* q;
  uint8_t* scales;
  int64_t rows;
  int32_t cols;
  int32_t rank_rows;  // rows per rank window (with a plan)
  int32_t per_wg;     // rows per workgroup, with a plan at most 64
  int32_t lanes;      // lanes per row, a power of two
  int32_t words;      // scale bytes are stored four at a time
};

// Eight values: codes under the block's scale; the four lanes of a quad hold
// one block.
template <bool BF16>
__device__ __forceinline__ uint32_t to_codes(const vec4u (&v)[2], uint32_t* scale_byte) {
  uint32_t m = 0;
  if (BF16) {
    // the larger magnitude of each half as whole numbers: the order of floats
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo = max(lo, v[0][i] & 0x7FFFu);
      hi = max(hi, v[0][i] & 0x7FFF0000u);
    }
    m = max(lo << 16, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(v[0][i] & 0x7FFFFFFFu, v[1][i] & 0x7FFFFFFFu));
  }
  const uint32_t e = quad_max_u32(m) >> 23;
  const uint32_t c = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
  *scale_byte = c;
  if (c == 255u) return 0;
  // 2^(c - 127) as a float; c = 0 is the subnormal 2^-127
  const float scale = __uint_as_float(c == 0u ? 0x00400000u : c << 23);
  uint32_t out = 0;
  if (BF16) {
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf16x2(v[0][0]), scale, 0);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf16x2(v[0][1]), scale, 1);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf16x2(v[0][2]), scale, 2);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf16x2(v[0][3]), scale, 3);
  } else {
    const auto f = [&](int i) { return __uint_as_float(v[i / 4][i % 4]); };
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f(0), f(1), scale, 0);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f(2), f(3), scale, 1);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f(4), f(5), scale, 2);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f(6), f(7), scale, 3);
  }
  return out;
}

// Scale bytes of a row of whole 16-lane runs go out four at a time where they
// lie on whole words.
__device__ __forceinline__ void store_scale(const Mx4Args& a, int64_t at, int c, uint32_t s) {
  if (a.words) {
    const uint32_t word = quad_bytes(s);
    if ((c & 15) == 0) *reinterpret_cast<uint32_t*>(a.scales + at / 4) = word;
  } else if ((c & 3) == 0) {
    a.scales[at / 4] = (uint8_t)s;
  }
}

// A row, four vectors of a lane in flight at a time.
template <bool BF16, bool Quantise>
__device__ __forceinline__ void convert(const Mx4Args& a, int64_t row, int lane) {
  constexpr int U = 4;
  const int vecs = a.cols / 8;
  for (int c0 = lane; c0 < vecs; c0 += U * a.lanes) {
    if (Quantise) {
      vec4u v[U][2];
      const vec4u* x = static_cast<const vec4u*>(a.x);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * a.lanes;
        if (c >= vecs) break;
        const int64_t at = row * vecs + c;
        if (BF16) {
          v[u][0] = __builtin_nontemporal_load(&x[at]);
        } else {
          v[u][0] = x[2 * at];
          v[u][1] = x[2 * at + 1];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * a.lanes;
        if (c >= vecs) break;
        const int64_t at = row * vecs + c;
        uint32_t s;
        const uint32_t codes = to_codes<BF16>(v[u], &s);
        reinterpret_cast<uint32_t*>(a.q)[at] = codes;
        store_scale(a, at, c, s);
      }
    } else {
      uint32_t q[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * a.lanes;
        if (c >= vecs) break;
        const int64_t at = row * vecs + c;
        q[u] = reinterpret_cast<const uint32_t*>(a.q)[at];
        b[u] = a.scales[at / 4];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * a.lanes;
        if (c >= vecs) break;
        const int64_t at = row * vecs + c;
        const float scale = __uint_as_float(b[u] == 255u ? 0x7FC00000u
                                            : b[u] == 0u ? 0x00400000u : b[u] << 23);
        vec4u* y = static_cast<vec4u*>(a.y);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // e2m1 bits s ee m as a float of exponent ee - 1, or half of m
          const uint32_t n = (q[u] >> (4 * i)) & 15u, ee = (n >> 1) & 3u;
          const float mag = ee == 0u ? 0.5f * (float)(n & 1u)
                                     : __uint_as_float((ee + 126u) << 23 | (n & 1u) << 22);
          f[i] = ((n & 8u) != 0u ? -mag : mag) * scale;
        }
        if (BF16) {
          __builtin_nontemporal_store(vec4u{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                        pack_bf16(f[6], f[7])}, &y[at]);
        } else {
          y[2 * at] = vec4u{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                            __float_as_uint(f[3])};
          y[2 * at + 1] = vec4u{__float_as_uint(f[4]), __float_as_uint(f[5]),
                                __float_as_uint(f[6]), __float_as_uint(f[7])};
        }
      }
    }
  }
}

template <bool BF16, bool Quantise>
__device__ __forceinline__ void clear(const Mx4Args& a, int64_t row, int lane) {
  const int64_t vecs = a.cols / 8;
  const vec4u zero = {0u, 0u, 0u, 0u};
  for (int c = lane; c < vecs; c += a.lanes) {
    const int64_t at = row * vecs + c;
    if (Quantise) {
      reinterpret_cast<uint32_t*>(a.q)[at] = 0u;
      store_scale(a, at, c, 0u);
    } else if (BF16) {
      static_cast<vec4u*>(a.y)[at] = zero;
    } else {
      static_cast<vec4u*>(a.y)[2 * at] = zero;
      static_cast<vec4u*>(a.y)[2 * at + 1] = zero;
    }
  }
}

template <bool BF16, bool Quantise, bool Planned>
__global__ void __launch_bounds__(256) k_mx4(Mx4Args a, Groups g) {
  __shared__ unsigned long long m[2];
  const int lane = threadIdx.x & (a.lanes - 1);
  const int step = 256 / a.lanes;
  if (Planned) {
    if (g.status[0] != 0) return;
    const int u = blockIdx.y, r0 = blockIdx.x * a.per_wg;
    const int n = min(a.per_wg, a.rank_rows - r0);
    unsigned long long real, pad;
    row_masks(g, u, r0, n, m, &real, &pad);
    for (int i = threadIdx.x / a.lanes; i < n; i += step) {
      const int64_t row = (int64_t)u * a.rank_rows + r0 + i;
      if ((real >> i) & 1ull)
        convert<BF16, Quantise>(a, row, lane);
      else if ((pad >> i) & 1ull)
        clear<BF16, Quantise>(a, row, lane);
    }
  } else {
    const int64_t r0 = (int64_t)blockIdx.x * a.per_wg;
    const int n = (int)min((int64_t)a.per_wg, a.rows - r0);
    for (int i = threadIdx.x / a.lanes; i < n; i += step)
      convert<BF16, Quantise>(a, r0 + i, lane);
  }
}

template <bool Quantise>
moon_status launch(Mx4Args a, int32_t dtype, const moon_plan_arrays* plan, hipStream_t s) {
  const void* values = Quantise ? a.x : a.y;
  if (values == nullptr || a.q == nullptr || a.scales == nullptr || !is_aligned(values, 16) ||
      !is_aligned(a.q, 16) || (dtype != MOON_DTYPE_F32 && dtype != MOON_DTYPE_BF16) ||
      a.rows < 1 || a.cols < 32 || a.cols % 32 != 0)
    return MOON_ERR_INVALID_ARG;
  if (a.cols > 65536 || a.rows >= (int64_t)1 << 31) return MOON_ERR_UNSUPPORTED;
  Groups g = {};
  if (plan != nullptr) {
    const moon_status st = make_groups(plan, &g);
    if (st != MOON_OK) return st;
    if (a.rows != (int64_t)g.R * g.NvS) return MOON_ERR_INVALID_ARG;
    a.rank_rows = g.NvS;
  }
  a.lanes = kLanes;
  while (a.lanes > 4 && a.lanes / 2 >= a.cols / 8) a.lanes /= 2;
  a.words = a.cols % 128 == 0 && is_aligned(a.scales, 4);
  // Rows per workgroup: many small workgroups finish evenly (4 rows each take
  // 5 % less time than 16 at 65536 x 7168), at most 64 rows (the plan's row masks
  // are one word) for long thin arrays.
  a.per_wg = (int)std::max<int64_t>(1, std::min<int64_t>(64, a.rows / 16384));
  a.per_wg = std::max(a.per_wg, std::min(64, 256 / a.lanes));
  // A launch has fewer than 2^32 threads: from 2^30 rows on more rows each.
  if (plan == nullptr) a.per_wg = std::max(a.per_wg, (int)(a.rows >> 23) + 1);
  const bool bf = dtype == MOON_DTYPE_BF16;
  if (plan != nullptr) {
    const dim3 grid((g.NvS + a.per_wg - 1) / a.per_wg, g.R);
    if (bf)
      hipLaunchKernelGGL((k_mx4<true, Quantise, true>), grid, dim3(256), 0, s, a, g);
    else
      hipLaunchKernelGGL((k_mx4<false, Quantise, true>), grid, dim3(256), 0, s, a, g);
  } else {
    const dim3 grid((uint32_t)((a.rows + a.per_wg - 1) / a.per_wg));
    if (bf)
      hipLaunchKernelGGL((k_mx4<true, Quantise, false>), grid, dim3(256), 0, s, a, g);
    else
      hipLaunchKernelGGL((k_mx4<false, Quantise, false>), grid, dim3(256), 0, s, a, g);
  }
  return hipGetLastError() == hipSuccess ? MOON_OK : MOON_ERR_HIP;
}

}  // namespace
}  // namespace moon

extern "C" {

moon_status moon_mx4_quantize(const void* x, int32_t dtype, int64_t rows, int32_t cols,
                              const moon_plan_arrays* plan, uint8_t* q, uint8_t* scales,
                              hipStream_t stream) {
  moon::Mx4Args a = {};
  a.x = x;
  a.q = q;
  a.scales = scales;
  a.rows = rows;
  a.cols = cols;
  return moon::launch<true>(a, dtype, plan, stream);
}

moon_status moon_mx4_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows,
                                int32_t cols, const moon_plan_arrays* plan, int32_t dtype,
                                void* y, hipStream_t stream) {
  moon::Mx4Args a = {};
  a.y = y;
  a.q = const_cast<uint8_t*>(q);
  a.scales = const_cast<uint8_t*>(scales);
  a.rows = rows;
  a.cols = cols;
  return moon::launch<false>(a, dtype, plan, stream);
}

}  // extern "C"
