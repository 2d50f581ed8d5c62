// moon_expert.hip — the experts' products over a plan's groups with rows and
// weights in microscaled 4-bit floating point (MXFP4).
//
//   gemm    y[row][n] = sum_k x[row][k] * W_g[n][k]
//   swiglu  h[row][f] = w[row] * G / (1 + e^-G) * U,  G and U the products
//                       with the gate and the up weights of f
// for every row of every group g of every rank, W_g the weights of the group's
// expert (a rank's own experts, or the prefetched copy in the group's slot).
// Values and scales go into the matrix cores as they are stored: one
// v_mfma_scale_f32_16x16x128 multiplies 16 weight rows by 16 window rows over
// 128 values, each lane holding the 32 values of one scale block, exact
// products summed in fp32.  The result is rounded once, to bf16.
//
// The weights are the matrix operand whose rows land in a lane's four
// registers, so a lane owns four neighbouring outputs of one window row and
// stores them as one 8-byte word.
#include <algorithm>

#include "moon_rows.h"

namespace moon {
namespace {

typedef int vec8i __attribute__((ext_vector_type(8)));
typedef float vec4f __attribute__((ext_vector_type(4)));

struct Weight {
  const uint8_t *eq, *es, *sq, *ss;  // experts' codes and scales, slots' codes and scales
};

struct ExpertArgs {
  const uint8_t *xq, *xs;
  Weight w[2];
  const float* row_w;
  uint16_t* y;
  int32_t K, N;  // values per row; outputs per row
};

// Codes and scales of one weight matrix for entry j of rank u.
__device__ __forceinline__ void weight_of(const Groups& g, const Weight& w, int u, int j,
                                          int64_t n, int64_t k, const uint8_t** q,
                                          const uint8_t** s) {
  const int64_t i = j < g.Eg ? u * g.Eg + j : (int64_t)u * g.B + (j - g.Eg);
  *q = (j < g.Eg ? w.eq : w.sq) + i * n * (k / 2);
  *s = (j < g.Eg ? w.es : w.ss) + i * n * (k / 32);
}

__device__ __forceinline__ vec4f mfma4(vec4u a, vec4u b, vec4f c, uint32_t sa, uint32_t sb) {
  const vec8i av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const vec8i bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

__device__ __forceinline__ vec2u round4(vec4f v) {
  const vec2u o = {pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
  return o;
}

__device__ __forceinline__ vec4f gated(vec4f g, vec4f u, float w) {
  vec4f o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = w * (g[i] * sigmoid_f32(g[i]) * u[i]);
  return o;
}

// Padding rows [a, b) of columns [n0, n0 + width) to zero; a whole workgroup.
__device__ __forceinline__ void zero_rows(uint16_t* y, int64_t row0, int rows, int N, int n0,
                                          int width) {
  const int vecs = min(width, N - n0) / 8;
  const vec4u zero = {0u, 0u, 0u, 0u};
  for (int i = threadIdx.x; i < rows * vecs; i += blockDim.x)
    *reinterpret_cast<vec4u*>(y + (row0 + i / vecs) * N + n0 + i % vecs * 8) = zero;
}

// Few rows per group: the weights are read once and bound the time.  A
// workgroup takes 32 outputs of one group; its four waves split K, each
// streaming 512 values at a time straight into the matrix cores, and add up
// in LDS.
template <int MT, bool Swiglu>
__global__ void __launch_bounds__(256) k_expert_stream(ExpertArgs a, Groups g) {
  constexpr int P = Swiglu ? 2 : 1, NT = 2;
  __shared__ vec4f red[4][P][NT][MT][kLanes];
  if (g.status[0] != 0) return;
  const int u = blockIdx.y / g.per, j = blockIdx.y % g.per;
  const Span sp = group_span(g, u, j);
  const int n0 = blockIdx.x * 16 * NT;
  const int64_t base = (int64_t)u * g.NvS;
  zero_rows(a.y, base + sp.real_end, sp.end - sp.real_end, a.N, n0, 16 * NT);
  const int lane = threadIdx.x & (kLanes - 1), w = threadIdx.x / kLanes;
  const int r16 = lane & 15, kb = lane >> 4;
  const int blocks = a.K / 32;
  const uint8_t *wq[P], *ws[P];
#pragma unroll
  for (int p = 0; p < P; ++p) weight_of(g, a.w[p], u, j, a.N, a.K, &wq[p], &ws[p]);
  for (int m0 = sp.begin; m0 < sp.real_end; m0 += 16 * MT) {
    const int left = sp.real_end - m0;
    vec4f acc[P][NT][MT];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[p][n][m] = vec4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = w * 16; c < blocks; c += 64) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = c + 4 * i + kb;
        const bool in = b < blocks;
        const int bb = in ? b : 0;
        vec4u xv[MT];
        uint32_t xsc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int64_t row = base + min(m0 + 16 * m + r16, sp.real_end - 1);
          xv[m] = *reinterpret_cast<const vec4u*>(a.xq + (row * blocks + bb) * 16);
          xsc[m] = a.xs[row * blocks + bb];
          if (!in) {
            xv[m] = vec4u{0u, 0u, 0u, 0u};
            xsc[m] = 127u;
          }
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int64_t row = min(n0 + 16 * n + r16, a.N - 1);
            vec4u wv = *reinterpret_cast<const vec4u*>(wq[p] + (row * blocks + bb) * 16);
            uint32_t wsc = ws[p][row * blocks + bb];
            if (!in) {
              wv = vec4u{0u, 0u, 0u, 0u};
              wsc = 127u;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
              if (16 * m < left) acc[p][n][m] = mfma4(wv, xv[m], acc[p][n][m], wsc, xsc[m]);
          }
      }
    }
    __syncthreads();  // the last tile's sums are read
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) red[w][p][n][m][lane] = acc[p][n][m];
    __syncthreads();
    for (int t = w; t < NT * MT; t += 4) {
      const int n = t % NT, m = t / NT;
      const int row = m0 + 16 * m + r16, col = n0 + 16 * n + 4 * kb;
      if (row >= sp.real_end || col >= a.N) continue;
      vec4f s[P];
#pragma unroll
      for (int p = 0; p < P; ++p)
        s[p] = (red[0][p][n][m][lane] + red[1][p][n][m][lane]) +
               (red[2][p][n][m][lane] + red[3][p][n][m][lane]);
      vec4f o = s[0];
      if (Swiglu) o = gated(s[0], s[P - 1], a.row_w != nullptr ? a.row_w[base + row] : 1.0f);
      *reinterpret_cast<vec2u*>(a.y + (base + row) * a.N + col) = round4(o);
    }
  }
}

moon_status check(const ExpertArgs& a, const moon_plan_arrays* plan, int products, Groups* g) {
  const moon_status st = make_groups(plan, g);
  if (st != MOON_OK) return st;
  if (a.xq == nullptr || a.xs == nullptr || a.y == nullptr || !is_aligned(a.xq, 16) ||
      !is_aligned(a.y, 16) || !is_aligned(a.row_w, 4) || a.K < 32 || a.K % 32 != 0 || a.N < 8 ||
      a.N % 8 != 0)
    return MOON_ERR_INVALID_ARG;
  for (int p = 0; p < products; ++p) {
    const Weight& w = a.w[p];
    if (w.eq == nullptr || w.es == nullptr || w.sq == nullptr || w.ss == nullptr ||
        !is_aligned(w.eq, 16) || !is_aligned(w.sq, 16))
      return MOON_ERR_INVALID_ARG;
  }
  if (a.K > 65536 || a.N > 65536) return MOON_ERR_UNSUPPORTED;
  return MOON_OK;
}

template <bool Swiglu>
moon_status launch(const ExpertArgs& a, const Groups& g, hipStream_t s) {
  const dim3 grid((a.N + 31) / 32, g.R * g.per);
  hipLaunchKernelGGL((k_expert_stream<4, Swiglu>), grid, dim3(256), 0, s, a, g);
  return hipGetLastError() == hipSuccess ? MOON_OK : MOON_ERR_HIP;
}

Weight weight(const moon_mx4_weight* w) {
  Weight o = {};
  if (w != nullptr) {
    o.eq = w->expert_q;
    o.es = w->expert_scales;
    o.sq = w->slot_q;
    o.ss = w->slot_scales;
  }
  return o;
}

}  // namespace
}  // namespace moon

extern "C" {

moon_status moon_expert_gemm_mx4(const moon_plan_arrays* plan, const uint8_t* xq,
                                 const uint8_t* xs, int32_t K, const moon_mx4_weight* w, int32_t N,
                                 void* y, hipStream_t stream) {
  moon::ExpertArgs a = {};
  a.xq = xq;
  a.xs = xs;
  a.w[0] = moon::weight(w);
  a.y = static_cast<uint16_t*>(y);
  a.K = K;
  a.N = N;
  moon::Groups g;
  const moon_status st = moon::check(a, plan, 1, &g);
  return st != MOON_OK ? st : moon::launch<false>(a, g, stream);
}

moon_status moon_expert_swiglu_mx4(const moon_plan_arrays* plan, const uint8_t* xq,
                                   const uint8_t* xs, int32_t K, const moon_mx4_weight* gate,
                                   const moon_mx4_weight* up, int32_t F, const float* row_weights,
                                   void* h, hipStream_t stream) {
  moon::ExpertArgs a = {};
  a.xq = xq;
  a.xs = xs;
  a.w[0] = moon::weight(gate);
  a.w[1] = moon::weight(up);
  a.row_w = row_weights;
  a.y = static_cast<uint16_t*>(h);
  a.K = K;
  a.N = F;
  moon::Groups g;
  const moon_status st = moon::check(a, plan, 2, &g);
  return st != MOON_OK ? st : moon::launch<true>(a, g, stream);
}

}  // extern "C"
