// moon_expert.hip — the experts' products over a plan's groups with rows and
// weights in microscaled 4-bit floating point (MXFP4).
//
//   gemm    y[row][n] = sum_k x[row][k] * W_g[n][k]
//   swiglu  h[row][f] = w[row] * G / (1 + e^-G) * U,  G and U the products
//                       with the gate and the up weights of f
// for every row of every group g of every rank, W_g the weights of the group's
// expert (a rank's own experts, or the prefetched copy in the group's slot).
// Values and scales go into the matrix cores as they are stored: a
// v_mfma_scale_f32 takes 32 values of a row and their scale per lane, and sums
// exact products in fp32.  The result is rounded once, to bf16.  The weights are
// the operand whose rows land in a lane's registers, so a lane owns
// neighbouring outputs of one window row.
//
// Two kernels: one streams the weights past a few rows, the other multiplies
// tiles of 256 by 256.
#include <algorithm>

#include "moon_rows.h"

namespace moon {
namespace {

typedef int vec8i __attribute__((ext_vector_type(8)));
typedef float vec4f __attribute__((ext_vector_type(4)));
typedef float vec16f __attribute__((ext_vector_type(16)));

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
  for (int64_t i = threadIdx.x; i < (int64_t)rows * vecs; i += blockDim.x)
    *reinterpret_cast<vec4u*>(y + (row0 + i / vecs) * N + n0 + i % vecs * 8) = zero;
}

// `bytes` bytes from p as a buffer: loads beyond them read nothing and give 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, (int)bytes, 0x00027000);
}

// 16 bytes per lane from a buffer straight into LDS, lane l at dst + 16 l.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t src, uint32_t at, vec4u* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16,
                                           (int)at, 0, 0, 0);
}

// Waits until at most n vector memory operations of this wave are in flight.
template <int n>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | ((n >> 4) << 14));
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- few rows per group: the weights are read once and bound the time ----

// A workgroup takes 64 weight rows of one group (with a gate 32 of each
// matrix) and its window rows, 16 * MT at a time.  K advances by 256 values, 128
// bytes of a row, a step; LDS holds four steps, loaded straight into it eight
// lanes a row, three steps ahead.  The 16-byte blocks of a row are stored
// swapped by its index, so ds_read_b128 of 16 rows meets no bank twice.  Each of
// the four waves owns 16 outputs; with a gate two, and the waves of a pair take
// turns along K and add up at the end.
template <int MT, bool Swiglu, bool Whole>
__global__ void __launch_bounds__(256) k_expert_stream(ExpertArgs a, Groups g) {
  constexpr int P = Swiglu ? 2 : 1;
  constexpr int kOut = 64 / P, kRows = 64 + 16 * MT, kXLoads = MT < 2 ? 1 : MT / 2;
  constexpr int kLoads = 2 + kXLoads;  // of a wave, a step
  __shared__ vec4u st0[kRows * 8], st1[kRows * 8], st2[kRows * 8], st3[kRows * 8];
  __shared__ vec4u sc[2][kRows];
  if (g.status[0] != 0) return;
  const int u = blockIdx.y / g.per, j = blockIdx.y % g.per;
  const Span sp = group_span(g, u, j);
  const int n0 = blockIdx.x * kOut;
  const int64_t base = (int64_t)u * g.NvS;
  zero_rows(a.y, base + sp.real_end, sp.end - sp.real_end, a.N, n0, kOut);
  const int tid = threadIdx.x, lane = tid & (kLanes - 1);
  const int w = __builtin_amdgcn_readfirstlane(tid / kLanes);
  const int r16 = lane & 15, kb = lane >> 4;
  const int blocks = a.K / 32, steps = (blocks + 7) / 8;
  const uint32_t row_bytes = 16u * blocks;
  const int nr = min(kOut, a.N - n0);  // weight rows of each matrix
  const uint8_t *wq[2], *ws[2];
  weight_of(g, a.w[0], u, j, a.N, a.K, &wq[0], &ws[0]);
  weight_of(g, a.w[P - 1], u, j, a.N, a.K, &wq[1], &ws[1]);
  const __amdgpu_buffer_rsrc_t wsrc =
      buffer(wq[Swiglu ? w >> 1 : 0] + (int64_t)n0 * row_bytes, nr * row_bytes);
  // A load takes eight rows; the block that this lane takes of its row, for the
  // first and the second half of 16 rows.
  const uint32_t blk16[2] = {16u * ((lane & 7) ^ (lane >> 4)), 16u * ((lane & 7) ^ (4 + (lane >> 4)))};
  const uint32_t wat = ((Swiglu ? w & 1 : w) * 16 + (lane >> 3)) * row_bytes;
  for (int m0 = sp.begin; m0 < sp.real_end; m0 += 16 * MT) {
    const int left = min(sp.real_end - m0, 16 * MT);
    const __amdgpu_buffer_rsrc_t xsrc = buffer(a.xq + (base + m0) * row_bytes, left * row_bytes);
    // Blocks behind a row's end are the next row's (or zeros): their scales, of
    // both operands, are 2^-127, and what they add vanishes in fp32.
    const auto fill = [&](vec4u* st, int step) {
      const uint32_t at = step < steps ? step * 128u : 0x80000000u;  // nothing behind the last
#pragma unroll
      for (int i = 0; i < 2; ++i)
        load_lds16(wsrc, wat + i * 8 * row_bytes + blk16[i] + at, st + (w * 2 + i) * kLanes);
#pragma unroll
      for (int i = 0; i < kXLoads; ++i) {
        const int blk = (MT < 2 ? w & 1 : w * kXLoads + i);  // eight rows
        load_lds16(xsrc, (blk * 8 + (lane >> 3)) * row_bytes + blk16[MT < 2 ? w & 1 : i & 1] + at,
                   st + 64 * 8 + blk * kLanes);
      }
    };
    // Scales of 512 values of this thread's row (weights, then window rows);
    // unless K is Whole turns of them, byte by byte at the row's end.
    const uint8_t* const wscale = tid < kOut ? ws[0] : ws[1];
    const uint8_t* const scale_row =
        tid < 64 ? wscale + (int64_t)(n0 + min(tid % kOut, nr - 1)) * blocks
                 : a.xs + (base + m0 + min(tid - 64, left - 1)) * blocks;
    const auto get_scales = [&](int turn) {
      vec4u v = {0u, 0u, 0u, 0u};
      if (Whole) {
        __builtin_memcpy(&v, scale_row + min(turn * 16, blocks - 16), 16);
        if (turn * 16 >= blocks) v = vec4u{0u, 0u, 0u, 0u};
        return v;
      }
      if (tid >= kRows) return v;
      if (turn * 16 + 16 <= blocks) {
        __builtin_memcpy(&v, scale_row + turn * 16, 16);
      } else {
#pragma unroll 1
        for (int k = 0; k < 16; ++k) {  // bytes move in from the top
          const int n = turn * 16 + k;
          const uint32_t in = n < blocks ? scale_row[n] : 0u;
          v.x = v.x >> 8 | v.y << 24;
          v.y = v.y >> 8 | v.z << 24;
          v.z = v.z >> 8 | v.w << 24;
          v.w = v.w >> 8 | in << 24;
        }
      }
      return v;
    };
    vec4f acc[P][MT];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[p][m] = vec4f{0.0f, 0.0f, 0.0f, 0.0f};
    vec4u even = get_scales(0), odd = get_scales(1);
    fill(st0, 0);
    fill(st1, 1);
    fill(st2, 2);
    if (tid < kRows) sc[0][tid] = even;
    const int in_frag = (r16 >> 3) * 64 + (r16 & 7) * 8;
    const int shift = 8 * kb;
    // Values 128 * sub .. of a step: products of the wave's fragments; d picks
    // the scales' word of the turn's four.
    const auto products = [&](const vec4u* st, const vec4u (&sv)[P], const vec4u (&sx)[MT], int sub,
                              int d) {
      const int c = (4 * sub + kb) ^ (r16 >> 1);
      vec4u wv[P], xv[MT];
#pragma unroll
      for (int p = 0; p < P; ++p)
        wv[p] = st[(Swiglu ? p * 2 + (w & 1) : w) * 128 + in_frag + c];
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[m] = st[512 + m * 128 + in_frag + c];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        if (16 * m < left)
#pragma unroll
          for (int p = 0; p < P; ++p)
            acc[p][m] = mfma4(wv[p], xv[m], acc[p][m], sv[p][d] >> shift, sx[m][d] >> shift);
    };
    const auto both = [&](const vec4u* st, const vec4u (&sv)[P], const vec4u (&sx)[MT], int half) {
      if (Swiglu) {
        const int sub = w >> 1;
        if (sub == 0)
          products(st, sv, sx, 0, 2 * half);
        else
          products(st, sv, sx, 1, 2 * half + 1);
      } else {
        products(st, sv, sx, 0, 2 * half);
        products(st, sv, sx, 1, 2 * half + 1);
      }
    };
    vec4u sv[P], sx[MT];
    const auto read_scales = [&](int buf) {
#pragma unroll
      for (int p = 0; p < P; ++p) sv[p] = sc[buf][(Swiglu ? p * 32 + (w & 1) * 16 : w * 16) + r16];
#pragma unroll
      for (int m = 0; m < MT; ++m) sx[m] = sc[buf][64 + m * 16 + r16];
    };
    // Four steps, two turns of scales, a round; the buffer before THIS has been
    // read by every wave once the barrier is passed and takes the step after
    // the two on their way.
#define MOON_STEP(S, THIS, FREE)                       \
  {                                                    \
    wait_vm<2 * kLoads>();                             \
    wait_lds();                                        \
    asm volatile("" ::: "memory");                     \
    __builtin_amdgcn_s_barrier();                      \
    asm volatile("" ::: "memory");                     \
    fill(FREE, s + S + 3);                             \
    if (S == 0 || S == 2) read_scales(S / 2);          \
    both(THIS, sv, sx, S & 1);                         \
  }
#pragma unroll 1
    for (int s = 0; s < steps; s += 4) {
      even = get_scales(s / 2 + 2);  // on their way for three steps
      MOON_STEP(0, st0, st3)
      MOON_STEP(1, st1, st0)
      if (tid < kRows) sc[1][tid] = odd;
      odd = get_scales(s / 2 + 3);
      MOON_STEP(2, st2, st1)
      MOON_STEP(3, st3, st2)
      if (tid < kRows) sc[0][tid] = even;
    }
#undef MOON_STEP
    wait_vm<0>();
    __syncthreads();
    if (Swiglu) {
      vec4f* const red = reinterpret_cast<vec4f*>(st0);
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (w >= 2) red[(((w & 1) * P + p) * MT + m) * kLanes + lane] = acc[p][m];
      __syncthreads();
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (w < 2) acc[p][m] += red[((w * P + p) * MT + m) * kLanes + lane];
    }
    if (!Swiglu || w < 2) {
      const int col = n0 + w * 16 + 4 * kb;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = 16 * m + r16;
        if (row < left && col < a.N) {
          const int64_t at = base + m0 + row;
          vec4f o = acc[0][m];
          if (Swiglu) o = gated(o, acc[P - 1][m], a.row_w != nullptr ? a.row_w[at] : 1.0f);
          *reinterpret_cast<vec2u*>(a.y + at * a.N + col) = round4(o);
        }
      }
    }
    __syncthreads();  // LDS is free for the next rows
  }
}

// ---- many rows per group: tiles of 256 weight rows by 256 window rows ----

constexpr int kTileWaves = 8;
constexpr int kTileThreads = kTileWaves * kLanes;
constexpr int kTile = 256;
constexpr int kMaxEntries = 1024;  // of the tile table

// The thread's index as a value the compiler knows nothing of: what follows
// from it is worked out where it is used, not kept in registers across the
// main loop, which needs them all.
__device__ __forceinline__ int fresh_thread_id() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// One tile of results; every field is the same in all lanes.
struct Tile {
  int u, j;          // rank and entry
  int row0, n0;      // first window row (local) and first output
  int rows;          // rows from row0 to the group's last route
  int pad;           // padding rows to clear behind them, 0 but for the last row tile
};

// Scale bytes of 512 values (16 blocks) as the matrix cores take them: word kb
// holds the blocks kb, 4 + kb, 8 + kb, 12 + kb, the lane group's block in each
// of four steps.
__device__ __forceinline__ vec4u transpose_scales(vec4u d) {
  const uint32_t a0 = __builtin_amdgcn_perm(d.y, d.x, 0x05010400u);  // x0 y0 x1 y1
  const uint32_t a1 = __builtin_amdgcn_perm(d.y, d.x, 0x07030602u);  // x2 y2 x3 y3
  const uint32_t b0 = __builtin_amdgcn_perm(d.w, d.z, 0x05010400u);
  const uint32_t b1 = __builtin_amdgcn_perm(d.w, d.z, 0x07030602u);
  const vec4u o = {__builtin_amdgcn_perm(b0, a0, 0x05040100u),
                   __builtin_amdgcn_perm(b0, a0, 0x07060302u),
                   __builtin_amdgcn_perm(b1, a1, 0x05040100u),
                   __builtin_amdgcn_perm(b1, a1, 0x07060302u)};
  return o;
}

template <int Step>
__device__ __forceinline__ vec16f mfma32(vec4u a, vec4u b, vec16f c, uint32_t sa, uint32_t sb) {
  const vec8i av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const vec8i bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, Step, (int)sa, Step,
                                                         (int)sb);
}

// Half a step of a wave (64 values): 8 products of its four weight and two row
// fragments f, while the fragments n of the next half come from LDS.  The
// schedule puts two reads before each of the first three pairs of products, so
// they have arrived when the half ends.
template <int Step>
__device__ __forceinline__ void half_step(const vec4u* wsrc, const vec4u* xsrc, const vec4u (&f)[6],
                                          vec4u (&n)[6], const uint32_t (&s)[6],
                                          vec16f (&acc)[4][2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) n[i] = wsrc[i * 2 * kLanes];
#pragma unroll
  for (int i = 0; i < 2; ++i) n[4 + i] = xsrc[i * 2 * kLanes];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i][k] = mfma32<Step>(f[i], f[4 + k], acc[i][k], s[i], s[4 + k]);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < 3) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
  }
}

// A workgroup of eight waves (two per SIMD) walks tiles of 256 weight rows by
// 256 window rows; each wave owns 128 by 64 of them (128 accumulators a lane,
// v_mfma_scale_f32_32x32x64).  K advances by 128 values a step, four steps to a
// turn of 512.  LDS holds four steps of both operands: a load straight into it
// writes 16 rows by four scale blocks in lane order, four lanes a row so that
// they share its 64 bytes (with a row per lane, 16 lines for 16 lanes, the
// first cache took twice the time of the products); the blocks of a row are
// stored swapped by its index, so that ds_read_b128 of 16 rows meets no bank
// twice.  Each step refills the buffer it has just emptied with the same step
// of the next turn, which may belong to the next tile: the loads run three
// steps ahead without a pause at tile borders.
//
// Gate and up products of 262144 rows, K=7168, F=2048 in 288 groups take 4.2 ms
// (3.7 PFLOP/s, 4.2 with the unused rows of the groups' last tiles, 12 % of the
// tiles' rows); a library's product of two 16384 x 16384 MXFP4 matrices reaches
// 3.2 PFLOP/s on the same card.  The matrix cores are busy 60 % of the cycles, and
// the clock, 2.4 GHz at most, is 1.5 to 1.7 GHz under this load (2.1 under slower
// variants of it).  Tried and slower:
// four waves of 128 by 128 (256 accumulators: spills, or waits that drain the
// loads), 128 bytes of a row a load with two steps ahead, loads into the caches
// further ahead, a raised wave priority, leaving out the products of rows that
// a last tile lacks.
// Products of K=1024 (98304 rows, N=2048, 97 groups) take 186 to 197 us; in one
// run 195, of which 123 without the epilogue and 148 with its stores dropped.  No
// faster there: the next tile's
// first steps not waiting for the stores, whole cache lines a store (205 us),
// non-temporal stores (202 us).
template <bool Swiglu, bool Whole>
__global__ void __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
    k_expert_tiles(ExpertArgs a, Groups g) {
  constexpr int kOut = Swiglu ? kTile / 2 : kTile;  // outputs per tile
  __shared__ vec4u st0[32 * kLanes], st1[32 * kLanes], st2[32 * kLanes], st3[32 * kLanes];
  __shared__ uint32_t sc[2][32 * kLanes];
  __shared__ int32_t first[kMaxEntries + 1];
  __shared__ int32_t wave_total[kTileWaves];
  __shared__ vec4u turned[kTileWaves][kLanes];
  if (g.status[0] != 0) return;
  const int tid = threadIdx.x, lane = tid & (kLanes - 1);
  const int w = __builtin_amdgcn_readfirstlane(tid / kLanes);
  const int chunk = (lane & 3) ^ (lane >> 4);  // scale block that this lane loads

  // Row tiles before every entry: a scan over the groups' sizes.
  const int entries = g.R * g.per, nt = (a.N + kOut - 1) / kOut;
  {
    const int each = (entries + kTileThreads - 1) / kTileThreads;
    int sum = 0;
    for (int i = 0; i < each; ++i) {
      const int e = tid * each + i;
      if (e >= entries) break;
      const Span s = group_span(g, e / g.per, e % g.per);
      // (padding without a route still has a tile, which clears it)
      const int t = max((s.real_end - s.begin + kTile - 1) / kTile, s.end > s.begin ? 1 : 0);
      first[e + 1] = t;
      sum += t;
    }
    int incl = sum;
    for (int k = 1; k < kLanes; k *= 2) {
      const int o = __shfl_up(incl, k);
      if (lane >= k) incl += o;
    }
    if (lane == kLanes - 1) wave_total[w] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int i = 0; i < w; ++i) before += wave_total[i];
    for (int i = 0; i < each; ++i) {
      const int e = tid * each + i;
      if (e >= entries) break;
      before += first[e + 1];
      first[e + 1] = before;
    }
    if (tid == 0) first[0] = 0;
    __syncthreads();
  }
  // Consecutive tiles share weights or rows, so each XCD (workgroups go round
  // the eight) takes one run of them: its L2 serves the sharing.
  const int total = first[entries] * nt;
  const int xcd = blockIdx.x & 7, xn = gridDim.x >> 3;
  const int t_end = (int)((int64_t)total * (xcd + 1) / 8);
  int t_load = (int)((int64_t)total * xcd / 8) + (int)(blockIdx.x >> 3);
  if (t_load >= t_end) return;

  // Tile t, which is never before the one asked for last: its entry is looked
  // for from there on.
  int entry = 0;
  const auto find = [&](int t) {
    const int mt = t / nt;
    while (first[entry + 1] <= mt) ++entry;
    entry = uniform(entry);
    const int before = uniform(first[entry]), m_tiles = uniform(first[entry + 1]) - before;
    const int in = t - before * nt, n = in / m_tiles, m = in - n * m_tiles;
    const Span sp = group_span(g, entry / g.per, entry % g.per);
    Tile o;
    o.u = entry / g.per;
    o.j = entry % g.per;
    o.n0 = n * kOut;
    o.row0 = sp.begin + m * kTile;
    o.rows = sp.real_end - o.row0;
    o.pad = m == m_tiles - 1 ? sp.end - sp.real_end : 0;
    return o;
  };

  const int blocks = a.K / 32, turns = (blocks + 15) / 16;
  // Load cursor: the wave's operand (waves 0 to 3 take the weights, two
  // fragments each, the others the window rows) and its scales as buffers that
  // end with the tile's last row, so rows behind it read as zeros.
  const bool is_w = w < 4;
  __amdgpu_buffer_rsrc_t src, src_scales;
  const uint8_t* src_scale;
  // Output that row m (0..31) of weight fragment f (0..7, four a wave) is for;
  // with a gate two gate fragments and the up fragments of the same outputs
  // alternate.  Row m = 8 q + 4 h + i of the product is register 4 q + i of the
  // lanes of half h.
  const auto weight_row = [&](int f, int m) {
    const int h = (m >> 2) & 1, r = (m >> 3) * 4 + (m & 3);
    return (Swiglu ? (f >> 2) * 64 + (f & 1) * 32 : f * 32) + h * 16 + r;
  };
  const uint32_t row_bytes = 16u * blocks;
  const auto point = [&](Tile& t) {
    t.row0 = uniform(t.row0);
    t.rows = uniform(t.rows);
    t.pad = uniform(t.pad);
    const uint8_t *wq[2], *ws[2];
    weight_of(g, a.w[0], t.u, t.j, a.N, a.K, &wq[0], &ws[0]);
    weight_of(g, a.w[Swiglu ? 1 : 0], t.u, t.j, a.N, a.K, &wq[1], &ws[1]);
    const int64_t base = (int64_t)t.u * g.NvS + t.row0;
    const int nr = min(a.N - t.n0, kOut), mr = min(t.rows, kTile);
    const uint32_t rows = is_w ? nr : mr;
    const uint8_t* const q = Swiglu && (w & 1) ? wq[1] : wq[0];
    const uint8_t* const sq = Swiglu && (w & 1) ? ws[1] : ws[0];
    src = buffer(is_w ? q + (int64_t)t.n0 * row_bytes : a.xq + base * row_bytes, rows * row_bytes);
    if (Whole) {
      src_scales = buffer(is_w ? sq + (int64_t)t.n0 * blocks : a.xs + base * blocks, rows * blocks);
    } else {  // a row per thread, in the order of the fragments
      const int tid = fresh_thread_id(), f = (tid >> 4) & 15, r = tid & 15;
      src_scale = is_w ? ((f >> 2) & 1 ? ws[1] : ws[0]) +
                             (int64_t)(t.n0 + min(weight_row(f >> 1, (f & 1) * 16 + r), nr - 1)) * blocks
                       : a.xs + (base + max(min(tid - kTile, mr - 1), 0)) * blocks;
    }
  };

  // Codes of one step.  Blocks behind a row's end are those of the next row (or
  // zeros): 4-bit codes are all finite, and the scales 2^-127 of both operands
  // there make what they add (below 2^-240) vanish in fp32.
  const int r16 = lane >> 2;
  const uint32_t code_at = (is_w ? weight_row(w * 2, r16) : (w - 4) * 64 + r16) * row_bytes +
                           16 * chunk;
  const auto fill = [&](vec4u* dst, int turn, int step) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // rows of block i, relative to the first's
      const int rows = is_w ? (i >> 1) * 32 + (i & 1) * 8 : i * 16;
      load_lds16(src, code_at + (rows * row_bytes + turn * 256 + step * 64),
                 dst + (w * 4 + i) * kLanes);
    }
  };
  // Scales of one turn: 16 bytes of the thread's row; unless K is Whole turns,
  // a row's last blocks byte by byte, with 2^-127 behind them.
  const int scale_at = (tid >> 4) * kLanes + (tid & 15);
  const auto get_scales = [&](int turn) {
    vec4u v;
    if (turn * 16 + 16 <= blocks) {
      __builtin_memcpy(&v, src_scale + turn * 16, 16);
    } else {
      v = vec4u{0u, 0u, 0u, 0u};
#pragma unroll 1
      for (int k = 0; k < 16; ++k) {  // bytes move in from the top
        const int n = turn * 16 + k;
        const uint32_t in = n < blocks ? src_scale[n] : 0u;
        v.x = v.x >> 8 | v.y << 24;
        v.y = v.y >> 8 | v.z << 24;
        v.z = v.z >> 8 | v.w << 24;
        v.w = v.w >> 8 | in << 24;
      }
    }
    return v;
  };
  const auto put_scales = [&](int b, vec4u v) {
    const vec4u t = transpose_scales(v);
#pragma unroll
    for (int k = 0; k < 4; ++k) sc[b][scale_at + 16 * k] = t[k];
  };

  // Scales of whole turns, two of them (32 bytes of a row) at a time straight
  // into LDS, as they lie in memory: two lanes a row, 512 rows.
  vec4u* const raw = reinterpret_cast<vec4u*>(&sc[0][0]);
  const uint32_t scales_at = (is_w ? weight_row(w * 2, lane >> 1) : (w - 4) * 64 + (lane >> 1)) *
                                 blocks + 16 * (lane & 1);
  const auto fill_scales = [&](int turn) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      load_lds16(src_scales, scales_at + (i * 32 * blocks + turn * 16), raw + (w * 2 + i) * kLanes);
  };

  // This wave's fragments (32 rows, two blocks of 16): weights (w & 1)*4 ..,
  // window rows 8 + (w >> 1)*2 ..; a lane holds row lane % 32 and, of the four
  // scale blocks of a step, 2 * half + lane / 32.
  vec16f acc[4][2];
  vec4u fa[6], fb[6];
  uint32_t sr[2][6], sr_next[2][6];
  const int wfrag = (w & 1) * 8 * kLanes, xfrag = (16 + (w >> 1) * 4) * kLanes;
  const int in_block = ((lane >> 4) & 1) * kLanes + (lane & 15) * 4;
  const int in0 = in_block + ((lane >> 5) ^ ((lane >> 2) & 3)), in1 = in0 ^ 2;
  const int scale_in = ((lane >> 4) & 1) * kLanes + (lane >> 5) * 16 + (lane & 15);
  // bytes h and 2 + h, the blocks of this half of the lanes, of two words
  const uint32_t pick = 0x06020400u + 0x01010101u * (lane >> 5);
  const auto read_scales = [&](int b, int turn, uint32_t(&s)[2][6]) {
    if (Whole) {
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        const vec4u d = raw[((i < 4 ? wfrag : xfrag) >> 1) + (i & 3) * kLanes +
                            (lane & 31) * 2 + (turn & 1)];
        const uint32_t lo = __builtin_amdgcn_perm(d.y, d.x, pick);
        const uint32_t hi = __builtin_amdgcn_perm(d.w, d.z, pick);
        s[0][i] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
        s[1][i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
      }
      return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 6; ++i)
        s[h][i] = sc[b][(i < 4 ? wfrag : xfrag) + scale_in + (i & 3) * 2 * kLanes + 32 * h];
  };

  {  // the first tile's entry, by halves
    const int mt = t_load / nt;
    int hi = entries;  // first[entry] <= mt < first[hi]
    while (hi - entry > 1) {
      const int mid = (entry + hi) / 2;
      if (first[mid] <= mt)
        entry = mid;
      else
        hi = mid;
    }
  }
  Tile cur = find(t_load), next;
  point(cur);
  {
    vec4u v = {};
    if (Whole)
      fill_scales(0);
    else
      v = get_scales(0);
    fill(st0, 0, 0);
    fill(st1, 0, 1);
    fill(st2, 0, 2);
    fill(st3, 0, 3);
    if (!Whole) put_scales(0, v);
  }
  wait_vm<0>();  // this wave's part is in LDS before the others read it
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 6; ++i)
    fa[i] = st0[(i < 4 ? wfrag : xfrag) + in0 + (i & 3) * 2 * kLanes];
  read_scales(0, 0, sr);
  int buf = 0;
  bool more = true;  // a tile is left to load
  while (true) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][k][r] = 0.0f;
    // The next tile is looked up now, so that what it needs from memory is here
    // when its loads begin.
    t_load += xn;
    more = t_load < t_end;
    next = cur;
    if (more) next = find(t_load);
#pragma unroll 1
    for (int turn = 0; turn < turns; ++turn) {
      // The turn to load: the next of this tile, or the first of the next
      // tile; behind the last one it is loaded again, for nothing.
      int turn_load = turn + 1;
      if (turn_load == turns) {
        turn_load = 0;
        if (more) point(next);
      }
      vec4u v = {};
      if (!Whole) v = get_scales(turn_load);
      // In the middle of a step its second half has been read (by every wave,
      // behind the barrier), so its buffer is free, and the next step's data,
      // all but the last two steps' loads (8 of this wave), has landed.
#define MOON_STEP(S, THIS, NEXT)                                                       \
  {                                                                                    \
    wait_lds();                                                                        \
    half_step<S>(THIS + wfrag + in1, THIS + xfrag + in1, fa, fb, sr[0], acc);                 \
    __builtin_amdgcn_sched_barrier(0);                                                 \
    wait_lds();                                                                        \
    wait_vm<8>();                                                                      \
    asm volatile("" ::: "memory");                                                     \
    __builtin_amdgcn_s_barrier();                                                      \
    asm volatile("" ::: "memory");                                                     \
    __builtin_amdgcn_sched_barrier(0);                                                 \
    if (Whole && S == 0 && (turn_load & 1) == 0) fill_scales(turn_load);               \
    fill(THIS, turn_load, S);                                                          \
    if (!Whole && S == 2) put_scales(buf ^ 1, v);                                      \
    if (S == 3) read_scales(buf ^ 1, turn_load, sr_next);                              \
    half_step<S>(NEXT + wfrag + in0, NEXT + xfrag + in0, fb, fa, sr[1], acc);                     \
    __builtin_amdgcn_sched_barrier(0);                                                 \
  }
      MOON_STEP(0, st0, st1)
      MOON_STEP(1, st1, st2)
      MOON_STEP(2, st2, st3)
      MOON_STEP(3, st3, st0)
#undef MOON_STEP
      buf ^= 1;
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        sr[0][i] = sr_next[0][i];
        sr[1][i] = sr_next[1][i];
      }
    }
    const int64_t base = (int64_t)cur.u * g.NvS + cur.row0;
    // A lane holds 16 neighbouring outputs of one row per fragment; through LDS,
    // 16 rows at a time, four lanes get a row's 64 bytes, so that a store writes
    // whole segments.
    const int lane = fresh_thread_id() & (kLanes - 1);
    const int row = lane & 31, col = cur.n0 + (w & 1) * (kOut / 2);
    vec4u* const put = &turned[w][(lane & 15) * 4];
    const int swap = (lane >> 2) & 3, half = lane >> 5;
    const int out_row = lane >> 2, out_col = ((lane & 3) ^ (lane >> 4)) * 8;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int m = (w >> 1) * 64 + k * 32;
      const float rw = Swiglu && a.row_w != nullptr && m + row < cur.rows
                           ? a.row_w[base + m + row] : 1.0f;
#pragma unroll
      for (int i = 0; i < (Swiglu ? 2 : 4); ++i) {
        vec4u v[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float o[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            o[r] = acc[i][k][8 * q + r];
            if (Swiglu) o[r] = rw * (o[r] * sigmoid_f32(o[r]) * acc[(i + 2) & 3][k][8 * q + r]);
          }
          v[q] = vec4u{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                       pack_bf16(o[6], o[7])};
        }
        vec4u p[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (((lane >> 4) & 1) == j) {
            put[(2 * half) ^ swap] = v[0];
            put[(2 * half + 1) ^ swap] = v[1];
          }
          wave_lds_sync();
          p[j] = turned[w][lane];
          wave_lds_sync();
        }
        const int c = col + 32 * i + out_col;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = m + 16 * j + out_row;
          if (r < cur.rows && c < a.N) *reinterpret_cast<vec4u*>(a.y + (base + r) * a.N + c) = p[j];
        }
      }
    }
    zero_rows(a.y, base + cur.rows, cur.pad, a.N, cur.n0, kOut);
    if (!more) break;
    cur = next;
  }
  wait_vm<0>();  // nothing may land in LDS after the workgroup has left
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
  // By the rows an expert gets on average, over K=2048, N=7168, E=256 (R=8, 288
  // groups; us by 16 rows at a time, by 64 and by tiles of 256):
  //   2 rows 320/367/415, 8 rows 420/472/537, 16 rows 477/474/550,
  //   32 rows 663/513/578, 64 rows 1107/647/591, 128 rows 2087/1041/667.
  // The counts themselves are on the GPU; any group is right in any kernel.
  // More entries than the tile table holds go by 64 rows at a time (R=32, E=512,
  // 128 rows an expert, K=2048, gate and up to N=1024: 513 us by tiles with 1024
  // entries, 690 with 1056).
  const int64_t rows = (int64_t)g.R * g.N;
  if (rows >= 48 * (int64_t)g.E && g.R * g.per <= kMaxEntries) {
    int dev = 0, cus = 256;
    if (hipGetDevice(&dev) == hipSuccess)
      (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    const int wgs = std::max(8, cus / 8 * 8);
    // whole turns of scales go straight into LDS, from whole 16 bytes
    bool whole = a.K % 512 == 0 && is_aligned(a.xs, 16);
    for (int p = 0; p < (Swiglu ? 2 : 1); ++p)
      whole = whole && is_aligned(a.w[p].es, 16) && is_aligned(a.w[p].ss, 16);
    if (whole)
      hipLaunchKernelGGL((k_expert_tiles<Swiglu, true>), dim3(wgs), dim3(kTileThreads), 0, s, a, g);
    else
      hipLaunchKernelGGL((k_expert_tiles<Swiglu, false>), dim3(wgs), dim3(kTileThreads), 0, s, a, g);
    return hipGetLastError() == hipSuccess ? MOON_OK : MOON_ERR_HIP;
  }
  // K that is not whole turns of 512 values has its row's last scales read byte
  // by byte, in either kind of kernel, and costs as much as the next whole K or
  // more (us; whole K last):
  //   16 rows at a time, R=8, E=256, S=16, N=7168: K=1056 350, 1408 408, 1536 325;
  //     2880 702, 3584 696
  //   tiles, R=8, E=256, S=4096, gate and up to N=2048: K=1056 1357, 1408 1380,
  //     1536 1250; 2880 2456, 3584 2297
  const dim3 grid(Swiglu ? (a.N + 31) / 32 : (a.N + 63) / 64, g.R * g.per);
  const bool few = rows <= 12 * (int64_t)g.E;
  if (a.K % 512 == 0) {
    if (few)
      hipLaunchKernelGGL((k_expert_stream<1, Swiglu, true>), grid, dim3(256), 0, s, a, g);
    else
      hipLaunchKernelGGL((k_expert_stream<4, Swiglu, true>), grid, dim3(256), 0, s, a, g);
  } else {
    if (few)
      hipLaunchKernelGGL((k_expert_stream<1, Swiglu, false>), grid, dim3(256), 0, s, a, g);
    else
      hipLaunchKernelGGL((k_expert_stream<4, Swiglu, false>), grid, dim3(256), 0, s, a, g);
  }
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
