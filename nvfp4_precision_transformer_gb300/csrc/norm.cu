// Root-mean-square norm with the residual's addition and an 8-bit output, and its gradient.
//
//   forward   s = x + residual;  rsigma = 1 / sqrt(mean(s^2) + eps);  y = (s * rsigma) * gamma
//             outputs: s, y in bf16, y in FP8 (per-tensor scale) or MXFP8 (1 x 32 blocks), rsigma
//   backward  xhat = s * rsigma, p = dy * gamma:
//             ds = rsigma * (p - xhat * mean(p * xhat)) (+ the residual stream's own gradient)
//             dgamma = sum over the rows of dy * xhat
//
// Both are bound by HBM (15872 x 4096 bf16 on 6.8 TB/s: forward with every output and MXFP8 88 us in the
// kernel, 6.65 TB/s; backward with dgamma's sums 82 us a call, 6.3 TB/s).  A row belongs to WPR warps
// (1 to 16), each lane holding up to four (backward: two) chunks of eight columns in registers, so
// every tensor is read once; the row's sum is a butterfly over the lanes and one exchange through
// shared memory between the row's warps.  Groups walk the rows with the grid's stride, the next row's
// loads in flight while one is reduced and written; gamma comes from L1 (backward: shared memory).  All
// sums are fp32 in a fixed order, so results do not depend on timing.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "convert.cuh"
#include "launch_setup.cuh"

namespace te {
namespace {

constexpr int kCh = 4;                       // chunks of eight columns per lane
constexpr int kWarpCols = 32 * 8 * kCh;      // columns of a row per warp
constexpr int64_t kMaxCols = 16 * kWarpCols;
constexpr int64_t kMaxPartials = 512;        // rows of partial column sums in the workspace

// Warps of a CTA when a row takes `wpr` of them, and the rows that it works on at a time.
__host__ __device__ constexpr int cta_warps(int wpr) { return wpr < 8 ? 8 : wpr; }
__host__ __device__ constexpr int cta_rows(int wpr) { return cta_warps(wpr) / wpr; }

// Eight consecutive elements, as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t w = i == 0 ? a.x : (i == 1 ? a.y : (i == 2 ? a.z : a.w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float2 pair(int i) const {
    return i == 0 ? make_float2(a.x, a.y) : (i == 1 ? make_float2(a.z, a.w)
                                                     : (i == 2 ? make_float2(b.x, b.y) : make_float2(b.z, b.w)));
  }
};

__device__ __forceinline__ uint32_t bf16x2(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2 (&v)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(v[0]), bf16x2(v[1]), bf16x2(v[2]), bf16x2(v[3]));
}
__device__ __forceinline__ void store8(float* p, const float2 (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
__device__ __forceinline__ void ld8(const float* p, float2 (&v)[4]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w);
  v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Sum over the WPR warps of a row, in warp order.  `red` has two slots (`turn` alternates
// between them), so that one barrier a row is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[WPR], int turn, int grp, int wr, int lane) {
  v = warp_sum(v);
  if (WPR == 1) return v;
  if (lane == 0) red[turn][wr] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * WPR) : "memory");
  float t = red[turn][0];
#pragma unroll
  for (int w = 1; w < WPR; ++w) t = __fadd_rn(t, red[turn][w]);
  return t;
}

struct NormArgs {
  const void* x;
  const void* res;
  const float* gamma;
  float eps;
  int64_t rows, cols;
  __nv_bfloat16* y;
  void* res_out;
  float* rsigma;
  uint8_t* q;
  const float* scale;      // FP8
  int e5m2;
  unsigned int* amax;
  float* scale_inv;
  int amax_whole;          // 1: the grid is one CTA, which writes the amax itself
  uint8_t* s_row;          // MXFP8
  int64_t kpad, rpad;
};

// The maximum of |y| is kept as bits (ordered as the non-negative floats are), so a NaN, whose
// bits are above infinity's, is not lost.
template <typename T, int WPR, bool MX>
__global__ void __launch_bounds__(32 * cta_warps(WPR), WPR <= 8 ? 2 : 1) rmsnorm_kernel(NormArgs a) {
  constexpr int GR = cta_rows(WPR);
  __shared__ float red[GR][2][WPR];
  __shared__ unsigned int top[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp / WPR, wr = warp % WPR;
  const int64_t C = a.cols;
  const int64_t step = static_cast<int64_t>(gridDim.x) * GR;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  const int col0 = (wr * kCh * 32 + lane) * 8;   // chunk t starts at col0 + 256 t
  dev::pdl_wait();
  dev::pdl_trigger();
  const float sc = !MX && a.scale ? *a.scale : 1.0f;
  unsigned int lmax = 0;

  Raw8<T> rx[kCh], rr[kCh];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int t = 0; t < kCh; ++t) {
      const int col = col0 + 256 * t;
      rx[t].zero();
      rr[t].zero();
      if (row < a.rows && col < C) {
        rx[t].load(x + row * C + col);
        if (res) rr[t].load(res + row * C + col);
      }
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * GR + grp;
  load(row);
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    float2 v[kCh][4];
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int t = 0; t < kCh; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[t][i] = res ? __fadd2_rn(rx[t].pair(i), rr[t].pair(i)) : rx[t].pair(i);
        sq = __ffma2_rn(v[t][i], v[t][i], sq);
      }
    load(row + step);   // the next row's loads are in flight while this one is reduced and written
    const float sum = row_sum<WPR>(__fadd_rn(sq.x, sq.y), red[grp], turn, grp, wr, lane);
    const float rs = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(C)), a.eps)));
    if (a.rsigma && wr == 0 && lane == 0) a.rsigma[row] = rs;
    const float2 rs2 = make_float2(rs, rs);
#pragma unroll
    for (int t = 0; t < kCh; ++t) {
      const int col = col0 + 256 * t;
      const bool live = col < C;
      const int64_t at = row * C + col;
      float2 g[4] = {}, y[4];
      if (live) ld8(a.gamma + col, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = __fmul2_rn(__fmul2_rn(v[t][i], rs2), g[i]);
      if (live && a.res_out) store8(static_cast<T*>(a.res_out) + at, v[t]);
      if (live && a.y) store8(a.y + at, y);
      unsigned int m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m = max(m, max(__float_as_uint(y[i].x) & 0x7FFFFFFFu, __float_as_uint(y[i].y) & 0x7FFFFFFFu));
      float mul = sc;
      if (MX) {
        // a block of 32 columns is four neighbouring lanes' chunks (cols % 32 == 0: all live or none)
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const int e = mx_exponent(__uint_as_float(m));
        mul = mx_mult(e);
        if (live && (lane & 3) == 0)
          a.s_row[scale_offset(static_cast<uint64_t>(row), static_cast<uint64_t>(col >> 5),
                               static_cast<uint64_t>(a.kpad))] = static_cast<uint8_t>(e + 127);
      } else if (live) {
        lmax = max(lmax, m);
      }
      if (live && a.q) {
        const float2 m2 = make_float2(mul, mul);
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 p = __fmul2_rn(y[2 * h], m2), r = __fmul2_rn(y[2 * h + 1], m2);
          w[h] = (!MX && a.e5m2) ? (cvt_e5m2x2(p.x, p.y) | (cvt_e5m2x2(r.x, r.y) << 16))
                                 : (cvt_e4m3x2(p.x, p.y) | (cvt_e4m3x2(r.x, r.y) << 16));
        }
        *reinterpret_cast<uint2*>(a.q + at) = make_uint2(w[0], w[1]);
      }
    }
    if (MX && wr == 0 && lane == 0)   // padding columns of this row's scales
      for (int64_t j = C / 32; j < a.kpad; ++j)
        a.s_row[scale_offset(static_cast<uint64_t>(row), static_cast<uint64_t>(j), static_cast<uint64_t>(a.kpad))] = 0;
  }
  if (MX) {
    // padding rows, four scale columns a word
    const int64_t words = (a.rpad - a.rows) * (a.kpad / 4);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < words;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
      *reinterpret_cast<uint32_t*>(a.s_row + scale_offset(static_cast<uint64_t>(a.rows + i / (a.kpad / 4)),
                                                          static_cast<uint64_t>(i % (a.kpad / 4) * 4),
                                                          static_cast<uint64_t>(a.kpad))) = 0u;
    return;
  }
  if (a.scale_inv && blockIdx.x == 0 && threadIdx.x == 0) *a.scale_inv = __fdiv_rn(1.0f, sc);
  if (a.amax) {
    lmax = __reduce_max_sync(0xFFFFFFFFu, lmax);
    if (lane == 0) top[warp] = lmax;
    __syncthreads();
    if (warp == 0) {
      lmax = __reduce_max_sync(0xFFFFFFFFu, lane < cta_warps(WPR) ? top[lane] : 0u);
      if (lane == 0) {
        if (a.amax_whole) {
          *a.amax = lmax;
        } else {
          atomicMax(a.amax, lmax);
        }
      }
    }
  }
}

struct NormBwdArgs {
  const __nv_bfloat16* dy;
  const void* s;
  const void* dres;
  const float* gamma;
  const float* rsigma;
  int64_t rows, cols;
  void* dx;
  float* partial;   // [gridDim.x, cols]
};

// Two chunks a lane and two CTAs per SM, with the next row in flight in bf16 (15872 x 4096, of one early build,
// 87.7 us; without it 105.1, four chunks 96.7, three CTAs 94.2 and, with it, spilled, 132.5).  In fp32
// the second row would take the registers of the second CTA's warps: 151 us without, 152 with it
// (30000 x 768: 59.9 / 74.7), four chunks 217.  Now: fp32 143 us and 54.
template <typename T, int WPR, int CH>
__global__ void __launch_bounds__(32 * cta_warps(WPR), WPR <= 8 ? 2 : 1) rmsnorm_bwd_kernel(NormBwdArgs a) {
  constexpr int GR = cta_rows(WPR);
  constexpr bool kAhead = sizeof(T) == 2 && CH == 2;   // the next row's loads before this row is reduced
  __shared__ float red[GR][2][WPR];
  extern __shared__ __align__(16) float cols_sum[];   // [GR - 1][cols], then gamma
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp / WPR, wr = warp % WPR;
  const int64_t C = a.cols;
  const int64_t step = static_cast<int64_t>(gridDim.x) * GR;
  const T* s = static_cast<const T*>(a.s);
  const T* dres = static_cast<const T*>(a.dres);
  const int col0 = (wr * CH * 32 + lane) * 8;
  float2 dg[CH][4];
#pragma unroll
  for (int t = 0; t < CH; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[t][i] = make_float2(0.f, 0.f);

  struct RowRegs {
    Raw8<__nv_bfloat16> d[CH];
    Raw8<T> x[CH], r[CH];
    float rs;
  };
  auto load = [&](RowRegs& q, int64_t row) {
    q.rs = row < a.rows ? a.rsigma[row] : 0.0f;
#pragma unroll
    for (int t = 0; t < CH; ++t) {
      const int col = col0 + 256 * t;
      q.d[t].zero();
      q.x[t].zero();
      q.r[t].zero();
      if (row < a.rows && col < C) {
        q.d[t].load(a.dy + row * C + col);
        q.x[t].load(s + row * C + col);
        if (dres) q.r[t].load(dres + row * C + col);
      }
    }
  };
  dev::pdl_wait();
  // gamma once into shared memory, the two halves of its chunks of eight apart (reads without bank conflicts):
  // loaded from L1 in every row it waits behind the stores, which ordinary loads do not pass (15872 x 4096 bf16
  // 98.8 us a call, in registers 84.8, so 82.2-82.9; 4000 x 16384 fp32, four chunks a lane, 229 from L1, so 165)
  float4* sgam = reinterpret_cast<float4*>(cols_sum + (GR - 1) * C);
  const int chunks = static_cast<int>(C >> 3);
  for (int i = threadIdx.x; i < 2 * chunks; i += blockDim.x)
    sgam[(i & 1) * chunks + (i >> 1)] = reinterpret_cast<const float4*>(a.gamma)[i];
  auto gamma8 = [&](int col, float2 (&g)[4]) {
    const float4 u = sgam[col >> 3], v = sgam[chunks + (col >> 3)];
    g[0] = make_float2(u.x, u.y), g[1] = make_float2(u.z, u.w);
    g[2] = make_float2(v.x, v.y), g[3] = make_float2(v.z, v.w);
  };
  RowRegs cur;
  int64_t row = static_cast<int64_t>(blockIdx.x) * GR + grp;
  if (kAhead) load(cur, row);
  __syncthreads();
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    RowRegs nxt;
    if (kAhead) load(nxt, row + step);
    else load(cur, row);
    const float2 rs2 = make_float2(cur.rs, cur.rs);
    float2 dot = make_float2(0.f, 0.f);
#pragma unroll
    for (int t = 0; t < CH; ++t) {
      const int col = col0 + 256 * t;
      float2 g[4] = {};
      if (col < C) gamma8(col, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 w = __fmul2_rn(cur.d[t].pair(i), __fmul2_rn(cur.x[t].pair(i), rs2));   // dy * xhat
        dg[t][i] = __fadd2_rn(dg[t][i], w);
        dot = __ffma2_rn(w, g[i], dot);
      }
    }
    const float sum = row_sum<WPR>(__fadd_rn(dot.x, dot.y), red[grp], turn, grp, wr, lane);
    const float c = -__fdiv_rn(sum, static_cast<float>(C));
    const float2 c2 = make_float2(c, c);
#pragma unroll
    for (int t = 0; t < CH; ++t) {
      const int col = col0 + 256 * t;
      if (col >= C) break;
      float2 g[4], o[4];
      gamma8(col, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = __fmul2_rn(cur.d[t].pair(i), g[i]);
        const float2 d = __ffma2_rn(__fmul2_rn(cur.x[t].pair(i), rs2), c2, p);
        o[i] = __ffma2_rn(d, rs2, cur.r[t].pair(i));
      }
      store8(static_cast<T*>(a.dx) + row * C + col, o);
    }
    if (kAhead) cur = nxt;
  }
  dev::pdl_trigger();
  // the CTA's column sums: the row groups in order
  if (GR > 1) {
    if (grp > 0) {
#pragma unroll
      for (int t = 0; t < CH; ++t)
        if (col0 + 256 * t < C) store8(cols_sum + (grp - 1) * C + col0 + 256 * t, dg[t]);
    }
    __syncthreads();
    if (grp > 0) return;
    for (int k = 0; k < GR - 1; ++k)
#pragma unroll
      for (int t = 0; t < CH; ++t) {
        const int col = col0 + 256 * t;
        if (col >= C) break;
        const float4 u = *reinterpret_cast<const float4*>(cols_sum + k * C + col);
        const float4 w = *reinterpret_cast<const float4*>(cols_sum + k * C + col + 4);
        dg[t][0] = __fadd2_rn(dg[t][0], make_float2(u.x, u.y));
        dg[t][1] = __fadd2_rn(dg[t][1], make_float2(u.z, u.w));
        dg[t][2] = __fadd2_rn(dg[t][2], make_float2(w.x, w.y));
        dg[t][3] = __fadd2_rn(dg[t][3], make_float2(w.z, w.w));
      }
  }
#pragma unroll
  for (int t = 0; t < CH; ++t)
    if (col0 + 256 * t < C) store8(a.partial + static_cast<int64_t>(blockIdx.x) * C + col0 + 256 * t, dg[t]);
}

// dgamma[c] = the sum of the partial rows in a fixed order: 32 columns x 32 row lanes a CTA, every
// load of a lane in flight at once (304 rows x 4096: with 8 lanes 8 us, as much as it hid).
__global__ void __launch_bounds__(1024) dgamma_kernel(const float* partial, int n, int64_t C, float* dgamma) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  dev::pdl_wait();   // the partial sums are complete
  dev::pdl_trigger();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float t = 0.0f;
  if (c < C) {
    float v[16];   // n <= 512
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = w + 32 * k;
      v[k] = r < n ? partial[static_cast<int64_t>(r) * C + c] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) t = __fadd_rn(t, v[k]);
  }
  part[w][lane] = t;
  __syncthreads();
  t = warp_sum(part[lane][w]);   // warp w: column w
  if (lane == 0 && static_cast<int64_t>(blockIdx.x) * 32 + w < C) dgamma[static_cast<int64_t>(blockIdx.x) * 32 + w] = t;
}

// Warps per row (at most 16): the fewest whose lanes hold `cols` columns in `ch` chunks each.
int warps_per_row(int64_t cols, int ch) {
  int w = 1;
  while (w < 16 && w * 32 * 8 * ch < cols) w *= 2;
  return w;
}

// CTAs of the persistent walk over `rows`.
int walk_grid(int64_t rows, int wpr) {
  const int64_t want = (rows + cta_rows(wpr) - 1) / cta_rows(wpr);
  const int64_t fit = static_cast<int64_t>(wpr <= 8 ? 2 : 1) * num_sms();
  const int64_t most = fit < kMaxPartials ? fit : kMaxPartials;
  return static_cast<int>(want < most ? (want > 0 ? want : 1) : most);
}

template <typename T, bool MX>
te_status launch_norm(NormArgs& a, cudaStream_t st) {
  const int wpr = warps_per_row(a.cols, kCh);
  int grid = walk_grid(a.rows, wpr);
  if (MX) {
    // padding rows of the scales beside few rows: a CTA per 2048 words of them
    const int64_t want = ((a.rpad - a.rows) * (a.kpad / 4) + 2047) / 2048;
    if (want > grid) grid = static_cast<int>(want < num_sms() ? want : num_sms());
  }
  if (a.amax) {
    a.amax_whole = grid == 1;
    if (grid > 1) {
      const te_status s = zero_amax(a.amax, st);
      if (s != TE_OK) return s;
    }
  }
  void (*kernel)(NormArgs) = wpr == 1   ? rmsnorm_kernel<T, 1, MX>
                             : wpr == 2 ? rmsnorm_kernel<T, 2, MX>
                             : wpr == 4 ? rmsnorm_kernel<T, 4, MX>
                             : wpr == 8 ? rmsnorm_kernel<T, 8, MX>
                                        : rmsnorm_kernel<T, 16, MX>;
  const dim3 block(static_cast<unsigned>(32 * cta_warps(wpr)), 1, 1);
  const cudaError_t e = launch_dependent(kernel, dim3(static_cast<unsigned>(grid), 1, 1), block, 0, st, a);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

template <typename T>
te_status launch_norm_bwd(const NormBwdArgs& a, int wpr, int grid, cudaStream_t st) {
  void (*kernel)(NormBwdArgs) = wpr == 1                    ? rmsnorm_bwd_kernel<T, 1, 2>
                                : wpr == 2                  ? rmsnorm_bwd_kernel<T, 2, 2>
                                : wpr == 4                  ? rmsnorm_bwd_kernel<T, 4, 2>
                                : wpr == 8                  ? rmsnorm_bwd_kernel<T, 8, 2>
                                : a.cols <= 16 * 32 * 8 * 2 ? rmsnorm_bwd_kernel<T, 16, 2>
                                                            : rmsnorm_bwd_kernel<T, 16, 4>;
  const size_t smem = static_cast<size_t>(cta_rows(wpr)) * static_cast<size_t>(a.cols) * sizeof(float);
  if (a.cols > 16 * 32 * 8 * 2) {   // up to 64 KB of gamma
    static PerDevice<SharedMemory> ready;
    te_status s = TE_OK;
    if (!ready.get(&s, [](SharedMemory* m) {
          return allow_shared_memory(m, kernel_address(rmsnorm_bwd_kernel<T, 16, 4>), kMaxCols * sizeof(float));
        }))
      return s;
  }
  return record_cuda(launch_dependent(kernel, dim3(static_cast<unsigned>(grid), 1, 1),
                                      dim3(static_cast<unsigned>(32 * cta_warps(wpr)), 1, 1), smem, st, a));
}

te_status check_norm(const void* x, te_dtype in, int64_t rows, int64_t cols, const float* gamma, float eps,
                     const void* residual, const void* res_out, const void* y) {
  if (in != TE_BF16 && in != TE_F32) return TE_ERR_DTYPE;
  if (rows < 0 || cols <= 0 || cols % 16 || cols > kMaxCols || rows > (int64_t(1) << 31)) return TE_ERR_SHAPE;
  if (!(eps >= 0.0f) || !isfinite(eps)) return TE_ERR_ARG;
  if (gamma == nullptr || (rows > 0 && x == nullptr)) return TE_ERR_NULL;
  if (!aligned16(x) || !aligned16(gamma) || !aligned16(residual) || !aligned16(res_out) || !aligned16(y))
    return TE_ERR_ALIGN;
  return TE_OK;
}

NormArgs norm_args(const void* x, int64_t rows, int64_t cols, const void* residual, const float* gamma, float eps,
                   void* y, void* res_out, float* rsigma) {
  NormArgs a = {};
  a.x = x;
  a.res = residual;
  a.gamma = gamma;
  a.eps = eps;
  a.rows = rows;
  a.cols = cols;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.res_out = res_out;
  a.rsigma = rsigma;
  return a;
}

}  // namespace
}  // namespace te

using namespace te;

extern "C" {

te_status te_rmsnorm_fp8(const void* x, te_dtype in_dtype, int64_t rows, int64_t cols, const void* residual,
                         const float* gamma, float eps, te_dtype fmt, const float* scale, uint8_t* q_row, void* y,
                         void* res_out, float* rsigma, float* amax_out, float* scale_inv_out, void* stream) {
  te_status s = check_norm(x, in_dtype, rows, cols, gamma, eps, residual, res_out, y);
  if (s != TE_OK) return s;
  if (fmt != TE_E4M3 && fmt != TE_E5M2) return TE_ERR_DTYPE;
  if ((q_row || scale_inv_out) && scale == nullptr) return TE_ERR_NULL;
  if (!aligned16(q_row)) return TE_ERR_ALIGN;
  NormArgs a = norm_args(x, rows, cols, residual, gamma, eps, y, res_out, rsigma);
  a.q = q_row;
  a.scale = scale;
  a.e5m2 = fmt == TE_E5M2;
  a.amax = reinterpret_cast<unsigned int*>(amax_out);
  a.scale_inv = scale_inv_out;
  if (rows == 0 && !amax_out && !scale_inv_out) return TE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return in_dtype == TE_BF16 ? launch_norm<__nv_bfloat16, false>(a, st) : launch_norm<float, false>(a, st);
}

te_status te_rmsnorm_mxfp8(const void* x, te_dtype in_dtype, int64_t rows, int64_t cols, const void* residual,
                           const float* gamma, float eps, uint8_t* q_row, uint8_t* s_row, void* y, void* res_out,
                           float* rsigma, void* stream) {
  te_status s = check_norm(x, in_dtype, rows, cols, gamma, eps, residual, res_out, y);
  if (s != TE_OK) return s;
  if (cols % 32) return TE_ERR_SHAPE;
  if (rows == 0) return TE_OK;
  if (q_row == nullptr || s_row == nullptr) return TE_ERR_NULL;
  if (!aligned16(q_row) || !aligned16(s_row)) return TE_ERR_ALIGN;
  NormArgs a = norm_args(x, rows, cols, residual, gamma, eps, y, res_out, rsigma);
  a.q = q_row;
  a.s_row = s_row;
  a.kpad = (cols / 32 + 3) / 4 * 4;
  a.rpad = (rows + 127) / 128 * 128;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return in_dtype == TE_BF16 ? launch_norm<__nv_bfloat16, true>(a, st) : launch_norm<float, true>(a, st);
}

size_t te_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return static_cast<size_t>(rows < kMaxPartials ? rows : kMaxPartials) * static_cast<size_t>(cols) * sizeof(float);
}

te_status te_rmsnorm_bwd(const void* dy, const void* s, te_dtype in_dtype, int64_t rows, int64_t cols,
                         const float* gamma, const float* rsigma, const void* dres, void* dx, float* dgamma,
                         float* workspace, size_t workspace_bytes, void* stream) {
  if (in_dtype != TE_BF16 && in_dtype != TE_F32) return TE_ERR_DTYPE;
  if (rows < 0 || cols <= 0 || cols % 16 || cols > kMaxCols || rows > (int64_t(1) << 31)) return TE_ERR_SHAPE;
  if (gamma == nullptr || dgamma == nullptr) return TE_ERR_NULL;
  if (rows > 0 && (!dy || !s || !rsigma || !dx || !workspace)) return TE_ERR_NULL;
  if (workspace_bytes < te_rmsnorm_bwd_workspace_bytes(rows, cols)) return TE_ERR_SHAPE;
  if (!aligned16(dy) || !aligned16(s) || !aligned16(gamma) || !aligned16(dres) || !aligned16(dx) ||
      !aligned16(workspace))
    return TE_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (cudaMemsetAsync(dgamma, 0, static_cast<size_t>(cols) * sizeof(float), st) != cudaSuccess)
      return record_cuda(cudaGetLastError());
    return TE_OK;
  }
  NormBwdArgs a = {static_cast<const __nv_bfloat16*>(dy), s, dres, gamma, rsigma, rows, cols, dx, workspace};
  const int wpr = warps_per_row(cols, 2);
  const int grid = walk_grid(rows, wpr);
  const te_status launched = in_dtype == TE_BF16 ? launch_norm_bwd<__nv_bfloat16>(a, wpr, grid, st)
                                                 : launch_norm_bwd<float>(a, wpr, grid, st);
  if (launched != TE_OK) return launched;
  count_launch();
  // the sums' launch overlaps the end of the first kernel
  const cudaError_t e = launch_dependent(dgamma_kernel, dim3(static_cast<unsigned>((cols + 31) / 32), 1, 1),
                                         dim3(1024, 1, 1), 0, st, static_cast<const float*>(workspace), grid, cols,
                                         dgamma);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

}  // extern "C"
