// LayerNorm with the residual's addition and an 8-bit output, and its gradient.
//
//   forward   s = x + residual;  mu = mean(s);  rsigma = 1 / sqrt(mean((s - mu)^2) + eps);
//             y = ((s - mu) * rsigma) * gamma + beta
//             outputs: s, y in bf16, y in FP8 (per-tensor scale) or MXFP8 (1 x 32 blocks), mu, rsigma
//   backward  xhat = (s - mu) * rsigma, p = dy * gamma:
//             ds = rsigma * (p - mean(p) - xhat * mean(p * xhat)) (+ the residual stream's own gradient)
//             dgamma = sum over the rows of dy * xhat,  dbeta = sum over the rows of dy
//
// Both are bound by HBM, and a row lies in registers as in norm.cu, so every tensor is read once.  The
// variance takes no second exchange between the row's warps: each of them has the sum and the sum of squares
// about its own mean (two butterflies), and n_w, sum_w and M2_w of the warps give (a lane each)
//   mu = sum of sum_w / C,   sum of (s - mu)^2 = sum of (M2_w + n_w (mu_w - mu)^2),
// without the cancellation of sum(s^2) - C mu^2.  All sums are fp32 in a fixed order.
//
// 15872 x 4096 bf16: x + residual to s, y, MXFP8 94 us (587 MB, 6.2 TB/s), x to bf16 53 (260 MB, 4.9) and to FP8 51 to 52
// (195 MB, 3.8): the arithmetic of a row is no longer hidden where a row moves so little; backward with dres 85 us with the
// columns' sums (520 MB, 6.1).  gamma and beta read again for each row, from L1: kept in shared memory the first took
// 101.5 us.  Two rows ahead: no gain.  At 128 registers the forward kernels of fp32 rows store up to 88 bytes a thread, the
// backward ones past 8192 columns 52 (bf16) and 96 (fp32), the others none.
#include "norm_rows.cuh"

namespace te {
namespace {

// Sums of two values over the WPR warps of a row, in warp order, behind one barrier (see row_sum).
template <int WPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 (*red)[WPR], int turn, int grp, int wr, int lane) {
  v = make_float2(warp_sum(v.x), warp_sum(v.y));
  if (WPR == 1) return v;
  if (lane == 0) red[turn][wr] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * WPR) : "memory");
  float2 t = red[turn][0];
#pragma unroll
  for (int w = 1; w < WPR; ++w) t = __fadd2_rn(t, red[turn][w]);
  return t;
}

struct LnArgs {
  const void* x;
  const void* res;
  const float* gamma;
  const float* beta;
  float eps;
  int64_t rows, cols;
  __nv_bfloat16* y;
  void* res_out;
  float* mu;
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
__global__ void __launch_bounds__(32 * cta_warps(WPR), WPR <= 8 ? 2 : 1) layernorm_rows_kernel(LnArgs a) {
  constexpr int GR = cta_rows(WPR);
  __shared__ float2 red[GR][2][WPR];
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
  // (one tensor after the other: FP8 of 15872 x 4096 bf16 55.4 -> 52.0 us, with a residual and MXFP8 95.9 -> 94.5)
  auto load = [&](Raw8<T> (&r)[kCh], const T* p, int64_t row) {
#pragma unroll
    for (int t = 0; t < kCh; ++t) {
      const int col = col0 + 256 * t;
      r[t].zero();
      if (row < a.rows && col < C) r[t].load(p + row * C + col);
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * GR + grp;
  load(rx, x, row);
  if (res) load(rr, res, row);
  // columns of warp w of the row
  auto columns = [&](int w) {
    const int64_t n = C - static_cast<int64_t>(w) * kWarpCols;
    return static_cast<float>(n < 0 ? 0 : (n < kWarpCols ? n : kWarpCols));
  };
  // (reciprocals once: a row's divisions cost as much as all of the rest, FP8 of 15872 x 4096 bf16 61.4 -> 52.9 us)
  auto inverse = [](float n) { return n > 0.0f ? __fdiv_rn(1.0f, n) : 0.0f; };
  const float inv_c = inverse(static_cast<float>(C)), inv_mine = inverse(columns(wr));
  const float n_lane = columns(lane % WPR), inv_lane = inverse(n_lane);   // of the warp whose sums this lane takes
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    float2 v[kCh][4];
    float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int t = 0; t < kCh; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[t][i] = res ? __fadd2_rn(rx[t].pair(i), rr[t].pair(i)) : rx[t].pair(i);
        sum2 = __fadd2_rn(sum2, v[t][i]);
      }
    // the next row's loads are in flight while this one is reduced and written
    if (res) {
      load(rx, x, row + step);
      load(rr, res, row + step);
    } else {
      load(rx, x, row + step);
    }
    const float sum = warp_sum(__fadd_rn(sum2.x, sum2.y));
    const float mw = __fmul_rn(sum, inv_mine);
    const float2 neg = make_float2(-mw, -mw);
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int t = 0; t < kCh; ++t) {
      if (col0 + 256 * t >= C) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 d = __fadd2_rn(v[t][i], neg);
        sq = __ffma2_rn(d, d, sq);
      }
    }
    const float m2w = warp_sum(__fadd_rn(sq.x, sq.y));
    float mu = mw, m2 = m2w;
    if (WPR > 1) {
      if (lane == 0) red[grp][turn][wr] = make_float2(sum, m2w);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * WPR) : "memory");
      // lane l takes warp l % WPR's sums, and the lanes add them in a butterfly
      const float2 p = red[grp][turn][lane % WPR];
      float total = p.x;
#pragma unroll
      for (int o = WPR / 2; o > 0; o >>= 1) total = __fadd_rn(total, __shfl_xor_sync(0xFFFFFFFFu, total, o));
      mu = __fmul_rn(total, inv_c);
      const float d = __fmaf_rn(p.x, inv_lane, -mu);
      m2 = __fmaf_rn(__fmul_rn(n_lane, d), d, p.y);
#pragma unroll
      for (int o = WPR / 2; o > 0; o >>= 1) m2 = __fadd_rn(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, o));
    }
    const float rs = rsqrtf(__fmaf_rn(m2, inv_c, a.eps));
    if (wr == 0 && lane == 0) {
      if (a.mu) a.mu[row] = mu;
      if (a.rsigma) a.rsigma[row] = rs;
    }
    const float2 rs2 = make_float2(rs, rs), mu2 = make_float2(-mu, -mu);
#pragma unroll
    for (int t = 0; t < kCh; ++t) {
      const int col = col0 + 256 * t;
      const bool live = col < C;
      const int64_t at = row * C + col;
      float2 g[4] = {}, b[4] = {}, y[4];
      if (live) {
        ld8(a.gamma + col, g);
        ld8(a.beta + col, b);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[t][i], mu2), rs2), g[i], b[i]);
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
        const float2 m2v = make_float2(mul, mul);
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 p = __fmul2_rn(y[2 * h], m2v), r = __fmul2_rn(y[2 * h + 1], m2v);
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

struct LnBwdArgs {
  const __nv_bfloat16* dy;
  const void* s;
  const void* dres;
  const float* gamma;
  const float* mu;
  const float* rsigma;
  int64_t rows, cols;
  void* dx;
  float* partial;   // [gridDim.x, 2, cols]: dgamma's, then dbeta's
};

// Two chunks a lane (four from 8193 columns on) and two CTAs per SM, with the next row in flight in bf16, as
// norm.cu's backward pass has them.
template <typename T, int WPR, int CH>
__global__ void __launch_bounds__(32 * cta_warps(WPR), WPR <= 8 ? 2 : 1) layernorm_bwd_kernel(LnBwdArgs a) {
  constexpr int GR = cta_rows(WPR);
  constexpr bool kAhead = sizeof(T) == 2 && CH == 2;   // the next row's loads before this row is reduced
  // dres chunk by chunk when it is added, from L2, where its registers are not there (4000 x 16384 fp32 273 -> 185 us)
  constexpr bool kLate = CH == 4 && sizeof(T) == 4;
  __shared__ float2 red[GR][2][WPR];
  extern __shared__ __align__(16) float cols_sum[];   // [GR - 1][2][cols], then gamma
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp / WPR, wr = warp % WPR;
  const int64_t C = a.cols;
  const int64_t step = static_cast<int64_t>(gridDim.x) * GR;
  const T* s = static_cast<const T*>(a.s);
  const T* dres = static_cast<const T*>(a.dres);
  const int col0 = (wr * CH * 32 + lane) * 8;
  float2 dg[CH][4], db[CH][4];
#pragma unroll
  for (int t = 0; t < CH; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[t][i] = db[t][i] = make_float2(0.f, 0.f);

  struct RowRegs {
    Raw8<__nv_bfloat16> d[CH];
    Raw8<T> x[CH], r[CH];
    float mu, rs;
  };
  auto load = [&](RowRegs& q, int64_t row) {
    q.mu = row < a.rows ? a.mu[row] : 0.0f;
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
        if (dres) {
          if (kLate) asm volatile("prefetch.global.L2 [%0];" ::"l"(dres + row * C + col));
          else q.r[t].load(dres + row * C + col);
        }
      }
    }
  };
  dev::pdl_wait();
  // gamma once into shared memory, the two halves of its chunks of eight apart (reads without bank conflicts)
  float4* sgam = reinterpret_cast<float4*>(cols_sum + 2 * (GR - 1) * C);
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
  const float inv_c = __fdiv_rn(-1.0f, static_cast<float>(C));
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    RowRegs nxt;
    if (kAhead) load(nxt, row + step);
    else load(cur, row);
    const float2 rs2 = make_float2(cur.rs, cur.rs), mu2 = make_float2(-cur.mu, -cur.mu);
    float2 dot = make_float2(0.f, 0.f), sum = dot;
#pragma unroll
    for (int t = 0; t < CH; ++t) {
      const int col = col0 + 256 * t;
      if (col >= C) break;
      float2 g[4];
      gamma8(col, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 dy = cur.d[t].pair(i);
        const float2 w = __fmul2_rn(dy, __fmul2_rn(__fadd2_rn(cur.x[t].pair(i), mu2), rs2));   // dy * xhat
        dg[t][i] = __fadd2_rn(dg[t][i], w);
        db[t][i] = __fadd2_rn(db[t][i], dy);
        dot = __ffma2_rn(w, g[i], dot);
        sum = __ffma2_rn(dy, g[i], sum);
      }
    }
    const float2 both = row_sum2<WPR>(make_float2(__fadd_rn(dot.x, dot.y), __fadd_rn(sum.x, sum.y)), red[grp], turn, grp,
                                      wr, lane);
    const float c1 = __fmul_rn(both.x, inv_c), c2 = __fmul_rn(both.y, inv_c);
    const float2 c12 = make_float2(c1, c1), c22 = make_float2(c2, c2);
#pragma unroll
    for (int t = 0; t < CH; ++t) {
      const int col = col0 + 256 * t;
      if (col >= C) break;
      float2 g[4], o[4];
      gamma8(col, g);
      if (kLate && dres) cur.r[t].load(dres + row * C + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = __ffma2_rn(cur.d[t].pair(i), g[i], c22);
        const float2 d = __ffma2_rn(__fmul2_rn(__fadd2_rn(cur.x[t].pair(i), mu2), rs2), c12, p);
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
      for (int t = 0; t < CH; ++t) {
        const int col = col0 + 256 * t;
        if (col >= C) break;
        store8(cols_sum + 2 * (grp - 1) * C + col, dg[t]);
        store8(cols_sum + (2 * (grp - 1) + 1) * C + col, db[t]);
      }
    }
    __syncthreads();
    if (grp > 0) return;
    for (int k = 0; k < GR - 1; ++k)
#pragma unroll
      for (int t = 0; t < CH; ++t) {
        const int col = col0 + 256 * t;
        if (col >= C) break;
        float2 u[4];
        ld8(cols_sum + 2 * k * C + col, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[t][i] = __fadd2_rn(dg[t][i], u[i]);
        ld8(cols_sum + (2 * k + 1) * C + col, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) db[t][i] = __fadd2_rn(db[t][i], u[i]);
      }
  }
  float* mine = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * C;
#pragma unroll
  for (int t = 0; t < CH; ++t) {
    const int col = col0 + 256 * t;
    if (col >= C) break;
    store8(mine + col, dg[t]);
    store8(mine + C + col, db[t]);
  }
}

// dgamma and dbeta = the sums of the partial rows (n <= 512) in a fixed order: 32 columns x 32 row lanes a CTA,
// every load of a lane in flight at once.  Column c of [n, 2 C] belongs to dgamma, then to dbeta.
__global__ void __launch_bounds__(1024) ln_param_grad_kernel(const float* partial, int n, int64_t C, float* dgamma,
                                                             float* dbeta) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  dev::pdl_wait();   // the partial sums are complete
  dev::pdl_trigger();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float t = 0.0f;
  if (c < 2 * C) {
    float v[16];   // n <= 512
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = w + 32 * k;
      v[k] = r < n ? partial[static_cast<int64_t>(r) * 2 * C + c] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) t = __fadd_rn(t, v[k]);
  }
  part[w][lane] = t;
  __syncthreads();
  t = warp_sum(part[lane][w]);   // warp w: column w
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + w;
  if (lane == 0 && col < 2 * C) *(col < C ? dgamma + col : dbeta + (col - C)) = t;
}

template <typename T, bool MX>
te_status launch_layernorm(LnArgs& a, cudaStream_t st) {
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
  void (*kernel)(LnArgs) = wpr == 1   ? layernorm_rows_kernel<T, 1, MX>
                           : wpr == 2 ? layernorm_rows_kernel<T, 2, MX>
                           : wpr == 4 ? layernorm_rows_kernel<T, 4, MX>
                           : wpr == 8 ? layernorm_rows_kernel<T, 8, MX>
                                      : layernorm_rows_kernel<T, 16, MX>;
  const dim3 block(static_cast<unsigned>(32 * cta_warps(wpr)), 1, 1);
  const cudaError_t e = launch_dependent(kernel, dim3(static_cast<unsigned>(grid), 1, 1), block, 0, st, a);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

template <typename T>
te_status launch_layernorm_bwd(const LnBwdArgs& a, int wpr, int grid, cudaStream_t st) {
  void (*kernel)(LnBwdArgs) = wpr == 1                    ? layernorm_bwd_kernel<T, 1, 2>
                              : wpr == 2                  ? layernorm_bwd_kernel<T, 2, 2>
                              : wpr == 4                  ? layernorm_bwd_kernel<T, 4, 2>
                              : wpr == 8                  ? layernorm_bwd_kernel<T, 8, 2>
                              : a.cols <= 16 * 32 * 8 * 2 ? layernorm_bwd_kernel<T, 16, 2>
                                                          : layernorm_bwd_kernel<T, 16, 4>;
  const size_t smem = static_cast<size_t>(2 * cta_rows(wpr) - 1) * static_cast<size_t>(a.cols) * sizeof(float);
  if (a.cols > 16 * 32 * 8 * 2) {   // up to 64 KB of gamma
    static PerDevice<SharedMemory> ready;
    te_status s = TE_OK;
    if (!ready.get(&s, [](SharedMemory* m) {
          return allow_shared_memory(m, kernel_address(layernorm_bwd_kernel<T, 16, 4>), kMaxCols * sizeof(float));
        }))
      return s;
  }
  return record_cuda(launch_dependent(kernel, dim3(static_cast<unsigned>(grid), 1, 1),
                                      dim3(static_cast<unsigned>(32 * cta_warps(wpr)), 1, 1), smem, st, a));
}

te_status check_layernorm(const void* x, te_dtype in, int64_t rows, int64_t cols, const float* gamma, const float* beta,
                          float eps, const void* residual, const void* res_out, const void* y) {
  if (in != TE_BF16 && in != TE_F32) return TE_ERR_DTYPE;
  if (rows < 0 || cols <= 0 || cols % 16 || cols > kMaxCols || rows > (int64_t(1) << 31)) return TE_ERR_SHAPE;
  if (!(eps >= 0.0f) || !isfinite(eps)) return TE_ERR_ARG;
  if (gamma == nullptr || beta == nullptr || (rows > 0 && x == nullptr)) return TE_ERR_NULL;
  if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(residual) || !aligned16(res_out) ||
      !aligned16(y))
    return TE_ERR_ALIGN;
  return TE_OK;
}

LnArgs layernorm_args(const void* x, int64_t rows, int64_t cols, const void* residual, const float* gamma,
                      const float* beta, float eps, void* y, void* res_out, float* mu, float* rsigma) {
  LnArgs a = {};
  a.x = x;
  a.res = residual;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.rows = rows;
  a.cols = cols;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.res_out = res_out;
  a.mu = mu;
  a.rsigma = rsigma;
  return a;
}

}  // namespace
}  // namespace te

using namespace te;

extern "C" {

te_status te_add_layernorm_fp8(const void* x, te_dtype in_dtype, int64_t rows, int64_t cols, const void* residual,
                               const float* gamma, const float* beta, float eps, te_dtype fmt, const float* scale,
                               uint8_t* q_row, void* y, void* res_out, float* mu, float* rsigma, float* amax_out,
                               float* scale_inv_out, void* stream) {
  te_status s = check_layernorm(x, in_dtype, rows, cols, gamma, beta, eps, residual, res_out, y);
  if (s != TE_OK) return s;
  if (fmt != TE_E4M3 && fmt != TE_E5M2) return TE_ERR_DTYPE;
  if ((q_row || scale_inv_out) && scale == nullptr) return TE_ERR_NULL;
  if (!aligned16(q_row)) return TE_ERR_ALIGN;
  LnArgs a = layernorm_args(x, rows, cols, residual, gamma, beta, eps, y, res_out, mu, rsigma);
  a.q = q_row;
  a.scale = scale;
  a.e5m2 = fmt == TE_E5M2;
  a.amax = reinterpret_cast<unsigned int*>(amax_out);
  a.scale_inv = scale_inv_out;
  if (rows == 0 && !amax_out && !scale_inv_out) return TE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return in_dtype == TE_BF16 ? launch_layernorm<__nv_bfloat16, false>(a, st) : launch_layernorm<float, false>(a, st);
}

te_status te_add_layernorm_mxfp8(const void* x, te_dtype in_dtype, int64_t rows, int64_t cols, const void* residual,
                                 const float* gamma, const float* beta, float eps, uint8_t* q_row, uint8_t* s_row,
                                 void* y, void* res_out, float* mu, float* rsigma, void* stream) {
  te_status s = check_layernorm(x, in_dtype, rows, cols, gamma, beta, eps, residual, res_out, y);
  if (s != TE_OK) return s;
  if (cols % 32) return TE_ERR_SHAPE;
  if (rows == 0) return TE_OK;
  if (q_row == nullptr || s_row == nullptr) return TE_ERR_NULL;
  if (!aligned16(q_row) || !aligned16(s_row)) return TE_ERR_ALIGN;
  LnArgs a = layernorm_args(x, rows, cols, residual, gamma, beta, eps, y, res_out, mu, rsigma);
  a.q = q_row;
  a.s_row = s_row;
  a.kpad = (cols / 32 + 3) / 4 * 4;
  a.rpad = (rows + 127) / 128 * 128;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return in_dtype == TE_BF16 ? launch_layernorm<__nv_bfloat16, true>(a, st) : launch_layernorm<float, true>(a, st);
}

size_t te_layernorm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return static_cast<size_t>(rows < kMaxPartials ? rows : kMaxPartials) * 2 * static_cast<size_t>(cols) * sizeof(float);
}

te_status te_layernorm_bwd(const void* dy, const void* s, te_dtype in_dtype, int64_t rows, int64_t cols,
                           const float* gamma, const float* mu, const float* rsigma, const void* dres, void* dx,
                           float* dgamma, float* dbeta, float* workspace, size_t workspace_bytes, void* stream) {
  if (in_dtype != TE_BF16 && in_dtype != TE_F32) return TE_ERR_DTYPE;
  if (rows < 0 || cols <= 0 || cols % 16 || cols > kMaxCols || rows > (int64_t(1) << 31)) return TE_ERR_SHAPE;
  if (gamma == nullptr || dgamma == nullptr || dbeta == nullptr) return TE_ERR_NULL;
  if (rows > 0 && (!dy || !s || !mu || !rsigma || !dx || !workspace)) return TE_ERR_NULL;
  if (workspace_bytes < te_layernorm_bwd_workspace_bytes(rows, cols)) return TE_ERR_SHAPE;
  if (!aligned16(dy) || !aligned16(s) || !aligned16(gamma) || !aligned16(dres) || !aligned16(dx) ||
      !aligned16(workspace))
    return TE_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    const size_t bytes = static_cast<size_t>(cols) * sizeof(float);
    if (cudaMemsetAsync(dgamma, 0, bytes, st) != cudaSuccess || cudaMemsetAsync(dbeta, 0, bytes, st) != cudaSuccess)
      return record_cuda(cudaGetLastError());
    return TE_OK;
  }
  LnBwdArgs a = {static_cast<const __nv_bfloat16*>(dy), s, dres, gamma, mu, rsigma, rows, cols, dx, workspace};
  const int wpr = warps_per_row(cols, 2);
  const int grid = walk_grid(rows, wpr);
  const te_status launched = in_dtype == TE_BF16 ? launch_layernorm_bwd<__nv_bfloat16>(a, wpr, grid, st)
                                                 : launch_layernorm_bwd<float>(a, wpr, grid, st);
  if (launched != TE_OK) return launched;
  count_launch();
  // the sums' launch overlaps the end of the first kernel
  const cudaError_t e = launch_dependent(ln_param_grad_kernel, dim3(static_cast<unsigned>((2 * cols + 31) / 32), 1, 1),
                                         dim3(1024, 1, 1), 0, st, static_cast<const float*>(workspace), grid, cols,
                                         dgamma, dbeta);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

}  // extern "C"
