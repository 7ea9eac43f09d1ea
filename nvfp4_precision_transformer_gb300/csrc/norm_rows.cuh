// What the row norms (norm.cu, layernorm.cu) share: a row in the registers of 1 to 16 warps, eight columns at
// a time, its sums over the row's warps, and the persistent walk over the rows.
#pragma once

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

}  // namespace
}  // namespace te
