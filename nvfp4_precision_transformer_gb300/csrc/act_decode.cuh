// The linear with bias, activation and residual for up to eight tokens of a small w (act_decodes, below), BF16 and FP8:
// w is read once from HBM and everything else is small, so the kernel is a stream over w.
//
// One persistent CTA of 16 warps per SM keeps x in shared memory and has an equal share of w's rows (within one:
// with whole 16-row units the SMs that have one unit more would be alone at the end), which it takes up to 16 rows
// at a time as the 16-row operand of mma.m16n8 (tokens are its n).  The 16 warps split K; a lane's 16-byte piece of
// a weight row is loaded straight into the registers the instruction reads it from (the order of k inside a block is
// free, as long as x follows it), four blocks ahead and across units, so the loads never wait for the arithmetic.
// Each unit ends with the warps' partial sums added in warp order through shared memory.
#pragma once

#include "gated_stream.cuh"

namespace te {
namespace {

// A call with few tokens (this file and act_stream.cuh).
struct FewArgs {
  const uint8_t* x;      // [T, K]
  const uint8_t* w;      // [N, K]
  int T, K, N, act;
  const float* alpha_a;
  const float* alpha_b;
  const float* bias;
  const void* res;
  __nv_bfloat16* z;
  void* y;
  int y_f32;
  uint8_t* q;
  const float* q_scale;   // FP8
  int q_e5m2;
  unsigned int* amax;
  float* scale_inv;
  // block-scaled operands: scales in the tensor-core layout, their padded columns, and those of an MXFP8 q
  const uint8_t* sx;
  const uint8_t* sw;
  int64_t s_kpad;
  uint8_t* s_q;
  int64_t q_kpad;
};

__device__ __forceinline__ float few_residual(const FewArgs& a, int64_t at) {
  if (!a.res) return 0.0f;
  return a.y_f32 ? static_cast<const float*>(a.res)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.res)[at]);
}
// z and y of one element (q is the caller's).
__device__ __forceinline__ void few_store(const FewArgs& a, int64_t at, float z, float v, float res) {
  if (a.z) a.z[at] = __float2bfloat16_rn(z);
  if (a.y) {
    const float y = a.res ? __fadd_rn(v, res) : v;
    if (a.y_f32) static_cast<float*>(a.y)[at] = y;
    else static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(y);
  }
}
__device__ __forceinline__ uint8_t few_code(const FewArgs& a, float v, float scale) {
  return static_cast<uint8_t>(a.q_e5m2 ? cvt_e5m2x2(v * scale, 0.0f) : cvt_e4m3x2(v * scale, 0.0f));
}

constexpr int kActDecTokens = 8;
constexpr int kActDecX = 32 * 1024;   // bytes of x

// x's T rows, then the partial sums of two units: [turn][warp][lane].
__host__ inline size_t act_decode_smem(int T, int K, int elem) {
  return static_cast<size_t>(T) * decode_row_bytes(K, elem) + 2 * kDecWarps * 512;
}

template <int W, int X>
__global__ void __launch_bounds__(32 * kDecWarps, 1) act_decode_kernel(FewArgs a) {
  constexpr int EB = W == kDecBF16 ? 2 : 1;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, t = lane & 3;
  const int row_bytes = a.K * EB;
  const int blocks = (row_bytes + 63) >> 6;
  const int srow = decode_row_bytes(a.K, EB);
  float4* red = reinterpret_cast<float4*>(dec_smem + a.T * srow);
  const int steps = (blocks + kDecWarps * kDecAhead - 1) / (kDecWarps * kDecAhead);
  // this CTA's rows of w, in units of at most 16
  const int lo = static_cast<int>(static_cast<int64_t>(a.N) * blockIdx.x / gridDim.x);
  const int rows = static_cast<int>(static_cast<int64_t>(a.N) * (blockIdx.x + 1) / gridDim.x) - lo;
  const int units = (rows + 15) >> 4;
  auto unit_lo = [&](int u) { return lo + rows * u / units; };

  // Pieces of unit `unit`, step `step`: block (step * kDecAhead + i) * kDecWarps + warp of its rows r and r + 8.
  uint4 wa[kDecAhead], wb[kDecAhead];
  auto fetch = [&](int unit, int step) {
    const bool live = unit < units;
    const int u0 = live ? unit_lo(unit) : 0, n = live ? unit_lo(unit + 1) - u0 : 0;
    const uint8_t* p = a.w + static_cast<int64_t>(u0 + r) * row_bytes;
    const uint8_t* p8 = p + static_cast<int64_t>(8) * row_bytes;
#pragma unroll
    for (int i = 0; i < kDecAhead; ++i) {
      const int at = ((step * kDecAhead + i) * kDecWarps + warp) * 64 + t * 16;
      wa[i] = wb[i] = make_uint4(0u, 0u, 0u, 0u);
      if (at < row_bytes) {
        if (r < n) wa[i] = ld_stream(p + at);
        if (r + 8 < n) wb[i] = ld_stream(p8 + at);
      }
    }
  };
  dev::pdl_wait();
  dev::pdl_trigger();
  fetch(0, 0);

  // x into shared memory, 16 bytes of it at a time; the last block's tail is zero
  const int pieces = blocks * 4;
  for (int i = threadIdx.x; i < a.T * pieces; i += blockDim.x) {
    const int n = i / pieces, p = i - n * pieces;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (p * 16 < row_bytes) v = *reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(n) * row_bytes + p * 16);
    *reinterpret_cast<uint4*>(dec_smem + n * srow + p * 16) = v;
  }
  const float alpha = (a.alpha_a ? *a.alpha_a : 1.0f) * (a.alpha_b ? *a.alpha_b : 1.0f);
  const float qs = a.q ? *a.q_scale : 1.0f;
  unsigned int top = 0;
  __syncthreads();

  const uint8_t* xrow = dec_smem + r * srow + t * 16;
  for (int unit = 0; unit < units; ++unit) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int step = 0; step < steps; ++step) {
      uint4 ca[kDecAhead], cb[kDecAhead];
#pragma unroll
      for (int i = 0; i < kDecAhead; ++i) ca[i] = wa[i], cb[i] = wb[i];
      const bool last = step + 1 == steps;
      fetch(last ? unit + 1 : unit, last ? 0 : step + 1);
      // (the tensor cores round their sums towards zero: only eight instructions' worth before they are added up here)
      float4 part = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kDecAhead; ++i) {
        const int block = (step * kDecAhead + i) * kDecWarps + warp;
        if (block >= blocks) break;
        uint4 b = make_uint4(0u, 0u, 0u, 0u);   // tokens past the last
        if (r < a.T) b = *reinterpret_cast<const uint4*>(xrow + block * 64);
        mma_dec<W, X>(part, ca[i].x, cb[i].x, ca[i].y, cb[i].y, b.x, b.y);
        mma_dec<W, X>(part, ca[i].z, cb[i].z, ca[i].w, cb[i].w, b.z, b.w);
      }
      acc.x += part.x, acc.y += part.y, acc.z += part.z, acc.w += part.w;
    }
    // (the units' sums take turns in two buffers, so that one barrier a unit is enough)
    float4* mine = red + (unit & 1) * kDecWarps * 32;
    mine[warp * 32 + lane] = acc;
    __syncthreads();
    // lane (r, t) has tokens 2 t and 2 t + 1 of rows r (warp 0) and r + 8 (warp 1)
    if (warp < 2) {
      const float2* p = reinterpret_cast<const float2*>(mine + lane) + warp;
      float2 s = p[0];
#pragma unroll
      for (int k = 1; k < kDecWarps; ++k) s = __fadd2_rn(s, p[k * 64]);
      const int u0 = unit_lo(unit), row = r + 8 * warp;
      if (row < unit_lo(unit + 1) - u0) {
        const int col = u0 + row;
        const float b = a.bias ? a.bias[col] : 0.0f;
        const float2 z2 = __ffma2_rn(s, both(alpha), both(b));
        const float2 v2 = act_value(z2, a.act);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int tok = 2 * t + j;
          if (tok < a.T) {
            const int64_t at = static_cast<int64_t>(tok) * a.N + col;
            const float v = j ? v2.y : v2.x;
            few_store(a, at, j ? z2.y : z2.x, v, few_residual(a, at));
            if (a.q) {
              top = max(top, __float_as_uint(v) & 0x7FFFFFFFu);
              a.q[at] = few_code(a, v, qs);
            }
          }
        }
      }
    }
  }
  if (a.amax && warp < 2) {
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) atomicMax(a.amax, top);
  }
  if (a.scale_inv && blockIdx.x == 0 && threadIdx.x == 0) *a.scale_inv = __fdiv_rn(1.0f, qs);
}

template <int W, int X>
te_status launch_act_decode(const FewArgs& a, cudaStream_t st) {
  static PerDevice<SharedMemory> ready;
  te_status s = TE_OK;
  if (!ready.get(&s, [](SharedMemory* m) {
        return allow_shared_memory(m, kernel_address(act_decode_kernel<W, X>), 64 * 1024);
      }))
    return s;
  // a CTA for every eight rows where there are few
  const int units = (a.N + 7) / 8;
  const int grid = units < num_sms() ? units : num_sms();
  const size_t smem = act_decode_smem(a.T, a.K, W == kDecBF16 ? 2 : 1);
  if (a.amax) {
    s = zero_amax(a.amax, st);
    if (s != TE_OK) return s;
  }
  const cudaError_t e = launch_dependent(act_decode_kernel<W, X>, dim3(static_cast<unsigned>(grid), 1, 1),
                                         dim3(32 * kDecWarps, 1, 1), smem, st, a);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

// Whether this kernel takes the call, or the one of act_stream.cuh (us, this / that):
//   T = 1, BF16: K = 512, N = 512 2.4 / 3.7, K = 768, N = 2048 2.7 / 4.1, K = N = 2048 3.1 / 5.1, K = 1024, N = 4096 3.9 /
//   4.6, K = 2048, N = 4096 (16 MB) 5.3 / 5.4, K = N = 4096 8.6 / 8.6, K = 4096, N = 16384 24.9 / 24.3; FP8 K = 768,
//   N = 2048 2.7 / 3.9, K = N = 2048 2.9 / 4.3, K = 1024, N = 4096 3.9 / 4.0, K = N = 4096 6.5 / 5.4;
//   short rows, many of them: K = 256, N = 8192 BF16 5.6 / 4.0, FP8 5.8 / 2.9;
//   T = 2, 4 and 8 of a long row: BF16 K = 8192, N = 256 6.0, 7.0 and 9.0 / 6.7, K = 3200, N = 1600 4.0, 4.5 and 5.3 / 5.0;
//   FP8 K = 8192, N = 256 4.8, 5.3 and 6.2 / 5.1.
// No tensor memory to set up and loads that go out at once make it the faster one where w is small; a unit of 16 rows
// costs as much for a short row, and what x takes of shared memory and of the loads is felt beside few rows.
inline bool act_decodes(int64_t T, int64_t K, int64_t N, int elem) {
  const int64_t row = K * elem;
  return T <= kActDecTokens && N * row <= (12 << 20) && N <= 4 * row && T * row <= kActDecX;
}

}  // namespace
}  // namespace te
