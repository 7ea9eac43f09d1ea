// The gated projections of a few tokens (decoding): the two weight halves are read once from HBM and
// everything else is small, so the kernel is a stream over w.
//
// One persistent CTA of 16 warps per SM keeps x in shared memory.  A unit of work is eight columns of
// h: eight gate rows and the eight up rows beside them are one 16-row operand of mma.m16n8 (tokens
// are its n), whose accumulator layout puts g and u of the same element in the same thread.  The 16
// warps split K; a lane's 16-byte piece of a weight row is loaded straight into the registers the
// instruction reads it from (the order of k inside a block is free, as long as x follows it), four
// blocks ahead and across units, so the loads never wait for the arithmetic.  Each unit ends with the
// warps' partial sums added in warp order through shared memory.
//
// One token, K = 4096, F = 16384: BF16 42.4 us (6.33 TB/s; gemm_kernel, whose SMs all read the one line
// of x at the same time, 84.0), FP8 24.3 us (5.52 TB/s; 43.4).
#pragma once

#include "gemm.cuh"

namespace te {
namespace {

constexpr int kDecWarps = 16;
constexpr int kDecAhead = 4;          // blocks of 64 bytes of K per warp and step
constexpr int kDecMaxTiles = 4;       // tiles of eight tokens

enum DecW { kDecBF16 = 0, kDecE4M3 = 1, kDecE5M2 = 2 };

struct DecodeArgs {
  const uint8_t* x;      // [T, K] bf16 or FP8
  const uint8_t* w;      // [2 F, K]
  int T, K, F, act;
  const float* alpha_a;
  const float* alpha_b;
  __nv_bfloat16* h;
  __nv_bfloat16* gu;
  uint8_t* q;
  const float* q_scale;
  int q_e5m2;
  unsigned int* amax;
  float* scale_inv;
  // block-scaled operands (gated_stream_block.cuh): scales in the tensor-core layout, their padded
  // columns, and those of an MXFP8 h
  const uint8_t* sx;
  const uint8_t* sw;
  int64_t s_kpad;
  uint8_t* s_h;
};

// (An ordinary load that leaves L1 alone: the read-only path is not for a kernel that is set up beside
// the one before it, see pdl_wait.)
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// One instruction over 32 bytes of K of each row: weights (operand A) of type W, x of type X.
#define TE_DEC_MMA(TYPES)                                                                                           \
  asm volatile("mma.sync.aligned." TYPES " {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"          \
               : "+f"(c.x), "+f"(c.y), "+f"(c.z), "+f"(c.w)                                                          \
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
template <int W, int X>
__device__ __forceinline__ void mma_dec(float4& c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  if (W == kDecBF16) TE_DEC_MMA("m16n8k16.row.col.f32.bf16.bf16.f32");
  else if (W == kDecE4M3 && X == kDecE4M3) TE_DEC_MMA("m16n8k32.row.col.f32.e4m3.e4m3.f32");
  else if (W == kDecE4M3) TE_DEC_MMA("m16n8k32.row.col.f32.e4m3.e5m2.f32");
  else if (X == kDecE4M3) TE_DEC_MMA("m16n8k32.row.col.f32.e5m2.e4m3.f32");
  else TE_DEC_MMA("m16n8k32.row.col.f32.e5m2.e5m2.f32");
}
#undef TE_DEC_MMA

// Bytes of a token's row of x in shared memory: whole blocks, an odd number of them, so that
// neighbouring rows lie in different halves of the banks.
__host__ __device__ inline int decode_row_bytes(int K, int elem) { return (((K * elem + 63) / 64) | 1) * 64; }
__host__ inline size_t decode_smem(int T, int K, int elem) {
  const int tiles = (T + 7) / 8;
  return static_cast<size_t>(tiles) * 8 * decode_row_bytes(K, elem) + static_cast<size_t>(kDecWarps) * tiles * 512;
}

template <int W, int X, int NT>
__global__ void __launch_bounds__(32 * kDecWarps, 1) gated_decode_kernel(DecodeArgs a) {
  constexpr int EB = W == kDecBF16 ? 2 : 1;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, t = lane & 3;
  const int row_bytes = a.K * EB;
  const int blocks = (row_bytes + 63) >> 6;
  const int srow = decode_row_bytes(a.K, EB);
  float4* red = reinterpret_cast<float4*>(dec_smem + NT * 8 * srow);   // [warp][tile][lane]
  const int units = a.F >> 3;
  const int steps = (blocks + kDecWarps * kDecAhead - 1) / (kDecWarps * kDecAhead);

  // Pieces of unit `unit`, step `step`: block (step * kDecAhead + i) * kDecWarps + warp.
  uint4 wg[kDecAhead], wu[kDecAhead];
  auto fetch = [&](int unit, int step) {
    const uint8_t* g = a.w + static_cast<int64_t>(unit * 8 + r) * row_bytes;
    const uint8_t* u = g + static_cast<int64_t>(a.F) * row_bytes;
#pragma unroll
    for (int i = 0; i < kDecAhead; ++i) {
      const int at = ((step * kDecAhead + i) * kDecWarps + warp) * 64 + t * 16;
      wg[i] = wu[i] = make_uint4(0u, 0u, 0u, 0u);
      if (unit < units && at < row_bytes) {
        wg[i] = ld_stream(g + at);
        wu[i] = ld_stream(u + at);
      }
    }
  };
  dev::pdl_wait();
  dev::pdl_trigger();
  int unit = static_cast<int>(blockIdx.x);
  fetch(unit, 0);

  // x into shared memory, 16 bytes of it at a time; rows past T and the last block's tail are zero
  const int pieces = blocks * 4;
  for (int i = threadIdx.x; i < NT * 8 * pieces; i += blockDim.x) {
    const int n = i / pieces, p = i - n * pieces;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (n < a.T && p * 16 < row_bytes)
      v = *reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(n) * row_bytes + p * 16);
    *reinterpret_cast<uint4*>(dec_smem + n * srow + p * 16) = v;
  }
  const float alpha = (a.alpha_a ? *a.alpha_a : 1.0f) * (a.alpha_b ? *a.alpha_b : 1.0f);
  const float qs = a.q ? *a.q_scale : 1.0f;
  unsigned int top = 0;
  __syncthreads();

  const uint8_t* xrow = dec_smem + r * srow + t * 16;
  for (; unit < units; unit += static_cast<int>(gridDim.x)) {
    float4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int step = 0; step < steps; ++step) {
      uint4 cg[kDecAhead], cu[kDecAhead];
#pragma unroll
      for (int i = 0; i < kDecAhead; ++i) cg[i] = wg[i], cu[i] = wu[i];
      const bool last = step + 1 == steps;
      fetch(last ? unit + static_cast<int>(gridDim.x) : unit, last ? 0 : step + 1);
#pragma unroll
      for (int i = 0; i < kDecAhead; ++i) {
        const int block = (step * kDecAhead + i) * kDecWarps + warp;
        if (block >= blocks) break;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 b = *reinterpret_cast<const uint4*>(xrow + n * 8 * srow + block * 64);
          mma_dec<W, X>(acc[n], cg[i].x, cu[i].x, cg[i].y, cu[i].y, b.x, b.y);
          mma_dec<W, X>(acc[n], cg[i].z, cu[i].z, cg[i].w, cu[i].w, b.z, b.w);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) red[(warp * NT + n) * 32 + lane] = acc[n];
    __syncthreads();
    if (warp < NT) {
      // tile `warp` of tokens: lane (f, t) has tokens 2 t and 2 t + 1 of column f
      float4 s = red[warp * 32 + lane];
#pragma unroll
      for (int k = 1; k < kDecWarps; ++k) {
        const float4 p = red[(k * NT + warp) * 32 + lane];
        s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
      }
      const int f = unit * 8 + r;
      const float2 g2 = __fmul2_rn(make_float2(s.x, s.y), both(alpha));
      const float2 u2 = __fmul2_rn(make_float2(s.z, s.w), both(alpha));
      const float2 h2 = __fmul2_rn(gate_act(g2, a.act), u2);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = warp * 8 + 2 * t + j;
        if (n < a.T) {
          const float g = j ? g2.y : g2.x, u = j ? u2.y : u2.x, hv = j ? h2.y : h2.x;
          if (a.gu) {
            a.gu[n * 2 * a.F + f] = __float2bfloat16_rn(g);
            a.gu[n * 2 * a.F + a.F + f] = __float2bfloat16_rn(u);
          }
          if (a.h) a.h[n * a.F + f] = __float2bfloat16_rn(hv);
          if (a.q) {
            top = max(top, __float_as_uint(hv) & 0x7FFFFFFFu);
            a.q[n * a.F + f] = static_cast<uint8_t>(a.q_e5m2 ? cvt_e5m2x2(hv * qs, 0.0f) : cvt_e4m3x2(hv * qs, 0.0f));
          }
        }
      }
    }
    __syncthreads();   // the partial sums have been read
  }
  if (a.amax && warp < NT) {
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) atomicMax(a.amax, top);
  }
  if (a.scale_inv && blockIdx.x == 0 && threadIdx.x == 0) *a.scale_inv = __fdiv_rn(1.0f, qs);
}

template <int W, int X, int NT>
te_status launch_decode(const DecodeArgs& a, cudaStream_t st) {
  static PerDevice<SharedMemory> ready;
  te_status s = TE_OK;
  if (!ready.get(&s, [](SharedMemory* m) {
        return allow_shared_memory(m, kernel_address(gated_decode_kernel<W, X, NT>), 232448);
      }))
    return s;
  const int units = a.F / 8;
  const int grid = units < num_sms() ? units : num_sms();
  const size_t smem = decode_smem(a.T, a.K, W == kDecBF16 ? 2 : 1);
  const dim3 g(static_cast<unsigned>(grid), 1, 1), block(32 * kDecWarps, 1, 1);
  if (a.amax) {
    s = zero_amax(a.amax, st);
    if (s != TE_OK) return s;
  }
  const cudaError_t e = launch_dependent(gated_decode_kernel<W, X, NT>, g, block, smem, st, a);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

template <int W, int X>
te_status launch_decode(const DecodeArgs& a, cudaStream_t st) {
  switch ((a.T + 7) / 8) {
    case 1: return launch_decode<W, X, 1>(a, st);
    case 2: return launch_decode<W, X, 2>(a, st);
    case 3: return launch_decode<W, X, 3>(a, st);
    default: return launch_decode<W, X, 4>(a, st);
  }
}

// Whether this kernel takes the call, or the one of gated_stream.cuh (us, this / that):
//   T = 1, BF16: K = 4096, F = 1024 6.0 / 7.5, F = 4096 14.2 / 14.9, F = 16384 42.4 / 47.2; K = 5120,
//   F = 1024 7.6 / 8.5, F = 4096 18.1 / 16.6; K = 8192, F = 1024 9.9 / 11.0, F = 4096 25.9 / 24.1;
//   K = 2048, F = 16384 22.9 / 25.5; K = 1024, F = 4096 6.2 / 6.6, F = 16384 15.2 / 15.0; K = 512,
//   F = 4096 4.9 / 5.2, F = 16384 12.2 / 9.7;
//   T = 1, FP8: K = 4096, F = 1024 4.3 / 5.6, F = 16384 24.3 / 25.2; K = 2048, F = 4096 6.7 / 6.6, F = 16384
//   16.5 / 14.9; K = 512, F = 4096 4.8 / 4.4, F = 16384 11.8 / 7.3;
//   T = 2 to 8 as one token: T = 2 and 8, BF16 K = 4096, F = 1024 6.0 and 6.2 / 7.5 and 7.6, F = 16384 42.7 and
//   43.4 / 47.3 and 44.0, K = 2048, F = 16384 23.1 and 23.5 / 24.8 and 24.7, K = 8192, F = 1024 10.0 and 10.3 /
//   11.0 and 11.1, K = 512, F = 4096 5.0 and 5.0 / 5.3 and 5.3; FP8 K = 4096, F = 1024 4.3 and 4.4 / 5.6 and
//   5.7, F = 16384 24.4 and 24.5 / 25.3 and 24.7, K = 8192, F = 1024 6.6 and 6.8 / 7.5 and 7.6;
//   T = 16: BF16 K = 768, F = 2048 4.3 / 5.5, K = 1024, F = 4096 6.8 / 6.9, F = 8192 9.7 / 9.2, K = 2048,
//   F = 1024 5.7 / 5.8; FP8 K = 768, F = 2048 3.7 / 5.1, K = 1024, F = 2048 4.1 / 5.0, F = 4096 5.9 / 5.5;
//   T = 24: BF16 K = 1024, F = 2048 5.5 / 5.8, K = 2048, F = 1024 6.8 / 6.2; FP8 K = 2048, F = 1024 4.9 / 5.2.
// No tensor memory to set up and loads that go out at once make it the faster one up to eight tokens, but
// for many columns of a short K (each column's sum over the warp's lanes is then most of its work) and for
// few warps on a long K.  Beyond, its matrix rate (512 multiply-adds a clock and SM) and its shared memory
// for x, taken from the L1 that the loads in flight pass through, cost more than that saves unless both x
// and w are small.
inline bool decodes(int64_t T, int64_t K, int64_t F, int elem) {
  if (T > 8 * kDecMaxTiles || K > (1 << 17)) return false;
  const int64_t row = K * elem;
  if (T > 8) {
    if (T * row >= (1 << 16) || F > 2048 * elem) return false;
  } else if (K > 4096 ? F > 1024 : (row < 4096 && F > 2048 && F > 4 * row)) {
    return false;
  }
  return decode_smem(static_cast<int>(T), static_cast<int>(K), elem) <= 232448;
}

}  // namespace
}  // namespace te
