// The gated projections of up to 128 tokens that the kernel of gated_decode.cuh does not take: still a
// stream over the weights, but with too much matrix work for mma.sync.  The operands change places
// against gemm_kernel: the weights are the 128-row operand of the MMA (64 gate rows and the 64 up rows
// beside them) and the tokens its N (32, 64 or 128), so a stage is 16 KB of weights and 4, 8 or 16 KB of
// x, and ten (eight, six) of them fit where gemm_kernel has six with as much x as weights: 160 KB of weights in
// flight per SM.  One CTA per SM, no pairs: tiles of 64 columns of h, and a CTA with one tile more than
// another has that much more of the bandwidth at the end.  From 65 tokens on only where the tiles are
// shared (stream_takes has the rule).
//
// warp 0 TMA producer, warp 1 MMA issuer, warps 2-5 epilogue.  Accumulator lanes 0-63 hold g and 64-127
// u of the tile's columns, tokens along the TMEM columns: the g warps hand the second half of the
// tokens to the u warps through shared memory and get the first half's u back, and each thread then
// has one column of h for half of the tokens; neighbouring lanes write neighbouring columns.  (Tiles of
// 128 columns without the exchange, as gated_stream_block.cuh has them, are as fast at F = 16384 but
// leave more SMs idle at smaller F: 24 tokens, K = F = 4096 BF16 18.7 us here, 25.3 so, with one CTA a
// tile.)  Where the tiles leave SMs idle, clusters of 2, 4 or 8 CTAs share a tile's K (below).
//
// 24 tokens, K = 4096, F = 16384: BF16 44.1 us (6.09 TB/s; gemm_kernel 51.5), FP8 24.8 us (5.41 TB/s;
// 33.2); 64 tokens 46.9 / 49.6 and 27.2 / 27.6.  gemm_kernel's six stages turn round in about 1.7 us
// (load, MMA, commit), which bounds what an SM can have in flight; these turn round in less and are more.
#pragma once

#include "gated_decode.cuh"
#include "launch_setup.cuh"

namespace te {
namespace {

constexpr int kStrThreads = 32 * 6;
constexpr int64_t kStrMaxTokens = 128;   // 64 where a tile's K is not shared
constexpr int kStrMaxStages = 12;

template <int NP>   // tokens, padded
struct StrCfg {
  static constexpr int kA = 128 * 128, kB = NP * 128;
  static constexpr int kExchange = NP * 64 * 4;
  static constexpr int kFit = (232448 - 1024 - 512 - kExchange) / (kA + kB);
  static constexpr int kStages = kFit < kStrMaxStages ? kFit : kStrMaxStages;
  static constexpr int kSmemB = kStages * kA;
  static constexpr int kSmemX = kSmemB + kStages * kB;
  static constexpr int kSmemBar = kSmemX + kExchange;
  static constexpr int kSmemTotal = kSmemBar + 512 + 1024;
  static constexpr int kCols = 2 * NP;   // two accumulators
  static_assert(kSmemTotal <= 232448 && (2 * kStages + 5) * 8 + 16 <= 512, "shared memory");
  static_assert(NP == 32 || NP == 64 || NP == 128, "whole tcgen05.ld chunks, power-of-two TMEM columns");
  static_assert(NP / 4 * 128 * 16 <= kSmemX, "the shared accumulators' parts");
};

// A CTA's walk: its first tile and the step to the next, and its part of the k-tiles where a cluster shares
// a tile's K (SPLIT).  Each role makes its own: kept in registers from the start of the kernel on, the same
// numbers cost 0.3 us a call.
template <bool SPLIT>
struct Walk {
  int split, part, tile, step, k_lo, k_num;
  __device__ __forceinline__ explicit Walk(int k_tiles)
      : split(1), part(0), tile(static_cast<int>(blockIdx.x)), step(static_cast<int>(gridDim.x)), k_lo(0),
        k_num(k_tiles) {
    if constexpr (SPLIT) {
      asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(split));
      part = static_cast<int>(dev::cluster_ctarank());
      tile /= split;
      step /= split;
      k_lo = k_tiles * part / split;
      k_num = k_tiles * (part + 1) / split - k_lo;
    }
  }
};

// What the CTAs of a cluster send one another: four tokens of a row of an accumulator in 16 bytes, the
// tokens of group i going to CTA i % split, where the parts of CTA 0, 1, ... of its j-th group lie in
// rows of `rows`.
__device__ __forceinline__ uint32_t kpart_offset(int from, int j, int per, int rows, int row) {
  return static_cast<uint32_t>(((from * per + j) * rows + row) * 16);
}
// Tokens 4 i to 4 i + 3 of this thread's row to their owner's buffer (at the start of shared memory).
template <int N>
__device__ __forceinline__ void kpart_send(const uint32_t (&acc)[N], int at, uint32_t buffer, int split, int part, int group,
                                           int per, int rows, int row) {
  const int owner = group & (split - 1), j = group / split;
  dev::st_shared_cluster_v4(
      dev::mapa_shared(buffer + kpart_offset(part, j, per, rows, row), static_cast<uint32_t>(owner)), acc[at],
      acc[at + 1], acc[at + 2], acc[at + 3]);
}

// SPLIT: a cluster of `split` CTAs has one tile and each of them a part of K; they add their accumulators
// through distributed shared memory, every one of them for its groups of four tokens and in the CTAs'
// order, so the result does not depend on timing.
template <int KIND, int NP, bool SPLIT>
__global__ void __launch_bounds__(kStrThreads, 1)
    gated_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ DecodeArgs a, uint32_t idesc, int k_tiles, int* err) {
  using C = StrCfg<NP>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = dev::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::kSmemB;
  float* ex = reinterpret_cast<float*>(smem + C::kSmemX);   // [token][64 columns]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kSmemBar);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (a.F + 63) / 64;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      dev::mbar_init(&full[s], 1);
      dev::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      dev::mbar_init(&acc_full[s], 1);
      dev::mbar_init(&acc_empty[s], 4);
    }
    dev::mbar_init(drain, 1);
    *abort_flag = 0;
    dev::fence_barrier_init();
    dev::prefetch_tmap(&tmW);
    dev::prefetch_tmap(&tmX);
  }
  if (warp == 1) dev::tmem_alloc(tmem_slot, C::kCols);
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  dev::pdl_wait();
  dev::pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      const Walk<SPLIT> w(k_tiles);
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      for (int tile = w.tile; tile < tiles && ok; tile += w.step) {
        for (int kt = 0; kt < w.k_num; ++kt) {
          if (!dev::mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          dev::mbar_expect_tx(&full[stage], C::kA + C::kB);
          dev::tma_load_2d(sA + stage * C::kA, &tmW, &full[stage], (w.k_lo + kt) * 128, tile * 64);
          dev::tma_load_2d(sA + stage * C::kA + 64 * 128, &tmW, &full[stage], (w.k_lo + kt) * 128, a.F + tile * 64);
          dev::tma_load_2d(sB + stage * C::kB, &tmX, &full[stage], (w.k_lo + kt) * 128, 0);
          ++issued;
          if (++stage == S) stage = 0, phase ^= 1u;
        }
      }
      if (!ok) {
        // bounded wait for the copies in flight, the latest S at most
        volatile int dummy = 0;
        for (int i = issued > S ? issued - S : 0; i < issued; ++i)
          dev::mbar_wait(&full[i % S], static_cast<uint32_t>(i / S) & 1u, &dummy, err);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const Walk<SPLIT> w(k_tiles);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = w.tile; tile < tiles && ok; tile += w.step, ++it) {
        const int as = it & 1;
        if (!dev::mbar_wait(&acc_empty[as], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, abort_flag, err)) break;
        dev::tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(as * NP);
        for (int kt = 0; kt < w.k_num; ++kt) {
          if (!dev::mbar_wait(&full[stage], phase, abort_flag, err)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t sa = dev::smem_u32(sA + stage * C::kA), sb = dev::smem_u32(sB + stage * C::kB);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t ad = dev::smem_desc(sa + 32 * ks, 0, 1024, 2), bd = dev::smem_desc(sb + 32 * ks, 0, 1024, 2);
            if (KIND == kBF16) dev::mma_f16(d, ad, bd, idesc, (kt | ks) != 0);
            else dev::mma_f8f6f4(d, ad, bd, idesc, (kt | ks) != 0);
          }
          dev::tc_commit(&empty[stage]);
          if (++stage == S) stage = 0, phase ^= 1u;
        }
        if (!ok) break;
        dev::tc_commit(&acc_full[as]);
      }
      dev::tc_commit(drain);
      volatile int dummy = 0;
      dev::mbar_wait(drain, 0, &dummy, err);
    }
  } else {
    const Walk<SPLIT> w(k_tiles);
    const int quarter = warp & 3;
    const bool up = quarter >= 2;                 // lanes 64-127 of the accumulator: u
    const int fl = (quarter & 1) * 32 + lane;     // column of the tile
    const float alpha = (a.alpha_a ? *a.alpha_a : 1.0f) * (a.alpha_b ? *a.alpha_b : 1.0f);
    const float qs = a.q ? *a.q_scale : 1.0f;
    unsigned int top = 0;
    // g and u of tokens t0 and t0 + 1, column f
    auto emit = [&](float2 g, float2 u, int t0, int f) {
      const float2 h = __fmul2_rn(gate_act(g, a.act), u);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + j;
        if (t < a.T && f < a.F) {
          const float gv = j ? g.y : g.x, uv = j ? u.y : u.x, hv = j ? h.y : h.x;
          if (a.gu) {
            a.gu[t * 2 * a.F + f] = __float2bfloat16_rn(gv);
            a.gu[t * 2 * a.F + a.F + f] = __float2bfloat16_rn(uv);
          }
          if (a.h) a.h[t * a.F + f] = __float2bfloat16_rn(hv);
          if (a.q) {
            top = max(top, __float_as_uint(hv) & 0x7FFFFFFFu);
            a.q[t * a.F + f] = static_cast<uint8_t>(a.q_e5m2 ? cvt_e5m2x2(hv * qs, 0.0f) : cvt_e4m3x2(hv * qs, 0.0f));
          }
        }
      }
    };
    int it = 0;
    bool ok = true;
    for (int tile = w.tile; tile < tiles; tile += w.step, ++it) {
      const int as = it & 1;
      if (!dev::mbar_wait(&acc_full[as], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, err)) ok = false;
      if (!SPLIT) {
        // the four warps leave together: the exchange below has barriers of all of them
        int all_ok;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
            : "=r"(all_ok)
            : "r"(static_cast<int>(ok))
            : "memory");
        if (!all_ok) break;
      }
      dev::tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(as * NP);
      if constexpr (SPLIT) {
        // every load of the cluster has landed and every MMA has read it: the rings are free
        __syncwarp();
        dev::cluster_sync();
        const int per = NP / 4 / w.split, row = quarter * 32 + lane;
#pragma unroll
        for (int c = 0; c < NP / 32; ++c) {
          if (32 * c >= a.T) break;
          uint32_t acc[32];
          dev::tmem_ld_32x32b_x32(taddr + 32 * c, acc);
          dev::tmem_ld_wait();
          dev::reg_fence(acc);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (32 * c + 4 * i < a.T)
              kpart_send(acc, 4 * i, dev::smem_u32(smem), w.split, w.part, 8 * c + i, per, 128, row);
        }
        dev::tc_fence_before();
        dev::cluster_sync();
        if (!ok) break;
        const int col = row & 63, hi = row >> 6;   // this thread: a column, two tokens of the four
        for (int j = 0; j < per; ++j) {
          const int t0 = 4 * (j * w.split + w.part);
          if (t0 >= a.T) break;
          float2 g = make_float2(0.0f, 0.0f), u = g;
          for (int from = 0; from < w.split; ++from) {
            const uint8_t* p = smem + kpart_offset(from, j, per, 128, col) + 8 * hi;
            g = __fadd2_rn(g, *reinterpret_cast<const float2*>(p));
            u = __fadd2_rn(u, *reinterpret_cast<const float2*>(p + 64 * 16));
          }
          emit(__fmul2_rn(g, both(alpha)), __fmul2_rn(u, both(alpha)), t0 + 2 * hi, tile * 64 + col);
        }
        break;
      }
      uint32_t acc[NP / 32][32];
#pragma unroll
      for (int c = 0; c < NP / 32; ++c) dev::tmem_ld_32x32b_x32(taddr + 32 * c, acc[c]);
      dev::tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < NP / 32; ++c) dev::reg_fence(acc[c]);
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&acc_empty[as]);
      // g warps give away the second half of the tokens, u warps the first
#pragma unroll
      for (int n = 0; n < NP / 2; ++n) {
        const int give = up ? n : n + NP / 2;
        ex[give * 64 + fl] = __uint_as_float(up ? acc[n / 32][n % 32] : acc[(n + NP / 2) / 32][(n + NP / 2) % 32]);
      }
      asm volatile("bar.sync 2, 128;" ::: "memory");
      const int f = tile * 64 + fl;
#pragma unroll
      for (int n = 0; n < NP / 2; n += 2) {
        const int n0 = up ? n + NP / 2 : n;
        const float2 mine = make_float2(
            __uint_as_float(up ? acc[(n + NP / 2) / 32][(n + NP / 2) % 32] : acc[n / 32][n % 32]),
            __uint_as_float(up ? acc[(n + NP / 2 + 1) / 32][(n + NP / 2 + 1) % 32] : acc[(n + 1) / 32][(n + 1) % 32]));
        const float2 got = make_float2(ex[n0 * 64 + fl], ex[(n0 + 1) * 64 + fl]);
        const float2 g = __fmul2_rn(up ? got : mine, both(alpha)), u = __fmul2_rn(up ? mine : got, both(alpha));
        emit(g, u, n0, f);
      }
      // (the exchange is written again only after the next tile's first barrier)
    }
    if (a.amax) {
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      if (lane == 0) atomicMax(a.amax, top);
    }
    if (a.scale_inv && blockIdx.x == 0 && threadIdx.x == 64) *a.scale_inv = __fdiv_rn(1.0f, qs);
  }

  if constexpr (SPLIT) {
    if (warp < 2) {   // the other warps' part in the epilogue's two barriers
      __syncwarp();
      dev::cluster_sync();
      dev::cluster_sync();
    }
  }
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  if (warp == 1) dev::tmem_dealloc(tmem_base, C::kCols);
}

// The CTAs that share a tile's K: as many of 2, 4 and 8 as the tiles leave SMs for and K has k-tiles for.
// most[i]: clusters of 2 << i CTAs that run at once.  One CTA a tile / shared, one token MXFP8 (24 tokens
// BF16): F = 2048, K = 2048 9.0 / 6.3 us (8.3 / 7.2), K = 4096 14.7 / 8.0 (17.3 / 9.7), K = 8192 26.0 / 11.5
// (30.6 / 14.8); F = 4096, K = 16384 48.8 / 25.0 (58.1 / 45.0).  The exchange takes about 1 us: MXFP8
// K = 768 (6 k-tiles) 5.4 / 4.9, K = 512 4.2 / 4.0, K = 256 (2) 3.4 / 3.7.
inline int stream_split(int tiles, int k_tiles, const int (&most)[3]) {
  for (int i = 2; i >= 0; --i)
    if (tiles <= most[i] && k_tiles >= (2 << i) && k_tiles > 2) return 2 << i;
  return 1;
}

// Whether a call runs here or in gemm_kernel, whose time hardly depends on the tokens while the exchange's
// and the outputs' part of this one's grows with them: up to 32 tokens always, beyond where K has the
// k-tiles to pay for them.  Here / there, us:
//   65 and 128 tokens: BF16 K = 4096, F = 2048 11.2 and 13.1 / 16.8, F = 4096 (split 2) 17.3 and 20.3 / 20.0,
//   K = 8192, F = 2048 16.2 and 18.4 / 28.6; FP8 K = F = 2048 7.5 and 9.2 / 9.3, K = F = 4096 (split 2) 12.1
//   and 15.1 / 14.1; MXFP8 K = F = 2048 (16 k-tiles) 9.5 and 12.2 / 10.2, K = 4096, F = 2048 11.5 and 14.2 /
//   15.4, F = 8192 (split 2) 19.2 and 23.2 / 18.2; NVFP4 K = 4096, F = 2048 (16) 9.4 and 11.7 / 11.0;
//   33 and 64 tokens, few k-tiles: BF16 K = 512, F = 4096 (split 2) 7.0 and 8.1 / 7.6, F = 16384 13.6 and
//   14.2 / 12.2; FP8 K = 1024, F = 16384 13.5 and 14.2 / 11.9; MXFP8 K = 1024, F = 4096 (split 4) 7.6 and 8.7 /
//   8.0, F = 8192 (split 2) 9.4 and 11.3 / 9.1, K = 2048, F = 16384 16.8 and 19.0 / 18.6; NVFP4 K = 1024,
//   F = 4096 6.5 and 7.4 / 7.0, K = 4096, F = 8192 (split 2) 12.2 and 13.6 / 12.7, F = 16384 18.1 and 18.2 / 19.4;
//   where the tokens cut, 48 and 49: BF16 K = 512, F = 4096 7.3 and 7.6 / 7.7; MXFP8 K = 1024, F = 4096 8.0 and
//   8.3 / 8.1, K = 2048, F = 8192 (split 2) 12.5 and 12.8 / 13.0, F = 16384 17.9 and 18.2 / 20.3 and 21.0 (64: 19.1 /
//   18.5); NVFP4 K = 1024, F = 4096 6.8 and 7.2 / 6.9, K = 4096, F = 8192 (split 2) 12.9 and 13.1 / 13.2;
//   80 and 81 (few k-tiles): MXFP8 K = F = 2048 9.9 and 10.2 / 10.2, NVFP4 K = 4096, F = 2048 9.7 and 10.1 / 10.9,
//   FP8 K = F = 2048 (16 k-tiles: all) 7.7 and 8.0 / 9.3; 96 and 97 (split 2): BF16 K = F = 4096 19.0 and 19.3 /
//   20.1, FP8 K = F = 4096 13.5 and 13.8 / 14.1.
// `idle`: the tiles leave SMs for a split.
inline bool stream_takes(int kind, int64_t T, int k_tiles, int split, bool idle) {
  const bool block = kind == kMXFP8 || kind == kNVFP4;
  if (T <= 32) return true;
  if (T <= 64) {
    if (!block) return split >= 4 || k_tiles >= 16 || (split == 2 && k_tiles >= 4 && T <= 48);
    const bool long_k = k_tiles >= (kind == kMXFP8 ? 16 : 8);   // K >= 2048
    if (k_tiles >= 32) return true;
    if (split == 1) return !idle && (kind == kNVFP4 || T <= 48);
    return split == 2 ? long_k && T <= 48 : long_k || T <= 48;
  }
  const int enough = block ? 32 : 16;
  if (split >= 4) return k_tiles >= enough || (2 * k_tiles >= enough && T <= 80);
  return split == 2 && !block && k_tiles >= 32 && T <= 96;
}

// launch_dependent of clusters of `split` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_dependent_clusters(void (*kernel)(Params...), int split, dim3 grid, dim3 block, size_t smem,
                                      cudaStream_t st, Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(split), 1u, 1u};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// *taken: whether the call runs here.
template <int KIND, int NP>
te_status launch_stream(const DecodeArgs& a, uint32_t xfmt, uint32_t wfmt, cudaStream_t st, bool* taken) {
  using C = StrCfg<NP>;
  constexpr bool kSharedOnly = NP == 128;
  *taken = true;
  static PerDevice<StreamSetup> setups;
  te_status s = TE_OK;
  const StreamSetup* setup = setups.get(&s, [](StreamSetup* m) {
    return m->set(kernel_address(gated_stream_kernel<KIND, NP, kSharedOnly>),
                  kernel_address(gated_stream_kernel<KIND, NP, true>), kStrThreads, C::kSmemTotal);
  });
  if (setup == nullptr) return s;
  const uint64_t row_bytes = static_cast<uint64_t>(a.K) * (KIND == kBF16 ? 2 : 1);
  const int tiles = (a.F + 63) / 64;
  const int k_tiles = static_cast<int>((row_bytes + 127) / 128);
  const int split = stream_split(tiles, k_tiles, setup->most);
  if (!stream_takes(KIND, a.T, k_tiles, split, tiles <= setup->most[0])) {
    *taken = false;
    return TE_OK;
  }
  CUtensorMap tw, tx;
  s = make_tmap_2d(&tw, a.w, row_bytes, 2 * static_cast<uint64_t>(a.F), 64);
  if (s != TE_OK) return s;
  s = make_tmap_2d(&tx, a.x, row_bytes, static_cast<uint64_t>(a.T), NP);
  if (s != TE_OK) return s;
  int* err = device_error_word();
  if (err == nullptr) return record_cuda(cudaErrorInvalidDevice);
  // the weights are operand A: M = 128, N = NP
  uint32_t idesc = make_idesc(KIND, wfmt, xfmt, 128);
  idesc = (idesc & ~(0x3Fu << 17)) | (static_cast<uint32_t>(NP >> 3) << 17);
  const int grid = split > 1 ? split * tiles : (tiles < num_sms() ? tiles : num_sms());
  if (a.amax && (s = zero_amax(a.amax, st)) != TE_OK) return s;
  const dim3 g(static_cast<unsigned>(grid), 1, 1), block(kStrThreads, 1, 1);
  const cudaError_t e =
      split > 1 ? launch_dependent_clusters(gated_stream_kernel<KIND, NP, true>, split, g, block, C::kSmemTotal, st, tw,
                                            tx, a, idesc, k_tiles, err)
                : launch_dependent(gated_stream_kernel<KIND, NP, kSharedOnly>, g, block, C::kSmemTotal, st, tw, tx, a, idesc,
                                   k_tiles, err);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

template <int KIND>
te_status launch_stream(const DecodeArgs& a, uint32_t xfmt, uint32_t wfmt, cudaStream_t st, bool* taken) {
  return a.T <= 32   ? launch_stream<KIND, 32>(a, xfmt, wfmt, st, taken)
         : a.T <= 64 ? launch_stream<KIND, 64>(a, xfmt, wfmt, st, taken)
                     : launch_stream<KIND, 128>(a, xfmt, wfmt, st, taken);
}

}  // namespace
}  // namespace te
