// The gated projections of up to 128 tokens with block-scaled operands (MXFP8, NVFP4): the kernel of
// gated_stream.cuh with the weights as the 128-row operand and the tokens as N, but a tile of 128
// columns of h: a whole 128-row group of the gate's scales and one of the up projection's, each its own
// MMA into its own accumulator, so that a thread finds g and u of its column in the same lane and
// nothing is exchanged.  A stage holds 32 KB of weights; the scale atoms come by bulk copy with it, and
// a copier warp moves them into the stage's tensor-memory slot (gemm_kernel's scheme).
//
// warp 0 producer, warp 1 MMA issuer, warps 2-5 epilogue (lane = column of h; a warp's 32 columns are
// one MXFP8 block of h), warp 6 scale copier.
//
// One token, K = 4096, F = 16384: MXFP8 23.9 us (5.79 TB/s; gemm_kernel 43.2), NVFP4 15.6 us (4.84 TB/s;
// 27.1); 32 tokens 26.4 / 32.7 and 15.9 / 21.3.  128 tiles leave 24 SMs idle; what is left beside that is
// set-up and the first loads' latency (about 4 us).
#pragma once

#include "gated_stream.cuh"

namespace te {
namespace {

constexpr int kStbThreads = 32 * 7;

template <int KIND, int NP>
struct StbCfg {
  static constexpr int kAtoms = KIND == kMXFP8 ? 1 : 4;          // scale atoms per 128 rows and k-tile
  static constexpr int kSf = kAtoms * 512;
  static constexpr int kA = 128 * 128, kB = NP * 128;
  static constexpr int kStage = 2 * kA + kB + 3 * kSf;
  static constexpr int kFit = (232448 - 1024 - 512) / kStage;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kSmemB = kStages * 2 * kA;
  static constexpr int kSmemSf = kSmemB + kStages * kB;
  static constexpr int kSmemBar = kSmemSf + kStages * 3 * kSf;
  static constexpr int kSmemTotal = kSmemBar + 512 + 1024;
  static constexpr int kSfBase = NP == 128 ? 256 : 128, kSfCols = 12 * kAtoms;    // TMEM columns of a stage's scales: g, u, x
  static_assert(kSmemTotal <= 232448 && (3 * kStages + 3) * 8 + 16 <= 512, "shared memory");
  static_assert(NP / 4 * 256 * 16 <= kSmemSf, "the shared accumulators' parts");
  static_assert(2 * NP <= kSfBase && kSfBase + kStages * kSfCols <= 512, "TMEM");
};

// g and u of tokens t0 and t0 + 1 (the same in the whole warp), column f0 + lane: every output.
template <int KIND>
__device__ __forceinline__ void stb_emit(const DecodeArgs& a, float2 g2, float2 u2, int t0, int f0, int lane) {
  const float2 h2 = __fmul2_rn(gate_act(g2, a.act), u2);
  const int f = f0 + lane;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t t = t0 + j;
    if (t >= a.T) break;
    const float gv = j ? g2.y : g2.x, uv = j ? u2.y : u2.x, hv = j ? h2.y : h2.x;
    if (a.gu) {
      a.gu[t * 2 * a.F + f] = __float2bfloat16_rn(gv);
      a.gu[t * 2 * a.F + a.F + f] = __float2bfloat16_rn(uv);
    }
    if (a.h) a.h[t * a.F + f] = __float2bfloat16_rn(hv);
    if (KIND == kMXFP8 && a.q) {
      const int e = mx_exponent(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(hv) & 0x7FFFFFFFu)));
      a.q[t * a.F + f] = static_cast<uint8_t>(cvt_e4m3x2(hv * mx_mult(e), 0.0f));
      if (lane == 0)
        a.s_h[scale_offset(static_cast<uint64_t>(t), static_cast<uint64_t>(f0 >> 5),
                           static_cast<uint64_t>(a.F >> 5))] = static_cast<uint8_t>(e + 127);
    }
  }
}

template <int KIND, int NP, bool SPLIT>   // SPLIT: as in gated_stream_kernel
__global__ void __launch_bounds__(kStbThreads, 1)
    gated_stream_block_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                              const __grid_constant__ DecodeArgs a, uint32_t idesc, int k_tiles, int* err) {
  using C = StbCfg<KIND, NP>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = dev::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sB = smem + C::kSmemB;
  uint8_t* sSf = smem + C::kSmemSf;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kSmemBar);
  uint64_t* empty = full + S;
  uint64_t* sf_ready = empty + S;
  uint64_t* acc_full = sf_ready + S;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = a.F >> 7;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      dev::mbar_init(&full[s], 1);
      dev::mbar_init(&empty[s], 1);
      dev::mbar_init(&sf_ready[s], 1);
    }
    dev::mbar_init(acc_full, 1);
    dev::mbar_init(acc_empty, 4);
    dev::mbar_init(drain, 1);
    *abort_flag = 0;
    dev::fence_barrier_init();
    dev::prefetch_tmap(&tmW);
    dev::prefetch_tmap(&tmX);
  }
  if (warp == 1) dev::tmem_alloc(tmem_slot, 512);
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  dev::pdl_wait();
  dev::pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      const Walk<SPLIT> w(k_tiles);
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      const int64_t katoms = a.s_kpad >> 2;   // scale atoms of a 128-row group
      for (int tile = w.tile; tile < tiles && ok; tile += w.step) {
        for (int kt = 0; kt < w.k_num; ++kt) {
          if (!dev::mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          uint64_t* bar = &full[stage];
          uint8_t* sf = sSf + stage * 3 * C::kSf;
          const int64_t katom = static_cast<int64_t>(w.k_lo + kt) * C::kAtoms;
          dev::mbar_expect_tx(bar, C::kStage);
          dev::bulk_load(sf, a.sw + (tile * katoms + katom) * 512, C::kSf, bar);
          dev::bulk_load(sf + C::kSf, a.sw + ((tiles + tile) * katoms + katom) * 512, C::kSf, bar);
          dev::bulk_load(sf + 2 * C::kSf, a.sx + katom * 512, C::kSf, bar);
          dev::tma_load_2d(smem + stage * 2 * C::kA, &tmW, bar, (w.k_lo + kt) * 128, tile * 128);
          dev::tma_load_2d(smem + stage * 2 * C::kA + C::kA, &tmW, bar, (w.k_lo + kt) * 128, a.F + tile * 128);
          dev::tma_load_2d(sB + stage * C::kB, &tmX, bar, (w.k_lo + kt) * 128, 0);
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
  } else if (warp == 6) {
    if (lane == 0) {
      const Walk<SPLIT> w(k_tiles);
      int stage = 0, last = -1;
      uint32_t phase = 0, last_phase = 0;
      bool ok = true;
      for (int tile = w.tile; tile < tiles && ok; tile += w.step) {
        for (int kt = 0; kt < w.k_num; ++kt) {
          // full of this phase also means that the MMAs that read the slot before have completed
          if (!dev::mbar_wait(&full[stage], phase, abort_flag, err)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t t = tmem_base + C::kSfBase + static_cast<uint32_t>(stage * C::kSfCols);
          const uint32_t s = dev::smem_u32(sSf + stage * 3 * C::kSf);
#pragma unroll
          for (int j = 0; j < C::kAtoms; ++j)
#pragma unroll
            for (int o = 0; o < 3; ++o)
              dev::tc_cp_32x128b_x4(t + 4 * (o * C::kAtoms + j), dev::smem_desc(s + o * C::kSf + 512 * j, 0, 128, 0));
          dev::tc_commit(&sf_ready[stage]);
          last = stage;
          last_phase = phase;
          if (++stage == S) stage = 0, phase ^= 1u;
        }
      }
      if (!ok && last >= 0) {
        // bounded wait for this thread's last copies before TMEM can be released
        volatile int dummy = 0;
        dev::mbar_wait(&sf_ready[last], last_phase, &dummy, err);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const Walk<SPLIT> w(k_tiles);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = w.tile; tile < tiles && ok; tile += w.step, ++it) {
        if (!dev::mbar_wait(acc_empty, (static_cast<uint32_t>(it) & 1u) ^ 1u, abort_flag, err)) break;
        dev::tc_fence_after();
        for (int kt = 0; kt < w.k_num; ++kt) {
          // the scales in tensor memory: the stage's operands have landed too, on the same barrier
          if (!dev::mbar_wait(&full[stage], phase, abort_flag, err) ||
              !dev::mbar_wait(&sf_ready[stage], phase, abort_flag, err)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t sb = dev::smem_u32(sB + stage * C::kB);
          const uint32_t sf = tmem_base + C::kSfBase + static_cast<uint32_t>(stage * C::kSfCols);
          const uint32_t sfb = sf + 8 * C::kAtoms;
#pragma unroll
          for (int o = 0; o < 2; ++o) {   // g, then u
            const uint32_t sa = dev::smem_u32(smem + stage * 2 * C::kA + o * C::kA);
            const uint32_t sfa = sf + 4 * o * C::kAtoms, d = tmem_base + static_cast<uint32_t>(o * NP);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              const uint64_t ad = dev::smem_desc(sa + 32 * ks, 0, 1024, 2), bd = dev::smem_desc(sb + 32 * ks, 0, 1024, 2);
              if (KIND == kMXFP8)   // scale byte `ks` of each 32-bit scale column
                dev::mma_mxf8f6f4(d, ad, bd, idesc | (static_cast<uint32_t>(ks) << 29) | (static_cast<uint32_t>(ks) << 4),
                                  sfa, sfb, (kt | ks) != 0);
              else
                dev::mma_mxf4nvf4(d, ad, bd, idesc, sfa + 4 * ks, sfb + 4 * ks, (kt | ks) != 0);
            }
          }
          dev::tc_commit(&empty[stage]);
          if (++stage == S) stage = 0, phase ^= 1u;
        }
        if (!ok) break;
        dev::tc_commit(acc_full);
      }
      dev::tc_commit(drain);
      volatile int dummy = 0;
      dev::mbar_wait(drain, 0, &dummy, err);
    }
  } else {
    const Walk<SPLIT> w(k_tiles);
    const int quarter = warp & 3;
    const float alpha = (a.alpha_a ? *a.alpha_a : 1.0f) * (a.alpha_b ? *a.alpha_b : 1.0f);
    int it = 0;
    for (int tile = w.tile; tile < tiles; tile += w.step, ++it) {
      const bool ok = __all_sync(0xFFFFFFFFu, dev::mbar_wait(acc_full, static_cast<uint32_t>(it) & 1u, abort_flag, err));
      if (!SPLIT && !ok) break;
      dev::tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
      const int f0 = tile * 128 + quarter * 32;
      if constexpr (SPLIT) {
        // every load of the cluster has landed and every MMA has read it: the rings are free
        dev::cluster_sync();
        const int per = NP / 4 / w.split, row = quarter * 32 + lane;
        const uint32_t buffer = dev::smem_u32(smem);
#pragma unroll
        for (int c = 0; c < NP / 32; ++c) {
          if (32 * c >= a.T && c > 0) break;
          uint32_t g[32], u[32];
          dev::tmem_ld_32x32b_x32(taddr + 32 * c, g);
          dev::tmem_ld_32x32b_x32(taddr + NP + 32 * c, u);
          dev::tmem_ld_wait();
          dev::reg_fence(g);
          dev::reg_fence(u);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (32 * c + 4 * i < a.T) {
              kpart_send(g, 4 * i, buffer, w.split, w.part, 8 * c + i, per, 256, row);
              kpart_send(u, 4 * i, buffer, w.split, w.part, 8 * c + i, per, 256, 128 + row);
            }
        }
        dev::cluster_sync();
        if (!ok) break;
        for (int j = 0; j < per; ++j) {
          const int t0 = 4 * (j * w.split + w.part);
          if (t0 >= a.T) break;
          float2 g[2] = {}, u[2] = {};
          for (int from = 0; from < w.split; ++from) {
            const uint8_t* p = smem + kpart_offset(from, j, per, 256, row);
            const float4 gv = *reinterpret_cast<const float4*>(p);
            const float4 uv = *reinterpret_cast<const float4*>(p + 128 * 16);
            g[0] = __fadd2_rn(g[0], make_float2(gv.x, gv.y));
            g[1] = __fadd2_rn(g[1], make_float2(gv.z, gv.w));
            u[0] = __fadd2_rn(u[0], make_float2(uv.x, uv.y));
            u[1] = __fadd2_rn(u[1], make_float2(uv.z, uv.w));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
            stb_emit<KIND>(a, __fmul2_rn(g[i], both(alpha)), __fmul2_rn(u[i], both(alpha)), t0 + 2 * i, f0, lane);
        }
        break;
      }
#pragma unroll
      for (int c = 0; c < NP / 32; ++c) {
        if (32 * c >= a.T && c > 0) break;
        uint32_t g[32], u[32];
        dev::tmem_ld_32x32b_x32(taddr + 32 * c, g);
        dev::tmem_ld_32x32b_x32(taddr + NP + 32 * c, u);
        dev::tmem_ld_wait();
        dev::reg_fence(g);
        dev::reg_fence(u);
        if (c == NP / 32 - 1 || 32 * (c + 1) >= a.T) {   // the last of the accumulators that is read
          dev::tc_fence_before();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(acc_empty);
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 g2 = __fmul2_rn(pair_of(g, i), both(alpha)), u2 = __fmul2_rn(pair_of(u, i), both(alpha));
          stb_emit<KIND>(a, g2, u2, 32 * c + i, f0, lane);
        }
      }
    }
    if (KIND == kMXFP8 && a.q) {
      // padding rows T to 127 of h's scales, four scale columns a word
      const int kw = a.F >> 7;
      const int64_t words = static_cast<int64_t>(128 - a.T) * kw;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + (threadIdx.x - 64); i < words;
           i += static_cast<int64_t>(gridDim.x) * 128)
        *reinterpret_cast<uint32_t*>(a.s_h + scale_offset(static_cast<uint64_t>(a.T + i / kw),
                                                          static_cast<uint64_t>(i % kw * 4),
                                                          static_cast<uint64_t>(a.F >> 5))) = 0u;
    }
  }

  if constexpr (SPLIT) {
    if (warp < 2 || warp == 6) {   // the other warps' part in the epilogue's two barriers
      __syncwarp();
      dev::cluster_sync();
      dev::cluster_sync();
    }
  }
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  if (warp == 1) dev::tmem_dealloc(tmem_base, 512);
}

template <int KIND, int NP>
te_status launch_stream_block(const DecodeArgs& a, uint32_t xfmt, uint32_t wfmt, cudaStream_t st, bool* taken) {
  using C = StbCfg<KIND, NP>;
  constexpr bool kSharedOnly = NP == 128;
  *taken = true;
  static PerDevice<StreamSetup> setups;
  te_status s = TE_OK;
  const StreamSetup* setup = setups.get(&s, [](StreamSetup* m) {
    return m->set(kernel_address(gated_stream_block_kernel<KIND, NP, kSharedOnly>),
                  kernel_address(gated_stream_block_kernel<KIND, NP, true>), kStbThreads, C::kSmemTotal);
  });
  if (setup == nullptr) return s;
  const uint64_t row_bytes = static_cast<uint64_t>(a.K) / (KIND == kMXFP8 ? 1 : 2);
  const int tiles = a.F / 128;
  const int k_tiles = static_cast<int>((row_bytes + 127) / 128);
  const int split = stream_split(tiles, k_tiles, setup->most);
  if (!stream_takes(KIND, a.T, k_tiles, split, tiles <= setup->most[0])) {
    *taken = false;
    return TE_OK;
  }
  CUtensorMap tw, tx;
  s = make_tmap_2d(&tw, a.w, row_bytes, 2 * static_cast<uint64_t>(a.F), 128);
  if (s != TE_OK) return s;
  s = make_tmap_2d(&tx, a.x, row_bytes, static_cast<uint64_t>(a.T), NP);
  if (s != TE_OK) return s;
  int* err = device_error_word();
  if (err == nullptr) return record_cuda(cudaErrorInvalidDevice);
  // the weights are operand A: M = 128, N = NP
  uint32_t idesc = make_idesc(KIND, wfmt, xfmt, 128);
  idesc = (idesc & ~(0x3Fu << 17)) | (static_cast<uint32_t>(NP >> 3) << 17);
  const int grid = split > 1 ? split * tiles : (tiles < num_sms() ? tiles : num_sms());
  const dim3 g(static_cast<unsigned>(grid), 1, 1), block(kStbThreads, 1, 1);
  const cudaError_t e =
      split > 1 ? launch_dependent_clusters(gated_stream_block_kernel<KIND, NP, true>, split, g, block, C::kSmemTotal,
                                            st, tw, tx, a, idesc, k_tiles, err)
                : launch_dependent(gated_stream_block_kernel<KIND, NP, kSharedOnly>, g, block, C::kSmemTotal, st, tw, tx, a,
                                   idesc, k_tiles, err);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

template <int KIND>
te_status launch_stream_block(const DecodeArgs& a, uint32_t xfmt, uint32_t wfmt, cudaStream_t st, bool* taken) {
  return a.T <= 32   ? launch_stream_block<KIND, 32>(a, xfmt, wfmt, st, taken)
         : a.T <= 64 ? launch_stream_block<KIND, 64>(a, xfmt, wfmt, st, taken)
                     : launch_stream_block<KIND, 128>(a, xfmt, wfmt, st, taken);
}

}  // namespace
}  // namespace te
