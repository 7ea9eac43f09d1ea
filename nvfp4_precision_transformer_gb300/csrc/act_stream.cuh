// The linear with bias, activation and residual for up to 128 tokens that the kernel of act_decode.cuh does not
// take, every operand kind: still a stream over the weights, but with too much matrix work for mma.sync.  The
// operands change places against gemm_kernel: up to 128 rows of w are the 128-row operand of the MMA and the tokens
// its N (32, 64 or 128), so a stage is 16 KB of weights and 4, 8 or 16 KB of x (and, block-scaled, the scale atoms of
// both), and as many stages as fit keep loads in flight.  One CTA per SM, no pairs.
//
// warp 0 TMA producer, warp 1 MMA issuer, warps 2-5 epilogue, warp 6 (block-scaled kinds) copies the scale atoms to
// tensor memory.  An accumulator lane is a column of y and the tokens lie along the TMEM columns, so neighbouring
// lanes write neighbouring columns, and a warp's 32 columns are one MXFP8 block of q.  Where the tiles leave SMs
// idle, clusters of 2, 4 or 8 CTAs share a tile's K and add their parts through distributed shared memory, each of
// them for its groups of four tokens and in the CTAs' order, so the result does not depend on timing.
#pragma once

#include "act_decode.cuh"

namespace te {
namespace {

constexpr int64_t kAstMaxTokens = 128;

template <int KIND, int NP>   // tokens, padded
struct AstCfg {
  static constexpr bool kBlock = KIND >= kMXFP8;
  static constexpr int kAtoms = KIND == kMXFP8 ? 1 : (KIND == kNVFP4 ? 4 : 0);   // scale atoms per 128 rows and k-tile
  static constexpr int kSf = kAtoms * 512;
  static constexpr int kA = 128 * 128, kB = NP * 128;
  static constexpr int kStage = kA + kB + 2 * kSf;
  static constexpr int kFit = (232448 - 1024 - 512) / kStage;
  static constexpr int kSfBase = NP == 128 ? 256 : 128, kSfCols = 8 * kAtoms;    // TMEM columns of a stage's scales
  static constexpr int kMost = KIND == kNVFP4 ? (512 - kSfBase) / kSfCols : 12;
  static constexpr int kStages = kFit < kMost ? kFit : kMost;
  static constexpr int kSmemB = kStages * kA;
  static constexpr int kSmemSf = kSmemB + kStages * kB;
  static constexpr int kSmemBar = kSmemSf + kStages * 2 * kSf;
  static constexpr int kSmemTotal = kSmemBar + 512 + 1024;
  static constexpr int kCols = kBlock ? 512 : 2 * NP;   // two accumulators, and the scales
  static constexpr int kThreads = 32 * (kBlock ? 7 : 6);
  static_assert(kSmemTotal <= 232448 && (3 * kStages + 5) * 8 + 16 <= 512, "shared memory");
  static_assert(NP == 32 || NP == 64 || NP == 128, "whole tcgen05.ld chunks, power-of-two TMEM columns");
  static_assert(!kBlock || (2 * NP <= kSfBase && kSfBase + kStages * kSfCols <= 512), "TMEM");
  static_assert(NP / 4 * 128 * 16 <= kSmemSf, "the shared accumulators' parts");
};

// Four tokens from t0 of column n (live: the column is one of y's): every output.  The whole warp, the same t0.
template <int KIND>
__device__ __forceinline__ void ast_emit(const FewArgs& a, const float4& acc, float alpha, float bias, float qs, int t0,
                                         int n, bool live, int lane, unsigned int& top) {
  const float2 za = __ffma2_rn(make_float2(acc.x, acc.y), both(alpha), both(bias));
  const float2 zb = __ffma2_rn(make_float2(acc.z, acc.w), both(alpha), both(bias));
  const float2 va = act_value(za, a.act), vb = act_value(zb, a.act);
  const float z[4] = {za.x, za.y, zb.x, zb.y}, v[4] = {va.x, va.y, vb.x, vb.y};
  float res[4];   // all of them before the first store: y may be residual
#pragma unroll
  for (int j = 0; j < 4; ++j)
    res[j] = live && t0 + j < a.T ? few_residual(a, static_cast<int64_t>(t0 + j) * a.N + n) : 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t t = t0 + j;
    if (t >= a.T) break;
    const int64_t at = t * a.N + n;
    if (live) few_store(a, at, z[j], v[j], res[j]);
    if (!a.q) continue;
    if (KIND == kMXFP8) {
      // (N is a multiple of 32: a warp's columns are all live or none)
      const int e = mx_exponent(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[j]) & 0x7FFFFFFFu)));
      if (live) a.q[at] = static_cast<uint8_t>(cvt_e4m3x2(v[j] * mx_mult(e), 0.0f));
      const int64_t block = (n - lane) >> 5;
      if (lane == 0 && block < a.q_kpad)   // past the last column: padding
        a.s_q[scale_offset(static_cast<uint64_t>(t), static_cast<uint64_t>(block), static_cast<uint64_t>(a.q_kpad))] =
            live ? static_cast<uint8_t>(e + 127) : uint8_t(0);
    } else if (live) {
      top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      a.q[at] = few_code(a, v[j], qs);
    }
  }
}

// rows: of w in a tile (128 for the block-scaled kinds, whose scales come in groups of 128 rows).
template <int KIND, int NP, bool SPLIT>
__global__ void __launch_bounds__(AstCfg<KIND, NP>::kThreads, 1)
    act_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ FewArgs a, uint32_t idesc, int rows, int tiles, int k_tiles, int* err) {
  using C = AstCfg<KIND, NP>;
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
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      dev::mbar_init(&full[s], 1);
      dev::mbar_init(&empty[s], 1);
      dev::mbar_init(&sf_ready[s], 1);
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
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      const int64_t katoms = a.s_kpad >> 2;   // scale atoms of a 128-row group
      const uint32_t tx = static_cast<uint32_t>(rows * 128 + C::kB + 2 * C::kSf);
      for (int tile = w.tile; tile < tiles && ok; tile += w.step) {
        for (int kt = 0; kt < w.k_num; ++kt) {
          if (!dev::mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          uint64_t* bar = &full[stage];
          dev::mbar_expect_tx(bar, tx);
          if (C::kBlock) {
            uint8_t* sf = sSf + stage * 2 * C::kSf;
            const int64_t katom = static_cast<int64_t>(w.k_lo + kt) * C::kAtoms;
            dev::bulk_load(sf, a.sw + (tile * katoms + katom) * 512, C::kSf, bar);
            dev::bulk_load(sf + C::kSf, a.sx + katom * 512, C::kSf, bar);
          }
          dev::tma_load_2d(smem + stage * C::kA, &tmW, bar, (w.k_lo + kt) * 128, tile * rows);
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
          const uint32_t s = dev::smem_u32(sSf + stage * 2 * C::kSf);
#pragma unroll
          for (int j = 0; j < C::kAtoms; ++j)
#pragma unroll
            for (int o = 0; o < 2; ++o)
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
        const int as = it & 1;
        if (!dev::mbar_wait(&acc_empty[as], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, abort_flag, err)) break;
        dev::tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(as * NP);
        for (int kt = 0; kt < w.k_num; ++kt) {
          if (!dev::mbar_wait(&full[stage], phase, abort_flag, err) ||
              (C::kBlock && !dev::mbar_wait(&sf_ready[stage], phase, abort_flag, err))) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t sa = dev::smem_u32(smem + stage * C::kA), sb = dev::smem_u32(sB + stage * C::kB);
          const uint32_t sfa = tmem_base + C::kSfBase + static_cast<uint32_t>(stage * C::kSfCols);
          const uint32_t sfb = sfa + 4 * C::kAtoms;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t ad = dev::smem_desc(sa + 32 * ks, 0, 1024, 2), bd = dev::smem_desc(sb + 32 * ks, 0, 1024, 2);
            const uint32_t on = (kt | ks) != 0;
            if (KIND == kBF16) dev::mma_f16(d, ad, bd, idesc, on);
            else if (KIND == kFP8) dev::mma_f8f6f4(d, ad, bd, idesc, on);
            else if (KIND == kMXFP8)   // scale byte `ks` of each 32-bit scale column
              dev::mma_mxf8f6f4(d, ad, bd, idesc | (static_cast<uint32_t>(ks) << 29) | (static_cast<uint32_t>(ks) << 4), sfa,
                                sfb, on);
            else dev::mma_mxf4nvf4(d, ad, bd, idesc, sfa + 4 * ks, sfb + 4 * ks, on);
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
    const int row = quarter * 32 + lane;          // of the tile
    const float alpha = (a.alpha_a ? *a.alpha_a : 1.0f) * (a.alpha_b ? *a.alpha_b : 1.0f);
    const float qs = KIND != kMXFP8 && a.q ? *a.q_scale : 1.0f;
    unsigned int top = 0;
    int it = 0;
    for (int tile = w.tile; tile < tiles; tile += w.step, ++it) {
      const int as = it & 1;
      const int n = tile * rows + row;
      const bool live = row < rows && n < a.N;
      const float bias = live && a.bias ? a.bias[n] : 0.0f;
      const bool ok = __all_sync(0xFFFFFFFFu, dev::mbar_wait(&acc_full[as], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, err));
      if (!SPLIT && !ok) break;
      dev::tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(as * NP);
      if constexpr (SPLIT) {
        // every load of the cluster has landed and every MMA has read it: the rings are free
        dev::cluster_sync();
        const int per = NP / 4 / w.split;
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
        for (int j = 0; j < per; ++j) {
          const int t0 = 4 * (j * w.split + w.part);
          if (t0 >= a.T) break;
          float2 lo = make_float2(0.0f, 0.0f), hi = lo;
          for (int from = 0; from < w.split; ++from) {
            const float4 p = *reinterpret_cast<const float4*>(smem + kpart_offset(from, j, per, 128, row));
            lo = __fadd2_rn(lo, make_float2(p.x, p.y));
            hi = __fadd2_rn(hi, make_float2(p.z, p.w));
          }
          ast_emit<KIND>(a, make_float4(lo.x, lo.y, hi.x, hi.y), alpha, bias, qs, t0, n, live, lane, top);
        }
        break;
      }
#pragma unroll
      for (int c = 0; c < NP / 32; ++c) {
        if (32 * c >= a.T && c > 0) break;
        uint32_t acc[32];
        dev::tmem_ld_32x32b_x32(taddr + 32 * c, acc);
        dev::tmem_ld_wait();
        dev::reg_fence(acc);
        if (c == NP / 32 - 1 || 32 * (c + 1) >= a.T) {   // the last of the accumulator that is read
          dev::tc_fence_before();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(&acc_empty[as]);
        }
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          if (32 * c + i >= a.T) break;
          const float4 v = make_float4(__uint_as_float(acc[i]), __uint_as_float(acc[i + 1]), __uint_as_float(acc[i + 2]),
                                       __uint_as_float(acc[i + 3]));
          ast_emit<KIND>(a, v, alpha, bias, qs, 32 * c + i, n, live, lane, top);
        }
      }
    }
    if (KIND == kMXFP8 && a.q) {
      // padding rows T to 127 of q's scales, four scale columns a word
      const int kw = static_cast<int>(a.q_kpad >> 2);
      const int64_t words = static_cast<int64_t>(128 - a.T) * kw;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + (threadIdx.x - 64); i < words;
           i += static_cast<int64_t>(gridDim.x) * 128)
        *reinterpret_cast<uint32_t*>(a.s_q + scale_offset(static_cast<uint64_t>(a.T + i / kw),
                                                          static_cast<uint64_t>(i % kw * 4),
                                                          static_cast<uint64_t>(a.q_kpad))) = 0u;
    }
    if (a.amax) {
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      if (lane == 0) atomicMax(a.amax, top);
    }
    if (a.scale_inv && blockIdx.x == 0 && threadIdx.x == 64) *a.scale_inv = __fdiv_rn(1.0f, qs);
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
  if (warp == 1) dev::tmem_dealloc(tmem_base, C::kCols);
}

// *taken: whether the call runs here.
template <int KIND, int NP>
te_status launch_act_stream(const FewArgs& a, uint32_t xfmt, uint32_t wfmt, cudaStream_t st, bool* taken) {
  using C = AstCfg<KIND, NP>;
  constexpr bool kSharedOnly = NP == 128;
  *taken = true;
  static PerDevice<StreamSetup> setups;
  te_status s = TE_OK;
  const StreamSetup* setup = setups.get(&s, [](StreamSetup* m) {
    return m->set(kernel_address(act_stream_kernel<KIND, NP, kSharedOnly>),
                  kernel_address(act_stream_kernel<KIND, NP, true>), C::kThreads, C::kSmemTotal);
  });
  if (setup == nullptr) return s;
  const uint64_t row_bytes = KIND == kBF16 ? 2 * static_cast<uint64_t>(a.K) : static_cast<uint64_t>(a.K) / (KIND == kNVFP4 ? 2 : 1);
  const int rows = 128;
  const int tiles = (a.N + rows - 1) / rows;
  const int k_tiles = static_cast<int>((row_bytes + 127) / 128);
  const int split = stream_split(tiles, k_tiles, setup->most);
  if (kSharedOnly && split == 1) {
    *taken = false;
    return TE_OK;
  }
  CUtensorMap tw, tx;
  s = make_tmap_2d(&tw, a.w, row_bytes, static_cast<uint64_t>(a.N), static_cast<uint32_t>(rows));
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
  const dim3 g(static_cast<unsigned>(grid), 1, 1), block(C::kThreads, 1, 1);
  const cudaError_t e =
      split > 1 ? launch_dependent_clusters(act_stream_kernel<KIND, NP, true>, split, g, block, C::kSmemTotal, st, tw, tx, a,
                                            idesc, rows, tiles, k_tiles, err)
                : launch_dependent(act_stream_kernel<KIND, NP, kSharedOnly>, g, block, C::kSmemTotal, st, tw, tx, a, idesc,
                                   rows, tiles, k_tiles, err);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

template <int KIND>
te_status launch_act_stream(const FewArgs& a, uint32_t xfmt, uint32_t wfmt, cudaStream_t st, bool* taken) {
  return a.T <= 32   ? launch_act_stream<KIND, 32>(a, xfmt, wfmt, st, taken)
         : a.T <= 64 ? launch_act_stream<KIND, 64>(a, xfmt, wfmt, st, taken)
                     : launch_act_stream<KIND, 128>(a, xfmt, wfmt, st, taken);
}

}  // namespace
}  // namespace te
