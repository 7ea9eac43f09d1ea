// The linear with bias, activation and residual for the tokens of a decoding batch or a short sequence (up to 128
// tokens where the kernel of act_decode.cuh does not take the call, up to 2048 where act_streams says so), every operand
// kind: bound by the weights that it reads, with too much matrix work for mma.sync.  The operands change places against
// gemm_kernel: 128 rows of w are the 128-row operand of the MMA and the tokens its N (32, 64 or 128, and from 129 tokens
// on groups of 128), so a stage is 16 KB of weights and 4, 8 or 16 KB of x (and, block-scaled, the scale atoms of both),
// and as many stages as fit keep loads in flight.  One CTA per SM, no pairs: two CTAs with half the stages each gained
// nothing.
//
// warp 0 TMA producer, warp 1 MMA issuer, four or (from 33 tokens on) eight epilogue warps, and for the block-scaled
// kinds one that copies the scale atoms to tensor memory.  An accumulator lane is a column of y and the tokens lie along
// the TMEM columns, so neighbouring lanes write neighbouring columns, and a warp's 32 columns are one MXFP8 block of q.
// Where the tiles leave SMs idle, clusters of 2, 4 or 8 CTAs share a tile's K and add their parts through distributed
// shared memory, each of them for its groups of four tokens and in the CTAs' order, so the result does not depend on
// timing.
//
// BF16, 1 token, K = 16384, N = 4096 24.6 us (134 MB, 5.5 TB/s); FP8, 24 tokens, K = 4096, N = 16384 15.2 us (67 MB,
// 4.5); gemm_kernel takes 26 and more for the second.
#pragma once

#include "act_decode.cuh"

namespace te {
namespace {

constexpr int64_t kAstMaxTokens = 2048;

template <int KIND, int NP>   // tokens, padded
struct AstCfg {
  static constexpr bool kBlock = KIND >= kMXFP8;
  static constexpr int kAtoms = KIND == kMXFP8 ? 1 : (KIND == kNVFP4 ? 4 : 0);   // scale atoms per 128 rows and k-tile
  static constexpr int kSf = kAtoms * 512;
  static constexpr int kA = 128 * 128, kB = NP * 128;
  static constexpr int kStage = kA + kB + 2 * kSf;
  static constexpr int kFit = (232448 - 1024 - 512) / kStage;
  static constexpr int kSfBase = 2 * NP, kSfCols = 8 * kAtoms;    // TMEM columns of a stage's scales
  static constexpr int kMost = KIND == kNVFP4 ? (512 - kSfBase) / kSfCols : 12;
  static constexpr int kStages = kFit < kMost ? kFit : kMost;
  static constexpr int kSmemB = kStages * kA;
  static constexpr int kSmemSf = kSmemB + kStages * kB;
  static constexpr int kSmemBar = kSmemSf + kStages * 2 * kSf;
  static constexpr int kSmemTotal = kSmemBar + 512 + 1024;
  static constexpr int kUsedCols = 2 * NP + (kBlock ? kStages * kSfCols : 0);   // two accumulators, and the scales
  static constexpr int kCols = kUsedCols <= 64 ? 64 : (kUsedCols <= 128 ? 128 : (kUsedCols <= 256 ? 256 : 512));
  static constexpr int kHalves = NP == 32 ? 1 : 2;   // epilogue warps of a quarter of the accumulator: halves of the tokens
  static constexpr int kEpi = 4 * kHalves;
  static constexpr int kCopier = 2 + kEpi;
  static constexpr int kThreads = 32 * (2 + kEpi + (kBlock ? 1 : 0));
  static_assert(kSmemTotal <= 232448 && (3 * kStages + 5) * 8 + 16 <= 512, "shared memory");
  static_assert(NP == 32 || NP == 64 || NP == 128, "whole tcgen05.ld chunks, power-of-two TMEM columns");
  static_assert(kUsedCols <= 512, "TMEM");
  static_assert(NP / 4 * 128 * 16 <= kSmemSf, "the shared accumulators' parts");
};

// NT tokens from t0 of column n (live: the column is one of y's): every output.  The whole warp, the same t0.
template <int KIND, int NT>
__device__ __forceinline__ void ast_emit(const FewArgs& a, uint32_t (&v)[NT], float alpha, float bias, float qs, int t0,
                                         int n, bool live, int lane, unsigned int& top) {
  const int count = min(NT, a.T - t0);
  const int64_t at = static_cast<int64_t>(t0) * a.N + n;
#pragma unroll
  for (int i = 0; i < NT; i += 2) {
    const float2 z = __ffma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), both(alpha), both(bias));
    v[i] = __float_as_uint(z.x), v[i + 1] = __float_as_uint(z.y);
  }
  if (a.z && live) {
    __nv_bfloat16* p = a.z + at;
#pragma unroll
    for (int i = 0; i < NT; ++i, p += a.N)
      if (i < count) *p = __float2bfloat16_rn(__uint_as_float(v[i]));
  }
  if constexpr (NT == 32) {
    act_chunk(v, a.act);
  } else {
#pragma unroll
    for (int i = 0; i < NT; i += 2) {
      const float2 x = act_value(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), a.act);
      v[i] = __float_as_uint(x.x), v[i + 1] = __float_as_uint(x.y);
    }
  }
  if (a.q) {   // (no residual beside it)
    uint8_t* p = a.q + at;
#pragma unroll
    for (int i = 0; i < NT; ++i, p += a.N) {
      if (i >= count) break;
      const float x = __uint_as_float(v[i]);
      if (KIND == kMXFP8) {
        // (N is a multiple of 32: a warp's columns are all live or none)
        const int e = mx_exponent(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, v[i] & 0x7FFFFFFFu)));
        if (live) *p = static_cast<uint8_t>(cvt_e4m3x2(x * mx_mult(e), 0.0f));
        const int64_t block = (n - lane) >> 5;
        if (lane == 0 && block < a.q_kpad)   // past the last column: padding
          a.s_q[scale_offset(static_cast<uint64_t>(t0 + i), static_cast<uint64_t>(block), static_cast<uint64_t>(a.q_kpad))] =
              live ? static_cast<uint8_t>(e + 127) : uint8_t(0);
      } else if (live) {
        top = max(top, v[i] & 0x7FFFFFFFu);
        *p = few_code(a, x, qs);
      }
    }
  }
  if (!a.y || !live) return;
  if (a.res) {
    // all of them before the first store: y may be residual
    float r[NT];
    if (a.y_f32) {
      const float* p = static_cast<const float*>(a.res) + at;
#pragma unroll
      for (int i = 0; i < NT; ++i, p += a.N) r[i] = i < count ? *p : 0.0f;
    } else {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.res) + at;
#pragma unroll
      for (int i = 0; i < NT; ++i, p += a.N) r[i] = i < count ? __bfloat162float(*p) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) v[i] = __float_as_uint(__fadd_rn(__uint_as_float(v[i]), r[i]));
  }
  if (a.y_f32) {
    float* p = static_cast<float*>(a.y) + at;
#pragma unroll
    for (int i = 0; i < NT; ++i, p += a.N)
      if (i < count) *p = __uint_as_float(v[i]);
  } else {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.y) + at;
#pragma unroll
    for (int i = 0; i < NT; ++i, p += a.N)
      if (i < count) *p = __float2bfloat16_rn(__uint_as_float(v[i]));
  }
}

// seg: k-tiles that are added up in tensor memory (0: all; kSegments in gemm.cuh has the reason and the rule); the
// two accumulators take turns with segments as with tiles.
template <int KIND, int NP, bool SPLIT>
__global__ void __launch_bounds__(AstCfg<KIND, NP>::kThreads, 1)
    act_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ FewArgs a, uint32_t idesc, int tiles, int k_tiles, int seg, int* err) {
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
  // a tile: 128 rows of w times NP tokens; those of the same rows follow one another
  const int groups = NP == 128 ? (a.T + 127) >> 7 : 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      dev::mbar_init(&full[s], 1);
      dev::mbar_init(&empty[s], 1);
      dev::mbar_init(&sf_ready[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      dev::mbar_init(&acc_full[s], 1);
      dev::mbar_init(&acc_empty[s], C::kEpi);
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
      for (int tile = w.tile; tile < tiles && ok; tile += w.step) {
        const int wt = tile / groups, xt = tile - wt * groups;
        for (int kt = 0; kt < w.k_num; ++kt) {
          if (!dev::mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          uint64_t* bar = &full[stage];
          dev::mbar_expect_tx(bar, C::kStage);
          if (C::kBlock) {
            uint8_t* sf = sSf + stage * 2 * C::kSf;
            const int64_t katom = static_cast<int64_t>(w.k_lo + kt) * C::kAtoms;
            dev::bulk_load(sf, a.sw + (wt * katoms + katom) * 512, C::kSf, bar);
            dev::bulk_load(sf + C::kSf, a.sx + (xt * katoms + katom) * 512, C::kSf, bar);
          }
          dev::tma_load_2d(smem + stage * C::kA, &tmW, bar, (w.k_lo + kt) * 128, wt * 128);
          dev::tma_load_2d(sB + stage * C::kB, &tmX, bar, (w.k_lo + kt) * 128, xt * NP);
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
  } else if (warp == C::kCopier) {
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
      const int segs = seg > 0 ? (w.k_num + seg - 1) / seg : 1;
      for (int tile = w.tile; tile < tiles && ok; tile += w.step)
      for (int sg = 0; sg < segs && ok; ++sg, ++it) {
        const int as = it & 1;
        if (!dev::mbar_wait(&acc_empty[as], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, abort_flag, err)) {
          ok = false;
          break;
        }
        dev::tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(as * NP);
        const int k_beg = sg > 0 ? part_begin(w.k_num, sg, segs) : 0;
        const int k_end = sg + 1 < segs ? part_begin(w.k_num, sg + 1, segs) : w.k_num;
        for (int kt = k_beg; kt < k_end; ++kt) {
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
            const uint32_t on = ((kt - k_beg) | ks) != 0;
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
    const int half = (warp - 2) >> 2;             // of the tokens
    const int row = quarter * 32 + lane;          // of the tile
    constexpr int kMine = NP / C::kHalves;        // this warp's tokens
    const float alpha = (a.alpha_a ? *a.alpha_a : 1.0f) * (a.alpha_b ? *a.alpha_b : 1.0f);
    const float qs = KIND != kMXFP8 && a.q ? *a.q_scale : 1.0f;
    unsigned int top = 0;
    const int segs = seg > 0 ? (w.k_num + seg - 1) / seg : 1;
    int it = 0;
    for (int tile = w.tile; tile < tiles; tile += w.step, ++it) {
      const int wt = tile / groups;
      const int n = wt * 128 + row, first = (tile - wt * groups) * NP;   // this thread's column, the tile's first token
      const bool live = n < a.N;
      const float bias = live && a.bias ? a.bias[n] : 0.0f;
      uint32_t acc[kMine / 32][32];
      bool ok = true;
      for (int sg = 0; sg < segs; ++sg) {
        if (sg > 0) {
          // the segment before has been taken over
          dev::tc_fence_before();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(&acc_empty[it & 1]);
          ++it;
        }
        ok = __all_sync(0xFFFFFFFFu,
                        dev::mbar_wait(&acc_full[it & 1], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, err));
        if (!ok) break;
        dev::tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                               static_cast<uint32_t>((it & 1) * NP + half * kMine);
        if (sg == 0) {
#pragma unroll
          for (int c = 0; c < kMine / 32; ++c) dev::tmem_ld_32x32b_x32(taddr + 32 * c, acc[c]);
          dev::tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < kMine / 32; ++c) dev::reg_fence(acc[c]);
        } else {
#pragma unroll
          for (int c = 0; c < kMine / 32; ++c) {
            uint32_t part[32];
            dev::tmem_ld_32x32b_x32(taddr + 32 * c, part);
            dev::tmem_ld_wait();
            dev::reg_fence(part);
#pragma unroll
            for (int i = 0; i < 32; i += 2) set_pair(acc[c], i, __fadd2_rn(pair_of(acc[c], i), pair_of(part, i)));
          }
        }
      }
      if (!SPLIT && !ok) break;
      if constexpr (SPLIT) {
        // every load of the cluster has landed and every MMA has read it: the rings are free
        dev::cluster_sync();
        const int per = NP / 4 / w.split;
        if (ok) {
#pragma unroll
          for (int i = 0; i < kMine / 4; ++i)
            if (first + half * kMine + 4 * i < a.T)
              kpart_send(acc[i / 8], 4 * (i % 8), dev::smem_u32(smem), w.split, w.part, half * (kMine / 4) + i, per, 128, row);
        }
        dev::tc_fence_before();
        dev::cluster_sync();
        if (!ok) break;
        for (int j = half; j < per; j += C::kHalves) {
          const int t0 = first + 4 * (j * w.split + w.part);
          if (t0 >= a.T) break;
          float2 lo = make_float2(0.0f, 0.0f), hi = lo;
          for (int from = 0; from < w.split; ++from) {
            const float4 p = *reinterpret_cast<const float4*>(smem + kpart_offset(from, j, per, 128, row));
            lo = __fadd2_rn(lo, make_float2(p.x, p.y));
            hi = __fadd2_rn(hi, make_float2(p.z, p.w));
          }
          uint32_t v[4] = {__float_as_uint(lo.x), __float_as_uint(lo.y), __float_as_uint(hi.x), __float_as_uint(hi.y)};
          ast_emit<KIND, 4>(a, v, alpha, bias, qs, t0, n, live, lane, top);
        }
        break;
      }
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&acc_empty[it & 1]);
#pragma unroll
      for (int c = 0; c < kMine / 32; ++c) {
        const int t0 = first + half * kMine + 32 * c;
        if (t0 < a.T) ast_emit<KIND, 32>(a, acc[c], alpha, bias, qs, t0, n, live, lane, top);
      }
    }
    if (KIND == kMXFP8 && a.q) {
      // padding rows of q's scales (T to a multiple of 128), four scale columns a word
      const int kw = static_cast<int>(a.q_kpad >> 2);
      const int64_t words = static_cast<int64_t>((128 - a.T % 128) % 128) * kw;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * (32 * C::kEpi) + (threadIdx.x - 64); i < words;
           i += static_cast<int64_t>(gridDim.x) * (32 * C::kEpi))
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
    if (warp < 2 || warp == C::kCopier) {   // the other warps' part in the epilogue's two barriers
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

// The CTAs that share a tile's K: stream_split's rule up to 64 tokens.  With 128 the exchange takes about 3.5 us and a
// k-tile 0.2, so that the k-tiles saved have to be 18 (us, one CTA / shared: BF16 K = 1024, N = 4096, 256 tokens
// 8.1 / 9.6, K = N = 2048 11.4 / 8.4, K = N = 4096 18.6 / 16.1).
template <int NP>
int act_split(int tiles, int k_tiles, const int (&most)[3]) {
  if constexpr (NP < 128) {
    return stream_split(tiles, k_tiles, most);
  } else {
    for (int i = 2; i >= 0; --i)
      if (tiles <= most[i] && k_tiles - k_tiles / (2 << i) >= 18) return 2 << i;
    return 1;
  }
}

// Whether a call of more than 128 tokens runs here or in gemm_kernel, whose tiles are four times as large: by how long
// each takes, in units of 10 ns: the k-tiles of its waves of tiles (a wave behind the first no less than its epilogue)
// beside what a call costs (here 4.5 us and 3.5 of an exchange; there 9.3 and 3).  us, here / there:
//   256 tokens: K = 768, N = 2048 BF16 7.3 / 11.2, MXFP8 7.5 / 10.5; K = N = 2048 BF16 8.4 / 13.5, NVFP4 8.0 / 10.7;
//   K = N = 4096 BF16 16.1 / 19.6, FP8 11.5 / 17.2, MXFP8 12.8 / 18.2; K = 16384, N = 4096 BF16 37.0 / 45.9, MXFP8
//   26.3 / 51.5, NVFP4 19.7 / 32.3; 512 tokens: K = N = 4096 BF16 18.9 / 21.6, MXFP8 13.8 / 19.2, K = 16384, N = 4096
//   BF16 59.2 / 48.9, MXFP8 38.7 / 51.6; two waves here: K = 4096, N = 12288, 300 tokens BF16 33.1 / 47.8, MXFP8 23.0 /
//   32.9, 129 tokens BF16 33.9 / 29.6; K = N = 4096, 768 tokens BF16 32.8 / 22.9, FP8 19.3 / 19.3; several waves of a
//   short K: K = 1024, N = 16384 MXFP8 700 tokens 22.1 / 27.0, 2048 47.1 / 56.0, BF16 1024 tokens 33.8 / 36.5.
template <int KIND>
bool act_streams(int64_t T, int64_t N, int tiles, int k_tiles, int split) {
  if (T <= 128) return true;
  const int sms = num_sms();
  const int ts = KIND == kMXFP8 ? 28 : (KIND == kNVFP4 ? 35 : 22), tp = KIND == kMXFP8 ? 33 : (KIND == kNVFP4 ? 36 : 28);
  auto time = [](int64_t k, int64_t waves, int64_t epilogue) { return k + (waves - 1) * (k > epilogue ? k : epilogue); };
  const int64_t here = 450 + (split > 1 ? 350 + static_cast<int64_t>(ts) * k_tiles / split
                                        : time(static_cast<int64_t>(ts) * k_tiles, (tiles + sms - 1) / sms, 290));
  const int64_t pair_tiles = (T + 255) / 256 * ((N + 255) / 256), pairs = sms / 2;
  int shared = 1;   // pairs to a tile there
  if (KIND <= kFP8 && pair_tiles <= pairs / 9 && k_tiles >= 24) shared = 4;
  else if (KIND <= kFP8 && pair_tiles <= pairs * 4 / 9 && k_tiles >= 48) shared = 2;
  const int64_t there = 930 + (shared > 1 ? 300 : 0) +
                        time(static_cast<int64_t>(tp) * k_tiles / shared, (pair_tiles + pairs - 1) / pairs, 560);
  return here < there;
}

// *taken: whether the call runs here.
template <int KIND, int NP>
te_status launch_act_stream(const FewArgs& a, uint32_t xfmt, uint32_t wfmt, cudaStream_t st, bool* taken) {
  *taken = true;
  using C = AstCfg<KIND, NP>;
  static PerDevice<StreamSetup> setups;
  te_status s = TE_OK;
  const StreamSetup* setup = setups.get(&s, [](StreamSetup* m) {
    return m->set(kernel_address(act_stream_kernel<KIND, NP, false>),
                  kernel_address(act_stream_kernel<KIND, NP, true>), C::kThreads, C::kSmemTotal);
  });
  if (setup == nullptr) return s;
  const uint64_t row_bytes = KIND == kBF16 ? 2 * static_cast<uint64_t>(a.K) : static_cast<uint64_t>(a.K) / (KIND == kNVFP4 ? 2 : 1);
  const int groups = NP == 128 ? (a.T + 127) / 128 : 1;
  const int tiles = (a.N + 127) / 128 * groups;
  const int k_tiles = static_cast<int>((row_bytes + 127) / 128);
  const int split = act_split<NP>(tiles, k_tiles, setup->most);
  if (!act_streams<KIND>(a.T, a.N, tiles, k_tiles, split)) {
    *taken = false;
    return TE_OK;
  }
  CUtensorMap tw, tx;
  s = make_tmap_2d(&tw, a.w, row_bytes, static_cast<uint64_t>(a.N), 128);
  if (s != TE_OK) return s;
  s = make_tmap_2d(&tx, a.x, row_bytes, static_cast<uint64_t>(a.T), NP);
  if (s != TE_OK) return s;
  int* err = device_error_word();
  if (err == nullptr) return record_cuda(cudaErrorInvalidDevice);
  // the weights are operand A: M = 128, N = NP
  uint32_t idesc = make_idesc(KIND, wfmt, xfmt, 128);
  idesc = (idesc & ~(0x3Fu << 17)) | (static_cast<uint32_t>(NP >> 3) << 17);
  const int grid = split > 1 ? split * tiles : (tiles < num_sms() ? tiles : num_sms());
  const int seg = KIND == kBF16 && !a.y_f32 ? 0 : kSegment<KIND>;   // as in gemm_kernel
  if (a.amax && (s = zero_amax(a.amax, st)) != TE_OK) return s;
  const dim3 g(static_cast<unsigned>(grid), 1, 1), block(C::kThreads, 1, 1);
  const cudaError_t e =
      split > 1 ? launch_dependent_clusters(act_stream_kernel<KIND, NP, true>, split, g, block, C::kSmemTotal, st, tw, tx, a,
                                            idesc, tiles, k_tiles, seg, err)
                : launch_dependent(act_stream_kernel<KIND, NP, false>, g, block, C::kSmemTotal, st, tw, tx, a, idesc,
                                   tiles, k_tiles, seg, err);
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
