// Entry points of the gated feed-forward projections: h = act(x Wg^T) * (x Wu^T) in one kernel, and
// its backward pass.  The kernels are gemm_kernel with the gated epilogues (gemm.cuh), and those of
// gated_decode.cuh, gated_stream.cuh and gated_stream_block.cuh for few tokens.
#include "gated_stream_block.cuh"

namespace te {
namespace {

// amax = 0 and 1 / scale where there is no row to compute them beside.
__global__ void publish_empty_kernel(const float* scale, float* amax, float* scale_inv) {
  if (amax) *amax = 0.0f;
  if (scale_inv) *scale_inv = __fdiv_rn(1.0f, *scale);
}

bool fp8_format(te_dtype f) { return f == TE_E4M3 || f == TE_E5M2; }
uint32_t fp8_code(te_dtype f) { return f == TE_E5M2 ? 1u : 0u; }

te_status check_sizes(int act, int64_t T, int64_t F, int64_t F_mult, int64_t K, int64_t K_mult) {
  if (act != TE_ACT_SILU && act != TE_ACT_GELU) return TE_ERR_ARG;
  if (T < 0 || F <= 0 || K <= 0 || F % F_mult || K % K_mult) return TE_ERR_SHAPE;
  if (T > (int64_t(1) << 30) || F > (int64_t(1) << 29) || K > (int64_t(1) << 30)) return TE_ERR_SHAPE;
  return TE_OK;
}

// The bf16 halves of [T, 2 F].
te_status halves(CUtensorMap* lo, CUtensorMap* hi, const void* p, int64_t T, int64_t F) {
  te_status s = make_tmap_2d_view64(lo, p, static_cast<uint64_t>(F) * 2, static_cast<uint64_t>(F) * 4,
                                    static_cast<uint64_t>(T));
  if (s != TE_OK) return s;
  return make_tmap_2d_view64(hi, static_cast<const uint8_t*>(p) + F * 2, static_cast<uint64_t>(F) * 2,
                             static_cast<uint64_t>(F) * 4, static_cast<uint64_t>(T));
}

// Describes the bf16 outputs.
te_status bf16_outputs(GatedArgs* ep, void* h, void* gu, int64_t T, int64_t F, int act) {
  ep->F = static_cast<int>(F);
  ep->act = act;
  ep->has_h = h != nullptr;
  ep->has_gu = gu != nullptr;
  if (h) {
    te_status s = make_tmap_2d_view64(&ep->h, h, static_cast<uint64_t>(F) * 2, static_cast<uint64_t>(F) * 2,
                                      static_cast<uint64_t>(T));
    if (s != TE_OK) return s;
  }
  return gu ? halves(&ep->g, &ep->u, gu, T, F) : TE_OK;
}

te_status check_operands(const void* a, const void* b) {
  if (!a || !b) return TE_ERR_NULL;
  return aligned16(a) && aligned16(b) ? TE_OK : TE_ERR_ALIGN;
}

te_status dgrad_args(GatedArgs* ep, const void* gu, void* dgu, int64_t T, int64_t F, int act) {
  if (!gu || !dgu) return TE_ERR_NULL;
  if (!aligned16(gu) || !aligned16(dgu)) return TE_ERR_ALIGN;
  ep->F = static_cast<int>(F);
  ep->act = act;
  te_status s = halves(&ep->g, &ep->u, gu, T, F);
  return s != TE_OK ? s : halves(&ep->h, &ep->q, dgu, T, F);
}

}  // namespace
}  // namespace te

using namespace te;

extern "C" {

te_status te_gated_gemm_bf16(const void* x, const void* w, int act, void* h, void* gu, int64_t T, int64_t K, int64_t F,
                             void* stream) {
  te_status s = check_sizes(act, T, F, 16, K, 16);
  if (s != TE_OK || T == 0) return s;
  if (!h && !gu) return TE_ERR_NULL;
  if ((s = check_operands(x, w)) != TE_OK) return s;
  if (!aligned16(h) || !aligned16(gu)) return TE_ERR_ALIGN;
  if (T <= kStrMaxTokens) {
    const DecodeArgs a = {static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(w), static_cast<int>(T),
                          static_cast<int>(K), static_cast<int>(F), act, nullptr, nullptr,
                          static_cast<__nv_bfloat16*>(h), static_cast<__nv_bfloat16*>(gu), nullptr, nullptr, 0, nullptr,
                          nullptr};
    if (decodes(T, K, F, 2)) return launch_decode<kDecBF16, kDecBF16>(a, static_cast<cudaStream_t>(stream));
    bool taken;
    s = launch_stream<kBF16>(a, 1u, 1u, static_cast<cudaStream_t>(stream), &taken);
    if (taken || s != TE_OK) return s;
  }
  GatedArgs ep = {};
  if ((s = bf16_outputs(&ep, h, gu, T, F, act)) != TE_OK) return s;
  return launch_gemm<kBF16, 2, kGated, true>(x, w, K * 2, nullptr, nullptr, 0, nullptr, nullptr, nullptr, nullptr,
                                             TE_BF16, 0, T, 2 * F, K, 1u, 1u, static_cast<cudaStream_t>(stream), 0, 0, ep,
                                             kPdlChain);
}

te_status te_gated_gemm_fp8(const uint8_t* x, te_dtype fx, const uint8_t* w, te_dtype fw, const float* x_scale_inv,
                            const float* w_scale_inv, int act, void* h, void* gu, uint8_t* q_h, te_dtype h_fmt,
                            const float* h_scale, float* h_amax, float* h_scale_inv, int64_t T, int64_t K, int64_t F,
                            void* stream) {
  if (!fp8_format(fx) || !fp8_format(fw) || (q_h && !fp8_format(h_fmt))) return TE_ERR_DTYPE;
  te_status s = check_sizes(act, T, F, 16, K, 16);
  if (s != TE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (h_scale_inv && !h_scale) return TE_ERR_NULL;
    if (!h_amax && !h_scale_inv) return TE_OK;
    publish_empty_kernel<<<1, 1, 0, st>>>(h_scale, h_amax, h_scale_inv);
    count_launch();
    return launch_status();
  }
  if (!h && !gu && !q_h) return TE_ERR_NULL;
  if (q_h ? !h_scale : (h_amax || h_scale_inv)) return TE_ERR_NULL;   // the amax and 1 / scale go with q_h
  if (!x_scale_inv || !w_scale_inv) return TE_ERR_NULL;
  if ((s = check_operands(x, w)) != TE_OK) return s;
  if (!aligned16(h) || !aligned16(gu) || !aligned16(q_h)) return TE_ERR_ALIGN;
  if (T <= kStrMaxTokens) {
    const DecodeArgs a = {x, w, static_cast<int>(T), static_cast<int>(K), static_cast<int>(F), act,
                          x_scale_inv, w_scale_inv, static_cast<__nv_bfloat16*>(h), static_cast<__nv_bfloat16*>(gu), q_h,
                          h_scale, h_fmt == TE_E5M2, reinterpret_cast<unsigned int*>(h_amax), h_scale_inv};
    if (decodes(T, K, F, 1)) {
      if (fw == TE_E4M3)
        return fx == TE_E4M3 ? launch_decode<kDecE4M3, kDecE4M3>(a, st) : launch_decode<kDecE4M3, kDecE5M2>(a, st);
      return fx == TE_E4M3 ? launch_decode<kDecE5M2, kDecE4M3>(a, st) : launch_decode<kDecE5M2, kDecE5M2>(a, st);
    }
    bool taken;
    s = launch_stream<kFP8>(a, fp8_code(fx), fp8_code(fw), st, &taken);
    if (taken || s != TE_OK) return s;
  }
  GatedArgs ep = {};
  if ((s = bf16_outputs(&ep, h, gu, T, F, act)) != TE_OK) return s;
  if (q_h) {
    ep.has_q = 1;
    ep.q_e5m2 = h_fmt == TE_E5M2;
    ep.q_scale = h_scale;
    ep.amax = reinterpret_cast<unsigned int*>(h_amax);
    ep.scale_inv = h_scale_inv;
    s = make_tmap_2d_view64(&ep.q, q_h, static_cast<uint64_t>(F), static_cast<uint64_t>(F), static_cast<uint64_t>(T));
    if (s != TE_OK) return s;
    s = make_tmap_2d_plain(&ep.q32, q_h, static_cast<uint64_t>(F), static_cast<uint64_t>(T), 32u, 32u);
    if (s != TE_OK) return s;
  }
  if (h_amax && (s = zero_amax(h_amax, st)) != TE_OK) return s;
  return launch_gemm<kFP8, 2, kGated, true>(x, w, K, nullptr, nullptr, 0, x_scale_inv, w_scale_inv, nullptr, nullptr,
                                            TE_BF16, 0, T, 2 * F, K, fp8_code(fx), fp8_code(fw), st, 0, 0, ep,
                                            kPdlChain);
}

te_status te_gated_gemm_mxfp8(const uint8_t* x, te_dtype fx, const uint8_t* sx, const uint8_t* w, te_dtype fw,
                              const uint8_t* sw, int act, void* h, void* gu, uint8_t* q_h, uint8_t* s_h, int64_t T,
                              int64_t K, int64_t F, void* stream) {
  if (!fp8_format(fx) || !fp8_format(fw)) return TE_ERR_DTYPE;
  te_status s = check_sizes(act, T, F, 128, K, 32);
  if (s != TE_OK || T == 0) return s;
  if ((!h && !gu && !q_h) || (q_h == nullptr) != (s_h == nullptr)) return TE_ERR_NULL;
  if ((s = check_operands(x, w)) != TE_OK) return s;
  if ((s = check_operands(sx, sw)) != TE_OK) return s;
  if (!aligned16(h) || !aligned16(gu) || !aligned16(q_h) || !aligned16(s_h)) return TE_ERR_ALIGN;
  if (T <= kStrMaxTokens) {
    DecodeArgs a = {x, w, static_cast<int>(T), static_cast<int>(K), static_cast<int>(F), act};
    a.h = static_cast<__nv_bfloat16*>(h);
    a.gu = static_cast<__nv_bfloat16*>(gu);
    a.q = q_h;
    a.sx = sx;
    a.sw = sw;
    a.s_kpad = (K / 32 + 3) / 4 * 4;
    a.s_h = s_h;
    bool taken;
    s = launch_stream_block<kMXFP8>(a, fp8_code(fx), fp8_code(fw), static_cast<cudaStream_t>(stream), &taken);
    if (taken || s != TE_OK) return s;
  }
  GatedArgs ep = {};
  if ((s = bf16_outputs(&ep, h, gu, T, F, act)) != TE_OK) return s;
  if (q_h) {
    ep.has_q = 1;
    ep.s_h = s_h;
    ep.s_kpad = F / 32;
    ep.s_rows = static_cast<int>((T + 127) / 128 * 128);
    s = make_tmap_2d_view64(&ep.q, q_h, static_cast<uint64_t>(F), static_cast<uint64_t>(F), static_cast<uint64_t>(T));
    if (s != TE_OK) return s;
  }
  return launch_gemm<kMXFP8, 2, kGated>(x, w, K, sx, sw, (K / 32 + 3) / 4, nullptr, nullptr, nullptr, nullptr, TE_BF16,
                                        0, T, 2 * F, K, fp8_code(fx), fp8_code(fw), static_cast<cudaStream_t>(stream), 0,
                                        0, ep, kPdlChain);
}

te_status te_gated_gemm_nvfp4(const uint8_t* x, const uint8_t* sx, const float* gx, const uint8_t* w, const uint8_t* sw,
                              const float* gw, int act, void* h, void* gu, int64_t T, int64_t K, int64_t F,
                              void* stream) {
  te_status s = check_sizes(act, T, F, 128, K, 32);
  if (s != TE_OK || T == 0) return s;
  if ((!h && !gu) || !gx || !gw) return TE_ERR_NULL;
  if ((s = check_operands(x, w)) != TE_OK) return s;
  if ((s = check_operands(sx, sw)) != TE_OK) return s;
  if (!aligned16(h) || !aligned16(gu)) return TE_ERR_ALIGN;
  if (T <= kStrMaxTokens) {
    DecodeArgs a = {x, w, static_cast<int>(T), static_cast<int>(K), static_cast<int>(F), act, gx, gw};
    a.h = static_cast<__nv_bfloat16*>(h);
    a.gu = static_cast<__nv_bfloat16*>(gu);
    a.sx = sx;
    a.sw = sw;
    a.s_kpad = (K / 16 + 15) / 16 * 16;
    bool taken;
    s = launch_stream_block<kNVFP4>(a, 1u, 1u, static_cast<cudaStream_t>(stream), &taken);
    if (taken || s != TE_OK) return s;
  }
  GatedArgs ep = {};
  if ((s = bf16_outputs(&ep, h, gu, T, F, act)) != TE_OK) return s;
  return launch_gemm<kNVFP4, 2, kGated>(x, w, K / 2, sx, sw, (K / 16 + 15) / 16 * 4, gx, gw, nullptr, nullptr, TE_BF16,
                                        0, T, 2 * F, K, 1u, 1u, static_cast<cudaStream_t>(stream), 0, 0, ep, kPdlChain);
}

te_status te_gated_dgrad_fp8(const uint8_t* dy, te_dtype fd, const uint8_t* w2, te_dtype fw, const float* dy_scale_inv,
                             const float* w2_scale_inv, const void* gu, int act, void* dgu, int64_t T, int64_t F,
                             int64_t N, void* stream) {
  if (!fp8_format(fd) || !fp8_format(fw)) return TE_ERR_DTYPE;
  te_status s = check_sizes(act, T, F, 16, N, 16);
  if (s != TE_OK || T == 0) return s;
  if (!dy_scale_inv || !w2_scale_inv) return TE_ERR_NULL;
  if ((s = check_operands(dy, w2)) != TE_OK) return s;
  GatedArgs ep = {};
  if ((s = dgrad_args(&ep, gu, dgu, T, F, act)) != TE_OK) return s;
  return launch_gemm<kFP8, 2, kDgrad, true>(dy, w2, N, nullptr, nullptr, 0, dy_scale_inv, w2_scale_inv, nullptr, nullptr,
                                      TE_BF16, 0, T, F, N, fp8_code(fd), fp8_code(fw),
                                      static_cast<cudaStream_t>(stream), 0, 0, ep, kPdlChain);
}

te_status te_gated_dgrad_mxfp8(const uint8_t* dy, te_dtype fd, const uint8_t* sd, const uint8_t* w2, te_dtype fw,
                               const uint8_t* sw, const void* gu, int act, void* dgu, int64_t T, int64_t F, int64_t N,
                               void* stream) {
  if (!fp8_format(fd) || !fp8_format(fw)) return TE_ERR_DTYPE;
  te_status s = check_sizes(act, T, F, 16, N, 32);
  if (s != TE_OK || T == 0) return s;
  if ((s = check_operands(dy, w2)) != TE_OK) return s;
  if ((s = check_operands(sd, sw)) != TE_OK) return s;
  GatedArgs ep = {};
  if ((s = dgrad_args(&ep, gu, dgu, T, F, act)) != TE_OK) return s;
  return launch_gemm<kMXFP8, 2, kDgrad>(dy, w2, N, sd, sw, (N / 32 + 3) / 4, nullptr, nullptr, nullptr, nullptr, TE_BF16,
                                        0, T, F, N, fp8_code(fd), fp8_code(fw), static_cast<cudaStream_t>(stream), 0,
                                        0, ep, kPdlChain);
}

te_status te_gated_dgrad_nvfp4(const uint8_t* dy, const uint8_t* sd, const float* gd, const uint8_t* w2,
                               const uint8_t* sw, const float* gw, const void* gu, int act, void* dgu, int64_t T,
                               int64_t F, int64_t N, void* stream) {
  te_status s = check_sizes(act, T, F, 16, N, 32);
  if (s != TE_OK || T == 0) return s;
  if (!gd || !gw) return TE_ERR_NULL;
  if ((s = check_operands(dy, w2)) != TE_OK) return s;
  if ((s = check_operands(sd, sw)) != TE_OK) return s;
  GatedArgs ep = {};
  if ((s = dgrad_args(&ep, gu, dgu, T, F, act)) != TE_OK) return s;
  return launch_gemm<kNVFP4, 2, kDgrad>(dy, w2, N / 2, sd, sw, (N / 16 + 15) / 16 * 4, gd, gw, nullptr, nullptr, TE_BF16,
                                        0, T, F, N, 1u, 1u, static_cast<cudaStream_t>(stream), 0, 0, ep, kPdlChain);
}

te_status te_gated_bwd_bf16(const void* x, const void* w, const void* w2, const void* dy, const void* gu, int act,
                            void* dgu, void* dx, void* dw, te_dtype dw_dtype, int accumulate, int64_t T, int64_t K,
                            int64_t F, int64_t N, void* stream) {
  te_status s = check_sizes(act, T, F, 16, N, 16);
  if (s != TE_OK) return s;
  if ((dx || dw) && (K <= 0 || K % 16 || K > (int64_t(1) << 30))) return TE_ERR_SHAPE;
  if (dw && dw_dtype != TE_BF16 && dw_dtype != TE_F32) return TE_ERR_DTYPE;
  if (accumulate != 0 && accumulate != 1) return TE_ERR_ARG;
  if (dw && accumulate && dw_dtype != TE_F32) return TE_ERR_DTYPE;
  if (!aligned16(dx) || !aligned16(dw)) return TE_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    const size_t bytes = static_cast<size_t>(2 * F * K) * (dw_dtype == TE_F32 ? 4 : 2);
    if (dw && !accumulate && cudaMemsetAsync(dw, 0, bytes, st) != cudaSuccess) return record_cuda(cudaGetLastError());
    return TE_OK;
  }
  if ((s = check_operands(dy, w2)) != TE_OK) return s;
  if (dx && (s = check_operands(w, w)) != TE_OK) return s;
  if (dw && (s = check_operands(x, x)) != TE_OK) return s;
  GatedArgs ep = {};
  if ((s = dgrad_args(&ep, gu, dgu, T, F, act)) != TE_OK) return s;
  // dh = dY W2 (W2 [N, F] read MN-major), dg and du in its epilogue.  The next kernel is set up while
  // this one drains, and dW, which reads the same dGU, runs beside dX wherever that leaves SMs idle
  // (1001 tokens, K = N = 768, F = 2048: dX has 12 tiles for 76 pairs).
  s = launch_gemm<kBF16, 2, kDgrad, true>(dy, w2, N * 2, nullptr, nullptr, 0, nullptr, nullptr, nullptr, nullptr,
                                          TE_BF16, 0, T, F, N, 1u, 1u, st, 0, 1, ep, kPdlChain);
  // dX = dGU W (W [2 F, K] MN-major);  dW = dGU^T X (both MN-major).  They contract dg and du as stored, rounded
  // to bf16: the tensor cores take no wider operand, and a second one for what the rounding drops would double
  // their work.  Their outputs are then 0.0023 off (relative Frobenius), two roundings, where one leaves 0.0017.  dX's tiles are shared between CTA
  // pairs only as far as dW's fit beside them, where they fit at all.
  int share = 4;
  if (dx && dw) {
    const int64_t tx = (T + 255) / 256 * ((K + 255) / 256), tw = (2 * F + 255) / 256 * ((K + 255) / 256);
    const int64_t free_pairs = num_sms() / 2 - tw;
    if (tx <= free_pairs) share = 4 * tx <= free_pairs ? 4 : (2 * tx <= free_pairs ? 2 : 1);
  }
  if (s == TE_OK && dx)
    s = gemm_bf16_tokens(dgu, 0, w, 1, dx, TE_BF16, 0, T, K, 2 * F, st, kPdlChain, share);
  if (s == TE_OK && dw)
    s = gemm_bf16_tokens(dgu, 1, x, 1, dw, dw_dtype, accumulate, 2 * F, K, T, st, dx ? kPdlWaitAtEnd : kPdlChain);
  return s;
}

}  // extern "C"
