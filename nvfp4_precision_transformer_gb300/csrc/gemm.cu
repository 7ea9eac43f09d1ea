// Entry points of the plain GEMMs: D = alpha * A B^T (+ bias).  The kernel is in gemm.cuh.
#include "gemm.cuh"

namespace te {
namespace {

te_status check_gemm(const void* A, const void* B, const void* D, te_dtype out, int accumulate, int64_t M, int64_t N,
                     int64_t K, int64_t k_multiple) {
  if (out != TE_BF16 && out != TE_F32) return TE_ERR_DTYPE;
  if (accumulate != 0 && accumulate != 1) return TE_ERR_ARG;
  if (accumulate && out != TE_F32) return TE_ERR_DTYPE;
  if (M < 0 || N < 0 || K <= 0 || M % 16 || N % 16 || K % k_multiple) return TE_ERR_SHAPE;
  if (M > (int64_t(1) << 30) || N > (int64_t(1) << 30) || K > (int64_t(1) << 30)) return TE_ERR_SHAPE;
  if (M * N == 0) return TE_OK;
  if (!A || !B || !D) return TE_ERR_NULL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(D)) return TE_ERR_ALIGN;
  return TE_OK;
}

inline bool fp8_fmt(te_dtype f) { return f == TE_E4M3 || f == TE_E5M2; }
inline uint32_t f8_code(te_dtype f) { return f == TE_E5M2 ? 1u : 0u; }

}  // namespace

te_status gemm_bf16_tokens(const void* A, int a_mn, const void* B, int b_mn, void* D, te_dtype out, int accumulate,
                           int64_t M, int64_t N, int64_t K, cudaStream_t st, int pdl, int max_split) {
  return launch_gemm<kBF16, 2, kPlain, true>(A, B, K * 2, nullptr, nullptr, 0, nullptr, nullptr, nullptr, D, out,
                                             accumulate, M, N, K, 1u, 1u, st, a_mn, b_mn, NoEpiArgs(), pdl, max_split);
}

}  // namespace te

using namespace te;

extern "C" {

te_status te_gemm_bf16(const void* A, te_layout a_layout, const void* B, te_layout b_layout, const float* bias, void* D,
                       te_dtype out_dtype, int accumulate, int64_t M, int64_t N, int64_t K, void* stream) {
  if ((a_layout != TE_K_MAJOR && a_layout != TE_MN_MAJOR) || (b_layout != TE_K_MAJOR && b_layout != TE_MN_MAJOR))
    return TE_ERR_ARG;
  te_status s = check_gemm(A, B, D, out_dtype, accumulate, M, N, K, 16);
  if (s != TE_OK || M * N == 0) return s;
  return launch_gemm<kBF16, 2>(A, B, K * 2, nullptr, nullptr, 0, nullptr, nullptr, bias, D, out_dtype, accumulate, M, N,
                               K, 1u, 1u, static_cast<cudaStream_t>(stream), a_layout == TE_MN_MAJOR,
                               b_layout == TE_MN_MAJOR);
}

te_status te_gemm_fp8(const uint8_t* A, te_dtype fa, const uint8_t* B, te_dtype fb, const float* a_scale_inv,
                      const float* b_scale_inv, const float* bias, void* D, te_dtype out_dtype, int accumulate,
                      int64_t M, int64_t N, int64_t K, void* stream) {
  if (!fp8_fmt(fa) || !fp8_fmt(fb)) return TE_ERR_DTYPE;
  te_status s = check_gemm(A, B, D, out_dtype, accumulate, M, N, K, 16);
  if (s != TE_OK || M * N == 0) return s;
  if (!a_scale_inv || !b_scale_inv) return TE_ERR_NULL;
  return launch_gemm<kFP8, 2>(A, B, K, nullptr, nullptr, 0, a_scale_inv, b_scale_inv, bias, D, out_dtype, accumulate, M,
                              N, K, f8_code(fa), f8_code(fb), static_cast<cudaStream_t>(stream));
}

te_status te_gemm_mxfp8(const uint8_t* A, te_dtype fa, const uint8_t* sA, const uint8_t* B, te_dtype fb,
                        const uint8_t* sB, const float* bias, void* D, te_dtype out_dtype, int accumulate,
                        int64_t M, int64_t N, int64_t K, void* stream) {
  if (!fp8_fmt(fa) || !fp8_fmt(fb)) return TE_ERR_DTYPE;
  te_status s = check_gemm(A, B, D, out_dtype, accumulate, M, N, K, 32);
  if (s != TE_OK || M * N == 0) return s;
  if (!sA || !sB) return TE_ERR_NULL;
  if (!aligned16(sA) || !aligned16(sB)) return TE_ERR_ALIGN;
  const int64_t katoms = ((K / 32 + 3) / 4);
  return launch_gemm<kMXFP8, 2>(A, B, K, sA, sB, katoms, nullptr, nullptr, bias, D, out_dtype, accumulate, M, N, K,
                                f8_code(fa), f8_code(fb), static_cast<cudaStream_t>(stream));
}

te_status te_gemm_nvfp4(const uint8_t* A, const uint8_t* sA, const float* gA, const uint8_t* B, const uint8_t* sB,
                        const float* gB, const float* bias, void* D, te_dtype out_dtype, int accumulate,
                        int64_t M, int64_t N, int64_t K, void* stream) {
  te_status s = check_gemm(A, B, D, out_dtype, accumulate, M, N, K, 32);
  if (s != TE_OK || M * N == 0) return s;
  if (!sA || !sB || !gA || !gB) return TE_ERR_NULL;
  if (!aligned16(sA) || !aligned16(sB)) return TE_ERR_ALIGN;
  const int64_t katoms = ((K / 16 + 15) / 16) * 4;
  return launch_gemm<kNVFP4, 2>(A, B, K / 2, sA, sB, katoms, gA, gB, bias, D, out_dtype, accumulate, M, N, K, 1u, 1u,
                                static_cast<cudaStream_t>(stream));
}

}  // extern "C"
