// Entry points of the linear with bias, activation and residual in its epilogue, y = act(x W^T + b) + residual,
// and of its backward pass.  The kernels are gemm_kernel with the epilogues of act_epilogue.inc, and those of
// act_decode.cuh and act_stream.cuh for few tokens.
#include "act_stream.cuh"

namespace te {
namespace {

// amax = 0 and 1 / scale where there is no row to compute them beside.
__global__ void publish_empty_act_kernel(const float* scale, float* amax, float* scale_inv) {
  if (amax) *amax = 0.0f;
  if (scale_inv) *scale_inv = __fdiv_rn(1.0f, *scale);
}

bool fp8_format(te_dtype f) { return f == TE_E4M3 || f == TE_E5M2; }
uint32_t fp8_code(te_dtype f) { return f == TE_E5M2 ? 1u : 0u; }

te_status check_sizes(int act, int64_t T, int64_t K, int64_t K_mult, int64_t N, int64_t N_mult) {
  if (act != TE_ACT_NONE && act != TE_ACT_RELU && act != TE_ACT_SILU && act != TE_ACT_GELU) return TE_ERR_ARG;
  if (T < 0 || N <= 0 || K <= 0 || N % N_mult || K % K_mult) return TE_ERR_SHAPE;
  if (T > (int64_t(1) << 30) || N > (int64_t(1) << 29) || K > (int64_t(1) << 30)) return TE_ERR_SHAPE;
  return TE_OK;
}

te_status check_operands(const void* a, const void* b) {
  if (!a || !b) return TE_ERR_NULL;
  return aligned16(a) && aligned16(b) ? TE_OK : TE_ERR_ALIGN;
}

// Boxes of 32 rows x 64 bytes of a [T, N] tensor whose elements have `size` bytes.
te_status boxes(CUtensorMap* map, const void* p, int64_t T, int64_t N, int size) {
  const uint64_t row = static_cast<uint64_t>(N) * static_cast<uint64_t>(size);
  return make_tmap_2d_view64(map, p, row, row, static_cast<uint64_t>(T));
}

// What every forward call has: checked before anything is enqueued.
struct Outputs {
  const float* bias;
  int act;
  const void* residual;
  void* z;
  void* y;
  te_dtype y_dtype;
  uint8_t* q;
};
te_status check_outputs(const Outputs& o) {
  if (!o.z && !o.y && !o.q) return TE_ERR_NULL;
  if (o.y && o.y_dtype != TE_BF16 && o.y_dtype != TE_F32) return TE_ERR_DTYPE;
  if (o.residual && !o.y) return TE_ERR_NULL;
  if (o.residual && o.q) return TE_ERR_UNSUPPORTED;
  if (!aligned16(o.bias) || !aligned16(o.residual) || !aligned16(o.z) || !aligned16(o.y) || !aligned16(o.q))
    return TE_ERR_ALIGN;
  return TE_OK;
}

te_status act_args(ActArgs* ep, const Outputs& o, int64_t T, int64_t N) {
  ep->N = static_cast<int>(N);
  ep->act = o.act;
  ep->bias = o.bias;
  ep->has_y = o.y != nullptr;
  ep->has_z = o.z != nullptr;
  ep->has_res = o.residual != nullptr;
  ep->has_q = o.q != nullptr;
  ep->y_f32 = o.y != nullptr && o.y_dtype == TE_F32;
  const int size = ep->y_f32 ? 4 : 2;
  te_status s = TE_OK;
  if (o.y && (s = boxes(&ep->y, o.y, T, N, size)) != TE_OK) return s;
  if (o.residual && (s = boxes(&ep->res, o.residual, T, N, size)) != TE_OK) return s;
  if (o.z && (s = boxes(&ep->z, o.z, T, N, 2)) != TE_OK) return s;
  if (o.q) {
    if ((s = boxes(&ep->q, o.q, T, N, 1)) != TE_OK) return s;
    s = make_tmap_2d_plain(&ep->q32, o.q, static_cast<uint64_t>(N), static_cast<uint64_t>(T), 32u, 32u);
  }
  return s;
}

// The same for the kernels of few tokens.
FewArgs few_args(const void* x, const void* w, const Outputs& o, int64_t T, int64_t K, int64_t N) {
  FewArgs a = {};
  a.x = static_cast<const uint8_t*>(x);
  a.w = static_cast<const uint8_t*>(w);
  a.T = static_cast<int>(T);
  a.K = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.act = o.act;
  a.bias = o.bias;
  a.res = o.residual;
  a.z = static_cast<__nv_bfloat16*>(o.z);
  a.y = o.y;
  a.y_f32 = o.y != nullptr && o.y_dtype == TE_F32;
  a.q = o.q;
  return a;
}

// dbias[c] = the sum of the partial rows (one for each 32 tokens) in a fixed order: 32 columns x 32 row lanes a
// CTA.  It is set up, and may run, beside a kernel that does not write them (`beside`: it then waits for that one
// at its end, see kPdlWaitAtEnd); its loads go past L1, which may hold an earlier call's sums.
__global__ void __launch_bounds__(1024) act_dbias_kernel(const float* partial, int64_t n, int64_t N, float* dbias,
                                                         int beside) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (!beside) dev::pdl_wait();
  dev::pdl_trigger();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float t = 0.0f;
  if (c < N) {
    for (int64_t r0 = w; r0 < n; r0 += 32 * 8) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t r = r0 + 32 * k;
        v[k] = 0.0f;
        if (r < n) asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v[k]) : "l"(partial + r * N + c) : "memory");
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) t = __fadd_rn(t, v[k]);
    }
  }
  part[w][lane] = t;
  __syncthreads();
  t = part[lane][w];   // warp w: column w
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t = __fadd_rn(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + w;
  if (lane == 0 && col < N) dbias[col] = t;
  if (beside) dev::pdl_wait();
}

te_status reduce_dbias(const float* partial, int64_t T, int64_t N, float* dbias, int beside, cudaStream_t st) {
  const cudaError_t e = launch_dependent(act_dbias_kernel, dim3(static_cast<unsigned>((N + 31) / 32), 1, 1),
                                         dim3(1024, 1, 1), 0, st, partial, (T + 31) / 32, N, dbias, beside);
  if (e != cudaSuccess) return record_cuda(e);
  count_launch();
  return launch_status();
}

size_t partial_bytes(int64_t T, int64_t F) {
  if (T <= 0 || F <= 0) return 0;
  return static_cast<size_t>((T + 31) / 32) * static_cast<size_t>(F) * sizeof(float);
}

// The backward pass's own tensors: their checks, and their description for a call with tokens.
struct Grads {
  const void* z;
  int act;
  void* dz;
  float* dbias;
  float* workspace;
  size_t workspace_bytes;
};
te_status check_grads(const Grads& g, int64_t T, int64_t F) {
  if (reinterpret_cast<uintptr_t>(g.dbias) & 3u) return TE_ERR_ALIGN;
  if (T == 0) return TE_OK;
  if (!g.dz || (!g.z && g.act != TE_ACT_NONE)) return TE_ERR_NULL;
  if (!aligned16(g.z) || !aligned16(g.dz)) return TE_ERR_ALIGN;
  if (g.dbias) {
    if (!g.workspace) return TE_ERR_NULL;
    if (g.workspace_bytes < partial_bytes(T, F)) return TE_ERR_SHAPE;
    if (!aligned16(g.workspace)) return TE_ERR_ALIGN;
  }
  return TE_OK;
}
te_status grads_args(ActArgs* ep, const Grads& g, int64_t T, int64_t F) {
  ep->N = static_cast<int>(F);
  ep->act = g.act;
  ep->partial = g.dbias ? g.workspace : nullptr;
  ep->has_z = g.act != TE_ACT_NONE;
  const te_status s = boxes(&ep->y, g.dz, T, F, 2);
  return s == TE_OK && g.act != TE_ACT_NONE ? boxes(&ep->z, g.z, T, F, 2) : s;
}

// dW [F, K] (+)= dZ^T X (both MN-major).  In fp32 by the forward pass's kernel, whose residual is what dW holds where it
// is added to: its sum over the tokens is cut into segments, as every fp32 output's (kSegments in gemm.cuh; 16384 tokens
// in one piece are 2e-5 short, where all terms have one sign 3.7e-5 and more).  The whole pass with dw in fp32 takes 4100
// us at 15872 tokens, K = N = 4096, F = 16384, uncut 3910; at 4096 tokens, K = F = 4096, N = 1024 224 and 212.
te_status weight_grad(const void* dz, const void* x, void* dw, te_dtype dt, int accumulate, int64_t T, int64_t K, int64_t F,
                      cudaStream_t st, int pdl) {
  if (dt != TE_F32) return gemm_bf16_tokens(dz, 1, x, 1, dw, dt, 0, F, K, T, st, pdl);
  ActArgs ep = {};
  const Outputs o = {nullptr, TE_ACT_NONE, accumulate ? dw : nullptr, nullptr, dw, TE_F32, nullptr};
  const te_status s = act_args(&ep, o, F, K);
  if (s != TE_OK) return s;
  return launch_gemm<kBF16, 2, kAct, true>(dz, x, T * 2, nullptr, nullptr, 0, nullptr, nullptr, nullptr, nullptr, TE_F32, 0,
                                           F, K, T, 1u, 1u, st, 1, 1, ep, pdl, 4, kSegment<kBF16>);
}

// No tokens: dbias = 0.
te_status empty_dbias(float* dbias, int64_t F, cudaStream_t st) {
  if (dbias && cudaMemsetAsync(dbias, 0, static_cast<size_t>(F) * sizeof(float), st) != cudaSuccess)
    return record_cuda(cudaGetLastError());
  return TE_OK;
}

}  // namespace
}  // namespace te

using namespace te;

extern "C" {

te_status te_act_gemm_bf16(const void* x, const void* w, const float* bias, int act, const void* residual, void* z,
                           void* y, te_dtype y_dtype, int64_t T, int64_t K, int64_t N, void* stream) {
  te_status s = check_sizes(act, T, K, 16, N, 16);
  if (s != TE_OK || T == 0) return s;
  const Outputs o = {bias, act, residual, z, y, y_dtype, nullptr};
  if ((s = check_outputs(o)) != TE_OK) return s;
  if ((s = check_operands(x, w)) != TE_OK) return s;
  if (T <= kAstMaxTokens) {
    const FewArgs a = few_args(x, w, o, T, K, N);
    if (act_decodes(T, K, N, 2)) return launch_act_decode<kDecBF16, kDecBF16>(a, static_cast<cudaStream_t>(stream));
    bool taken;
    s = launch_act_stream<kBF16>(a, 1u, 1u, static_cast<cudaStream_t>(stream), &taken);
    if (taken || s != TE_OK) return s;
  }
  ActArgs ep = {};
  if ((s = act_args(&ep, o, T, N)) != TE_OK) return s;
  return launch_gemm<kBF16, 2, kAct, true>(x, w, K * 2, nullptr, nullptr, 0, nullptr, nullptr, nullptr, nullptr, TE_BF16,
                                           0, T, N, K, 1u, 1u, static_cast<cudaStream_t>(stream), 0, 0, ep, kPdlChain, 4,
                                           ep.y_f32 ? kSegment<kBF16> : 0);
}

te_status te_act_gemm_fp8(const uint8_t* x, te_dtype fx, const uint8_t* w, te_dtype fw, const float* x_scale_inv,
                          const float* w_scale_inv, const float* bias, int act, const void* residual, void* z, void* y,
                          te_dtype y_dtype, uint8_t* q, te_dtype q_fmt, const float* q_scale, float* q_amax,
                          float* q_scale_inv, int64_t T, int64_t K, int64_t N, void* stream) {
  if (!fp8_format(fx) || !fp8_format(fw) || (q && !fp8_format(q_fmt))) return TE_ERR_DTYPE;
  te_status s = check_sizes(act, T, K, 16, N, 16);
  if (s != TE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (q_scale_inv && !q_scale) return TE_ERR_NULL;
    if (!q_amax && !q_scale_inv) return TE_OK;
    publish_empty_act_kernel<<<1, 1, 0, st>>>(q_scale, q_amax, q_scale_inv);
    count_launch();
    return launch_status();
  }
  const Outputs o = {bias, act, residual, z, y, y_dtype, q};
  if ((s = check_outputs(o)) != TE_OK) return s;
  if (q ? !q_scale : (q_amax || q_scale_inv)) return TE_ERR_NULL;   // the amax and 1 / scale go with q
  if (!x_scale_inv || !w_scale_inv) return TE_ERR_NULL;
  if ((s = check_operands(x, w)) != TE_OK) return s;
  if (T <= kAstMaxTokens) {
    FewArgs a = few_args(x, w, o, T, K, N);
    a.alpha_a = x_scale_inv;
    a.alpha_b = w_scale_inv;
    a.q_scale = q_scale;
    a.q_e5m2 = q_fmt == TE_E5M2;
    a.amax = reinterpret_cast<unsigned int*>(q_amax);
    a.scale_inv = q_scale_inv;
    if (act_decodes(T, K, N, 1)) {
      if (fw == TE_E4M3)
        return fx == TE_E4M3 ? launch_act_decode<kDecE4M3, kDecE4M3>(a, st) : launch_act_decode<kDecE4M3, kDecE5M2>(a, st);
      return fx == TE_E4M3 ? launch_act_decode<kDecE5M2, kDecE4M3>(a, st) : launch_act_decode<kDecE5M2, kDecE5M2>(a, st);
    }
    bool taken;
    s = launch_act_stream<kFP8>(a, fp8_code(fx), fp8_code(fw), st, &taken);
    if (taken || s != TE_OK) return s;
  }
  ActArgs ep = {};
  if ((s = act_args(&ep, o, T, N)) != TE_OK) return s;
  if (q) {
    ep.q_e5m2 = q_fmt == TE_E5M2;
    ep.q_scale = q_scale;
    ep.amax = reinterpret_cast<unsigned int*>(q_amax);
    ep.scale_inv = q_scale_inv;
  }
  if (q_amax && (s = zero_amax(q_amax, st)) != TE_OK) return s;
  return launch_gemm<kFP8, 2, kAct, true>(x, w, K, nullptr, nullptr, 0, x_scale_inv, w_scale_inv, nullptr, nullptr,
                                          TE_BF16, 0, T, N, K, fp8_code(fx), fp8_code(fw), st, 0, 0, ep, kPdlChain, 4,
                                          kSegment<kFP8>);
}

te_status te_act_gemm_mxfp8(const uint8_t* x, te_dtype fx, const uint8_t* sx, const uint8_t* w, te_dtype fw,
                            const uint8_t* sw, const float* bias, int act, const void* residual, void* z, void* y,
                            te_dtype y_dtype, uint8_t* q, uint8_t* s_q, int64_t T, int64_t K, int64_t N, void* stream) {
  if (!fp8_format(fx) || !fp8_format(fw)) return TE_ERR_DTYPE;
  te_status s = check_sizes(act, T, K, 32, N, q ? 32 : 16);
  if (s != TE_OK || T == 0) return s;
  const Outputs o = {bias, act, residual, z, y, y_dtype, q};
  if ((q == nullptr) != (s_q == nullptr)) return TE_ERR_NULL;
  if ((s = check_outputs(o)) != TE_OK) return s;
  if ((s = check_operands(x, w)) != TE_OK) return s;
  if ((s = check_operands(sx, sw)) != TE_OK) return s;
  if (!aligned16(s_q)) return TE_ERR_ALIGN;
  if (T <= kAstMaxTokens) {
    FewArgs a = few_args(x, w, o, T, K, N);
    a.sx = sx;
    a.sw = sw;
    a.s_kpad = (K / 32 + 3) / 4 * 4;
    a.s_q = s_q;
    a.q_kpad = (N / 32 + 3) / 4 * 4;
    bool taken;
    s = launch_act_stream<kMXFP8>(a, fp8_code(fx), fp8_code(fw), static_cast<cudaStream_t>(stream), &taken);
    if (taken || s != TE_OK) return s;
  }
  ActArgs ep = {};
  if ((s = act_args(&ep, o, T, N)) != TE_OK) return s;
  ep.s_q = s_q;
  ep.s_kpad = (N / 32 + 3) / 4 * 4;
  ep.s_rows = static_cast<int>((T + 127) / 128 * 128);
  return launch_gemm<kMXFP8, 2, kAct>(x, w, K, sx, sw, (K / 32 + 3) / 4, nullptr, nullptr, nullptr, nullptr, TE_BF16, 0,
                                      T, N, K, fp8_code(fx), fp8_code(fw), static_cast<cudaStream_t>(stream), 0, 0, ep,
                                      kPdlChain, 4, kSegment<kMXFP8>);
}

te_status te_act_gemm_nvfp4(const uint8_t* x, const uint8_t* sx, const float* gx, const uint8_t* w, const uint8_t* sw,
                            const float* gw, const float* bias, int act, const void* residual, void* z, void* y,
                            te_dtype y_dtype, int64_t T, int64_t K, int64_t N, void* stream) {
  te_status s = check_sizes(act, T, K, 32, N, 16);
  if (s != TE_OK || T == 0) return s;
  const Outputs o = {bias, act, residual, z, y, y_dtype, nullptr};
  if ((s = check_outputs(o)) != TE_OK) return s;
  if (!gx || !gw) return TE_ERR_NULL;
  if ((s = check_operands(x, w)) != TE_OK) return s;
  if ((s = check_operands(sx, sw)) != TE_OK) return s;
  if (T <= kAstMaxTokens) {
    FewArgs a = few_args(x, w, o, T, K, N);
    a.alpha_a = gx;
    a.alpha_b = gw;
    a.sx = sx;
    a.sw = sw;
    a.s_kpad = (K / 16 + 15) / 16 * 16;
    bool taken;
    s = launch_act_stream<kNVFP4>(a, 1u, 1u, static_cast<cudaStream_t>(stream), &taken);
    if (taken || s != TE_OK) return s;
  }
  ActArgs ep = {};
  if ((s = act_args(&ep, o, T, N)) != TE_OK) return s;
  return launch_gemm<kNVFP4, 2, kAct>(x, w, K / 2, sx, sw, (K / 16 + 15) / 16 * 4, gx, gw, nullptr, nullptr, TE_BF16, 0,
                                      T, N, K, 1u, 1u, static_cast<cudaStream_t>(stream), 0, 0, ep, kPdlChain);
}

size_t te_act_dbias_workspace_bytes(int64_t T, int64_t F) { return partial_bytes(T, F); }

te_status te_act_dgrad_fp8(const uint8_t* dy, te_dtype fd, const uint8_t* w2, te_dtype fw, const float* dy_scale_inv,
                           const float* w2_scale_inv, const void* z, int act, void* dz, float* dbias, float* workspace,
                           size_t workspace_bytes, int64_t T, int64_t F, int64_t N, void* stream) {
  if (!fp8_format(fd) || !fp8_format(fw)) return TE_ERR_DTYPE;
  te_status s = check_sizes(act, T, N, 16, F, 16);
  if (s != TE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Grads g = {z, act, dz, dbias, workspace, workspace_bytes};
  if ((s = check_grads(g, T, F)) != TE_OK) return s;
  if (T == 0) return empty_dbias(dbias, F, st);
  if (!dy_scale_inv || !w2_scale_inv) return TE_ERR_NULL;
  if ((s = check_operands(dy, w2)) != TE_OK) return s;
  ActArgs ep = {};
  if ((s = grads_args(&ep, g, T, F)) != TE_OK) return s;
  s = launch_gemm<kFP8, 2, kActGrad, true>(dy, w2, N, nullptr, nullptr, 0, dy_scale_inv, w2_scale_inv, nullptr, nullptr,
                                           TE_BF16, 0, T, F, N, fp8_code(fd), fp8_code(fw), st, 0, 0, ep, kPdlChain, 4,
                                           kSegment<kFP8>);
  return s != TE_OK || !dbias ? s : reduce_dbias(workspace, T, F, dbias, 0, st);
}

te_status te_act_dgrad_mxfp8(const uint8_t* dy, te_dtype fd, const uint8_t* sd, const uint8_t* w2, te_dtype fw,
                             const uint8_t* sw, const void* z, int act, void* dz, float* dbias, float* workspace,
                             size_t workspace_bytes, int64_t T, int64_t F, int64_t N, void* stream) {
  if (!fp8_format(fd) || !fp8_format(fw)) return TE_ERR_DTYPE;
  te_status s = check_sizes(act, T, N, 32, F, 16);
  if (s != TE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Grads g = {z, act, dz, dbias, workspace, workspace_bytes};
  if ((s = check_grads(g, T, F)) != TE_OK) return s;
  if (T == 0) return empty_dbias(dbias, F, st);
  if ((s = check_operands(dy, w2)) != TE_OK) return s;
  if ((s = check_operands(sd, sw)) != TE_OK) return s;
  ActArgs ep = {};
  if ((s = grads_args(&ep, g, T, F)) != TE_OK) return s;
  s = launch_gemm<kMXFP8, 2, kActGrad>(dy, w2, N, sd, sw, (N / 32 + 3) / 4, nullptr, nullptr, nullptr, nullptr, TE_BF16,
                                       0, T, F, N, fp8_code(fd), fp8_code(fw), st, 0, 0, ep, kPdlChain, 4, kSegment<kMXFP8>);
  return s != TE_OK || !dbias ? s : reduce_dbias(workspace, T, F, dbias, 0, st);
}

te_status te_act_dgrad_nvfp4(const uint8_t* dy, const uint8_t* sd, const float* gd, const uint8_t* w2, const uint8_t* sw,
                             const float* gw, const void* z, int act, void* dz, float* dbias, float* workspace,
                             size_t workspace_bytes, int64_t T, int64_t F, int64_t N, void* stream) {
  te_status s = check_sizes(act, T, N, 32, F, 16);
  if (s != TE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Grads g = {z, act, dz, dbias, workspace, workspace_bytes};
  if ((s = check_grads(g, T, F)) != TE_OK) return s;
  if (T == 0) return empty_dbias(dbias, F, st);
  if (!gd || !gw) return TE_ERR_NULL;
  if ((s = check_operands(dy, w2)) != TE_OK) return s;
  if ((s = check_operands(sd, sw)) != TE_OK) return s;
  ActArgs ep = {};
  if ((s = grads_args(&ep, g, T, F)) != TE_OK) return s;
  s = launch_gemm<kNVFP4, 2, kActGrad>(dy, w2, N / 2, sd, sw, (N / 16 + 15) / 16 * 4, gd, gw, nullptr, nullptr, TE_BF16,
                                       0, T, F, N, 1u, 1u, st, 0, 0, ep, kPdlChain);
  return s != TE_OK || !dbias ? s : reduce_dbias(workspace, T, F, dbias, 0, st);
}

te_status te_act_bwd_bf16(const void* x, const void* w, const void* w2, const void* dy, const void* z, int act, void* dz,
                          float* dbias, float* workspace, size_t workspace_bytes, void* dx, void* dw, te_dtype dw_dtype,
                          int accumulate, int64_t T, int64_t K, int64_t F, int64_t N, void* stream) {
  te_status s = check_sizes(act, T, N, 16, F, 16);
  if (s != TE_OK) return s;
  if ((dx || dw) && (K <= 0 || K % 16 || K > (int64_t(1) << 30))) return TE_ERR_SHAPE;
  if (dw && dw_dtype != TE_BF16 && dw_dtype != TE_F32) return TE_ERR_DTYPE;
  if (dw && dw_dtype == TE_F32 && K > (int64_t(1) << 29)) return TE_ERR_SHAPE;   // (columns are counted in bytes)
  if (accumulate != 0 && accumulate != 1) return TE_ERR_ARG;
  if (dw && accumulate && dw_dtype != TE_F32) return TE_ERR_DTYPE;
  if (!aligned16(dx) || !aligned16(dw)) return TE_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Grads g = {z, act, dz, dbias, workspace, workspace_bytes};
  if ((s = check_grads(g, T, F)) != TE_OK) return s;
  if (T == 0) {
    const size_t bytes = static_cast<size_t>(F * K) * (dw_dtype == TE_F32 ? 4 : 2);
    if (dw && !accumulate && cudaMemsetAsync(dw, 0, bytes, st) != cudaSuccess) return record_cuda(cudaGetLastError());
    return empty_dbias(dbias, F, st);
  }
  if ((s = check_operands(dy, w2)) != TE_OK) return s;
  if (dx && (s = check_operands(w, w)) != TE_OK) return s;
  if (dw && (s = check_operands(x, x)) != TE_OK) return s;
  ActArgs ep = {};
  if ((s = grads_args(&ep, g, T, F)) != TE_OK) return s;
  // dh = dY W2 (W2 [N, F] read MN-major), dz in its epilogue.  The kernels after it read dz and the partial sums
  // and nothing of one another, so dbias and dW run beside dX wherever that leaves SMs idle.
  s = launch_gemm<kBF16, 2, kActGrad, true>(dy, w2, N * 2, nullptr, nullptr, 0, nullptr, nullptr, nullptr, nullptr,
                                            TE_BF16, 0, T, F, N, 1u, 1u, st, 0, 1, ep, kPdlChain, 4, kSegment<kBF16>);
  // dX = dZ W (W [F, K] MN-major);  dW = dZ^T X (both MN-major), on dz as stored, rounded to bf16: the tensor cores
  // take no wider operand (dx and dw in bf16 are off by 2.3e-3 relative, from a dz in fp32 they would be by 1.7e-3).
  // dX's tiles are shared between CTA pairs only as far as dW's fit beside them, where they fit at all.
  int share = 4;
  if (dx && dw) {
    const int64_t tx = (T + 255) / 256 * ((K + 255) / 256), tw = (F + 255) / 256 * ((K + 255) / 256);
    const int64_t free_pairs = num_sms() / 2 - tw;
    if (tx <= free_pairs) share = 4 * tx <= free_pairs ? 4 : (2 * tx <= free_pairs ? 2 : 1);
  }
  if (s == TE_OK && dx) s = gemm_bf16_tokens(dz, 0, w, 1, dx, TE_BF16, 0, T, K, F, st, kPdlChain, share);
  if (s == TE_OK && dw)
    s = weight_grad(dz, x, dw, dw_dtype, accumulate, T, K, F, st, dx ? kPdlWaitAtEnd | kPdlTrigger : kPdlChain);
  // (behind dW, which lets it start: between the two it would hold SMs that dW needs until dX ends, 39.5 us for 31 at
  // 1001 tokens, K = N = 768, F = 2048)
  if (s == TE_OK && dbias) s = reduce_dbias(workspace, T, F, dbias, dx != nullptr || dw != nullptr, st);
  return s;
}

}  // extern "C"
