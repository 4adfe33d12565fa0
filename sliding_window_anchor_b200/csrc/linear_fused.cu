// linear_fused.cu — the products that stand between the SWA∥RMA layers of the
// model (EdgeRock-4B 开源：72 MiB 固定 KV, §架构：递归、局部窗口与记忆锚点三件套:
// 32 layers, of which eight are SWA∥RMA): a linear product with bias, activation
// and residual, and the gated feed-forward product.
//
//   er_linear_fused: y = act(x·wᵀ + bias) + residual
//   er_gated_linear: y = act(x·w_gateᵀ) ⊙ (x·w_upᵀ)
//
// x, w, bias BF16; the sums, the activation and the product stay in FP32 and
// are rounded once, into y.
#include "common.cuh"

namespace er {
namespace {

struct FusedParams {
  const uint16_t* x;
  const uint16_t *w, *w2;  // w2: the second projection of the gated product, or NULL
  const uint16_t* bias;
  const void* residual;
  void* y;
  int T, F, K;
  int64_t ldx, ldr, ldy;
  int act, f32;
};

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case ER_ACT_SILU:
      return v / (1.f + expf(-v));
    case ER_ACT_GELU:
      return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    case ER_ACT_GELU_TANH:
      return 0.5f * v * (1.f + tanhf(0.79788456080286536f * (v + 0.044715f * v * v * v)));
    default:
      return v;
  }
}

// 64 tokens x 64 features per block of 16 x 16 threads, FP32 FMAs.
template <bool GATED>
__global__ void __launch_bounds__(256) k_fused_tile(const FusedParams P) {
  __shared__ float xs[16][65], ws[16][65], us[GATED ? 16 : 1][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int t0 = blockIdx.y * 64, f0 = blockIdx.x * 64;
  float a[4][4] = {}, u[4][4] = {};
  for (int k0 = 0; k0 < P.K; k0 += 16) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int r = i >> 4, k = i & 15;
      const bool kin = k0 + k < P.K;
      xs[k][r] = kin && t0 + r < P.T ? bf1(P.x[(t0 + r) * P.ldx + k0 + k]) : 0.f;
      const bool fin = kin && f0 + r < P.F;
      const size_t at = (size_t)(f0 + r) * P.K + k0 + k;
      ws[k][r] = fin ? bf1(P.w[at]) : 0.f;
      if (GATED) us[k][r] = fin ? bf1(P.w2[at]) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
          a[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], a[i][j]);
          if (GATED) u[i][j] = fmaf(xs[k][ty + 16 * i], us[k][tx + 16 * j], u[i][j]);
        }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + ty + 16 * i, f = f0 + tx + 16 * j;
      if (t >= P.T || f >= P.F) continue;
      float v = a[i][j];
      if (P.bias) v += bf1(P.bias[f]);
      v = activate(v, P.act);
      if (GATED) v *= u[i][j];
      if (P.residual)
        v += P.f32 ? static_cast<const float*>(P.residual)[t * P.ldr + f]
                   : bf1(static_cast<const uint16_t*>(P.residual)[t * P.ldr + f]);
      if (P.f32)
        static_cast<float*>(P.y)[t * P.ldy + f] = v;
      else
        static_cast<uint16_t*>(P.y)[t * P.ldy + f] = f2bf(v);
    }
}

int launch_fused(const FusedParams& P, cudaStream_t st) {
  const dim3 grid((P.F + 63) / 64, (P.T + 63) / 64);
  if (P.w2)
    k_fused_tile<true><<<grid, 256, 0, st>>>(P);
  else
    k_fused_tile<false><<<grid, 256, 0, st>>>(P);
  count_launches(1);
  return launch_status();
}

bool sizes_ok(int32_t T, int32_t F, int32_t K, int32_t ldx, int32_t act, int32_t y_fp32,
              int32_t ldy) {
  return T >= 0 && F >= 1 && K >= 8 && K % 8 == 0 && ldx >= K && ldx % 8 == 0 && ldy >= F &&
         act >= ER_ACT_NONE && act <= ER_ACT_GELU_TANH && (y_fp32 == 0 || y_fp32 == 1);
}

}  // namespace
}  // namespace er

using namespace er;

extern "C" {

int er_linear_fused(const er_bf16* x, int32_t ldx, int32_t T, const er_bf16* w, int32_t F,
                    int32_t K, const er_bf16* bias, int32_t act, const void* residual,
                    int32_t ldr, void* y, int32_t y_fp32, int32_t ldy, int32_t* dev_error,
                    er_stream_t stream) {
  if (!sizes_ok(T, F, K, ldx, act, y_fp32, ldy) || (residual && ldr < F)) return ER_EINVAL;
  if (T == 0) return ER_OK;
  const uintptr_t el = y_fp32 ? 3u : 1u;
  if (!x || !w || !y || !aligned16(x) || !aligned16(w) || ((uintptr_t)y & el) ||
      ((uintptr_t)residual & el) || ((uintptr_t)bias & 1u))
    return ER_EINVAL;
  FusedParams P{x, w, nullptr, bias, residual, y, T, F, K, ldx, ldr, ldy, act, y_fp32};
  return launch_fused(P, (cudaStream_t)stream);
}

int er_gated_linear(const er_bf16* x, int32_t ldx, int32_t T, const er_bf16* w_gate,
                    const er_bf16* w_up, int32_t F, int32_t K, int32_t act, void* y,
                    int32_t y_fp32, int32_t ldy, int32_t* dev_error, er_stream_t stream) {
  if (!sizes_ok(T, F, K, ldx, act, y_fp32, ldy)) return ER_EINVAL;
  if (T == 0) return ER_OK;
  if (!x || !w_gate || !w_up || !y || !aligned16(x) || !aligned16(w_gate) || !aligned16(w_up) ||
      ((uintptr_t)y & (y_fp32 ? 3u : 1u)))
    return ER_EINVAL;
  FusedParams P{x, w_gate, w_up, nullptr, nullptr, y, T, F, K, ldx, 0, ldy, act, y_fp32};
  return launch_fused(P, (cudaStream_t)stream);
}

}  // extern "C"
