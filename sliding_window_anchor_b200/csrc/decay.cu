// decay.cu — linear attention with a decay for each head, for the recurrent
// layers that stand between the SWA∥RMA layers of the model (EdgeRock-4B 开源：72 MiB
// 固定 KV, §架构：递归、局部窗口与记忆锚点三件套: recurrent layers hold a matrix
// of fixed size for each head, whatever the stream's length).
//
//   S_t = e^{g_t} S_{t-1} + k_t v_tᵀ,   o_t = scale · S_tᵀ q_t
//
// per value head, S FP32 [k_dim][v_dim]; value head h reads the q and k of head
// h / (v_heads / k_heads).
#include "common.cuh"

namespace er {
namespace {

struct DecayParams {
  float* state;
  int s_max;
  const int32_t* seq_ids;
  const int32_t* cu;  // [B + 1], or NULL: sequence b is row b
  int B, T;
  int HK, HV, DK, DV;
  const uint16_t *q, *k, *v;
  int64_t ldq, ldk, ldv, ldg, ldo;
  const float* g;
  float scale;
  uint16_t* o;
  int32_t* err;
};

// The rows [begin, end) of sequence b; false when its state row or its rows
// are out of range, or an earlier sequence of the call has the same state row.
// Every thread of the block calls it.
__device__ __forceinline__ bool sequence_rows(const DecayParams& P, int b, int& row, int& begin,
                                              int& end) {
  row = P.seq_ids[b];
  begin = P.cu ? P.cu[b] : b;
  end = P.cu ? P.cu[b + 1] : b + 1;
  int same = 0;
  for (int j = threadIdx.x; j < b; j += blockDim.x) same |= P.seq_ids[j] == row;
  same = __syncthreads_or(same);
  if (same || row < 0 || row >= P.s_max || begin < 0 || end < begin || end > P.T) {
    if (threadIdx.x == 0) set_dev_error(P.err, ER_EINVAL);
    return false;
  }
  return true;
}

// One block per (32 columns of a value head's state, sequence), token by token;
// thread (r, c) holds rows r, r + 4, ... of column c.
template <int DK>
__global__ void __launch_bounds__(128) k_decay_tokens(const DecayParams P) {
  __shared__ float qs[DK], ks[DK], part[4][32];
  const int b = blockIdx.y, slices = P.DV / 32;
  const int h = blockIdx.x / slices, c0 = 32 * (blockIdx.x % slices);
  const int hk = h / (P.HV / P.HK);
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  int row, begin, end;
  if (!sequence_rows(P, b, row, begin, end)) return;
  float* S = P.state + (((size_t)row * P.HV + h) * DK) * P.DV + c0 + c;
  float s[DK / 4];
  for (int i = 0; i < DK / 4; ++i) s[i] = S[(size_t)(r + 4 * i) * P.DV];
  for (int t = begin; t < end; ++t) {
    for (int i = threadIdx.x; i < DK; i += 128) {
      qs[i] = bf1(P.q[t * P.ldq + hk * DK + i]);
      ks[i] = bf1(P.k[t * P.ldk + hk * DK + i]);
    }
    const float a = expf(P.g[t * P.ldg + h]);
    const float v = bf1(P.v[t * P.ldv + h * P.DV + c0 + c]);
    __syncthreads();
    float o = 0.f;
    for (int i = 0; i < DK / 4; ++i) {
      s[i] = fmaf(s[i], a, ks[r + 4 * i] * v);
      o = fmaf(qs[r + 4 * i], s[i], o);
    }
    part[r][c] = o;
    __syncthreads();
    if (r == 0)
      P.o[t * P.ldo + h * P.DV + c0 + c] =
          f2bf(P.scale * (part[0][c] + part[1][c] + part[2][c] + part[3][c]));
  }
  for (int i = 0; i < DK / 4; ++i) S[(size_t)(r + 4 * i) * P.DV] = s[i];
}

int launch_tokens(const DecayParams& P, cudaStream_t st) {
  const dim3 grid(P.HV * P.DV / 32, P.B);
  if (P.DK == 64)
    k_decay_tokens<64><<<grid, 128, 0, st>>>(P);
  else
    k_decay_tokens<128><<<grid, 128, 0, st>>>(P);
  count_launches(1);
  return launch_status();
}

bool shape_ok(const er_decay_shape* sh) {
  return sh && sh->k_heads >= 1 && sh->v_heads >= sh->k_heads && sh->v_heads <= 4096 &&
         sh->v_heads % sh->k_heads == 0 && (sh->k_dim == 64 || sh->k_dim == 128) &&
         (sh->v_dim == 64 || sh->v_dim == 128);
}

// The checks both calls share; fills P.
int fill(DecayParams& P, float* state, int32_t s_max, const int32_t* seq_ids, const int32_t* cu,
         int32_t B, int32_t T, const er_decay_shape* sh, const er_bf16* q, int32_t ldq,
         const er_bf16* k, int32_t ldk, const er_bf16* v, int32_t ldv, const float* g, int32_t ldg,
         float scale, er_bf16* o, int32_t ldo, int32_t* dev_error) {
  if (!shape_ok(sh) || s_max < 1 || B < 0 || B > 65535 || T < 0) return ER_EINVAL;
  const int qk = sh->k_heads * sh->k_dim, vo = sh->v_heads * sh->v_dim;
  if (ldq < qk || ldk < qk || ldv < vo || ldo < vo || ldq % 8 || ldk % 8 || ldv % 8 || ldo % 8 ||
      (ldg != 0 && ldg < sh->v_heads))
    return ER_EINVAL;
  if (B > s_max) return ER_ECAPACITY;
  if (B == 0) return ER_OK;
  if (!state || !seq_ids || !aligned16(state) || ((uintptr_t)seq_ids & 3u)) return ER_EINVAL;
  if (T > 0 && (!q || !k || !v || !g || !o || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
                !aligned16(o) || ((uintptr_t)g & 3u)))
    return ER_EINVAL;
  P = DecayParams{state, s_max, seq_ids, cu, B, T, sh->k_heads, sh->v_heads, sh->k_dim, sh->v_dim,
                  q, k, v, ldq, ldk, ldv, ldg, ldo, g, scale, o, dev_error};
  return ER_OK;
}

int error_word(DecayParams& P) {
  if (!P.err) P.err = call_error_word();
  return P.err ? ER_OK : ER_ECUDA;
}

}  // namespace
}  // namespace er

using namespace er;

extern "C" {

size_t er_decay_prefill_workspace_bytes(const er_decay_shape* shape, int32_t B, int32_t T) {
  if (!shape_ok(shape) || B < 1 || B > 65535 || T < 0) return 0;
  return 256;
}

int er_decay_decode(float* state, int32_t s_max, const int32_t* seq_ids, int32_t B,
                    const er_decay_shape* shape, const er_bf16* q, int32_t ldq, const er_bf16* k,
                    int32_t ldk, const er_bf16* v, int32_t ldv, const float* log_decay,
                    int32_t ldg, float scale, er_bf16* o, int32_t ldo, int32_t* dev_error,
                    er_stream_t stream) {
  DecayParams P;
  int rc = fill(P, state, s_max, seq_ids, nullptr, B, B, shape, q, ldq, k, ldk, v, ldv,
                      log_decay, ldg, scale, o, ldo, dev_error);
  if (rc != ER_OK || B == 0) return rc;
  if ((rc = error_word(P)) != ER_OK) return rc;
  return launch_tokens(P, (cudaStream_t)stream);
}

int er_decay_prefill(float* state, int32_t s_max, const int32_t* seq_ids,
                     const int32_t* cu_tokens, int32_t B, int32_t T, const er_decay_shape* shape,
                     const er_bf16* q, int32_t ldq, const er_bf16* k, int32_t ldk,
                     const er_bf16* v, int32_t ldv, const float* log_decay, int32_t ldg,
                     float scale, er_bf16* o, int32_t ldo, void* ws, size_t ws_bytes,
                     int32_t* dev_error, er_stream_t stream) {
  DecayParams P;
  int rc = fill(P, state, s_max, seq_ids, cu_tokens, B, T, shape, q, ldq, k, ldk, v, ldv,
                      log_decay, ldg, scale, o, ldo, dev_error);
  if (rc != ER_OK || B == 0 || T == 0) return rc;
  if (!cu_tokens || ((uintptr_t)cu_tokens & 3u) || !ws || ((uintptr_t)ws & 255u))
    return ER_EINVAL;
  if (ws_bytes < er_decay_prefill_workspace_bytes(shape, B, T)) return ER_ECAPACITY;
  if ((rc = error_word(P)) != ER_OK) return rc;
  return launch_tokens(P, (cudaStream_t)stream);
}

}  // extern "C"
