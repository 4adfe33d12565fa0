// decay.cu — linear attention with a decay for each head: a recurrent layer whose state
// is a matrix of fixed size for each head, whatever the stream's length.
//
//   S_t = e^{g_t} S_{t-1} + k_t v_tᵀ,   o_t = scale · S_tᵀ q_t
//
// per value head, S FP32 [k_dim][v_dim]; value head h reads the q and k of head
// h / (v_heads / k_heads).
//
// A general operator for hybrid stacks.  The recurrent layers of the model whose SWA∥RMA
// layers this library runs (EdgeRock-4B 开源：72 MiB 固定 KV, §架构：递归、局部窗口与
// 记忆锚点三件套) hold such a state, too, but update it by the delta rule
// (S ← (I - b k kᵀ) a S + b k vᵀ), which is not here.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "rounds.cuh"
#include "tc.cuh"

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
  // prompts: sequences of `few` tokens and fewer are k_decay_few's, the segments of L tokens of
  // longer ones k_decay_chunks'; *items: these segments' number at most (NULL: not known)
  int few, L;
  int32_t* items;
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

// ------------------------------------------------------------ single tokens
// One block per (sequence, value head, COLS columns of its state): the state streams
// through registers once, 16 bytes a thread and row; every thread's rows are
// requested before the first is used.  o's sums over the rows are joined in a fixed
// order.  HBM bounds it: 512 sequences of 32 heads of 128 x 128 take 344 us (2.2 GB read
// and written: 6.3 TB/s, 0.97 of a plain copy).
constexpr int DD_THREADS = 256;

template <int DK, int COLS>
__global__ void __launch_bounds__(DD_THREADS) k_decay_decode(const DecayParams P) {
  constexpr int LN = COLS / 4;         // threads of a row
  constexpr int RP = DD_THREADS / LN;  // rows of a pass
  constexpr int N = DK / RP;           // rows of a thread
  static_assert(N >= 1, "");
  __shared__ float qs[DK], ks[DK];
  __shared__ float4 part[DD_THREADS / 32][LN];
  grid_dep_wait();
  grid_dep_trigger();
  const int slices = P.DV / COLS;
  const int unit = blockIdx.x / slices, c0 = COLS * (blockIdx.x % slices);
  const int b = unit / P.HV, h = unit % P.HV, hk = h / (P.HV / P.HK);
  const int c = threadIdx.x % LN, r = threadIdx.x / LN;
  for (int i = threadIdx.x; i < DK; i += DD_THREADS) {
    qs[i] = bf1(P.q[b * P.ldq + hk * DK + i]);
    ks[i] = bf1(P.k[b * P.ldk + hk * DK + i]);
  }
  int row, begin, end;
  if (!sequence_rows(P, b, row, begin, end)) return;  // holds the block's barrier
  float* S = P.state + (((size_t)row * P.HV + h) * DK + r) * P.DV + c0 + 4 * c;
  float4 s[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    s[i] = *reinterpret_cast<const float4*>(S + (size_t)(RP * i) * P.DV);
  const float a = expf(P.g[b * P.ldg + h]);
  const uint2 vw = *reinterpret_cast<const uint2*>(P.v + b * P.ldv + h * P.DV + c0 + 4 * c);
  const float4 v = make_float4(bf_lo(vw.x), bf_hi(vw.x), bf_lo(vw.y), bf_hi(vw.y));
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float k = ks[r + RP * i], q = qs[r + RP * i];
    s[i].x = fmaf(s[i].x, a, k * v.x), o.x = fmaf(q, s[i].x, o.x);
    s[i].y = fmaf(s[i].y, a, k * v.y), o.y = fmaf(q, s[i].y, o.y);
    s[i].z = fmaf(s[i].z, a, k * v.z), o.z = fmaf(q, s[i].z, o.z);
    s[i].w = fmaf(s[i].w, a, k * v.w), o.w = fmaf(q, s[i].w, o.w);
    *reinterpret_cast<float4*>(S + (size_t)(RP * i) * P.DV) = s[i];
  }
#pragma unroll
  for (int m = LN; m < 32; m <<= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, m), o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, m), o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
  }
  if ((threadIdx.x & 31) < LN) part[threadIdx.x >> 5][threadIdx.x & 31] = o;
  __syncthreads();
  if (threadIdx.x < LN) {
    o = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < DD_THREADS / 32; ++w) {
      const float4 x = part[w][threadIdx.x];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
    }
    *reinterpret_cast<uint2*>(P.o + b * P.ldo + h * P.DV + c0 + 4 * threadIdx.x) =
        make_uint2(pack2_bf(P.scale * o.x, P.scale * o.y), pack2_bf(P.scale * o.z, P.scale * o.w));
  }
}

int launch_pdl(void (*fn)(const DecayParams), int blocks, int threads, const DecayParams& P,
               cudaStream_t st) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, P) != cudaSuccess) return ER_ECUDA;
  count_launches(1);
  return launch_status();
}

int launch_decode(const DecayParams& P, cudaStream_t st) {
  // whole rows of the state where they give every SM two blocks, else narrower ones
  const int units = P.B * P.HV;
  const bool wide = units >= 2 * num_sms();
  const int cols = wide ? P.DV : 32;
  const int blocks = units * (P.DV / cols);
  if (P.DK == 64)
    return launch_pdl(cols == 128  ? k_decay_decode<64, 128>
                      : cols == 64 ? k_decay_decode<64, 64>
                                   : k_decay_decode<64, 32>,
                      blocks, DD_THREADS, P, st);
  return launch_pdl(cols == 128  ? k_decay_decode<128, 128>
                    : cols == 64 ? k_decay_decode<128, 64>
                                 : k_decay_decode<128, 32>,
                    blocks, DD_THREADS, P, st);
}

// ------------------------------------------------------------ short sequences
// As for single tokens, with a loop over the sequence's tokens while the state is in registers:
// the state is read and written once, whatever their number.  A thread's rows follow one
// another; k and q of four tokens are in shared memory as pairs of equal values, for
// products on pairs of columns (fma.f32x2), while the next four tokens' rows are on their
// way.  HBM bounds it for single tokens (512 sequences, 32 heads of 128 x 128: 350 us), then
// more and more the tokens' own time, one after another in the two blocks that an SM holds:
// 512 of 4 take 490-510 us, of 16 1000.  Eight columns a thread, with half of the fetches from
// shared memory, took longer (550 and 1130 us).
constexpr int DF_TOKENS = 4;  // between two barriers

using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair_of(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 halves(f32x2 d) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from)
                 : "memory");
}

template <int DK, int COLS>
__global__ void __launch_bounds__(DD_THREADS, 2) k_decay_few(const DecayParams P) {
  constexpr int LN = COLS / 4;         // threads of a row
  constexpr int RP = DD_THREADS / LN;  // threads of a column
  constexpr int N = DK / RP;           // rows of a thread
  constexpr int WARPS = DD_THREADS / 32;
  static_assert(N >= 2 && N % 2 == 0, "");
  __shared__ __align__(16) f32x2 qs[DF_TOKENS][DK], ks[DF_TOKENS][DK];
  __shared__ __align__(16) uint16_t raw[2][DF_TOKENS][2 * DK + COLS];  // q, k and v
  __shared__ float log_decay[2][DF_TOKENS];
  __shared__ float4 part[DF_TOKENS][WARPS][LN];
  grid_dep_wait();
  grid_dep_trigger();
  const int slices = P.DV / COLS;
  const int unit = blockIdx.x / slices, c0 = COLS * (blockIdx.x % slices);
  const int b = unit / P.HV, h = unit % P.HV, hk = h / (P.HV / P.HK);
  const int c = threadIdx.x % LN, r = threadIdx.x / LN;
  int row, begin, end;
  if (blockIdx.x == 0 && P.items) {
    // for the launch behind this one, most of whose blocks may have nothing to do
    __shared__ unsigned long long items;
    if (threadIdx.x == 0) items = 0;
    __syncthreads();
    unsigned long long mine = 0;
    for (int j = threadIdx.x; j < P.B; j += DD_THREADS) {
      begin = P.cu[j], end = P.cu[j + 1];
      if (begin >= 0 && end <= P.T && end - begin > P.few) mine += (end - begin + P.L - 1) / P.L;
    }
    if (mine) atomicAdd(&items, mine);
    __syncthreads();
    if (threadIdx.x == 0) *P.items = (int)min(items, 0x7FFFFFFFull);
  }
  if (!sequence_rows(P, b, row, begin, end)) return;  // holds the block's barrier
  if (begin == end || end - begin > P.few) return;
  auto fetch = [&](int t0, int to) {
    constexpr int QU = DK / 8, UNITS = 2 * QU + COLS / 8;  // of 16 bytes
    const int m = min(DF_TOKENS, end - t0);
    for (int i = threadIdx.x; i < m * UNITS; i += DD_THREADS) {
      const int u = i / UNITS, x = i % UNITS, t = t0 + u;
      const uint16_t* from = x < QU       ? P.q + t * P.ldq + hk * DK + 8 * x
                             : x < 2 * QU ? P.k + t * P.ldk + hk * DK + 8 * (x - QU)
                                          : P.v + t * P.ldv + h * P.DV + c0 + 8 * (x - 2 * QU);
      copy_async<16>(&raw[to][u][8 * x], from);
    }
    if (threadIdx.x < m)
      copy_async<4>(&log_decay[to][threadIdx.x], P.g + (t0 + (int)threadIdx.x) * P.ldg + h);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(begin, 0);
  float* S = P.state + (((size_t)row * P.HV + h) * DK + N * r) * P.DV + c0 + 4 * c;
  f32x2 s[N][2];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(S + (size_t)i * P.DV);
    s[i][0] = x.x, s[i][1] = x.y;
  }
  int at = 0;
#pragma unroll 1
  for (int t0 = begin; t0 < end; t0 += DF_TOKENS, at ^= 1) {
    const int m = min(DF_TOKENS, end - t0);
    if (t0 + DF_TOKENS < end) {
      fetch(t0 + DF_TOKENS, at ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    for (int i = threadIdx.x; i < m * DK; i += DD_THREADS) {
      const int u = i / DK, x = i % DK;
      const float q = bf1(raw[at][u][x]), k = bf1(raw[at][u][DK + x]);
      qs[u][x] = pair_of(q, q);
      ks[u][x] = pair_of(k, k);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < DF_TOKENS; ++u) {
      if (u >= m) break;
      const uint2 vw = *reinterpret_cast<const uint2*>(&raw[at][u][2 * DK + 4 * c]);
      const f32x2 v0 = pair_of(bf_lo(vw.x), bf_hi(vw.x)), v1 = pair_of(bf_lo(vw.y), bf_hi(vw.y));
      const float e = expf(log_decay[at][u]);
      const f32x2 a = pair_of(e, e);
      f32x2 o0 = 0, o1 = 0;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&ks[u][N * r + i]);
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&qs[u][N * r + i]);
        s[i][0] = fma2(s[i][0], a, mul2(k.x, v0)), o0 = fma2(q.x, s[i][0], o0);
        s[i][1] = fma2(s[i][1], a, mul2(k.x, v1)), o1 = fma2(q.x, s[i][1], o1);
        s[i + 1][0] = fma2(s[i + 1][0], a, mul2(k.y, v0)), o0 = fma2(q.y, s[i + 1][0], o0);
        s[i + 1][1] = fma2(s[i + 1][1], a, mul2(k.y, v1)), o1 = fma2(q.y, s[i + 1][1], o1);
      }
      const float2 lo = halves(o0), hi = halves(o1);
      float4 o = make_float4(lo.x, lo.y, hi.x, hi.y);
#pragma unroll
      for (int x = LN; x < 32; x <<= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, x), o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, x), o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
      }
      if ((threadIdx.x & 31) < LN) part[u][threadIdx.x >> 5][threadIdx.x & 31] = o;
    }
    __syncthreads();
    if (threadIdx.x < m * LN) {
      const int u = threadIdx.x / LN, x = threadIdx.x % LN;
      float4 o = part[u][0][x];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) {
        const float4 y = part[u][w][x];
        o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
      }
      *reinterpret_cast<uint2*>(P.o + (t0 + u) * P.ldo + h * P.DV + c0 + 4 * x) = make_uint2(
          pack2_bf(P.scale * o.x, P.scale * o.y), pack2_bf(P.scale * o.z, P.scale * o.w));
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    *reinterpret_cast<ulonglong2*>(S + (size_t)i * P.DV) = make_ulonglong2(s[i][0], s[i][1]);
}

int launch_few(const DecayParams& P, cudaStream_t st) {
  // as for single tokens
  const int units = P.B * P.HV;
  const int cols = units >= 2 * num_sms() ? P.DV : 32;
  const int blocks = units * (P.DV / cols);
  if (P.DK == 64)
    return launch_pdl(cols == 128  ? k_decay_few<64, 128>
                      : cols == 64 ? k_decay_few<64, 64>
                                   : k_decay_few<64, 32>,
                      blocks, DD_THREADS, P, st);
  return launch_pdl(cols == 128  ? k_decay_few<128, 128>
                    : cols == 64 ? k_decay_few<128, 64>
                                 : k_decay_few<128, 32>,
                    blocks, DD_THREADS, P, st);
}

// ------------------------------------------------------------ prompts
// A sequence is walked in chunks of 128 tokens.  With G_i the sum of the log-decays of
// a chunk's tokens 0..i and S the state in front of it:
//   o_i = scale · (e^{G_i} Sᵀ q_i + Σ_{j<=i} (q_i·k_j) e^{G_i - G_j} v_j)
//   S  <- e^{G_127} S + Σ_j k_j (e^{G_127 - G_j} v_j)ᵀ
// as four tensor-core products (tcgen05): Q Kᵀ (masked and decayed in registers, back
// into TMEM as BF16), that times V, Q S (S as BF16), Kᵀ Ṽ.  What is rounded:
//  - the state's operand Ṽ goes in as three BF16 terms, which hold its FP32 values to
//    2^-24; with one or two an error of 2^-8 or 2^-16 would be carried to every later token.
//    The sums stay in FP32 in TMEM, where the chunk's decay is applied to them; what comes with
//    the additions inside the tensor cores leaves the state of long prompts 2e-6 to
//    4e-6 off.
//  - of o's terms each meets one rounding to BF16 (2^-8), like its result: the masked
//    products as the operand of V's, the state as that of Q's.  Two terms of each would
//    need twice the products and the TMEM columns that the state's terms take.
//  - G is summed in FP64.  An exponent goes to FP32: of a decay x since a token 2^-24 of x;
//    of the masked products, as a sum of two through a row of the same 32, 2^-24 of the
//    decay over up to 31 tokens each: with log-decays of 0 to -150 2^-11 at most (2^-11.5 of the
//    factor), with growth 2^-23 of what 31 tokens grow by.
//
// A CTA walks 64 columns of one value head through one segment of a sequence.
// Long sequences are cut into segments of L tokens that are walked at the same time:
// a first launch (STATES) finds what each segment's own tokens leave behind, a second one
// what the segments in front of each leave together, which its walk starts from.  There a
// segment's chunks are walked from its end, so that all decays are known and no
// product waits for another.
//
// What bounds it: 32768 tokens of 32 heads of 128 x 128 (16 of q and k) take 483-530 us (by the card
// and its power limit), of these STATES 0.31, the join 0.02 and the walk 0.67.  A walk's chunk takes about 4800 cycles: two
// chains (Q Kᵀ - decayed - times V, and the state out of TMEM - Q S - Kᵀ Ṽ) that meet in
// every chunk, each a row of waits of some hundred cycles, over 400 KB of shared-memory
// traffic (3100 cycles); a chunk of STATES takes 2040, as long as its decays' sums, its
// terms and its loads each take for themselves.
// The tensor cores are busy 16-25%.  Chunks of 64 tokens would have the same waits for half of
// the tokens; slices of 128 columns have no room beside two chunks of k and v in shared
// memory and three terms of the state in TMEM.
//
// Warps, by the TMEM lanes (32 · (warp % 4)..) that they can reach and by warp / 4: below
// warp / 4 = 4 one for each block of 32 x 32 of Q Kᵀ on and below the diagonal (lanes
// of block row r: r + 1 of them), the rest of these for TMA, the products and the
// decays; 4 and 5 — Ṽ and o; 6 — the state.  Non-finite values of v are kept out of the products of the
// tokens in front of them: they enter V as zero, the state as NaN, and o's column is
// NaN from that token on.
constexpr int CH = 128;
constexpr int DC_THREADS = 896;
constexpr int DC_TMA = 4, DC_MMA = 8, DC_GATES = 12;  // warps that have no block
constexpr uint64_t kDrainNs = 200000;

struct ChunkParams {
  CUtensorMap q_map, k_map, v_map;  // rows of [T][heads · dim], boxes 64 x 128
  CUtensorMap o_map;                // the same, boxes 32 x 32
  DecayParams d;
  float* W;     // [slots][HV][DK][DV] what a segment leaves, for sequences of two and more
  double* Wg;   // [slots][HV] a segment's log2 decay
};

struct alignas(16) Gates {
  float w[CH];  // e^{G_127 - G_j}; 0 behind the sequence
  float e[CH];  // |scale| · e^{G_i}
  // |scale| · e^{G_i - G_j} is 2^(row[i] + col[..][j]), through the first row r of i's
  // block of 32: log2 of |scale| · e^{G_i - G_r}, and for every block row log2 of
  // e^{G_r - G_j} for the columns up to its end
  float row[CH], col[32 * (1 + 2 + 3 + 4)];
  float tot;
};
__device__ __forceinline__ constexpr int col_at(int block) { return 16 * block * (block + 1); }

struct Item {
  int found, row, b, seg, nseg, slot, t0, t1;
};

// Segment `index` of the sequences that have LEAST segments and more (LEAST 3: the first one
// of sequence `index` of these), by one warp; reports bad rows.
template <int LEAST>
__device__ __forceinline__ void find_item(const DecayParams& P, int index, Item* out) {
  const int lane = threadIdx.x & 31;
  int acc = 0, slots = 0;
  long long tokens = 0;
  Item it{};
  int next[3];
  auto fetch = [&](int b) {
    next[0] = b < P.B ? P.cu[b] : 0;
    next[1] = b < P.B ? P.cu[b + 1] : 0;
    next[2] = b < P.B ? P.seq_ids[b] : 0;
  };
  fetch(lane);
#pragma unroll 1
  for (int b0 = 0; b0 < P.B; b0 += 32) {
    const int b = b0 + lane, begin = next[0], row = next[2];
    int end = next[1];
    fetch(b + 32);
    if (begin < 0 || end < begin || end > P.T || row < 0 || row >= P.s_max) {
      set_dev_error(P.err, ER_EINVAL);
      end = begin;
    }
    // together they have T tokens at most: the segments that the grid and the workspace
    // have room for
    long long len = tokens + (end - begin);
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, len, m);
      if (lane >= m) len += x - tokens;
    }
    tokens = __shfl_sync(0xffffffffu, len, 31);
    int segs = 0;
    if (len <= P.T)
      segs = end - begin > P.few ? (end - begin + P.L - 1) / P.L : 0;
    else if (end > begin)
      set_dev_error(P.err, ER_EINVAL);
    const int n = segs < LEAST ? 0 : LEAST == 3 ? 1 : segs;
    int sum = n, many = segs > 1 ? segs : 0;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, m), y = __shfl_up_sync(0xffffffffu, many, m);
      if (lane >= m) sum += x, many += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, acc + sum > index);
    if (hit) {
      const int l = __ffs(hit) - 1;
      // an earlier sequence with the same state row?
      const int same_as = __shfl_sync(0xffffffffu, row, l);
      bool same = lane < l && row == same_as;
      for (int j = lane; j < b0; j += 32) same |= P.seq_ids[j] == same_as;
      if (__any_sync(0xffffffffu, same)) {
        if (lane == 0) set_dev_error(P.err, ER_EINVAL), *out = it;
        return;
      }
      if (lane == l) {
        it.found = 1, it.row = row, it.b = b, it.nseg = segs;
        it.seg = LEAST == 3 ? 0 : index - (acc + sum - n);
        it.slot = slots + many - (segs > 1 ? segs : 0);
        it.t0 = begin + P.L * it.seg;
        it.t1 = min(end, it.t0 + P.L);
        *out = it;
      }
      return;
    }
    acc += __shfl_sync(0xffffffffu, sum, 31);
    slots += __shfl_sync(0xffffffffu, many, 31);
  }
  if (lane == 0) *out = it;
}

// Reports sequence b when it is empty, so that no block has an item of it, and its state row
// is listed before it; by one warp.
__device__ __noinline__ void check_empty(const DecayParams& P, int b) {
  if (b >= P.B || P.cu[b] != P.cu[b + 1]) return;
  const int row = P.seq_ids[b];
  bool same = false;
  for (int j = threadIdx.x & 31; j < b; j += 32) same |= P.seq_ids[j] == row;
  if (same) set_dev_error(P.err, ER_EINVAL);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x · 0 + y on two BF16 values.
__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(y));
  return d;
}

// The roles' loops run at the same time and share the SM's instruction cache: with
// everything unrolled and inlined (78 KB) they waited for instructions, so what runs
// rarely is a function, and loops stay loops where that costs little.
// The rest of a wait, bounded as mbar_wait: the hardware may hold the thread for the
// hinted time, so that a waiting warp issues little.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int32_t* err) {
  constexpr uint32_t kHintNs = 20000;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kHintNs)
        : "memory");
    if (ok) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      set_dev_error(err, ER_ETIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, int phase, int32_t* err) {
  return mbar_try_wait(bar, (uint32_t)phase & 1u) || wait_slow(bar, (uint32_t)phase & 1u, err);
}

// A row's infinite and NaN values among 32 columns of v: zero in v, NaN in the
// first term of Ṽ, and noted by column.
__device__ __noinline__ void mark_row(unsigned char* v, unsigned char* terms, int sw, int half,
                                      int j, int* colbad, int* anybad) {
#pragma unroll 1
  for (int x = 4 * half; x < 4 * half + 4; ++x)
#pragma unroll 1
    for (int m = 0; m < 8; ++m) {
      uint16_t* at = reinterpret_cast<uint16_t*>(v + 16 * (x ^ sw)) + m;
      if ((*at & 0x7F80u) != 0x7F80u) continue;
      *at = 0;
      reinterpret_cast<uint16_t*>(terms + 16 * (x ^ sw))[m] = 0x7FFF;
      atomicMin(&colbad[8 * x + m], j);
      *anybad = 1;
    }
}

template <int DK, bool STATES>
__global__ void __launch_bounds__(DC_THREADS, 1)
    k_decay_chunks(const __grid_constant__ ChunkParams P) {
  constexpr int QB = DK * 256;  // bytes of a chunk's q (or k) rows: 64-column blocks of 16 KB
  constexpr int VB = 16384;
  constexpr int RV = STATES ? 3 : 2;    // chunks of v in flight (of k two)
  constexpr int NV = STATES ? 2 : 1;    // buffers of Ṽ
  // TMEM columns: Q Kᵀ, and that masked, as BF16, in the first 16 columns of each 32; the
  // state's sums, one for each term of Ṽ; the masked products times V; Q S, twice
  constexpr uint32_t T_P = 0, T_S = 128, T_O = 320, T_OS = 384;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* vb = base + 2 * QB;
  unsigned char* vt = vb + RV * VB;         // Ṽ: three terms
  unsigned char* qb = vt + 3 * NV * VB;     // q
  unsigned char* sb = qb + (STATES ? 0 : QB);  // S in BF16, [DK][64]
  unsigned char* ob = sb + (STATES ? 0 : DK * 128);  // o on its way out
  struct Shared {
    Gates gate[2];
    int colbad[4][64];  // first token of a chunk with a non-finite v, by column
    int anybad[4];
    uint64_t k_full[2], k_empty[2], v_full[3], v_empty[3], gate_full[2], gate_empty[2];
    uint64_t vt_empty[2], last;  // STATES
    // one for each buffer of Ṽ: with one for both, a warp that is a chunk ahead would count
    // for one that is not there yet
    uint64_t vt_full[2];
    uint64_t o_full, o_empty[2], q_full, q_empty, p_full, pt_full, s_full, sb_full, done;
    double g_total;
    Item item;
    uint32_t tmem_base;
    volatile int failed;
  };
  Shared& B = *reinterpret_cast<Shared*>(ob + (STATES ? 0 : 16384));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const DecayParams& D = P.d;
  const int slices = D.DV / 64, per = D.HV * slices;
  const int h = blockIdx.x % per / slices, c0 = 64 * (blockIdx.x % slices);
  const int hk = h / (D.HV / D.HK);

  if (threadIdx.x == 64) {
    // launch arguments: no earlier kernel writes them
    tc::prefetch_map(&P.k_map);
    tc::prefetch_map(&P.v_map);
    if (!STATES) tc::prefetch_map(&P.q_map);
  }
  grid_dep_wait();
  grid_dep_trigger();
  if (D.items && (int)(blockIdx.x / per) >= *D.items) return;
  if (warp == 0) find_item<STATES ? 2 : 1>(D, blockIdx.x / per, &B.item);
  // where k_decay_few ran it has looked at every sequence; else there are B blocks at least
  if (!STATES && warp == 2 && !D.items && blockIdx.x % per == 0) check_empty(D, blockIdx.x / per);
  if (threadIdx.x == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.k_full[i], 1);
      mbar_init(&B.k_empty[i], 1);
      mbar_init(&B.gate_full[i], 1);
      mbar_init(&B.gate_empty[i], STATES ? 8 : 22);
      mbar_init(&B.vt_empty[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&B.v_full[i], 1);
      mbar_init(&B.v_empty[i], STATES ? 8 : 1);
    }
    mbar_init(&B.last, 1);
    mbar_init(&B.o_full, 1);
    mbar_init(&B.o_empty[0], 8);
    mbar_init(&B.o_empty[1], 8);
    mbar_init(&B.q_full, 1);
    mbar_init(&B.q_empty, 1);
    mbar_init(&B.p_full, 1);
    mbar_init(&B.pt_full, 10);
    mbar_init(&B.vt_full[0], 8);
    mbar_init(&B.vt_full[1], 8);
    mbar_init(&B.s_full, 1);
    mbar_init(&B.sb_full, 4);
    mbar_init(&B.done, 1);
    B.failed = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const Item it = B.item;
  if (!it.found) return;
  const size_t plane = (size_t)DK * D.DV;
  float* W0 = P.W + ((size_t)it.slot * D.HV + h) * plane;
  if (STATES && it.seg == it.nseg - 1) {
    // the last segment's walk writes the state's row, which the first one starts from: a
    // copy of it for that one takes the slot that no later segment needs
    const float* from = D.state + ((size_t)it.row * D.HV + h) * plane + c0;
    float* to = W0 + (size_t)it.seg * D.HV * plane + c0;
    for (int i = threadIdx.x; i < DK * 16; i += DC_THREADS) {
      const size_t at = (size_t)(i / 16) * D.DV + 4 * (i % 16);
      *reinterpret_cast<float4*>(to + at) = *reinterpret_cast<const float4*>(from + at);
    }
    return;
  }
  if (warp == DC_MMA) tc::tmem_alloc(&B.tmem_base, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = B.tmem_base;
  const int n = (it.t1 - it.t0 + CH - 1) / CH;

  // a wait of a whole warp: false (in every lane) when it gave up or another one did
  auto wait = [&](uint64_t* bar, int phase) {
    if (__all_sync(0xffffffffu, wait_bar(bar, phase, D.err))) return true;
    B.failed = 1;
    return false;
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp == DC_TMA) {
    // ------------------------------------------------------------- TMA
    if (tc::elect_one()) {
      bool ok = true;
      int vs = 0, vp = 1;  // v's slot and phase
      auto first_row = [&](int c) { return it.t0 + CH * (STATES ? n - 1 - c : c); };
      auto load_v = [&](int c) {
        ok = wait_bar(&B.v_empty[vs], vp, D.err);
        if (!ok) return;
        mbar_arrive_expect_tx(&B.v_full[vs], VB);
        tc::tma_load_2d(vb + vs * VB, &P.v_map, D.DV * h + c0, first_row(c), &B.v_full[vs]);
        if (++vs == RV) vs = 0, vp ^= 1;
      };
      load_v(0);
#pragma unroll 1
      for (int c = 0; ok && c < n; ++c) {
        const int s = c & 1, t = first_row(c);
        if (STATES && c + 1 < n) load_v(c + 1);
        ok = ok && wait_bar(&B.k_empty[s], (c >> 1) + 1, D.err);
        if (!ok) break;
        mbar_arrive_expect_tx(&B.k_full[s], QB);
#pragma unroll
        for (int x = 0; x < DK / 64; ++x)
          tc::tma_load_2d(base + s * QB + 16384 * x, &P.k_map, DK * hk + 64 * x, t, &B.k_full[s]);
        if (STATES) continue;
        ok = wait_bar(&B.q_empty, c + 1, D.err);
        if (!ok) break;
        mbar_arrive_expect_tx(&B.q_full, QB);
#pragma unroll
        for (int x = 0; x < DK / 64; ++x)
          tc::tma_load_2d(qb + 16384 * x, &P.q_map, DK * hk + 64 * x, t, &B.q_full);
        if (c + 1 < n) load_v(c + 1);
      }
      if (!ok) B.failed = 1;
    }
    __syncwarp();
  } else if (warp == DC_MMA) {
    // -------------------------------------------------------- products
    if (tc::elect_one()) {
      constexpr uint32_t id_p = tc::idesc_bf16(128, 128, false, false);
      constexpr uint32_t id_o = tc::idesc_bf16(128, 64, false, true);
      constexpr uint32_t id_s = tc::idesc_bf16(128, 192, true, true);
      // descriptors count 16-byte units: 16 of a K-major operand's K are 2 of them (64 of
      // K a block of 1024), 16 rows of an MN-major one 128
      const uint64_t k_major = tc::desc_sw128(smem_u32(base), 16, 1024);
      const uint64_t kt_desc = tc::desc_sw128(smem_u32(base), 16384, 1024);
      const uint64_t v_desc = tc::desc_sw128(smem_u32(vb), 8192, 1024);
      const uint64_t q_desc = tc::desc_sw128(smem_u32(qb), 16, 1024);
      const uint64_t s_desc = tc::desc_sw128(smem_u32(sb), 8192, 1024);
      const uint64_t vt_desc = tc::desc_sw128(smem_u32(vt), VB, 1024);
      bool ok = true;
      auto scores = [&](int c) {  // Q Kᵀ
        ok = wait_bar(&B.q_full, c, D.err) && wait_bar(&B.k_full[c & 1], c >> 1, D.err);
        if (!ok) return;
        tc::fence_after_sync();
        const uint64_t k = k_major + (c & 1) * (QB / 16);
#pragma unroll 2
        for (int kk = 0; kk < DK / 16; ++kk) {
          const int at = 1024 * (kk >> 2) + 2 * (kk & 3);
          tc::mma_bf16(tmem + T_P, q_desc + at, k + at, id_p, kk > 0);
        }
        tc::commit(&B.p_full);
      };
#pragma unroll 1
      for (int c = STATES ? 0 : -1; c < n; ++c) {
        const int s = c & 1;
        const int k_at = s * (QB / 16), v_at = s * (VB / 16);
        if (!STATES && c >= 0) {
          // Q S
          ok = wait_bar(&B.sb_full, c, D.err) && wait_bar(&B.o_empty[s], (c >> 1) + 1, D.err);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll 2
          for (int kk = 0; kk < DK / 16; ++kk)
            tc::mma_bf16(tmem + T_OS + 64 * s, q_desc + 1024 * (kk >> 2) + 2 * (kk & 3), s_desc + 128 * kk,
                         id_o, kk > 0);
          tc::commit(&B.q_empty);
        }
        if (c >= 0) {
          if (STATES) {
            ok = wait_bar(&B.k_full[s], c >> 1, D.err);
            if (!ok) break;
          }
          // S += Kᵀ Ṽ, its three terms side by side (K is read once; with k_dim 64, lanes
          // 64.. take v's rows for columns of k: never read)
          ok = wait_bar(&B.vt_full[c & (NV - 1)], c / NV, D.err);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t terms = vt_desc + (c & (NV - 1)) * (3 * VB / 16);
#pragma unroll 2
          for (int kk = 0; kk < CH / 16; ++kk)
            tc::mma_bf16(tmem + T_S, kt_desc + k_at + 128 * kk, terms + 128 * kk, id_s,
                         !STATES || c > 0 || kk > 0);
          if (STATES) {
            tc::commit(&B.vt_empty[s]);
            tc::commit(&B.k_empty[s]);
            continue;
          }
          tc::commit(&B.s_full);
          tc::commit(&B.k_empty[s]);  // Q Kᵀ is done too
          // the masked products times V
          ok = wait_bar(&B.pt_full, c, D.err) &&
               (c == 0 || wait_bar(&B.o_empty[s ^ 1], (c - 1) >> 1, D.err));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll 2
          for (int kk = 0; kk < CH / 16; ++kk)
            tc::mma_bf16_a_tmem(tmem + T_O, tmem + T_P + 32 * (kk >> 1) + 8 * (kk & 1),
                                v_desc + v_at + 128 * kk, id_o, kk > 0);
          tc::commit(&B.o_full);
          tc::commit(&B.v_empty[s]);
        }
        if (c + 1 < n) {
          scores(c + 1);
          if (!ok) break;
        }
      }
      if (!ok) B.failed = 1;
      if (STATES) tc::commit(&B.last);
      tc::commit(&B.done);
      wait_bar(&B.done, 0, D.err);  // nothing is on the tensor cores at exit
    }
    __syncwarp();
  } else if (warp == DC_GATES) {
    // ---------------------------------------------------------- decays
    constexpr double kLog2e = 1.4426950408889634;
    const float log_scale = log2f(fabsf(D.scale));
    double R = 0.0;  // STATES: the decay behind the chunk
    // the next chunk's log-decays are on their way while this one's are summed
    float next[4];
    auto fetch = [&](int c) {
      const int t = it.t0 + CH * (STATES ? n - 1 - c : c) + 4 * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) next[i] = t + i < it.t1 ? D.g[(t + i) * D.ldg + h] : 0.f;
    };
    fetch(0);
#pragma unroll 1
    for (int c = 0; c < n; ++c) {
      const int t = it.t0 + CH * (STATES ? n - 1 - c : c) + 4 * lane;
      float now[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) now[i] = next[i];
      if (c + 1 < n) fetch(c + 1);
      double G[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float g = now[i];
        if (g < -150.f) g = -150.f;  // e^-150 is 0 in FP32, and -inf has no differences
        G[i] = (double)g * kLog2e + (i ? G[i - 1] : 0.0);
      }
      double sum = G[3];
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, sum, m);
        if (lane >= m) sum += x;
      }
      // not sum - G[3]: a NaN of the lane's later tokens would reach its earlier ones
      const double before = __shfl_up_sync(0xffffffffu, sum, 1);
      const double front = lane ? before : 0.0, total = __shfl_sync(0xffffffffu, sum, 31);
      const double first = front + G[0], own = __shfl_sync(0xffffffffu, first, lane & ~7);
      double later[4];  // G at the blocks' first rows
#pragma unroll
      for (int q = 0; q < 4; ++q) later[q] = __shfl_sync(0xffffffffu, first, 8 * q);
      if (!wait(&B.gate_empty[c & 1], ((c >> 1) & 1) ^ 1)) break;
      Gates& g = B.gate[c & 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double x = front + G[i];
        g.w[4 * lane + i] = t + i < it.t1 ? ex2((float)(R + (total - x))) : 0.f;
        if (STATES) continue;
        g.e[4 * lane + i] = fabsf(D.scale) * ex2((float)x);
        g.row[4 * lane + i] = (float)(x - own) + log_scale;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (lane < 8 * q + 8) g.col[col_at(q) + 4 * lane + i] = (float)(later[q] - x);
      }
      if (lane == 0) g.tot = ex2((float)total);
      if (STATES) {
        R += total;
        if (lane == 0) B.g_total = R;
      }
      arrive(&B.gate_full[c & 1]);
    }
    if (STATES && lane == 0 && c0 == 0) P.Wg[(size_t)(it.slot + it.seg) * D.HV + h] = R;
  } else if (warp < 16) {
    // ------------------------- a block of Q Kᵀ, decayed and masked, to BF16
    const int quad = warp & 3, cb = warp >> 2, y = 32 * cb;
    if (!STATES && cb <= quad) {
      const uint32_t lanes = (uint32_t)(32 * quad) << 16;
      const int i = 32 * quad + lane;
#pragma unroll 1
      for (int c = 0; c < n; ++c) {
        if (!wait(&B.gate_full[c & 1], c >> 1) || !wait(&B.p_full, c)) break;
        tc::fence_after_sync();
        const Gates& g = B.gate[c & 1];
        uint32_t r[32], o[16];
        tc::tmem_ld32(tmem + lanes + T_P + y, r);
        tc::tmem_wait_ld();
        const float row = g.row[i];
        const float* col = &g.col[col_at(quad) + y];
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const float4 f = *reinterpret_cast<const float4*>(col + x);
          const float p0 = __uint_as_float(r[x]) * ex2(row + f.x);
          const float p1 = __uint_as_float(r[x + 1]) * ex2(row + f.y);
          const float p2 = __uint_as_float(r[x + 2]) * ex2(row + f.z);
          const float p3 = __uint_as_float(r[x + 3]) * ex2(row + f.w);
          o[x / 2] = pack2_bf(p0, p1);
          o[x / 2 + 1] = pack2_bf(p2, p3);
        }
        if (cb == quad) {
          // a column right of the diagonal is masked, whatever it holds
#pragma unroll
          for (int m = 0; m < 16; ++m)
            o[m] &= 2 * m + 1 <= lane ? 0xFFFFFFFFu : 2 * m == lane ? 0xFFFFu : 0u;
        }
        tc::tmem_st16(tmem + lanes + T_P + y, o);
        if (cb == quad) {
          // the blocks right of the diagonal one
          const uint32_t z[16] = {};
#pragma unroll 1
          for (int x = y + 32; x < CH; x += 32) tc::tmem_st16(tmem + lanes + T_P + x, z);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        arrive(&B.pt_full);
        if (lane == 0) mbar_arrive(&B.gate_empty[c & 1]);
      }
    }
  } else if (warp < 24) {
    // ------------------------------- Ṽ, then o: 32 columns of a row a thread
    const int quad = warp & 3, half = (warp - 16) >> 2, j = 32 * quad + lane;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int tid = threadIdx.x - 32 * 16;
    const uint32_t sign = D.scale < 0.f ? 0x80008000u : 0u;
    float e = 0.f;
    int vs = 0, vp = 0;  // v's slot and phase
    const auto meet = [] { named_bar_sync(1, 256); };
    int c = 0;
#pragma unroll 1
    for (; c <= n; ++c) {
      const float e_prev = e;
      if (c < n) {
        const int s = c & 1, t = it.t0 + CH * (STATES ? n - 1 - c : c) + j;
        if (!STATES) {
          if (tid < 64) B.colbad[c & 3][tid] = CH;
          if (tid == 64) B.anybad[c & 3] = 0;
          meet();
        }
        if (!wait(&B.v_full[vs], vp) || !wait(&B.gate_full[s], c >> 1)) break;
        const float w = B.gate[s].w[j];
        if (!STATES) e = B.gate[s].e[j];
        unsigned char* v = vb + vs * VB + 128 * j;
        unsigned char* to = vt + 3 * VB * (c & (NV - 1)) + 128 * j;
        const int sw = j & 7;
        // the rows of k behind a sequence are cleared below
        if (t - lane + 32 > it.t1 && !wait(&B.k_full[s], c >> 1)) break;
        if (!(STATES ? wait(&B.vt_empty[s], (c >> 1) + 1) : c == 0 || wait(&B.s_full, c - 1)))
          break;
        uint32_t odd = 0;  // NaN (in either half) once a value of v is infinite or NaN
#pragma unroll 2
        for (int y = 0; y < 4; ++y) {
          const int at = 16 * ((4 * half + y) ^ sw);
          uint4 word = make_uint4(0, 0, 0, 0);
          if (t < it.t1) {
            word = *reinterpret_cast<const uint4*>(v + at);
          } else {
            // behind the sequence: another one's rows, or nothing
            *reinterpret_cast<uint4*>(v + at) = word;
#pragma unroll
            for (int x = 0; x < DK / 64; ++x)
              *reinterpret_cast<uint4*>(base + s * QB + 16384 * x + 128 * j + at) = word;
          }
          const uint32_t in[4] = {word.x, word.y, word.z, word.w};
          uint32_t hi[4], mid[4], lo[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            float a = bf_lo(in[m]), b = bf_hi(in[m]);
            odd = times_zero(in[m], odd);
            a *= w, b *= w;
            hi[m] = pack2_bf(a, b);
            a -= bf_lo(hi[m]), b -= bf_hi(hi[m]);
            mid[m] = pack2_bf(a, b);
            lo[m] = pack2_bf(a - bf_lo(mid[m]), b - bf_hi(mid[m]));
          }
          *reinterpret_cast<uint4*>(to + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to + VB + at) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
          *reinterpret_cast<uint4*>(to + 2 * VB + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (odd & 0x7FFF7FFFu) mark_row(v, to, sw, half, j, B.colbad[c & 3], &B.anybad[c & 3]);
        tc::fence_async_smem();
        arrive(&B.vt_full[c & (NV - 1)]);
        if (lane == 0) {
          mbar_arrive(&B.gate_empty[s]);
          if (STATES) mbar_arrive(&B.v_empty[vs]);
        }
        if (++vs == RV) vs = 0, vp ^= 1;
      }
      if (!STATES && c > 0) {
        const int cc = c - 1, t = it.t0 + CH * cc + j;
        if (c == n) meet();  // the last chunk's marks
        if (!wait(&B.o_full, cc)) break;
        tc::fence_after_sync();
        const int col = 32 * half;
        // whole blocks of 32 rows go out by TMA from a warp's own 2 KB (16-byte chunk x of
        // row l at x ^ l / 2 % 4), the last ones of a sequence by plain stores
        unsigned char* mine = ob + 2048 * (warp - 16);
        const bool whole = t - lane + 32 <= it.t1;
        uint16_t* o = D.o + t * D.ldo + h * D.DV + c0 + col;
        if (lane == 0) tc::bulk_wait_read<0>();
        __syncwarp();
#pragma unroll 1
        for (int y = 0; y < 32; y += 16) {
          uint32_t a[16], b[16];
          tc::tmem_ld16(tmem + lanes + T_OS + 64 * (cc & 1) + col + y, a);
          tc::tmem_ld16(tmem + lanes + T_O + col + y, b);
          tc::tmem_wait_ld();
          uint32_t z[8];
#pragma unroll
          for (int m = 0; m < 8; ++m)
            z[m] = sign ^ pack2_bf(fmaf(e_prev, __uint_as_float(a[2 * m]), __uint_as_float(b[2 * m])),
                                   fmaf(e_prev, __uint_as_float(a[2 * m + 1]),
                                        __uint_as_float(b[2 * m + 1])));
          const int x = y / 8;
          if (whole) {
            unsigned char* l = mine + 64 * lane;
            const int sw = (lane >> 1) & 3;
            *reinterpret_cast<uint4*>(l + 16 * (x ^ sw)) = make_uint4(z[0], z[1], z[2], z[3]);
            *reinterpret_cast<uint4*>(l + 16 * ((x + 1) ^ sw)) =
                make_uint4(z[4], z[5], z[6], z[7]);
          } else if (t < it.t1) {
            *reinterpret_cast<uint4*>(o + y) = make_uint4(z[0], z[1], z[2], z[3]);
            *reinterpret_cast<uint4*>(o + y + 8) = make_uint4(z[4], z[5], z[6], z[7]);
          }
        }
        tc::fence_before_sync();
        arrive(&B.o_empty[cc & 1]);
        if (B.anybad[cc & 3]) {
          // a column is NaN from its first marked token on
#pragma unroll 1
          for (int u = 0; u < 32; ++u)
            if (B.colbad[cc & 3][col + u] <= j) {
              if (whole)
                reinterpret_cast<uint16_t*>(mine + 64 * lane +
                                            16 * ((u / 8) ^ ((lane >> 1) & 3)))[u & 7] = 0x7FFF;
              else if (t < it.t1)
                o[u] = 0x7FFF;
            }
        }
        if (whole) {
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tc::tma_store_2d(&P.o_map, D.DV * h + c0 + col, t, mine);
            tc::bulk_commit();
          }
        }
      }
    }
    if (!STATES) meet_rest(c, n, meet);
    if (!STATES && lane == 0) tc::bulk_wait_all();
  } else {
    // ------------------------------------------------------- the state
    const int quad = warp & 3, d = 32 * quad + lane;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const bool mine = 32 * quad < DK;
    float* row = D.state + (((size_t)it.row * D.HV + h) * DK + d) * D.DV + c0;
    float* left = W0 + (size_t)d * D.DV + c0;  // what segment 0 leaves behind
    // 16 columns at a time; `x` of the functions below is their first column
    float S[16];
    auto load = [&](const float* from, float f) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 y = *reinterpret_cast<const float4*>(from + i);
        S[i] = fmaf(f, y.x, S[i]), S[i + 1] = fmaf(f, y.y, S[i + 1]);
        S[i + 2] = fmaf(f, y.z, S[i + 2]), S[i + 3] = fmaf(f, y.w, S[i + 3]);
      }
    };
    auto from_tmem = [&](int x) {
      uint32_t hi[16], mid[16], lo[16];
      tc::tmem_ld16(tmem + lanes + T_S + x, hi);
      tc::tmem_ld16(tmem + lanes + T_S + 64 + x, mid);
      tc::tmem_ld16(tmem + lanes + T_S + 128 + x, lo);
      tc::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        S[i] = __uint_as_float(hi[i]) + (__uint_as_float(mid[i]) + __uint_as_float(lo[i]));
    };
    auto store = [&](float* to) {
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(to + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
    };
    bool ok = true;
    if (!STATES && mine) {
      // the state that the walk starts from, through TMEM like every later one: the row, its
      // copy in the last segment's slot, or what the segments in front leave together
      const float* from = it.nseg == 1 ? row : left + (size_t)((it.seg ? it.seg : it.nseg) - 1) *
                                                          D.HV * plane;
#pragma unroll 1
      for (int x = 0; x < 64; x += 32) {
        float4 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = *reinterpret_cast<const float4*>(from + x + 4 * i);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t r[16];
          const uint32_t zero[16] = {};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            r[4 * m] = __float_as_uint(y[4 * i + m].x), r[4 * m + 1] = __float_as_uint(y[4 * i + m].y);
            r[4 * m + 2] = __float_as_uint(y[4 * i + m].z);
            r[4 * m + 3] = __float_as_uint(y[4 * i + m].w);
          }
          tc::tmem_st16(tmem + lanes + T_S + x + 16 * i, r);
          tc::tmem_st16(tmem + lanes + T_S + 64 + x + 16 * i, zero);
          tc::tmem_st16(tmem + lanes + T_S + 128 + x + 16 * i, zero);
        }
      }
      tc::tmem_wait_st();
    }
#pragma unroll 1
    for (int c = 0; !STATES && c < n; ++c) {
      if (c > 0) {
        ok = wait(&B.s_full, c - 1);
        if (!ok) break;
        tc::fence_after_sync();
      }
      ok = wait(&B.gate_full[c & 1], c >> 1);
      if (!ok) break;
      if (mine) {
        const float tot = B.gate[c & 1].tot;
        const uint32_t zero[16] = {};
#pragma unroll 1
        for (int x = 0; x < 64; x += 16) {
          from_tmem(x);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(sb + 128 * d + 16 * ((x / 8 + i) ^ (d & 7))) = make_uint4(
                pack2_bf(S[8 * i], S[8 * i + 1]), pack2_bf(S[8 * i + 2], S[8 * i + 3]),
                pack2_bf(S[8 * i + 4], S[8 * i + 5]), pack2_bf(S[8 * i + 6], S[8 * i + 7]));
          uint32_t r[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(S[i] * tot);
          tc::tmem_st16(tmem + lanes + T_S + x, r);
          tc::tmem_st16(tmem + lanes + T_S + 64 + x, zero);
          tc::tmem_st16(tmem + lanes + T_S + 128 + x, zero);
        }
        tc::tmem_wait_st();
      }
      tc::fence_before_sync();
      tc::fence_async_smem();
      arrive(&B.sb_full);
      if (lane == 0) mbar_arrive(&B.gate_empty[c & 1]);
    }
    // STATES: g_total was written in front of the last gate_full, behind which is `last`
    if (ok) ok = STATES ? wait(&B.last, 0) : wait(&B.s_full, n - 1);
    if (ok && mine && !B.failed) {
      tc::fence_after_sync();
#pragma unroll 1
      for (int x = 0; x < 64; x += 16) {
        if (STATES) {
          from_tmem(x);
          if (it.seg == 0) load(row + x, ex2((float)B.g_total));
          store(left + (size_t)it.seg * D.HV * plane + x);
        } else if (it.seg == it.nseg - 1) {
          from_tmem(x);
          store(row + x);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (B.failed) {
    // a wait gave up: give copies that may still be in flight time to land
    const uint64_t tw = globaltimer_ns();
    while (globaltimer_ns() - tw < kDrainNs) {
    }
  }
  if (warp == DC_MMA) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// What each segment's own tokens leave behind becomes what all segments up to it leave
// together: W[g] += e^{G_g} W[g - 1], for the segments that a later one starts from.  Four
// values a thread, eight segments' loads in flight.
constexpr int DJ_THREADS = 256;
__global__ void __launch_bounds__(DJ_THREADS) k_decay_join(const ChunkParams P) {
  __shared__ Item item;
  const DecayParams& D = P.d;
  grid_dep_wait();
  grid_dep_trigger();
  const int plane = D.DK * D.DV, parts = plane / (4 * DJ_THREADS), per = D.HV * parts;
  if (threadIdx.x < 32) find_item<3>(D, blockIdx.x / per, &item);
  __syncthreads();
  const Item it = item;
  if (!it.found) return;
  const int h = blockIdx.x % per / parts, part = blockIdx.x % parts;
  const size_t step = (size_t)D.HV * plane;
  float* W = P.W + it.slot * step + (size_t)h * plane + 4 * (part * DJ_THREADS + threadIdx.x);
  const double* G = P.Wg + (size_t)it.slot * D.HV + h;
  float4 s = *reinterpret_cast<const float4*>(W);
  for (int g0 = 1; g0 < it.nseg - 1; g0 += 8) {
    float4 y[8];
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (g0 + i < it.nseg - 1) {
        y[i] = *reinterpret_cast<const float4*>(W + (g0 + i) * step);
        f[i] = ex2((float)G[(g0 + i) * D.HV]);
      }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (g0 + i < it.nseg - 1) {
        s.x = fmaf(f[i], s.x, y[i].x), s.y = fmaf(f[i], s.y, y[i].y);
        s.z = fmaf(f[i], s.z, y[i].z), s.w = fmaf(f[i], s.w, y[i].w);
        *reinterpret_cast<float4*>(W + (g0 + i) * step) = s;
      }
  }
}

// k twice; v twice, three terms of Ṽ, q, S and o (STATES: v three times, the terms twice);
// the rest, alignment.
constexpr int chunk_smem(int DK) {
  const int walk = 5 * 16384 + 256 * DK + 128 * DK + 16384, states = 9 * 16384;
  return 512 * DK + (walk > states ? walk : states) + 10240;
}

// Tokens of a segment: the cut with the least estimated time, of cuts that fill 1 to 8 rounds
// of the SMs, of none, and of one into the call's sequences.  The lengths are not known here: it
// is the time if one sequence has all tokens, plus that if all have as many.  Measured: a
// walk takes 5.5 us and 2.6 a chunk, one of the states' 2.5 and 1.1, their launch and the
// join's 7 and 0.2 a segment.  (32 heads of 128 x 128, by this and with four rounds and 512
// tokens at least: 1500 tokens 37 and 48 us, 4096 75 and 109, 8192 135 and 169, 32768 474 and 474;
// 8 heads of 64 x 64, 32768 tokens 70 and 110.)
int segment_tokens(int B, int T, int HV, int DV) {
  const int walks = HV * (DV / 64), sms = num_sms();
  const auto chunks = [](int tokens) { return std::max(1, (tokens + CH - 1) / CH); };
  const auto cost = [&](int n, int all, int len) {  // n sequences of `all` chunks
    const long long w = (long long)n * walks;
    const auto rounds = [&](int segs) { return (double)((w * segs + sms - 1) / sms); };
    const int segs = (all + len - 1) / len;
    if (segs == 1) return rounds(1) * (5.5 + 2.6 * all);
    return rounds(segs) * (5.5 + 2.6 * len) + 7.0 + 0.2 * segs +
           rounds(segs - 1) * (2.5 + 1.1 * len);
  };
  const int one = chunks(T), each = chunks((T + B - 1) / B);
  int best = one;
  double least = 1e300;
  const auto consider = [&](int len) {
    const double t = cost(1, one, len) + cost(B, each, len);
    if (t < least) least = t, best = len;
  };
  consider(one);
  consider(each);
  for (int r = 1; r <= 8; ++r) {
    const int segs = std::min(one, r * sms / walks);
    if (segs > 1) consider((one + segs - 1) / segs);
  }
  return CH * best;
}

// Segments of sequences that have two and more: a sequence of n > L tokens has
// ceil(n / L) < 2 n / L.
size_t segment_slots(int T, int L) { return T > L ? 2 * (size_t)T / L : 0; }

size_t prefill_bytes(int B, int T, int HV, int DK, int DV, float** W, double** Wg, int32_t** items,
                     void* base) {
  const size_t slots = segment_slots(T, segment_tokens(B, T, HV, DV));
  Carver c(base);
  float* w = c.take<float>(slots * HV * DK * DV);
  double* g = c.take<double>(slots * HV + 1);
  int32_t* n = c.take<int32_t>(1);
  if (W) *W = w, *Wg = g, *items = n;
  return c.used();
}

std::mutex g_attr_mu;
bool g_attr_done[64] = {false};

// Sequences of how many tokens k_decay_few takes.
int few_tokens(const DecayParams& D) {
  // Where heads fill the SMs, up to 32: 16 sequences of 16 tokens take 34 us (by chunks 57),
  // of 32 59 (57), of 60 106 (65); 512 of 32 1640 us (above 2200).  Else, with narrower slices, 16:
  // one of 8 tokens takes 4.3 us, of 16 6.6 (8.2).
  const int most = D.B * D.HV >= 2 * num_sms() ? 32 : 16;
  // its launch for nothing costs 2 us: only where the mean length is below a chunk's
  return D.T <= most || D.T < (int64_t)CH * D.B ? most : 0;
}

int launch_prefill(DecayParams D, void* ws, cudaStream_t st) {
  ChunkParams P{};
  int32_t* items;
  prefill_bytes(D.B, D.T, D.HV, D.DK, D.DV, &P.W, &P.Wg, &items, ws);
  D.L = segment_tokens(D.B, D.T, D.HV, D.DV);
  D.few = few_tokens(D);
  if (D.few) {
    D.items = items;
    const int rc = launch_few(D, st);
    if (rc != ER_OK || D.T <= D.few) return rc;
  }
  P.d = D;
  {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ER_ECUDA;
    std::lock_guard<std::mutex> lock(g_attr_mu);
    if (!g_attr_done[dev]) {
      const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
      if (cudaFuncSetAttribute(k_decay_chunks<64, false>, a, chunk_smem(64)) != cudaSuccess ||
          cudaFuncSetAttribute(k_decay_chunks<64, true>, a, chunk_smem(64)) != cudaSuccess ||
          cudaFuncSetAttribute(k_decay_chunks<128, false>, a, chunk_smem(128)) != cudaSuccess ||
          cudaFuncSetAttribute(k_decay_chunks<128, true>, a, chunk_smem(128)) != cudaSuccess)
        return ER_ECUDA;
      g_attr_done[dev] = true;
    }
  }
  if (!encode_rows(&P.q_map, D.q, false, D.HK * D.DK, D.T, D.ldq * 2, 64, CH) ||
      !encode_rows(&P.k_map, D.k, false, D.HK * D.DK, D.T, D.ldk * 2, 64, CH) ||
      !encode_rows(&P.v_map, D.v, false, D.HV * D.DV, D.T, D.ldv * 2, 64, CH) ||
      !encode_rows(&P.o_map, D.o, false, D.HV * D.DV, D.T, D.ldo * 2, 32, 32))
    return ER_ECUDA;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // sequences of more than n tokens are T / (n + 1) at most, and the segments of m sequences
  // m + T / L
  const auto sequences = [&](size_t n) { return std::min((size_t)D.B, D.T / (n + 1)); };
  const size_t per = D.HV * (D.DV / 64), cut = D.T > D.L ? D.T / D.L : 0;
  const size_t blocks = (sequences(D.few) + cut) * per;
  const size_t first = (sequences(D.L) + cut) * per;
  const size_t joins = sequences(2 * (size_t)D.L) * D.HV * (D.DK * D.DV / (4 * DJ_THREADS));
  if (blocks > 0x7FFFFFFFu || joins > 0x7FFFFFFFu) return ER_EINVAL;
  cfg.blockDim = dim3(DC_THREADS);
  cfg.dynamicSmemBytes = chunk_smem(D.DK);
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const bool wide = D.DK == 128;
  if (D.T > D.L) {
    cfg.gridDim = dim3((unsigned)first);
    if (cudaLaunchKernelEx(&cfg, wide ? k_decay_chunks<128, true> : k_decay_chunks<64, true>, P) !=
        cudaSuccess)
      return ER_ECUDA;
    count_launches(1);
  }
  if (joins) {
    cudaLaunchConfig_t join = cfg;
    join.gridDim = dim3((unsigned)joins);
    join.blockDim = dim3(DJ_THREADS);
    join.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&join, k_decay_join, P) != cudaSuccess) return ER_ECUDA;
    count_launches(1);
  }
  cfg.gridDim = dim3((unsigned)blocks);
  if (cudaLaunchKernelEx(&cfg, wide ? k_decay_chunks<128, false> : k_decay_chunks<64, false>, P) !=
      cudaSuccess)
    return ER_ECUDA;
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
  if (!shape_ok(sh) || s_max < 1 || B < 0 || B > 65535 || T < 0 || T > (1 << 30))
    return ER_EINVAL;
  const int qk = sh->k_heads * sh->k_dim, vo = sh->v_heads * sh->v_dim;
  if (ldq < qk || ldk < qk || ldv < vo || ldo < vo || ldq % 8 || ldk % 8 || ldv % 8 || ldo % 8 ||
      (ldg != 0 && ldg < sh->v_heads))
    return ER_EINVAL;
  if (B > s_max) return ER_ECAPACITY;
  if (B == 0) return ER_OK;
  if (!state || !seq_ids || !aligned16(state) || ((uintptr_t)seq_ids & 3u)) return ER_EINVAL;
  if (T > 0 && (!q || !k || !v || !g || !o || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
                !aligned16(o) || ((uintptr_t)g & 3u) || o == q || o == k || o == v ||
                (void*)o == state || (const void*)o == g))
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
  if (!shape_ok(shape) || B < 1 || B > 65535 || T < 0 || T > (1 << 30)) return 0;
  return prefill_bytes(B, T, shape->v_heads, shape->k_dim, shape->v_dim, nullptr, nullptr, nullptr,
                       nullptr);
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
  return launch_decode(P, (cudaStream_t)stream);
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
  return launch_prefill(P, ws, (cudaStream_t)stream);
}

}  // extern "C"
