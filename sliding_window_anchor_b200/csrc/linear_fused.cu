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
#include <mutex>

#include "common.cuh"
#include "tc.cuh"

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

// v / (1 + e^-z).  The quotient is __fdividef (2 ulp; 0 for a divisor above 2^126, where
// the value is below 2^-118): a division rounded to nearest takes a slow path for
// v = 0, the value of every row a tile has too many (gated, 9 tokens: 17 us a tile).
__device__ __forceinline__ float times_sigmoid(float v, float z) {
  return __fdividef(v, 1.f + __expf(-z));
}

// v · Φ(v).  The normal distribution's upper tail at x = |v| is t·P(t)·e^(-x²/2), t =
// 1 / (1 + 0.305 x), the form of Abramowitz & Stegun 26.2.17; P is fitted for the least relative
// error (2^-23.3) over x <= 13.2, behind which the tail is below the normal numbers.  No difference
// of near values for v < 0, where v/2 · (1 + erf(v / sqrt(2))) is off by 4% at -5 and 0 from
// -5.6 on.  Within (16 + 0.75 v²)·2^-23 of the value.  It takes as long as erff would;
// v/2 · erfcf(-v / sqrt(2)) is as near and took a tenth longer (gated 300 x 2*9000 x 2560 36.3
// against 32.8 us).
__device__ __forceinline__ float gelu(float v) {
  const float x = fabsf(v), t = __fdividef(1.f, fmaf(0.305f, x, 1.f));
  float p = 0.0366991982f;
  p = fmaf(p, t, -0.15298833f), p = fmaf(p, t, 0.185716912f), p = fmaf(p, t, -0.0379768424f);
  p = fmaf(p, t, 0.121021688f), p = fmaf(p, t, 0.103420869f), p = fmaf(p, t, 0.122466817f);
  p = fmaf(p, t, 0.121639736f);
  const float tail = t * p * exp2f(-0.72134752044448170f * (x * x));
  return v * (v < 0.f ? tail : 1.f - tail);
}

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case ER_ACT_SILU:
      return times_sigmoid(v, v);
    case ER_ACT_GELU:
      return gelu(v);
    case ER_ACT_GELU_TANH:
      // 1 + tanh(z) = 2 / (1 + e^-2z)
      return times_sigmoid(v, 1.5957691216057308f * (v + 0.044715f * v * v * v));
    default:
      return v;
  }
}

// One output value from its sums: v (+ u, the gated product's second one).
__device__ __forceinline__ float finish(const FusedParams& P, float v, float u, bool gated, int act,
                                        int t, int f) {
  if (P.bias) v += bf1(P.bias[f]);
  v = activate(v, act);
  if (gated) v *= u;
  if (P.residual)
    v += P.f32 ? static_cast<const float*>(P.residual)[t * P.ldr + f]
               : bf1(static_cast<const uint16_t*>(P.residual)[t * P.ldr + f]);
  return v;
}

__device__ __forceinline__ void store_one(const FusedParams& P, int t, int f, float v) {
  if (P.f32)
    static_cast<float*>(P.y)[t * P.ldy + f] = v;
  else
    static_cast<uint16_t*>(P.y)[t * P.ldy + f] = f2bf(v);
}

// Adds the residual to four values of token t, features f.., and stores them; `vec`: all
// four are there, in rows of y (and the residual) that are whole 16-byte units.
__device__ __forceinline__ void finish_four(const FusedParams& P, int el, bool vec, int t, int f,
                                            float4 v) {
  char* to = static_cast<char*>(P.y) + (t * P.ldy + f) * el;
  const char* add = static_cast<const char*>(P.residual) + (t * P.ldr + f) * el;
  if (vec && el == 4) {
    if (P.residual) {
      const float4 b = *reinterpret_cast<const float4*>(add);
      v.x += b.x, v.y += b.y, v.z += b.z, v.w += b.w;
    }
    *reinterpret_cast<float4*>(to) = v;
  } else if (vec) {
    if (P.residual) {
      const uint2 b = *reinterpret_cast<const uint2*>(add);
      v.x += bf_lo(b.x), v.y += bf_hi(b.x), v.z += bf_lo(b.y), v.w += bf_hi(b.y);
    }
    *reinterpret_cast<uint2*>(to) = make_uint2(pack2_bf(v.x, v.y), pack2_bf(v.z, v.w));
  } else {
#pragma unroll 1
    for (int j = 0; j < 4 && f + j < P.F; ++j) {
      float x = v.x;
      v.x = v.y, v.y = v.z, v.z = v.w;
      if (P.residual)
        x += el == 4 ? reinterpret_cast<const float*>(add)[j]
                     : bf1(reinterpret_cast<const uint16_t*>(add)[j]);
      if (el == 4)
        reinterpret_cast<float*>(to)[j] = x;
      else
        reinterpret_cast<uint16_t*>(to)[j] = f2bf(x);
    }
  }
}

// Bias of features f..f+15 (the same for every lane).
__device__ __forceinline__ void add_bias(float (&v)[16], const FusedParams& P, int f) {
  if (!P.bias) return;
  if (((uintptr_t)P.bias & 15u) == 0 && f + 16 <= P.F) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 b = __ldg(reinterpret_cast<const uint4*>(P.bias + f) + i);
      v[8 * i] += bf_lo(b.x), v[8 * i + 1] += bf_hi(b.x);
      v[8 * i + 2] += bf_lo(b.y), v[8 * i + 3] += bf_hi(b.y);
      v[8 * i + 4] += bf_lo(b.z), v[8 * i + 5] += bf_hi(b.z);
      v[8 * i + 6] += bf_lo(b.w), v[8 * i + 7] += bf_hi(b.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (f + i < P.F) v[i] += bf1(P.bias[f + i]);
  }
}

// Residual of token t, features f..f+15.  Plain loads: it may be y itself.
__device__ __forceinline__ void add_residual(float (&v)[16], const FusedParams& P, bool vec,
                                               int t, int f) {
  if (!P.residual) return;
  if (P.f32) {
    const float* r = static_cast<const float*>(P.residual) + t * P.ldr + f;
    if (vec && f + 16 <= P.F) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 b = reinterpret_cast<const float4*>(r)[i];
        v[4 * i] += b.x, v[4 * i + 1] += b.y, v[4 * i + 2] += b.z, v[4 * i + 3] += b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (f + i < P.F) v[i] += r[i];
    }
  } else {
    const uint16_t* r = static_cast<const uint16_t*>(P.residual) + t * P.ldr + f;
    if (vec && f + 16 <= P.F) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 b = reinterpret_cast<const uint4*>(r)[i];
        v[8 * i] += bf_lo(b.x), v[8 * i + 1] += bf_hi(b.x);
        v[8 * i + 2] += bf_lo(b.y), v[8 * i + 3] += bf_hi(b.y);
        v[8 * i + 4] += bf_lo(b.z), v[8 * i + 5] += bf_hi(b.z);
        v[8 * i + 6] += bf_lo(b.w), v[8 * i + 7] += bf_hi(b.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (f + i < P.F) v[i] += bf1(r[i]);
    }
  }
}

// Up to 32 staged rows (128 bytes each, chunk c of row l at c ^ l % 8) to y, whose rows are
// not 16-byte aligned: a row's elements by consecutive lanes.
__device__ __forceinline__ void copy_rows(const FusedParams& P, const unsigned char* stg, int t0,
                                          int f, int cols, int lane) {
  const int rows = min(32, P.T - t0);
  cols = min(cols, P.F - f);
  for (int l = 0; l < rows; ++l)
    for (int c = lane; c < cols; c += 32) {
      const size_t to = (t0 + l) * P.ldy + f + c;
      const int byte = c * (P.f32 ? 4 : 2);
      const unsigned char* from = stg + 128 * l + 16 * ((byte >> 4) ^ (l & 7)) + (byte & 15);
      if (P.f32)
        static_cast<float*>(P.y)[to] = *reinterpret_cast<const float*>(from);
      else
        static_cast<uint16_t*>(P.y)[to] = *reinterpret_cast<const uint16_t*>(from);
    }
}

// ------------------------------------------------------------ few tokens
// Up to 8 tokens the product is a read of the weights.  A warp owns 16 weight
// rows and a slice of K; per 32-wide step of K every lane loads 16 bytes of two
// rows (rows g and g + 8, columns 8c..8c+7 of the step, g = lane/4, c = lane%4)
// and 16 bytes of token g, and feeds them unchanged to two m16n8k16 products
// (a K column meets the same K column on both operands, so their order does not
// matter).  The K slices of a block's warps are added in a fixed order.  HBM bounds it, with
// the launch, the ramp and the few SMs that hold two blocks: with weights outside L2
// 1 x 2560 x 4096 takes 7.4 us (2.8 TB/s; 6.4 with them in L2), gated 1 x 2*6912 x 2560
// 15-18 us (70.8 MB; 3.9-4.7 TB/s).
constexpr int FV_TOKENS = 8;
constexpr int FV_MAXW = 8;

__device__ __forceinline__ uint4 ld_weights(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint4 ld_tokens(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// D += A·B, m16n8k16, BF16 operands, FP32 accumulators.
__device__ __forceinline__ void mma16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool GATED>
__global__ void __launch_bounds__(32 * FV_MAXW, 2) k_fused_few(const FusedParams P) {
  constexpr int NW = GATED ? 2 : 1;  // weights
  constexpr int U = 8 / NW;          // K steps in flight
  __shared__ float red[FV_MAXW][NW][4][32];
  const int S = blockDim.x >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int row0 = blockIdx.x * 16;
  const int KS = (P.K + 31) / 32;
  const int k_lo = KS * warp / S, k_hi = KS * (warp + 1) / S;
  const size_t ra = (size_t)min(row0 + g, P.F - 1) * P.K;
  const size_t rb = (size_t)min(row0 + g + 8, P.F - 1) * P.K;
  const uint16_t* wp[2] = {P.w, GATED ? P.w2 : P.w};
  const uint16_t* xp = P.x + min(g, P.T - 1) * P.ldx;
  const uint4 z = make_uint4(0, 0, 0, 0);
  float acc[NW][4] = {};
  grid_dep_wait();
  grid_dep_trigger();
  // U steps of weights and tokens are in flight, carried around the loop (loads that
  // are used in the iteration that issues them are moved down to their uses, one in
  // flight at a time); a step outside the slice or K loads its row's start and counts
  // as zero
  uint4 a[U][NW], b[U][NW], x[U];
  auto inside = [&](int step) { return step < k_hi && 32 * step + 8 * c < P.K; };
  auto load = [&](int k0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = inside(k0 + u) ? 32 * (k0 + u) + 8 * c : 0;
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        a[u][n] = ld_weights(wp[n] + ra + at);
        b[u][n] = ld_weights(wp[n] + rb + at);
      }
      x[u] = ld_tokens(xp + at);
    }
  };
  load(k_lo);
  for (int k0 = k_lo; k0 < k_hi; k0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = inside(k0 + u);
      const uint4 xu = in && g < P.T ? x[u] : z;
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        const uint4 au = in ? a[u][n] : z, bu = in ? b[u][n] : z;
        mma16816(acc[n], au.x, bu.x, au.y, bu.y, xu.x, xu.y);
        mma16816(acc[n], au.z, bu.z, au.w, bu.w, xu.z, xu.w);
      }
    }
    load(k0 + U);
  }
#pragma unroll
  for (int n = 0; n < NW; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][n][i][lane] = acc[n][i];
  __syncthreads();
  // value i of lane (g, c): row g + 8 (i / 2), token 2c + i % 2
  for (int e = threadIdx.x; e < 128; e += blockDim.x) {
    const int i = e >> 5, l = e & 31;
    const int f = row0 + (l >> 2) + 8 * (i >> 1), t = 2 * (l & 3) + (i & 1);
    if (t >= P.T || f >= P.F) continue;
    float v = 0.f, u = 0.f;
    for (int w = 0; w < S; ++w) {
      v += red[w][0][i][l];
      if (GATED) u += red[w][NW - 1][i][l];
    }
    store_one(P, t, f, finish(P, v, u, GATED, P.act, t, f));
  }
}

template <bool GATED>
int launch_few(const FusedParams& P, cudaStream_t st) {
  // K slices: about 8 warps per SM, a K step for each
  const int blocks = (P.F + 15) / 16, KS = (P.K + 31) / 32;
  int S = 1;
  while (S < FV_MAXW && blocks * S < 8 * num_sms() && 2 * S <= KS) S <<= 1;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(32 * S);
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k_fused_few<GATED>, P) != cudaSuccess) return ER_ECUDA;
  count_launches(1);
  return launch_status();
}

// ------------------------------------------------------------ many tokens
// CTA pairs (tcgen05 cta_group::2) compute tiles of 256 tokens (128 in each
// CTA's TMEM lanes) by BN weight rows, K in steps of 128 (two boxes of 64) through a
// ring of TMA stages.  Of a step each CTA fetches its 128 tokens and half of the BN
// weight rows; in the gated product the even CTA's half are rows of w_gate and
// the odd CTA's the same rows of w_up, so that a tile's columns j and j + BN/2
// are the gate and the up value of one feature, in one thread.
//
// A cluster is S pairs.  S = 1: pairs walk over the tiles, two accumulators in
// TMEM, so that a tile's epilogue runs beside the next one's products.  S > 1
// (few tiles): the pairs of a cluster each take a share of K of the cluster's
// one tile, leave their FP32 sums in shared memory, and each adds up a part of
// the tile over distributed shared memory, in the order of the shares.
//
// The tensor cores bound large products, with the power limit: 8192 x 10240 x 2560 takes 283 us
// (1.52 PFLOP/s; the library's product alone 304 beside it) to 343 in a long run of calls
// (1.25), gated 4096 x 2*10240 x 2560 274-326.  Middling ones are bound by what surrounds the
// tile: of 512 x 2560 x 4096 (17.5 us with weights outside L2, 23.1 with a residual from
// there too) 6.5 us are its products at the tensor cores' rate; the launch, the ring's first
// fill, the joining of the shares and the epilogue follow one another around them.
//
// Per CTA: warp 8 — TMA; warp 9 — TMEM and, in a pair's even CTA, the MMAs;
// warps 0-7 — the epilogue: warp w has the TMEM lanes (tokens) of quadrant w % 4
// and half w / 4 of the columns.
constexpr int DN_THREADS = 320;
constexpr int DN_EPI = 256;
constexpr int DN_A_BYTES = 128 * 128;
constexpr int DN_MAXST = 8;
constexpr int DN_SMEM = 232448;
constexpr int DN_STAGING = 8 * 4096;  // 4 KB per epilogue warp
constexpr uint64_t kDrainNs = 200000;

struct DenseParams {
  CUtensorMap x_map;        // x [T][K], box 64 x x_rows
  CUtensorMap w_map, w2_map;  // weights [F][K], box 64 x BN/2
  CUtensorMap y_map;        // y [T][F], box 128 bytes x 32 rows (when tma_y)
  FusedParams f;
  int n_m, n_n, KB, S;
  int x_rows;               // token rows a CTA fetches: 128, fewer when T has fewer
  int tma_y;
  int vec_r, vec_y;         // residual and y rows are whole 16-byte units
  int32_t* err;
};

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 r;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(a));
  return r;
}

// Tile order: eight token tiles side by side, then along the features, so that
// the pairs at work share weight rows and token rows in L2.
__device__ __forceinline__ void tile_at(const DenseParams& P, int tile, int& m, int& n) {
  constexpr int G = 8;
  const int band = tile / (G * P.n_n), first = band * G;
  const int rows = min(G, P.n_m - first), in = tile - band * G * P.n_n;
  m = first + in % rows;
  n = in / rows;
}

// ACT is a template argument: with a switch over the activations in the epilogue its
// instructions did not stay in the instruction cache (1400 cycles per 1024 values).
template <int BN, bool GATED, int ACT>
__global__ void __launch_bounds__(DN_THREADS, 1) k_dense(const __grid_constant__ DenseParams P) {
  constexpr int FT = GATED ? BN / 2 : BN;  // features of a tile
  constexpr int B_BYTES = BN / 2 * 128;
  constexpr int HALF = DN_A_BYTES + B_BYTES;  // 64 of K
  constexpr int STAGE = 2 * HALF;
  constexpr int NST = (DN_SMEM - 2048 - DN_STAGING) / STAGE < DN_MAXST
                          ? (DN_SMEM - 2048 - DN_STAGING) / STAGE
                          : DN_MAXST;
  static_assert(NST * STAGE + DN_STAGING >= 128 * BN * 4 + 3 * 32 * BN * 4 && BN <= 256,
                "a share's sums and the other shares' rows fit in front of the barriers");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  struct Bars {
    uint64_t full[NST], empty[NST], tfull[2], tempty[2], done, got;
    uint32_t tmem_base;
    volatile int failed;
  };
  unsigned char* staging = base + NST * STAGE;
  Bars& B = *reinterpret_cast<Bars*>(staging + DN_STAGING);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t crank = tc::cluster_rank();
  const uint32_t lead = crank & ~1u;
  const int rank = crank & 1, share = crank >> 1;
  const int n_tiles = P.n_m * P.n_n;
  const int n_clusters = gridDim.x / (2 * P.S), cluster = blockIdx.x / (2 * P.S);
  const int kb0 = P.KB * share / P.S, kb1 = P.KB * (share + 1) / P.S;

  if (threadIdx.x == 32 * 8) {
    // launch arguments: no earlier kernel writes them
    tc::prefetch_map(&P.x_map);
    tc::prefetch_map(&P.w_map);
    if (GATED) tc::prefetch_map(&P.w2_map);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&B.full[s], 1);   // the even CTA's arrival with both CTAs' byte count
      mbar_init(&B.empty[s], 1);  // the MMAs that read the stage have completed
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&B.tfull[b], 1);
      mbar_init(&B.tempty[b], 16);  // the epilogue warps of both CTAs
    }
    mbar_init(&B.done, 1);
    mbar_init(&B.got, 1);
    B.failed = 0;
    fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc_pair(&B.tmem_base, 2 * BN);
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  grid_dep_wait();  // nothing above touched the operands
  grid_dep_trigger();
  const uint32_t tmem = B.tmem_base;

  if (warp == 8) {
    if (tc::elect_one()) {
      int s = 0;
      uint32_t phase = 1;
      const CUtensorMap* wm = GATED && rank ? &P.w2_map : &P.w_map;
      const uint32_t full = tc::map_to_rank(&B.full[0], lead);
      bool ok = true;
      for (int tile = cluster; tile < n_tiles && ok && !B.failed; tile += n_clusters) {
        int m, n;
        tile_at(P, tile, m, n);
        const int t0 = 256 * m + 128 * rank;
        const int f0 = FT * n + (GATED ? 0 : BN / 2 * rank);
        // lanes whose tokens are not fetched hold what the stage held before: a lane's
        // sums are its own token's alone, and nothing past T is stored
        const bool some = t0 < P.f.T;
        // what both CTAs' copies of 64 of K bring; the even CTA's barrier counts them
        // all, and its own thread announces them
        const uint32_t bytes =
            2 * B_BYTES + 128u * P.x_rows * (256 * m + 128 < P.f.T ? 2u : 1u);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&B.empty[s], phase, P.err);
          if (!ok) break;
          unsigned char* st = base + (size_t)s * STAGE;
          const uint32_t fb = full + 8 * s;
          const bool two = 128 * kb + 64 < P.f.K;
          if (rank == 0) mbar_arrive_expect_tx(&B.full[s], two ? 2 * bytes : bytes);
          tc::tma_load_2d_pair(st + DN_A_BYTES, wm, 128 * kb, f0, fb);
          if (some) tc::tma_load_2d_pair(st, &P.x_map, 128 * kb, t0, fb);
          if (two) {
            tc::tma_load_2d_pair(st + HALF + DN_A_BYTES, wm, 128 * kb + 64, f0, fb);
            if (some) tc::tma_load_2d_pair(st + HALF, &P.x_map, 128 * kb + 64, t0, fb);
          }
          if (++s == NST) s = 0, phase ^= 1;
        }
      }
      if (!ok) B.failed = 1;
    }
    __syncwarp();
  } else if (warp == 9) {
    if (rank == 0 && tc::elect_one()) {
      constexpr uint32_t id = tc::idesc_bf16(256, BN, false, false);
      const uint16_t both = (uint16_t)(3u << lead);
      const uint64_t a_desc = tc::desc_sw128(smem_u32(base), 16, 1024);
      const uint64_t b_desc = tc::desc_sw128(smem_u32(base) + DN_A_BYTES, 16, 1024);
      int s = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = cluster; tile < n_tiles && ok && !B.failed; tile += n_clusters, ++it) {
        const int b = it & 1;
        ok = mbar_wait(&B.tempty[b], ((it >> 1) & 1) ^ 1, P.err);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t d = tmem + BN * b;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&B.full[s], phase, P.err);
          if (!ok) break;
          tc::fence_after_sync();
          // descriptors count 16-byte units: a stage, a half of it, 32 bytes (16 of K) a
          // product
          const uint64_t at = (uint64_t)(s * (STAGE / 16));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_pair_bf16(d, a_desc + at + 2 * kk, b_desc + at + 2 * kk, id,
                              (kb > kb0 || kk > 0) ? 1u : 0u);
          if (128 * kb + 64 < P.f.K) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc::mma_pair_bf16(d, a_desc + at + HALF / 16 + 2 * kk,
                                b_desc + at + HALF / 16 + 2 * kk, id, 1u);
          }
          tc::commit_pair_to(&B.empty[s], both);
          if (++s == NST) s = 0, phase ^= 1;
        }
        if (!ok) break;
        tc::commit_pair_to(&B.tfull[b], both);
      }
      if (!ok) B.failed = 1;
      tc::commit_pair(tc::map_to_rank(&B.done, crank));
      mbar_wait(&B.done, 0, P.err);  // nothing of the pair's is on the tensor cores at exit
    }
    __syncwarp();
  } else {
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    if (P.S == 1) {
      unsigned char* stg = staging + 4096 * warp;
      int it = 0;
      for (int tile = cluster; tile < n_tiles; tile += n_clusters, ++it) {
        const int b = it & 1;
        const bool ok = mbar_wait(&B.tfull[b], (it >> 1) & 1, P.err) && !B.failed;
        if (!__all_sync(0xffffffffu, ok)) {
          B.failed = 1;
          break;
        }
        tc::fence_after_sync();
        int m, n;
        tile_at(P, tile, m, n);
        const int t0 = 256 * m + 128 * rank + 32 * quad, t = t0 + lane;
        // Sixteen columns at a time (less code to fetch than for 32, for tiles that are few),
        // into the warp's staging rows of 128 bytes (16-byte chunk c of row l at c ^ l % 8),
        // from where whole rows go out: FP32 after 32 columns, BF16 after 64.
        const bool f32 = P.f.f32;
        const int group = f32 ? 2 : 4;
        constexpr int NC = FT / 32;  // in this warp's half of the tile's features
#pragma unroll 1
        for (int cb = 0; cb < NC; ++cb) {
          const int col = FT / 2 * half + 16 * cb, f = FT * n + col;
          uint32_t r[16], u[GATED ? 16 : 1];
          tc::tmem_ld16(tmem + lanes + BN * b + col, r);
          if constexpr (GATED) tc::tmem_ld16(tmem + lanes + BN * b + FT + col, u);
          tc::tmem_wait_ld();
          if (t0 >= P.f.T || f >= P.f.F) continue;  // no row, no column of y
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
          if constexpr (GATED) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = activate(v[i], ACT) * __uint_as_float(u[i]);
          } else {
            add_bias(v, P.f, f);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = activate(v[i], ACT);
            if (t < P.f.T) add_residual(v, P.f, P.vec_r, t, f);
          }
          const int part = cb % group;
          if (part == 0) {
            if (lane == 0) tc::bulk_wait_read<0>();
            __syncwarp();
          }
          if (f32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(stg + 128 * lane + 16 * ((4 * part + i) ^ (lane & 7))) =
                  make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint4 o;
              o.x = pack2_bf(v[8 * i], v[8 * i + 1]);
              o.y = pack2_bf(v[8 * i + 2], v[8 * i + 3]);
              o.z = pack2_bf(v[8 * i + 4], v[8 * i + 5]);
              o.w = pack2_bf(v[8 * i + 6], v[8 * i + 7]);
              *reinterpret_cast<uint4*>(stg + 128 * lane +
                                        16 * ((2 * part + i) ^ (lane & 7))) = o;
            }
          }
          if (part + 1 < group && f + 16 < P.f.F) continue;
          const int f_first = f - 16 * part;
          if (P.tma_y) {
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tc::tma_store_2d(&P.y_map, f_first, t0, stg);
              tc::bulk_commit();
            }
          } else {
            __syncwarp();
            copy_rows(P.f, stg, t0, f_first, 16 * (part + 1), lane);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(tc::map_to_rank(&B.tempty[b], lead));
      }
      if (lane == 0) tc::bulk_wait_all();
    } else {
      if (!__all_sync(0xffffffffu, mbar_wait(&B.tfull[0], 0, P.err))) B.failed = 1;
    }
  }
  if (P.S > 1) {
    // Share p finishes rows [rows p / S, rows (p + 1) / S) of its CTA's tokens.  A warp of
    // the epilogue writes its sums (32 tokens, half of the columns; [half][token][BN/2],
    // 16-byte chunk c of row t at c ^ t % 8) and copies the rows that other shares finish
    // to these, one bulk copy each.
    tc::cluster_sync();  // every CTA of the cluster is past its products
    int m, n;
    tile_at(P, cluster, m, n);
    const int t0 = 256 * m + 128 * rank;
    const int rows = max(0, min(128, P.f.T - t0));
    const int r0 = rows * share / P.S, r1 = rows * (share + 1) / P.S;
    const int slot = (rows + P.S - 1) / P.S;  // rows kept for another share's sums
    constexpr int HB = BN / 2;
    float* sums = reinterpret_cast<float*>(base);
    float* others = sums + 128 * BN;  // [share][half][slot][HB]
    if (threadIdx.x == 0)
      mbar_arrive_expect_tx(&B.got, (uint32_t)((P.S - 1) * (r1 - r0) * BN * 4));
    if (warp < 8 && !B.failed) {
      const int quad = warp & 3, half = warp >> 2, row = 32 * quad + lane;
      float* mine = sums + half * 128 * HB;
      tc::fence_after_sync();
#pragma unroll 1
      for (int col = 0; col < HB; col += 32) {
        uint32_t r[32];
        tc::tmem_ld32(tmem + ((uint32_t)(32 * quad) << 16) + HB * half + col, r);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(mine + HB * row + 4 * ((col / 4 + i) ^ (row & 7))) =
              make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
      }
      tc::fence_before_sync();
      tc::fence_async_smem();
      __syncwarp();
      if (lane < P.S && lane != share) {
        const int p = lane;
        const int q0 = max(rows * p / P.S, 32 * quad);
        const int q1 = min(rows * (p + 1) / P.S, 32 * quad + 32);
        if (q0 < q1) {
          float* at = others + ((size_t)(2 * (share - (share > p)) + half) * slot +
                                (q0 - rows * p / P.S)) * HB;
          tc::bulk_s2peer(tc::map_to_rank(at, 2 * p + rank), mine + HB * q0,
                          (uint32_t)((q1 - q0) * HB * 4),
                          tc::map_to_rank(&B.got, 2 * p + rank));
        }
      }
    }
    named_bar_sync(1, DN_THREADS);  // this CTA's own sums are in place
    if (threadIdx.x < DN_EPI && !mbar_wait(&B.got, 0, P.err)) B.failed = 1;
    if (threadIdx.x < DN_EPI && !B.failed) {
      // a thread keeps its four features and walks down the rows; a row's loads are issued
      // together (four shares' always, their sums by need: a branch between them made
      // each wait for the one before)
      constexpr int GR = FT / 4;
      static_assert(DN_EPI % GR == 0, "");
      const int c = threadIdx.x % GR, f = FT * n + 4 * c;
      const int c_in = c % (HB / 4), half = c / (HB / 4);  // gated: half 0, up in half 1
      float bias[4] = {};
      if (P.f.bias)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (f + j < P.f.F) bias[j] = bf1(P.f.bias[f + j]);
      const int S = P.S;
      uint32_t from[4], second[4];  // shared-memory addresses; the gated product's up sums
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const bool own = p == share || p >= S;
        const float* at = own ? sums + (half * 128 + r0) * HB
                              : others + (size_t)(2 * (p - (p > share)) + half) * slot * HB;
        from[p] = smem_u32(at);
        second[p] = from[p] + 4 * HB * (own ? 128 : slot);
      }
      const int el = P.f.f32 ? 4 : 2;
      const bool vec = f + 4 <= P.f.F && P.vec_y && (!P.f.residual || P.vec_r);
#pragma unroll 1
      for (int r = threadIdx.x / GR; r < r1 - r0 && f < P.f.F; r += DN_EPI / GR) {
        const uint32_t at = 4 * (HB * r + 4 * (c_in ^ ((r0 + r) & 7)));
        float4 a[4], b[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          a[p] = lds_f4(from[p] + at);
          if (GATED) b[p] = lds_f4(second[p] + at);
        }
        float4 v = make_float4(bias[0], bias[1], bias[2], bias[3]);
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < 4; ++p)
          if (p < S) {
            v.x += a[p].x, v.y += a[p].y, v.z += a[p].z, v.w += a[p].w;
            if (GATED) u.x += b[p].x, u.y += b[p].y, u.z += b[p].z, u.w += b[p].w;
          }
        v.x = activate(v.x, ACT), v.y = activate(v.y, ACT);
        v.z = activate(v.z, ACT), v.w = activate(v.w, ACT);
        if (GATED) v.x *= u.x, v.y *= u.y, v.z *= u.z, v.w *= u.w;
        finish_four(P.f, el, vec, t0 + r0 + r, f, v);
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
  tc::cluster_sync();  // nothing of the cluster's reads this CTA's memory any more
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, 2 * BN);
  }
}

// ------------------------------------------------------------ tokens as columns
// The same pairs the other way round: 256 weight rows are the MMA's rows (128 in each
// CTA's TMEM lanes), up to 512 tokens its columns, in one or two accumulators of `nacc`
// tokens.  A tile's tokens are then no more than there are (rounded up to 32 or 64), where
// tiles of 256 tokens would leave part of the last one empty, and a weight row is
// fetched once for all of them.  In the gated product a CTA's 128 rows are 64 of w_gate and
// the same 64 of w_up.  A pair has one tile.  Its sums go to shared memory, which the
// operands need no more, and from there out, four features of a token a thread.  The weights'
// stream and the tensor cores bound it about alike: gated 300 x 2*9000 x 2560 took 27 us
// where tiles of 256 tokens took 35 (92 MB of weights at 3.4 TB/s, 1.0 PFLOP/s); cards
// differ, 27-42 us with weights partly in L2 and 29-44 with weights outside it.
struct ColumnsParams {
  CUtensorMap x_map;          // x [T][K], box 64 x nacc / 2
  CUtensorMap w_map, w2_map;  // weights [F][K], box 64 x 128 (gated: 64)
  FusedParams f;
  int KB;                     // K steps of 128
  int nacc, accs;             // tokens of an accumulator, accumulators
  int stages;
  int vec_r, vec_y;           // residual and y rows are whole 16-byte units
  int32_t* err;
};
constexpr int CL_MAXST = 6;

template <bool GATED, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(DN_THREADS, 1)
    k_columns(const __grid_constant__ ColumnsParams P) {
  constexpr int FT = GATED ? 64 : 128;  // features of a CTA
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int N = P.nacc * P.accs;
  const int x_bytes = 64 * P.nacc;                       // an accumulator's tokens, 64 of K
  const int half_bytes = DN_A_BYTES + P.accs * x_bytes;  // 64 of K
  const int stage = 2 * half_bytes;
  struct Bars {
    uint64_t full[CL_MAXST], empty[CL_MAXST], tfull;
    uint32_t tmem_base;
    volatile int failed;
  };
  Bars& B = *reinterpret_cast<Bars*>(base + P.stages * stage);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = tc::cluster_rank();
  const int f0 = FT * blockIdx.x;  // the CTA's first feature

  if (threadIdx.x == 32 * 8) {
    // launch arguments: no earlier kernel writes them
    tc::prefetch_map(&P.x_map);
    tc::prefetch_map(&P.w_map);
    if (GATED) tc::prefetch_map(&P.w2_map);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) {
      mbar_init(&B.full[s], 1);
      mbar_init(&B.empty[s], 1);
    }
    mbar_init(&B.tfull, 1);
    B.failed = 0;
    fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc_pair(&B.tmem_base, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  grid_dep_wait();  // nothing above touched the operands
  grid_dep_trigger();
  const uint32_t tmem = B.tmem_base;

  if (warp == 8) {
    if (tc::elect_one()) {
      int s = 0;
      uint32_t phase = 1;
      const uint32_t full = tc::map_to_rank(&B.full[0], 0);
      for (int kb = 0; kb < P.KB; ++kb) {
        if (!mbar_wait(&B.empty[s], phase, P.err)) {
          B.failed = 1;
          break;
        }
        const uint32_t fb = full + 8 * s;
        const int parts = 128 * kb + 64 < P.f.K ? 2 : 1;
        if (rank == 0) mbar_arrive_expect_tx(&B.full[s], (uint32_t)(2 * parts * half_bytes));
        for (int part = 0; part < parts; ++part) {
          unsigned char* at = base + (size_t)s * stage + part * half_bytes;
          const int k = 128 * kb + 64 * part;
          tc::tma_load_2d_pair(at, &P.w_map, k, f0, fb);
          if (GATED) tc::tma_load_2d_pair(at + DN_A_BYTES / 2, &P.w2_map, k, f0, fb);
          for (int a = 0; a < P.accs; ++a)
            tc::tma_load_2d_pair(at + DN_A_BYTES + a * x_bytes, &P.x_map, k,
                                 P.nacc * a + P.nacc / 2 * rank, fb);
        }
        if (++s == P.stages) s = 0, phase ^= 1;
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    if (rank == 0 && tc::elect_one()) {
      const uint32_t id = tc::idesc_bf16(256, P.nacc, false, false);
      const uint64_t a_desc = tc::desc_sw128(smem_u32(base), 16, 1024);
      int s = 0;
      uint32_t phase = 0;
      for (int kb = 0; kb < P.KB; ++kb) {
        if (!mbar_wait(&B.full[s], phase, P.err)) {
          B.failed = 1;
          break;
        }
        tc::fence_after_sync();
        const int parts = 128 * kb + 64 < P.f.K ? 2 : 1;
        for (int part = 0; part < parts; ++part) {
          const uint64_t a = a_desc + (uint64_t)((s * stage + part * half_bytes) >> 4);
          for (int acc = 0; acc < P.accs; ++acc) {
            const uint64_t x = a + ((DN_A_BYTES + acc * x_bytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc::mma_pair_bf16(tmem + P.nacc * acc, a + 2 * kk, x + 2 * kk, id,
                                (kb > 0 || part > 0 || kk > 0) ? 1u : 0u);
          }
        }
        tc::commit_pair_to(&B.empty[s], 3);
        if (++s == P.stages) s = 0, phase ^= 1;
      }
      tc::commit_pair_to(&B.tfull, 3);
    }
    __syncwarp();
  }
  // every warp: the products are done with the operands
  bool ok = mbar_wait(&B.tfull, 0, P.err) && !B.failed;
  ok = __syncthreads_and(ok);
  tc::fence_after_sync();
  float* sums = reinterpret_cast<float*>(base);  // [token][128]
  const int most = P.stages * stage / 512 / 32 * 32;
  const int tokens = min(N, P.f.T);
  for (int t0 = 0; ok && t0 < tokens; t0 += most) {
    const int end = min(tokens, t0 + most);
    if (warp < 8) {
      const int quad = warp & 3;
#pragma unroll 1
      for (int c = t0 + 32 * (warp >> 2); c < end; c += 64) {
        uint32_t r[32];
        tc::tmem_ld32(tmem + ((uint32_t)(32 * quad) << 16) + c, r);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          sums[128 * (c - t0 + i) + 32 * quad + lane] = __uint_as_float(r[i]);
      }
    }
    __syncthreads();
    constexpr int GR = FT / 4;
    const int c4 = threadIdx.x % GR, f = f0 + 4 * c4;
    if (threadIdx.x < DN_EPI && f < P.f.F) {
      const int el = P.f.f32 ? 4 : 2;
      const bool vec = f + 4 <= P.f.F && P.vec_y && (!P.f.residual || P.vec_r);
      float bias[4] = {};
      if (!GATED && P.f.bias)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (f + j < P.f.F) bias[j] = bf1(P.f.bias[f + j]);
#pragma unroll 4
      for (int t = t0 + threadIdx.x / GR; t < end; t += DN_EPI / GR) {
        float4 v = *reinterpret_cast<const float4*>(sums + 128 * (t - t0) + 4 * c4);
        v.x = activate(v.x + bias[0], ACT), v.y = activate(v.y + bias[1], ACT);
        v.z = activate(v.z + bias[2], ACT), v.w = activate(v.w + bias[3], ACT);
        if (GATED) {
          const float4 u = *reinterpret_cast<const float4*>(sums + 128 * (t - t0) + 64 + 4 * c4);
          v.x *= u.x, v.y *= u.y, v.z *= u.z, v.w *= u.w;
        }
        finish_four(P.f, el, vec, t, f, v);
      }
    }
    __syncthreads();
  }
  if (!ok) {
    B.failed = 1;
    // a wait gave up: give copies that may still be in flight time to land
    const uint64_t tw = globaltimer_ns();
    while (globaltimer_ns() - tw < kDrainNs) {
    }
  }
  tc::fence_before_sync();
  tc::cluster_sync();  // nothing of the pair's reads this CTA's memory any more
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, 512);
  }
}

using ColumnsKernel = void (*)(const ColumnsParams);
const ColumnsKernel kColumns[2][4] = {
    {k_columns<false, 0>, k_columns<false, 1>, k_columns<false, 2>, k_columns<false, 3>},
    {k_columns<true, 0>, k_columns<true, 1>, k_columns<true, 2>, k_columns<true, 3>}};

using DenseKernel = void (*)(const DenseParams);
// [gated 256, 256, 128][activation]
const DenseKernel kDense[3][4] = {
    {k_dense<256, true, 0>, k_dense<256, true, 1>, k_dense<256, true, 2>, k_dense<256, true, 3>},
    {k_dense<256, false, 0>, k_dense<256, false, 1>, k_dense<256, false, 2>,
     k_dense<256, false, 3>},
    {k_dense<128, false, 0>, k_dense<128, false, 1>, k_dense<128, false, 2>,
     k_dense<128, false, 3>}};

// What a device holds at once: clusters of S pairs (they stay inside a GPC).
struct Room {
  int clusters[5];
};
std::mutex g_attr_mu;
bool g_attr_done[64] = {false};
Room g_room[64];

cudaLaunchConfig_t dense_config(cudaLaunchAttribute (&attr)[2], int clusters, int S,
                                cudaStream_t st) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * 2 * S);
  cfg.blockDim = dim3(DN_THREADS);
  cfg.dynamicSmemBytes = DN_SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

int dense_attributes(Room& room) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ER_ECUDA;
  std::lock_guard<std::mutex> lock(g_attr_mu);
  if (g_attr_done[dev]) {
    room = g_room[dev];
    return ER_OK;
  }
  for (auto& row : kDense)
    for (DenseKernel fn : row)
      if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, DN_SMEM) !=
          cudaSuccess)
        return ER_ECUDA;
  for (auto& row : kColumns)
    for (ColumnsKernel fn : row)
      if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, DN_SMEM) !=
          cudaSuccess)
        return ER_ECUDA;
  for (int S = 1; S <= 4; ++S) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = dense_config(attr, 1, S, nullptr);
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&g_room[dev].clusters[S], kDense[1][0], &cfg) !=
        cudaSuccess)
      return ER_ECUDA;
  }
  if (g_room[dev].clusters[1] < 1) return ER_ECUDA;
  room = g_room[dev];
  g_attr_done[dev] = true;
  return ER_OK;
}

// How a product is cut: tiles of 256 tokens by BN weight rows, K in S shares; or (BN = 0)
// tiles of 256 weight rows by `accs` times `nacc` tokens.
struct DensePlan {
  int BN, S, clusters;
  int nacc, accs;
};

// The cut with the least estimated cycles of a pair.  A K step of 128 costs the longer of
// its MMAs (4 cycles a column) and its fetches (measured: one SM's TMA brings about 60
// bytes per cycle in these boxes, about 24 of weights that come from HBM); joining shares
// costs the copies between the CTAs (measured: 16 bytes per cycle into a CTA) and two more
// barriers of the cluster; an epilogue that nothing runs beside about 12 cycles a column.
DensePlan choose_plan(int T, int F, int K, bool gated, const Room& room) {
  const int KB = (K + 127) / 128, n_m = (T + 255) / 256, rows = T < 128 ? T : 128;
  const auto step = [](double columns, double bytes, double weights, bool once) {
    const double mma = 4.0 * columns, fetch = bytes / 60.0, hbm = once ? weights / 24.0 : 0.0;
    return mma > fetch ? (mma > hbm ? mma : hbm) : (fetch > hbm ? fetch : hbm);
  };
  DensePlan best{256, 1, 1, 0, 0};
  double least = 1e300;
  for (int BN : {256, 128}) {
    if (gated && BN != 256) continue;
    const int FT = gated ? BN / 2 : BN, tiles = n_m * ((F + FT - 1) / FT);
    for (int S = 1; S <= 4 && S <= KB; ++S) {
      if (S > 1 && tiles > room.clusters[S]) break;
      const int clusters = tiles < room.clusters[S] ? tiles : room.clusters[S];
      const int waves = (tiles + clusters - 1) / clusters;
      const double join = 4000.0 + 4.0 * BN * rows * (S - 1) / S / 16.0;
      const double cost = waves * ((KB + S - 1) / S) *
                              step(BN, 256.0 * rows + 128.0 * BN, 128.0 * BN, n_m == 1) +
                          (S > 1 ? join : 12.0 * BN);
      if (cost < least) {
        least = cost;
        best = DensePlan{BN, S, clusters, 0, 0};
      }
    }
  }
  const int accs = T > 256 ? 2 : 1, nacc = ((T + accs - 1) / accs + 31) / 32 * 32;
  const int tiles = (F + (gated ? 127 : 255)) / (gated ? 128 : 256);
  if (T > FV_TOKENS && T <= 512 && tiles <= room.clusters[1]) {
    const int N = nacc * accs;
    const double cost = KB * step(N, 32768.0 + 128.0 * N, 32768.0, true) + 2000.0 + 12.0 * N;
    if (cost < least) best = DensePlan{0, 1, tiles, nacc, accs};
  }
  return best;
}

int launch_columns(const FusedParams& F, const DensePlan& plan, int32_t* err, cudaStream_t st) {
  const bool gated = F.w2 != nullptr;
  ColumnsParams P{};
  P.f = F;
  P.err = err;
  P.nacc = plan.nacc;
  P.accs = plan.accs;
  P.KB = (F.K + 127) / 128;
  const int stage = 2 * (DN_A_BYTES + 64 * plan.nacc * plan.accs);
  P.stages = (DN_SMEM - 2048) / stage;
  if (P.stages > CL_MAXST) P.stages = CL_MAXST;
  const int el = F.f32 ? 4 : 2;
  P.vec_r = aligned16(F.residual) && F.ldr * el % 16 == 0;
  P.vec_y = aligned16(F.y) && F.ldy * el % 16 == 0;
  const int box = gated ? 64 : 128;
  if (!encode_rows(&P.x_map, F.x, false, F.K, F.T, F.ldx * 2, 64, plan.nacc / 2) ||
      !encode_rows(&P.w_map, F.w, false, F.K, F.F, (uint64_t)F.K * 2, 64, box) ||
      (gated && !encode_rows(&P.w2_map, F.w2, false, F.K, F.F, (uint64_t)F.K * 2, 64, box)))
    return ER_ECUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * plan.clusters);
  cfg.blockDim = dim3(DN_THREADS);
  cfg.dynamicSmemBytes = DN_SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kColumns[gated ? 1 : 0][F.act], P) != cudaSuccess) return ER_ECUDA;
  count_launches(1);
  return launch_status();
}

int launch_dense(const FusedParams& F, int32_t* err, cudaStream_t st) {
  const bool gated = F.w2 != nullptr;
  Room room;
  const int rc = dense_attributes(room);
  if (rc != ER_OK) return rc;
  const DensePlan plan = choose_plan(F.T, F.F, F.K, gated, room);
  if (plan.BN == 0) return launch_columns(F, plan, err, st);
  DenseParams P{};
  P.f = F;
  const int FT = gated ? plan.BN / 2 : plan.BN;
  P.n_m = (F.T + 255) / 256;
  P.n_n = (F.F + FT - 1) / FT;
  P.KB = (F.K + 127) / 128;
  P.S = plan.S;
  P.err = err;
  const int el = F.f32 ? 4 : 2;
  // a TMA store rounds a clipped row up to 16 bytes
  P.tma_y = plan.S == 1 && aligned16(F.y) && F.ldy * el % 16 == 0 && F.F * el % 16 == 0;
  P.vec_r = aligned16(F.residual) && F.ldr * el % 16 == 0;
  P.vec_y = aligned16(F.y) && F.ldy * el % 16 == 0;
  P.x_rows = F.T >= 128 ? 128 : (F.T + 7) / 8 * 8;
  if (!encode_rows(&P.x_map, F.x, false, F.K, F.T, F.ldx * 2, 64, P.x_rows) ||
      !encode_rows(&P.w_map, F.w, false, F.K, F.F, (uint64_t)F.K * 2, 64, plan.BN / 2) ||
      (gated && !encode_rows(&P.w2_map, F.w2, false, F.K, F.F, (uint64_t)F.K * 2, 64, plan.BN / 2)) ||
      (P.tma_y && !encode_rows(&P.y_map, F.y, F.f32, F.F, F.T, F.ldy * el, 128 / el, 32)))
    return ER_ECUDA;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = dense_config(attr, plan.clusters, plan.S, st);
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kDense[gated ? 0 : plan.BN == 256 ? 1 : 2][F.act], P);
  if (e != cudaSuccess) return ER_ECUDA;
  count_launches(1);
  return launch_status();
}

int launch_fused(const FusedParams& P, int32_t* err, cudaStream_t st) {
  if (P.T <= FV_TOKENS) return P.w2 ? launch_few<true>(P, st) : launch_few<false>(P, st);
  return launch_dense(P, err, st);
}

bool sizes_ok(int32_t T, int32_t F, int32_t K, int32_t ldx, int32_t act, int32_t y_fp32,
              int32_t ldy) {
  constexpr int32_t kMost = 1 << 30;  // tile corners stay within 32 bits
  return T >= 0 && T <= kMost && F >= 1 && F <= kMost && K >= 8 && K <= kMost && K % 8 == 0 &&
         ldx >= K && ldx % 8 == 0 && ldy >= F && act >= ER_ACT_NONE &&
         act <= ER_ACT_GELU_TANH && (y_fp32 == 0 || y_fp32 == 1);
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
      ((uintptr_t)residual & el) || ((uintptr_t)bias & 1u) || y == x || y == w || y == bias ||
      (residual == y && ldr != ldy && T > 1))
    return ER_EINVAL;
  FusedParams P{x, w, nullptr, bias, residual, y, T, F, K, ldx, ldr, ldy, act, y_fp32};
  int32_t* err = dev_error ? dev_error : call_error_word();
  if (!err) return ER_ECUDA;
  return launch_fused(P, err, (cudaStream_t)stream);
}

int er_gated_linear(const er_bf16* x, int32_t ldx, int32_t T, const er_bf16* w_gate,
                    const er_bf16* w_up, int32_t F, int32_t K, int32_t act, void* y,
                    int32_t y_fp32, int32_t ldy, int32_t* dev_error, er_stream_t stream) {
  if (!sizes_ok(T, F, K, ldx, act, y_fp32, ldy)) return ER_EINVAL;
  if (T == 0) return ER_OK;
  if (!x || !w_gate || !w_up || !y || !aligned16(x) || !aligned16(w_gate) || !aligned16(w_up) ||
      ((uintptr_t)y & (y_fp32 ? 3u : 1u)) || y == x || y == w_gate || y == w_up)
    return ER_EINVAL;
  FusedParams P{x, w_gate, w_up, nullptr, nullptr, y, T, F, K, ldx, 0, ldy, act, y_fp32};
  int32_t* err = dev_error ? dev_error : call_error_word();
  if (!err) return ER_ECUDA;
  return launch_fused(P, err, (cudaStream_t)stream);
}

}  // extern "C"
