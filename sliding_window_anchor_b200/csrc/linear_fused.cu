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

// One output value from its sums: v (+ u, the gated product's second one).
__device__ __forceinline__ float finish(const FusedParams& P, float v, float u, bool gated, int t,
                                        int f) {
  if (P.bias) v += bf1(P.bias[f]);
  v = activate(v, P.act);
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

__device__ __forceinline__ void activate32(float (&v)[32], int act) {
  // one branch for the 32 values
  if (act == ER_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = activate(v[i], ER_ACT_SILU);
  } else if (act == ER_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = activate(v[i], ER_ACT_GELU);
  } else if (act == ER_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = activate(v[i], ER_ACT_GELU_TANH);
  }
}

// Bias of features f..f+31 (the same for every lane).
__device__ __forceinline__ void add_bias32(float (&v)[32], const FusedParams& P, int f) {
  if (!P.bias) return;
  if (((uintptr_t)P.bias & 15u) == 0 && f + 32 <= P.F) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 b = __ldg(reinterpret_cast<const uint4*>(P.bias + f) + i);
      v[8 * i] += bf_lo(b.x), v[8 * i + 1] += bf_hi(b.x);
      v[8 * i + 2] += bf_lo(b.y), v[8 * i + 3] += bf_hi(b.y);
      v[8 * i + 4] += bf_lo(b.z), v[8 * i + 5] += bf_hi(b.z);
      v[8 * i + 6] += bf_lo(b.w), v[8 * i + 7] += bf_hi(b.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (f + i < P.F) v[i] += bf1(P.bias[f + i]);
  }
}

// Residual of token t, features f..f+31.  Plain loads: it may be y itself.
__device__ __forceinline__ void add_residual32(float (&v)[32], const FusedParams& P, bool vec,
                                               int t, int f) {
  if (!P.residual) return;
  if (P.f32) {
    const float* r = static_cast<const float*>(P.residual) + t * P.ldr + f;
    if (vec && f + 32 <= P.F) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 b = reinterpret_cast<const float4*>(r)[i];
        v[4 * i] += b.x, v[4 * i + 1] += b.y, v[4 * i + 2] += b.z, v[4 * i + 3] += b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (f + i < P.F) v[i] += r[i];
    }
  } else {
    const uint16_t* r = static_cast<const uint16_t*>(P.residual) + t * P.ldr + f;
    if (vec && f + 32 <= P.F) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 b = reinterpret_cast<const uint4*>(r)[i];
        v[8 * i] += bf_lo(b.x), v[8 * i + 1] += bf_hi(b.x);
        v[8 * i + 2] += bf_lo(b.y), v[8 * i + 3] += bf_hi(b.y);
        v[8 * i + 4] += bf_lo(b.z), v[8 * i + 5] += bf_hi(b.z);
        v[8 * i + 6] += bf_lo(b.w), v[8 * i + 7] += bf_hi(b.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
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
// matter).  The K slices of a block's warps are added in a fixed order.
constexpr int FV_TOKENS = 8;
constexpr int FV_MAXW = 8;

__device__ __forceinline__ uint4 ld_weights(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
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
__global__ void __launch_bounds__(32 * FV_MAXW) k_fused_few(const FusedParams P) {
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
  for (int k0 = k_lo; k0 < k_hi; k0 += U) {
    uint4 a[NW][U], b[NW][U], x[U];
    // every load is issued; one outside the slice or K takes the row's start, and zero
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = 32 * (k0 + u) + 8 * c;
      const bool in = k0 + u < k_hi && k < P.K;
      const int at = in ? k : 0;
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        a[n][u] = ld_weights(wp[n] + ra + at);
        b[n][u] = ld_weights(wp[n] + rb + at);
      }
      x[u] = __ldg(reinterpret_cast<const uint4*>(xp + at));
      if (!in || g >= P.T) x[u] = z;
      if (!in) {
#pragma unroll
        for (int n = 0; n < NW; ++n) a[n][u] = b[n][u] = z;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        mma16816(acc[n], a[n][u].x, b[n][u].x, a[n][u].y, b[n][u].y, x[u].x, x[u].y);
        mma16816(acc[n], a[n][u].z, b[n][u].z, a[n][u].w, b[n][u].w, x[u].z, x[u].w);
      }
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
    store_one(P, t, f, finish(P, v, u, GATED, t, f));
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
// CTA's TMEM lanes) by BN weight rows, K in steps of 64 through a ring of TMA
// stages.  Of a step each CTA fetches its 128 tokens and half of the BN
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
  CUtensorMap x_map;        // x [T][K], box 64 x 128
  CUtensorMap w_map, w2_map;  // weights [F][K], box 64 x BN/2
  CUtensorMap y_map;        // y [T][F], box 128 bytes x 32 rows (when tma_y)
  FusedParams f;
  int n_m, n_n, KB, S;
  int tma_y;
  int vec_r;                // residual rows in 16-byte loads
  int32_t* err;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
  float4 r;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(a)
               : "memory");
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

template <int BN, bool GATED>
__global__ void __launch_bounds__(DN_THREADS, 1) k_dense(const __grid_constant__ DenseParams P) {
  constexpr int FT = GATED ? BN / 2 : BN;  // features of a tile
  constexpr int B_BYTES = BN / 2 * 128;
  constexpr int STAGE = DN_A_BYTES + B_BYTES;
  constexpr int NST = (DN_SMEM - 2048 - DN_STAGING) / STAGE < DN_MAXST
                          ? (DN_SMEM - 2048 - DN_STAGING) / STAGE
                          : DN_MAXST;
  static_assert(NST * STAGE >= 128 * BN * 4, "a share's sums fit in the stages");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  struct Bars {
    uint64_t full[NST], empty[NST], tfull[2], tempty[2], done;
    uint32_t tmem_base;
    volatile int failed;
  };
  unsigned char* staging = base + NST * STAGE;
  Bars& B = *reinterpret_cast<Bars*>(staging + DN_STAGING);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = tc::cluster_rank();
  const uint32_t lead = crank & ~1u, peer = crank ^ 1u;
  const int rank = crank & 1, share = crank >> 1;
  const int n_tiles = P.n_m * P.n_n;
  const int n_clusters = gridDim.x / (2 * P.S), cluster = blockIdx.x / (2 * P.S);
  const int kb0 = P.KB * share / P.S, kb1 = P.KB * (share + 1) / P.S;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&B.full[s], 2);   // each CTA's arrival with its byte count
      mbar_init(&B.empty[s], 1);  // the MMAs that read the stage have completed
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&B.tfull[b], 1);
      mbar_init(&B.tempty[b], 16);  // the epilogue warps of both CTAs
    }
    mbar_init(&B.done, 1);
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
    if (lane == 0) {
      int step = 0;
      const CUtensorMap* wm = GATED && rank ? &P.w2_map : &P.w_map;
      for (int tile = cluster; tile < n_tiles && !B.failed; tile += n_clusters) {
        int m, n;
        tile_at(P, tile, m, n);
        const int t0 = 256 * m + 128 * rank;
        const int f0 = FT * n + (GATED ? 0 : BN / 2 * rank);
        for (int kb = kb0; kb < kb1; ++kb, ++step) {
          const int s = step % NST;
          if (!mbar_wait(&B.empty[s], ((step / NST) & 1) ^ 1, P.err)) {
            B.failed = 1;
            break;
          }
          unsigned char* st = base + (size_t)s * STAGE;
          const uint32_t fb = tc::map_to_rank(&B.full[s], lead);
          tc::mbar_arrive_expect_tx_cluster(fb, STAGE);
          tc::tma_load_2d_pair(st + DN_A_BYTES, wm, 64 * kb, f0, fb);
          tc::tma_load_2d_pair(st, &P.x_map, 64 * kb, t0, fb);
        }
      }
    }
  } else if (warp == 9) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t id = tc::idesc_bf16(256, BN, false, false);
      int step = 0, it = 0;
      bool ok = true;
      for (int tile = cluster; tile < n_tiles && ok && !B.failed; tile += n_clusters, ++it) {
        const int b = it & 1;
        ok = mbar_wait(&B.tempty[b], ((it >> 1) & 1) ^ 1, P.err);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t d = tmem + BN * b;
        for (int kb = kb0; kb < kb1; ++kb, ++step) {
          const int s = step % NST;
          ok = mbar_wait(&B.full[s], (step / NST) & 1, P.err);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t a0 = smem_u32(base + (size_t)s * STAGE), b0 = a0 + DN_A_BYTES;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_pair_bf16_ss(d, tc::desc_sw128(a0 + 32 * kk, 16, 1024),
                                 tc::desc_sw128(b0 + 32 * kk, 16, 1024), id,
                                 (kb > kb0 || kk > 0) ? 1u : 0u);
          tc::commit_pair(tc::map_to_rank(&B.empty[s], crank));
          tc::commit_pair(tc::map_to_rank(&B.empty[s], peer));
        }
        if (!ok) break;
        tc::commit_pair(tc::map_to_rank(&B.tfull[b], crank));
        tc::commit_pair(tc::map_to_rank(&B.tfull[b], peer));
      }
      if (!ok) B.failed = 1;
      tc::commit_pair(tc::map_to_rank(&B.done, crank));
      mbar_wait(&B.done, 0, P.err);  // nothing of the pair's is on the tensor cores at exit
    }
  } else {
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    if (P.S == 1) {
      unsigned char* stg = staging + 4096 * warp;
      int it = 0;
      for (int tile = cluster; tile < n_tiles; tile += n_clusters, ++it) {
        const int b = it & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&B.tfull[b], (it >> 1) & 1, P.err)) || B.failed) {
          B.failed = 1;
          break;
        }
        tc::fence_after_sync();
        int m, n;
        tile_at(P, tile, m, n);
        const int t0 = 256 * m + 128 * rank + 32 * quad, t = t0 + lane;
        constexpr int NC = FT / 64;  // blocks of 32 columns in this warp's half
#pragma unroll 1
        for (int cb = 0; cb < NC; ++cb) {
          const int col = FT / 2 * half + 32 * cb, f = FT * n + col;
          uint32_t r[32], u[GATED ? 32 : 1];
          tc::tmem_ld32(tmem + lanes + BN * b + col, r);
          if constexpr (GATED) tc::tmem_ld32(tmem + lanes + BN * b + FT + col, u);
          tc::tmem_wait_ld();
          if (t0 >= P.f.T || f >= P.f.F) continue;  // no row, no column of y
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          if constexpr (GATED) {
            activate32(v, P.f.act);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= __uint_as_float(u[i]);
          } else {
            add_bias32(v, P.f, f);
            activate32(v, P.f.act);
            if (t < P.f.T) add_residual32(v, P.f, P.vec_r, t, f);
          }
          // the block into the warp's staging rows of 128 bytes (chunk c of row l
          // at c ^ l % 8), whole rows out: FP32 per block, BF16 per two blocks
          const bool f32 = P.f.f32;
          const bool first = f32 || (cb & 1) == 0;
          if (first) {
            if (lane == 0) tc::bulk_wait_read<0>();
            __syncwarp();
          }
          if (f32) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(stg + 128 * lane + 16 * (i ^ (lane & 7))) =
                  make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 o;
              o.x = pack_bf2(v[8 * i], v[8 * i + 1]);
              o.y = pack_bf2(v[8 * i + 2], v[8 * i + 3]);
              o.z = pack_bf2(v[8 * i + 4], v[8 * i + 5]);
              o.w = pack_bf2(v[8 * i + 6], v[8 * i + 7]);
              *reinterpret_cast<uint4*>(stg + 128 * lane +
                                        16 * ((4 * (cb & 1) + i) ^ (lane & 7))) = o;
            }
          }
          const bool last = f32 || (cb & 1) || f + 32 >= P.f.F;
          if (!last) continue;
          if (P.tma_y) {
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tc::tma_store_2d(&P.y_map, f32 ? f : f - 32 * (cb & 1), t0, stg);
              tc::bulk_commit();
            }
          } else {
            __syncwarp();
            copy_rows(P.f, stg, t0, f32 ? f : f - 32 * (cb & 1), f32 ? 32 : 32 + 32 * (cb & 1),
                      lane);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(tc::map_to_rank(&B.tempty[b], lead));
      }
      if (lane == 0) tc::bulk_wait_all();
    } else {
      // this share's sums: [128 tokens][BN], 16-byte chunk c of row t at c ^ t % 8
      const bool ok = mbar_wait(&B.tfull[0], 0, P.err);
      if (!ok) B.failed = 1;
      tc::fence_after_sync();
      const int row = 32 * quad + lane;
      if (__all_sync(0xffffffffu, ok)) {
        float* sums = reinterpret_cast<float*>(base);
#pragma unroll 1
        for (int cb = 0; cb < BN / 64; ++cb) {
          const int col = BN / 2 * half + 32 * cb;
          uint32_t r[32];
          tc::tmem_ld32(tmem + lanes + col, r);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(sums + BN * row + 4 * ((col / 4 + i) ^ (row & 7))) =
                make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
      }
      tc::fence_before_sync();
    }
  }
  if (P.S > 1) {
    tc::cluster_sync();  // every share's sums are in place
    int m, n;
    tile_at(P, cluster, m, n);
    const int t0 = 256 * m + 128 * rank;
    const int rows = min(128, P.f.T - t0);
    if (threadIdx.x < DN_EPI && rows > 0 && !B.failed) {
      const uint32_t mine = smem_u32(base);
      uint32_t at[4];
      for (int p = 0; p < 4; ++p)
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(at[p])
                     : "r"(mine), "r"(2 * min(p, P.S - 1) + rank));
      constexpr int GR = FT / 4;  // groups of four features in a row
      for (int i = share * DN_EPI + threadIdx.x; i < rows * GR; i += P.S * DN_EPI) {
        const int row = i / GR, c = i % GR;
        const int f = FT * n + 4 * c;
        if (f >= P.f.F) continue;
        float v[4] = {}, u[4] = {};
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if (p >= P.S) break;
          const float4 a = ld_cluster_f4(at[p] + 4 * (BN * row + 4 * (c ^ (row & 7))));
          v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
          if (GATED) {
            const float4 b = ld_cluster_f4(at[p] + 4 * (BN * row + 4 * ((GR + c) ^ (row & 7))));
            u[0] += b.x, u[1] += b.y, u[2] += b.z, u[3] += b.w;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (f + j < P.f.F)
            store_one(P.f, t0 + row, f + j, finish(P.f, v[j], u[j], GATED, t0 + row, f + j));
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

struct DensePlan {
  int BN, S, clusters;
};

// The tile width and the shares of K, by the estimated cycles of a pair.  A K step
// costs the longer of its MMAs (2 BN cycles) and its fetches (one SM takes about
// 65 bytes per cycle from L2, about 24 of them when they come from HBM).
DensePlan choose_plan(int T, int F, int K, bool gated) {
  const int pairs = num_sms() / 2, KB = (K + 63) / 64, n_m = (T + 255) / 256;
  DensePlan best{256, 1, 1};
  double least = 1e300;
  for (int BN : {256, 128}) {
    if (gated && BN != 256) continue;
    const int FT = gated ? BN / 2 : BN, tiles = n_m * ((F + FT - 1) / FT);
    for (int S = 1; S <= 4 && S <= KB; ++S) {
      if (S > 1 && tiles * S > pairs) break;
      const double mma = 2.0 * BN, fetch = (DN_A_BYTES + 64.0 * BN) / 65.0;
      const double hbm = n_m == 1 ? 64.0 * BN / 24.0 : 0.0;
      const double step = mma > fetch ? (mma > hbm ? mma : hbm) : (fetch > hbm ? fetch : hbm);
      const int clusters = S > 1 ? tiles : (tiles < pairs ? tiles : pairs);
      const int waves = (tiles + clusters - 1) / clusters;
      const double cost = waves * ((KB + S - 1) / S) * step + (S > 1 ? 3000.0 : 1500.0);
      if (cost < least) {
        least = cost;
        best = DensePlan{BN, S, clusters};
      }
    }
  }
  return best;
}

std::mutex g_attr_mu;
bool g_attr_done[64] = {false};

int dense_attributes() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ER_ECUDA;
  std::lock_guard<std::mutex> lock(g_attr_mu);
  if (g_attr_done[dev]) return ER_OK;
  for (auto* fn : {k_dense<256, false>, k_dense<128, false>, k_dense<256, true>})
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, DN_SMEM) !=
        cudaSuccess)
      return ER_ECUDA;
  g_attr_done[dev] = true;
  return ER_OK;
}

int launch_dense(const FusedParams& F, int32_t* err, cudaStream_t st) {
  const bool gated = F.w2 != nullptr;
  const DensePlan plan = choose_plan(F.T, F.F, F.K, gated);
  DenseParams P{};
  P.f = F;
  const int FT = gated ? plan.BN / 2 : plan.BN;
  P.n_m = (F.T + 255) / 256;
  P.n_n = (F.F + FT - 1) / FT;
  P.KB = (F.K + 63) / 64;
  P.S = plan.S;
  P.err = err;
  const int el = F.f32 ? 4 : 2;
  // a TMA store rounds a clipped row up to 16 bytes
  P.tma_y = plan.S == 1 && aligned16(F.y) && F.ldy * el % 16 == 0 && F.F * el % 16 == 0;
  P.vec_r = aligned16(F.residual) && F.ldr * el % 16 == 0;
  if (!encode_rows(&P.x_map, F.x, false, F.K, F.T, F.ldx * 2, 64, 128) ||
      !encode_rows(&P.w_map, F.w, false, F.K, F.F, (uint64_t)F.K * 2, 64, plan.BN / 2) ||
      (gated && !encode_rows(&P.w2_map, F.w2, false, F.K, F.F, (uint64_t)F.K * 2, 64, plan.BN / 2)) ||
      (P.tma_y && !encode_rows(&P.y_map, F.y, F.f32, F.F, F.T, F.ldy * el, 128 / el, 32)))
    return ER_ECUDA;
  const int rc = dense_attributes();
  if (rc != ER_OK) return rc;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * plan.S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.clusters * 2 * plan.S);
  cfg.blockDim = dim3(DN_THREADS);
  cfg.dynamicSmemBytes = DN_SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = gated ? cudaLaunchKernelEx(&cfg, k_dense<256, true>, P)
                        : plan.BN == 256 ? cudaLaunchKernelEx(&cfg, k_dense<256, false>, P)
                                         : cudaLaunchKernelEx(&cfg, k_dense<128, false>, P);
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
  return T >= 0 && T <= kMost && F >= 1 && F <= kMost && K >= 8 && K <= kMost && K % 8 == 0 && ldx >= K && ldx % 8 == 0 && ldy >= F &&
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
      ((uintptr_t)y & (y_fp32 ? 3u : 1u)))
    return ER_EINVAL;
  FusedParams P{x, w_gate, w_up, nullptr, nullptr, y, T, F, K, ldx, 0, ldy, act, y_fp32};
  int32_t* err = dev_error ? dev_error : call_error_word();
  if (!err) return ER_ECUDA;
  return launch_fused(P, err, (cudaStream_t)stream);
}

}  // extern "C"
