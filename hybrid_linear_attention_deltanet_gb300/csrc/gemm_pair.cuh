// Matrix products on the tensor cores with CTA pairs (tcgen05, cta_group::2),
// C[m][n] = sum_k A[m][k] B[n][k], and what follows them in the epilogue.
//
// A cluster of two CTAs computes a 256 x 256 tile of C: the even CTA the rows
// 0..127, the odd one the rows 128..255, each with all 256 columns in its
// tensor memory.  Per block of 128 bytes of K each CTA fetches its own 128
// rows of A and its own 128 of B's 256 rows (TMA, 128-byte swizzle) and the
// even CTA's one MMA thread multiplies all of it: 32 KB into each SM for
// 512 tensor cycles, half of what two single-CTA 128 x 256 tiles would fetch.
//
// Roles (12 warps): warp 0 fetches, warp 1 multiplies (even CTA only), warp 2
// owns the tensor memory, warps 4..11 take the accumulators out.  The grid is
// persistent and the tensor memory holds two accumulators, so a tile's
// epilogue runs while the next tile is multiplied.
//
// bf16 operands accumulate a whole tile in tensor memory.  8-bit operands
// carry one scale for every 128 elements of K, so there each K block is an
// accumulator of its own, which the epilogue warps scale and add into 128
// fp32 registers a thread while the next block is multiplied.
//
// Every wait has a limit: a wait that runs out flags GDN_ERR_TIMEOUT, and the
// CTA leaves after its copies and products in flight have had time to end.
#pragma once

#include <string.h>

#include "gdn_internal.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace gemm {

using namespace sm100;

// What the epilogue does with a tile.
enum Epilogue : int {
  kStore,      // C as bf16
  kStoreF32,   // C as fp32
  kGate,       // columns 0..127 are G, 128..255 U of the same 128 features: act(G) U
  kGateGrad    // the same G and U with dh: dG = dh U act'(G), dU = dh act(G)
};

// One product.  Its rows of A, or its K, may come in two halves with operands
// of their own (the two gradients of the weights; dG Wg + dU Wu).
struct Problem {
  CUtensorMap a[2], b[2];
  int32_t m_half;       // tiles of rows in each half of A (all of them: one half)
  int32_t m_tiles, n_tiles;
  int32_t k_half;       // K blocks in each half of K (all of them: one half)
  int32_t k_blocks;
  int32_t a_mn, b_mn;   // operand stored with its rows contiguous instead of its K
  int32_t M, N;         // valid rows (of each half) and columns
  void* out[2];
  int64_t ldc;
};

struct PairArgs {
  Problem p[2];
  int32_t problems;
  int32_t group_m;      // tiles of rows whose columns are visited together (L2 reuse)
  int32_t wide;         // outputs and row pitches are 32-byte aligned
  int32_t act;
  const __nv_bfloat16* dh;   // kGateGrad: [M][ldh]
  int64_t ldh;
  int32_t dh_wide;
  const float* sa;      // 8-bit: [M][sblocks] scales of A's rows
  const float* sb;      //        [ceil(N / 128)][sblocks] scales of B's blocks
  int32_t sblocks;
  unsigned* status;
};

constexpr int kPairThreads = 384;
constexpr int kStages = 6;
constexpr uint32_t kOperand = 128 * 128;             // bytes of A (and of B) a stage
constexpr uint32_t kStageBytes = 2 * kOperand;
constexpr uint32_t kPairSmem = kStages * kStageBytes + 1024;
constexpr uint64_t kWaitNs = 2000000000ull;

struct Tile {
  int p, half, m0, n0;   // problem, half of its rows, first row of the half, first column
};

// Tile t: groups of group_m row tiles, all columns of a group before the next
// group, so that the tiles in flight share their operands in L2.
__device__ __forceinline__ Tile tile_at(const PairArgs& g, int t) {
  Tile r;
  r.p = 0;
  const int first = g.p[0].m_tiles * g.p[0].n_tiles;
  if (t >= first) {
    r.p = 1;
    t -= first;
  }
  const Problem& p = g.p[r.p];
  const int per = g.group_m * p.n_tiles, grp = t / per, in = t - grp * per;
  const int left = p.m_tiles - grp * g.group_m, gm = left < g.group_m ? left : g.group_m;
  const int mt = grp * g.group_m + in % gm, nt = in / gm;
  r.half = mt >= p.m_half;
  r.m0 = (mt - (r.half ? p.m_half : 0)) * 256;
  r.n0 = nt * 256;
  return r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 32 bytes to global memory (one whole sector), 32-byte aligned
__device__ __forceinline__ void st32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// 32 consecutive columns of one row, columns past `valid` left out
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&v)[32], int valid,
                                          bool wide) {
  if (wide && valid >= 32) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1]);
    st32(p, w);
    st32(p + 16, w + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < valid) p[i] = __float2bfloat16_rn(v[i]);
  }
}
__device__ __forceinline__ void store_row(float* p, const float (&v)[32], int valid, bool wide) {
  if (wide && valid >= 32) {
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) st32(p + 8 * i, w + 8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < valid) p[i] = v[i];
  }
}

// The gate's activation and its derivative.
__device__ __forceinline__ float gate_sigmoid(float x) {
  return rcp_sfu(__fadd_rn(ex2_sfu(__fmul_rn(x, kNegLog2e)), 1.f));
}
__device__ __forceinline__ float gate_act(float x, int act) {
  const float s = gate_sigmoid(x);
  return act == GDN_GATE_SILU ? x * s : s;
}

template <bool kFp8, int kEpi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_gemm_kernel(const __grid_constant__ PairArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align_smem_1024(smem_raw);
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_base;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);    // the even CTA's expect_tx (both CTAs' bytes)
      mbar_init(&empty[i], 1);   // a commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);   // both CTAs' epilogue warps
    }
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc_pair(&tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // both CTAs' barriers exist before either uses the other's
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int n_tiles =
      g.p[0].m_tiles * g.p[0].n_tiles + (g.problems > 1 ? g.p[1].m_tiles * g.p[1].n_tiles : 0);
  const int t0 = blockIdx.x >> 1, step = gridDim.x >> 1;
  bool ok = true;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------- fetch
    int st = 0;
    uint32_t ph = 0;
    for (int t = t0; t < n_tiles && ok; t += step) {
      const Tile tl = tile_at(g, t);
      const Problem& p = g.p[tl.p];
      const int m0 = tl.m0 + 128 * (int)rank;
      // gated: both CTAs' halves of B are the same 128 features of Wg and Wu
      const int n0 = kEpi >= kGate ? tl.n0 / 2 : tl.n0 + 128 * (int)rank;
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        ok = mbar_wait(&empty[st], ph ^ 1u, kWaitNs);
        if (!ok) break;
        uint8_t* A = sm + st * kStageBytes;
        uint8_t* B = A + kOperand;
        if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * kStageBytes);
        const uint32_t bar = mapa_smem(&full[st], 0);
        const int h = kb >= p.k_half;
        const int k0 = (kb - (h ? p.k_half : 0)) * (kFp8 ? 128 : 64);
        const CUtensorMap* am = &p.a[h | tl.half];
        const CUtensorMap* bm = &p.b[kEpi >= kGate ? (int)rank : h];
        if (!kFp8 && p.a_mn) {
          tma_load_2d_pair(A, am, m0, k0, bar);
          tma_load_2d_pair(A + 8192, am, m0 + 64, k0, bar);
        } else {
          tma_load_2d_pair(A, am, k0, m0, bar);
        }
        if (!kFp8 && p.b_mn) {
          tma_load_2d_pair(B, bm, n0, k0, bar);
          tma_load_2d_pair(B + 8192, bm, n0 + 64, k0, bar);
        } else {
          tma_load_2d_pair(B, bm, k0, n0, bar);
        }
        if (++st == kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // -------------------------------------------------------- multiply
    int st = 0, buf = 0;
    uint32_t ph = 0, aph = 0;
    for (int t = t0; t < n_tiles && ok; t += step) {
      const Problem& p = g.p[tile_at(g, t).p];
      const uint32_t idesc =
          kFp8 ? idesc_e4m3(256, 256) : idesc_bf16(256, 256, p.a_mn, p.b_mn);
      // a K-major block advances 32 bytes an instruction inside the swizzled
      // row; one stored by rows advances 16 rows of K (2048 bytes)
      const uint32_t a_step = p.a_mn ? 2048 : 32, b_step = p.b_mn ? 2048 : 32;
      const uint32_t a_lbo = p.a_mn ? 8192 : 16, b_lbo = p.b_mn ? 8192 : 16;
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        const bool first = kFp8 || kb == 0, last = kFp8 || kb + 1 == p.k_blocks;
        if (first) {
          ok = mbar_wait(&acc_empty[buf], aph ^ 1u, kWaitNs);
          if (!ok) break;
        }
        ok = mbar_wait(&full[st], ph, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t A = smem_u32(sm + st * kStageBytes), B = A + kOperand;
        const uint32_t d = tmem + 256 * buf;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t ad = smem_desc(A + i * a_step, a_lbo, 1024, kSwizzle128B);
          const uint64_t bd = smem_desc(B + i * b_step, b_lbo, 1024, kSwizzle128B);
          if (kFp8) mma_f8_pair(d, ad, bd, idesc, i != 0);
          else mma_bf16_pair(d, ad, bd, idesc, !first || i != 0);
        }
        mma_commit_pair(&empty[st]);
        if (last) {
          mma_commit_pair(&acc_full[buf]);
          buf ^= 1;
          if (buf == 0) aph ^= 1u;
        }
        if (++st == kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t free_bar[2] = {mapa_smem(&acc_empty[0], 0), mapa_smem(&acc_empty[1], 0)};
    int buf = 0;
    uint32_t aph = 0;
    for (int t = t0; t < n_tiles && ok; t += step) {
      const Tile tl = tile_at(g, t);
      const Problem& p = g.p[tl.p];
      const int row = tl.m0 + 128 * (int)rank + 32 * q + lane;
      const bool live = row < p.M;
      if constexpr (kFp8) {
        // this thread's 128 columns belong to one block of the weights' scales
        const int n0 = tl.n0 + 128 * half;
        const float* sa = g.sa + (size_t)(live ? row : 0) * g.sblocks;
        const float* sb = g.sb + (size_t)(n0 < p.N ? n0 / 128 : 0) * g.sblocks;
        float acc[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) acc[i] = 0.f;
        float s = __ldg(sa) * __ldg(sb);
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          ok = mbar_wait(&acc_full[buf], aph, kWaitNs);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const float sn = kb + 1 < p.k_blocks ? __ldg(sa + kb + 1) * __ldg(sb + kb + 1) : 0.f;
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            uint32_t r[32];
            tmem_ld32(tmem + lanes + 256 * buf + 128 * half + c, r);
            tmem_ld_wait_regs(r);
            if (c == 96) {   // all of this warp's columns are out
              tc_fence_before();
              if (lane == 0) mbar_arrive_cluster(free_bar[buf]);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c + i] = fmaf(__uint_as_float(r[i]), s, acc[c + i]);
          }
          s = sn;
          buf ^= 1;
          if (buf == 0) aph ^= 1u;
        }
        if (!ok) break;
        if (live) {
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = acc[c + i];
            if (n0 + c < p.N) {
              const size_t o = (size_t)row * p.ldc + n0 + c;
              if (kEpi == kStoreF32) store_row((float*)p.out[0] + o, v, p.N - n0 - c, g.wide);
              else store_row((__nv_bfloat16*)p.out[0] + o, v, p.N - n0 - c, g.wide);
            }
          }
        }
      } else if constexpr (kEpi == kStore) {
        ok = mbar_wait(&acc_full[buf], aph, kWaitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t r[32];
          tmem_ld32(tmem + lanes + 256 * buf + 128 * half + c, r);
          tmem_ld_wait_regs(r);
          if (c == 96) {
            tc_fence_before();
            if (lane == 0) mbar_arrive_cluster(free_bar[buf]);
          }
          const int n = tl.n0 + 128 * half + c;
          if (live && n < p.N) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            store_row((__nv_bfloat16*)p.out[tl.half] + (size_t)row * p.ldc + n, v, p.N - n,
                      g.wide);
          }
        }
        buf ^= 1;
        if (buf == 0) aph ^= 1u;
      } else {
        // this thread's 64 features
        const int f0 = tl.n0 / 2 + 64 * half;
        uint32_t dh[kEpi == kGateGrad ? 32 : 1];   // 64 bf16, fetched before the wait
        if constexpr (kEpi == kGateGrad) {
          const __nv_bfloat16* d = g.dh + (size_t)(live ? row : 0) * g.ldh + f0;
          if (live && g.dh_wide && f0 + 64 <= p.N) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 w = __ldg(reinterpret_cast<const uint4*>(d) + i);
              dh[4 * i] = w.x; dh[4 * i + 1] = w.y; dh[4 * i + 2] = w.z; dh[4 * i + 3] = w.w;
            }
          } else {
            const unsigned short* u = reinterpret_cast<const unsigned short*>(d);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              uint32_t lo = 0, hi = 0;
              if (live && f0 + 2 * i < p.N) lo = __ldg(u + 2 * i);
              if (live && f0 + 2 * i + 1 < p.N) hi = __ldg(u + 2 * i + 1);
              dh[i] = lo | (hi << 16);
            }
          }
        }
        ok = mbar_wait(&acc_full[buf], aph, kWaitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t G[32], U[32];
          tmem_ld32(tmem + lanes + 256 * buf + 64 * half + c, G);
          tmem_ld32(tmem + lanes + 256 * buf + 128 + 64 * half + c, U);
          tmem_ld_wait_regs(G);
          tmem_ld_wait_regs(U);
          if (c == 32) {
            tc_fence_before();
            if (lane == 0) mbar_arrive_cluster(free_bar[buf]);
          }
          const int f = f0 + c;
          if (live && f < p.N) {
            const size_t o = (size_t)row * p.ldc + f;
            float v[32];
            if constexpr (kEpi == kGate) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                v[i] = gate_act(__uint_as_float(G[i]), g.act) * __uint_as_float(U[i]);
              store_row((__nv_bfloat16*)p.out[0] + o, v, p.N - f, g.wide);
            } else {
              float w[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const uint32_t d2 = dh[(c + i) >> 1];
                const float d = __uint_as_float((i & 1) ? d2 & 0xffff0000u : d2 << 16);
                const float x = __uint_as_float(G[i]), s = gate_sigmoid(x);
                const bool silu = g.act == GDN_GATE_SILU;
                const float slope = silu ? s * fmaf(x, 1.f - s, 1.f) : s * (1.f - s);
                v[i] = d * __uint_as_float(U[i]) * slope;
                w[i] = d * (silu ? x * s : s);
              }
              store_row((__nv_bfloat16*)p.out[0] + o, v, p.N - f, g.wide);
              store_row((__nv_bfloat16*)p.out[1] + o, w, p.N - f, g.wide);
            }
          }
        }
        buf ^= 1;
        if (buf == 0) aph ^= 1u;
      }
    }
  }
  if (!ok) {
    // copies and products in flight end within microseconds; give them longer
    flag_status(g.status, GDN_ERR_TIMEOUT);
    const uint64_t from = globaltimer_ns();
    while (globaltimer_ns() - from < 5000000ull) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // no CTA leaves while the other may still signal it
  if (warp == 2) tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------- host side
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// A matrix of `outer` rows of `inner` elements, `pitch` bytes apart, read in
// boxes of 128 bytes x box_rows rows with the 128-byte swizzle; what lies
// past its edges reads as zero.  Coordinates of the box start on 128 bytes.
inline bool matrix_map(CUtensorMap* m, const void* base, bool fp8, int64_t inner, int64_t outer,
                       int64_t pitch, uint32_t box_rows) {
  EncodeFn enc = encoder();
  if (!enc) return false;
  memset(m, 0, sizeof *m);
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)pitch};
  cuuint32_t box[2] = {fp8 ? 128u : 64u, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFp8, int kEpi>
cudaError_t launch_pair(const PairArgs& g, int sms, cudaStream_t st) {
  auto kern = pair_gemm_kernel<kFp8, kEpi>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem);
  if (e != cudaSuccess) return e;
  int64_t tiles = 0;
  for (int i = 0; i < g.problems; ++i) tiles += (int64_t)g.p[i].m_tiles * g.p[i].n_tiles;
  const int64_t pairs = sms / 2;
  kern<<<(unsigned)(2 * (tiles < pairs ? tiles : pairs)), kPairThreads, kPairSmem, st>>>(g);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace gemm
}  // namespace gdn
