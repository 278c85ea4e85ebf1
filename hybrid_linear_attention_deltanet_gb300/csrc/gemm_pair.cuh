// Matrix products on the tensor cores with CTA pairs (tcgen05, cta_group::2),
// C[m][n] = sum_k A[m][k] B[n][k], and what follows them in the epilogue.
//
// A cluster of two CTAs computes a 256 x 256 tile of C: the even CTA the rows
// 0..127, the odd one the rows 128..255, each with all 256 columns in its
// tensor memory.  Per block of 128 bytes of K each CTA fetches its own 128
// rows of A and its own 128 of B's 256 rows (TMA, 128-byte swizzle) and the
// even CTA's one MMA thread multiplies all of it: 32 KB into each SM for
// 512 tensor cycles, half of what two single-CTA 128 x 256 tiles would fetch.
// (Gated products take tiles of 192 columns, 8-bit ones of 128, where those fill
// the pairs better.)
//
// Roles: warp 0 fetches, warp 1 multiplies (even CTA only), warp 2 owns the
// tensor memory, warps 4 and up take the accumulators out.  The grid is
// persistent and the tensor memory holds two accumulators, so a tile's
// epilogue runs while the next tile is multiplied.  Results go through shared
// memory, 32 rows x 128 bytes a warp, and leave as TMA stores.
//
// bf16 operands accumulate a whole tile in tensor memory.  8-bit operands carry
// one scale for every 128 elements of K, so there each K block is an
// accumulator of its own, which the 8 epilogue warps scale and add into 128
// fp32 registers a thread while the next block is multiplied.
//
// What it measured (GB300).  bf16: 8192 x 2048 against 2 x 6144 rows keeps the
// tensor pipe 90 % busy (208 us cold); 32768 rows run 890 us at 1.85 PFLOP/s,
// and over seconds 955 us at the 1400 W limit with the SMs at 1.5 GHz, the rate
// of a plain library product there.  8 bits: 32768 x 2048 against 4608 rows
// 233 us, 2.65 PFLOP/s, tensor pipe 50 % busy (900 cycles a K block; 254 us over
// seconds, also at the power limit).  The epilogue's reads of tensor memory
// bound it: they share it with the products' sums and take twice their time
// alone.  (Same product, us: products without epilogue 184; loads and
// multiply-adds running free of any hand-over 254; hand-over without loads and
// multiply-adds 196, without multiply-adds 207.)  Not kept: 16 epilogue warps of
// 64 columns 262, two 128-column halves with four accumulators 250, 16-column
// loads 300, each block's first load before the last one's multiply-adds 262.
//
// Every wait has a limit: a wait that runs out flags GDN_ERR_TIMEOUT, and the
// CTA leaves after its copies and products in flight have had time to end.
#pragma once

#include <string.h>
#include <type_traits>

#include "gdn_internal.cuh"
#include "hostcheck.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace gemm {

using namespace sm100;

// What the epilogue does with a tile.
enum Epilogue : int {
  kStore,      // C as bf16
  kStoreF32,   // C as fp32
  kGate,       // columns of the first half are G, of the second U of the same features: act(G) U
  kGateGrad    // the same G and U with dh: dG = dh U act'(G), dU = dh act(G)
};

// One product.  Its rows of A, or its K, may come in two halves with operands
// of their own (the two gradients of the weights; dG Wg + dU Wu).
struct Problem {
  CUtensorMap a[2], b[2], c[2];
  int32_t c_tma;        // c is valid: rows of the outputs start on 16 bytes
  int32_t m_half;       // tiles of rows in each half of A (all of them: one half)
  int32_t m_tiles, n_tiles;
  int32_t k_half;       // K blocks in each half of K (all of them: one half)
  int32_t k_blocks;
  int32_t a_mn, b_mn;   // operand stored with its rows contiguous instead of its K
  int32_t k_parts;      // tiles share K among this many; more than 1: fp32 sums of each
                        // part at out + part * part_rows * ldc (kStore)
  int32_t part_rows;
  int32_t M, N;         // valid rows (of each half) and columns
  void* out[2];
  int64_t ldc;
};
inline int64_t tiles_of(const Problem& p) {
  return (int64_t)p.m_tiles * p.n_tiles * p.k_parts;
}

struct PairArgs {
  Problem p[2];
  int32_t problems;
  int32_t tiles[2];     // of each problem
  int32_t ahead;        // see tile_of
  int32_t group_m;      // tiles of rows whose columns are visited together (group_rows)
  int32_t act;
  const __nv_bfloat16* dh;   // kGateGrad: [M][ldh]
  int64_t ldh;
  int32_t dh_wide;
  const float* sa;      // 8-bit: [M][sblocks] scales of A's rows
  const float* sb;      //        [ceil(N / 128)][sblocks] scales of B's blocks
  int32_t sblocks;
  unsigned* status;
};

constexpr uint32_t kOperand = 128 * 128;             // bytes of A (and of B) a stage
constexpr uint32_t kStageBytes = 2 * kOperand;
constexpr int kGroup = 4;                            // K blocks whose scales travel together

constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kBounce = 32 * 128;               // a warp's staging: 32 rows x 128 bytes

template <bool kFp8>
struct Shape {
  // two groups of scales [kGroup][2 column blocks][128 rows]
  static constexpr uint32_t kScales = kFp8 ? 2 * kGroup * 256 * 4 : 0;
  static constexpr int kStages = kFp8 ? 5 : 6;       // what 227 KB hold
  static constexpr uint32_t kSmem =
      kStages * kStageBytes + kEpiWarps * kBounce + kScales + 1024;
};
constexpr uint64_t kWaitNs = 2000000000ull;

struct Tile {
  int p, half, m0, n0;   // problem, half of its rows, first row of the half, first column
  int part, k0, k1;      // part of K: its K blocks
};

// The k-th tile of pair i of `pairs`, or -1.  Problem 0, whose tiles are the
// longer, is dealt out first; the pairs that got one tile less of it (from r
// on) then take `ahead` rounds of problem 1 alone, about the time of the tile
// they were spared, and the last rounds reach everyone, those pairs first.
// (Dealing all tiles out in turn left 1111 tokens' gradients with pairs of 79
// and of 36 K blocks; these come to 61 and 54.)
__device__ __forceinline__ int tile_of(const PairArgs& g, int pairs, int i, int k) {
  const int r = g.tiles[0] % pairs, n0 = g.tiles[0] / pairs + (i < r);
  if (k < n0) return k * pairs + i;
  k -= n0;
  const int spared = pairs - r, first = g.ahead * spared;
  const int u = i < r ? first + k * pairs + spared + i
                      : k < g.ahead ? k * spared + i - r : first + (k - g.ahead) * pairs + i - r;
  return u < g.tiles[1] ? g.tiles[0] + u : -1;
}

// Tile t: groups of group_m row tiles, all columns of a group before the next
// group, so that the tiles in flight share their operands in L2.
template <int kTileN>
__device__ __forceinline__ Tile tile_at(const PairArgs& g, int t) {
  Tile r;
  r.p = 0;
  if (t >= g.tiles[0]) {
    r.p = 1;
    t -= g.tiles[0];
  }
  const Problem& p = g.p[r.p];
  r.part = 0;
  r.k0 = 0;
  r.k1 = p.k_blocks;
  if (p.k_parts > 1) {
    const int all = p.m_tiles * p.n_tiles;
    r.part = t / all;
    t -= r.part * all;
    r.k0 = (int)((int64_t)p.k_blocks * r.part / p.k_parts);
    r.k1 = (int)((int64_t)p.k_blocks * (r.part + 1) / p.k_parts);
  }
  const int per = g.group_m * p.n_tiles, grp = t / per, in = t - grp * per;
  const int left = p.m_tiles - grp * g.group_m, gm = left < g.group_m ? left : g.group_m;
  const int mt = grp * g.group_m + in % gm, nt = in / gm;
  r.half = mt >= p.m_half;
  r.m0 = (mt - (r.half ? p.m_half : 0)) * 256;
  r.n0 = nt * kTileN;
  return r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Offset of 16-byte piece `i` of row `r` in a warp's staging image with rows
// of kRow bytes, swizzled as TMA's mode of that many bytes does; lanes that
// write a piece of each row meet no bank conflicts.
template <int kRow = 128>
__device__ __forceinline__ uint32_t stage_piece(uint32_t r, uint32_t i) {
  return r * kRow + (kRow == 128 ? i ^ (r & 7u) : i ^ (r >> 1 & 3u)) * 16;
}
// 32 columns from `c0` of this lane's row into its warp's staging image.
template <typename T, int kRow = 128>
__device__ __forceinline__ void stage_put(uint8_t* buf, int lane, int c0, const float* v) {
  constexpr int kPer = 16 / (int)sizeof(T);   // elements a piece
#pragma unroll
  for (int i = 0; i < 32 / kPer; ++i) {
    uint4 w;
    if constexpr (sizeof(T) == 2)
      w = make_uint4(pack2(v[8 * i], v[8 * i + 1]), pack2(v[8 * i + 2], v[8 * i + 3]),
                     pack2(v[8 * i + 4], v[8 * i + 5]), pack2(v[8 * i + 6], v[8 * i + 7]));
    else
      w = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                     __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
    *reinterpret_cast<uint4*>(buf + stage_piece<kRow>(lane, c0 / kPer + i)) = w;
  }
}
// The staged 32 rows to their place, what lies past the edges of the output
// left out.  stage_free() must return before the next stage_put.  Rows that do
// not start on 16 bytes leave by single stores (32768 tokens, us, beside a width
// that starts on them: 8-bit product, 2048 -> 4609 301 and 4616 251; gated, 2048 ->
// 2 x 6145 930 and 6152 912).
template <typename T, int kRow = 128>
__device__ __forceinline__ void stage_out(const uint8_t* buf, int lane, const Problem& p, int half,
                                          int row0, int n0, int shift = 0) {
  if (row0 >= p.M || n0 >= p.N) return;
  if (p.c_tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&p.c[half], buf, n0, row0 + shift);
      bulk_commit();
    }
  } else {   // rows that start anywhere: a row at a time, 32 elements a step
    __syncwarp();
    constexpr int kCols = kRow / (int)sizeof(T), kPer = 16 / (int)sizeof(T);
    const int rows = p.M - row0 < 32 ? p.M - row0 : 32;
    T* out = (T*)p.out[half] + (size_t)row0 * p.ldc + n0;
#pragma unroll
    for (int i = 0; i < (kCols + 31) / 32; ++i) {
      const int c = lane + 32 * i;
      if (c >= kCols || n0 + c >= p.N) break;
#pragma unroll 8
      for (int r = 0; r < rows; ++r)
        out[(size_t)r * p.ldc + c] = *reinterpret_cast<const T*>(
            buf + stage_piece<kRow>(r, c / kPer) + (c % kPer) * sizeof(T));
    }
  }
}
__device__ __forceinline__ void stage_free(int lane) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
}

// The gate's activation and its derivative.
__device__ __forceinline__ float gate_sigmoid(float x) {
  return rcp_sfu(__fadd_rn(ex2_sfu(__fmul_rn(x, kNegLog2e)), 1.f));
}
__device__ __forceinline__ float gate_act(float x, int act) {
  const float s = gate_sigmoid(x);
  return act == GDN_GATE_SILU ? x * s : s;
}

// dG = dh U act'(G) and dU = dh act(G).  With e = exp(-|G|) and r = 1 / (1 + e)
// the sigmoids of G and of -G are r and e r, either way round: 1 - sigmoid(G)
// taken as a difference has lost a bf16's bits from G = 11 on.
__device__ __forceinline__ void gate_grad(float dh, float G, float U, int act, float& dG,
                                          float& dU) {
  const float e = ex2_sfu(__fmul_rn(fabsf(G), kNegLog2e));
  const float r = rcp_sfu(__fadd_rn(e, 1.f)), er = e * r;
  const float s = G < 0.f ? er : r, c = G < 0.f ? r : er;
  const bool silu = act == GDN_GATE_SILU;
  const float slope = silu ? s * fmaf(G, c, 1.f) : s * c;
  dG = dh * U * slope;
  dU = dh * (silu ? G * s : s);
}

// kTileN: 256 columns, or 192 (gated) or 128 (8 bits), see narrow_gated and
// narrow_fp8.
template <bool kFp8, int kEpi, int kTileN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_gemm_kernel(const __grid_constant__ PairArgs g) {
  constexpr int kStages = Shape<kFp8>::kStages;
  static_assert(kTileN == 256 || (kTileN == 192 && kEpi >= kGate && !kFp8) ||
                    (kTileN == 128 && kFp8), "");
  constexpr int kAccs = kTileN == 128 ? 4 : 2;       // accumulators in tensor memory
  constexpr uint32_t kAccCols = 512 / kAccs;
  // what arrives in both CTAs for a stage
  constexpr uint32_t kArrive = 2 * (kOperand + kOperand / 256 * kTileN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align_smem_1024(smem_raw);
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[kAccs], acc_empty[kAccs];
  __shared__ uint64_t sc_full[2], sc_empty[2];
  __shared__ uint32_t tmem_base;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // known to be uniform
  const uint32_t rank = cluster_ctarank();
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);    // the even CTA's expect_tx (both CTAs' bytes)
      mbar_init(&empty[i], 1);   // a commit
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiWarps);   // both CTAs' epilogue warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sc_full[i], 2);                 // the two warps that fetch scales
      mbar_init(&sc_empty[i], kEpiWarps);
    }
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc_pair(&tmem_base, 512);
  if (warp == 3 && lane == 0) {
    prefetch_tensormap(&g.p[0].a[0]);
    prefetch_tensormap(&g.p[0].b[kEpi >= kGate ? rank : 0]);
    if (g.p[0].c_tma) prefetch_tensormap(&g.p[0].c[0]);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // both CTAs' barriers exist before either uses the other's
  tc_fence_after();
  grid_release_next();
  grid_wait();
  const uint32_t tmem = tmem_base;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  bool ok = true;
  float* scales = reinterpret_cast<float*>(sm + kStages * kStageBytes + kEpiWarps * kBounce);

  // The fetching and the multiplying warp run their loops whole, with one
  // elected lane issuing: every address and descriptor then stays in uniform
  // registers.  (Loops run by one lane alone took 750 cycles a K block against
  // the 512 of its products.)
  if (warp < 4) {
    // 8 bits: 384 threads launch with 168 registers each, 64512 in all, which
    // is 128 x 72 + 256 x 216; the epilogue's 128 sums and 64 arriving columns
    // need more than 168 (32768 x 2048 -> 4608: 233 us with them, 243 without).  Both branches say
    // so themselves: behind a common branch the smaller limit holds for all.
    if constexpr (kFp8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // ---------------------------------------------------------- fetch
      const bool lead = elect_one();
      const uint32_t full0 = mapa_smem(&full[0], 0);   // the even CTA's barriers
      int st = 0;
      uint32_t ph = 0;
      for (int k = 0, t; ok && (t = tile_of(g, pairs, pair, k)) >= 0; ++k) {
        const Tile tl = tile_at<kTileN>(g, t);
        const Problem& p = g.p[tl.p];
        const int m0 = tl.m0 + 128 * (int)rank;
        // gated: both CTAs' halves of B are the same features of Wg and Wu
        const int n0 = kEpi >= kGate ? tl.n0 / 2 : tl.n0 + kTileN / 2 * (int)rank;
        const bool a_mn = !kFp8 && p.a_mn, b_mn = !kFp8 && p.b_mn;
        const int k_half = p.k_half;
        for (int kb = tl.k0; kb < tl.k1; ++kb) {
          ok = mbar_wait_warp(&empty[st], ph ^ 1u, kWaitNs);
          if (!ok) break;
          if (lead) {
            uint8_t* A = sm + st * kStageBytes;
            uint8_t* B = A + kOperand;
            if (rank == 0) mbar_arrive_expect_tx(&full[st], kArrive);
            const uint32_t bar = full0 + 8 * st;
            const int h = kb >= k_half;
            const int k0 = (kb - (h ? k_half : 0)) * (kFp8 ? 128 : 64);
            const CUtensorMap* am = &p.a[h | tl.half];
            const CUtensorMap* bm = &p.b[kEpi >= kGate ? (int)rank : h];
            if (a_mn) {
              tma_load_2d_pair(A, am, m0, k0, bar);
              tma_load_2d_pair(A + 8192, am, m0 + 64, k0, bar);
            } else {
              tma_load_2d_pair(A, am, k0, m0, bar);
            }
            if (b_mn) {
              tma_load_2d_pair(B, bm, n0, k0, bar);
              tma_load_2d_pair(B + 8192, bm, n0 + 64, k0, bar);
            } else {
              tma_load_2d_pair(B, bm, k0, n0, bar);
            }
          }
          __syncwarp();
          if (++st == kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
    } else if (warp == 1 && rank == 0) {
      // -------------------------------------------------------- multiply
      const bool lead = elect_one();
      const uint32_t sm0 = smem_u32(sm);
      int st = 0, buf = 0;
      uint32_t ph = 0, aph = 0;
      for (int k = 0, t; ok && (t = tile_of(g, pairs, pair, k)) >= 0; ++k) {
        const Tile tl = tile_at<kTileN>(g, t);
        const Problem& p = g.p[tl.p];
        const uint32_t idesc =
            kFp8 ? idesc_e4m3(256, kTileN) : idesc_bf16(256, kTileN, p.a_mn, p.b_mn);
        // a K-major block advances 32 bytes an instruction inside the swizzled
        // row; one stored by rows advances 16 rows of K (2048 bytes)
        const bool a_mn = !kFp8 && p.a_mn, b_mn = !kFp8 && p.b_mn;
        const uint64_t a_step = a_mn ? 2048 >> 4 : 32 >> 4, b_step = b_mn ? 2048 >> 4 : 32 >> 4;
        const uint64_t a0 = smem_desc(sm0, a_mn ? 8192 : 16, 1024, kSwizzle128B);
        const uint64_t b0 = smem_desc(sm0 + kOperand, b_mn ? 8192 : 16, 1024, kSwizzle128B);
        for (int kb = tl.k0; kb < tl.k1; ++kb) {
          const bool first = kFp8 || kb == tl.k0, last = kFp8 || kb + 1 == tl.k1;
          if (first) {
            ok = mbar_wait_warp(&acc_empty[buf], aph ^ 1u, kWaitNs);
            if (!ok) break;
          }
          ok = mbar_wait_warp(&full[st], ph, kWaitNs);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
            const uint64_t ad = a0 + (uint64_t)(st * (kStageBytes >> 4));
            const uint64_t bd = b0 + (uint64_t)(st * (kStageBytes >> 4));
            const uint32_t d = tmem + kAccCols * buf;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (kFp8) mma_f8_pair(d, ad + i * a_step, bd + i * b_step, idesc, i != 0);
              else mma_bf16_pair(d, ad + i * a_step, bd + i * b_step, idesc, !first || i != 0);
            }
            mma_commit_pair(&empty[st]);
            if (last) mma_commit_pair(&acc_full[buf]);
          }
          __syncwarp();
          if (last && ++buf == kAccs) {
            buf = 0;
            aph ^= 1u;
          }
          if (++st == kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
    } else if (kFp8 && (warp == 2 || warp == 3)) {
      // ---------------------------------------------------------- scales
      // s[j][h][r] = sa[row r][k0 + j] sb[column block h][k0 + j] of kGroup K
      // blocks at a time; a group is in registers while its slot is in use.
      int slot = 0;
      uint32_t ph = 0;
      for (int k = 0, t; ok && (t = tile_of(g, pairs, pair, k)) >= 0; ++k) {
        const Tile tl = tile_at<kTileN>(g, t);
        const Problem& p = g.p[tl.p];
        const int r0 = 64 * (warp - 2) + lane, nb = tl.n0 / 128;
        const float* sb0 = g.sb + (size_t)nb * g.sblocks;
        const float* sb1 = sb0 + (kTileN > 128 && tl.n0 + 128 < p.N ? g.sblocks : 0);
        const float* sa[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = tl.m0 + 128 * (int)rank + r0 + 32 * i;
          sa[i] = g.sa + (size_t)(row < p.M ? row : p.M - 1) * g.sblocks;
        }
        for (int kb = 0; kb < p.k_blocks; kb += kGroup) {
          float a[2][kGroup], b[2][kGroup];
#pragma unroll
          for (int j = 0; j < kGroup; ++j) {
            const int k = kb + j < p.k_blocks ? kb + j : kb;
            a[0][j] = ld_waited(sa[0] + k);
            a[1][j] = ld_waited(sa[1] + k);
            b[0][j] = ld_waited(sb0 + k);
            b[1][j] = ld_waited(sb1 + k);
          }
          ok = mbar_wait_warp(&sc_empty[slot], ph ^ 1u, kWaitNs);
          if (!ok) break;
          float* d = scales + slot * (kGroup * 256) + r0;
#pragma unroll
          for (int j = 0; j < kGroup; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              d[j * 256 + h * 128] = a[0][j] * b[h][j];
              d[j * 256 + h * 128 + 32] = a[1][j] * b[h][j];
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[slot]);
          slot ^= 1;
          if (slot == 0) ph ^= 1u;
        }
      }
    }
  } else {
    if constexpr (kFp8) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // -------------------------------------------------------- epilogue
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t free0 = mapa_smem(&acc_empty[0], 0);   // the even CTA's barriers
    uint8_t* bounce = sm + kStages * kStageBytes + (warp - 4) * kBounce;
    int buf = 0, slot = 0;
    uint32_t aph = 0, sph = 0;
    // this warp's columns of the accumulator are out of tensor memory
    auto release = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(free0 + 8 * buf);
    };
    auto advance = [&] {
      if (++buf == kAccs) {
        buf = 0;
        aph ^= 1u;
      }
    };
    for (int k = 0, t; ok && (t = tile_of(g, pairs, pair, k)) >= 0; ++k) {
      const Tile tl = tile_at<kTileN>(g, t);
      const Problem& p = g.p[tl.p];
      const int row0 = tl.m0 + 128 * (int)rank + 32 * q, row = row0 + lane;
      const bool live = row < p.M;
      if constexpr (kFp8) {
        // this thread's 128 or 64 columns are within one column block of the scales
        constexpr int kMine = kTileN / 2;
        const int n0 = tl.n0 + kMine * part;
        const float* sc = scales + (kMine == 128 ? 128 * part : 0) + 32 * q + lane;
        const int k_blocks = p.k_blocks;
        F2 acc[kMine / 2];
#pragma unroll
        for (int i = 0; i < kMine / 2; ++i) acc[i] = f2(0.f, 0.f);
        for (int kb = 0; kb < k_blocks; ++kb) {
          const int j = kb % kGroup;
          if (j == 0) {
            ok = mbar_wait_warp(&sc_full[slot], sph, kWaitNs);
            if (!ok) break;
          }
          const float s = sc[(slot * kGroup + j) * 256];
          ok = mbar_wait_warp(&acc_full[buf], aph, kWaitNs);
          if (!ok) break;
          tc_fence_after();
          // two 32-column pieces in turn: one is added while the next arrives;
          // all 64 columns of a narrow tile at once
          const uint32_t src = tmem + lanes + kAccCols * buf + kMine * part;
          uint32_t r[2][32];
          tmem_ld32(src, r[0]);
          if constexpr (kMine == 64) {
            tmem_ld32(src + 32, r[1]);
            tmem_ld_wait_regs(r[1]);
            release();
          }
#pragma unroll
          for (int c = 0; c < kMine / 32; ++c) {
            tmem_ld_wait_regs(r[c & 1]);
            if constexpr (kMine == 128) {
              if (c < 3) tmem_ld32(src + 32 * (c + 1), r[(c + 1) & 1]);
              else release();
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[16 * c + i] = f2_fma(f2(__uint_as_float(r[c & 1][2 * i]),
                                          __uint_as_float(r[c & 1][2 * i + 1])),
                                       f2(s, s), acc[16 * c + i]);
          }
          advance();
          if (j == kGroup - 1 || kb + 1 == k_blocks) {
            if (lane == 0) mbar_arrive(&sc_empty[slot]);   // read by the whole warp: release()'s
            slot ^= 1;                                     // __syncwarp came after
            if (slot == 0) sph ^= 1u;
          }
        }
        if (!ok) break;
        using T = typename std::conditional<kEpi == kStoreF32, float, __nv_bfloat16>::type;
        constexpr int kCols = 128 / (int)sizeof(T);   // 64 bf16 or 32 fp32
#pragma unroll
        for (int c = 0; c < kMine; c += 32) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 16; ++i) f2_split(acc[c / 2 + i], v[2 * i], v[2 * i + 1]);
          if (c % kCols == 0) stage_free(lane);
          stage_put<T>(bounce, lane, c % kCols, v);
          if ((c + 32) % kCols == 0) stage_out<T>(bounce, lane, p, 0, row0, n0 + c + 32 - kCols);
        }
      } else if constexpr (kEpi == kStore) {
        ok = mbar_wait_warp(&acc_full[buf], aph, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const int n0 = tl.n0 + 128 * part;
        const int shift = tl.part * p.part_rows;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t r[32];
          tmem_ld32(tmem + lanes + 256 * buf + 128 * part + c, r);
          tmem_ld_wait_regs(r);
          if (c == 96) release();
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          if (p.k_parts > 1) {
            stage_free(lane);
            stage_put<float>(bounce, lane, 0, v);
            stage_out<float>(bounce, lane, p, tl.half, row0, n0 + c, shift);
          } else {
            if (c % 64 == 0) stage_free(lane);
            stage_put<__nv_bfloat16>(bounce, lane, c % 64, v);
            if (c % 64 == 32)
              stage_out<__nv_bfloat16>(bounce, lane, p, tl.half, row0, n0 + c - 32);
          }
        }
        advance();
      } else {
        // this thread's 64 features; of 96 the second warps' 32
        constexpr bool kNarrow = kTileN == 192;
        const int f0 = tl.n0 / 2 + 64 * part;
        const bool half = kNarrow && part;
        uint32_t dh[kEpi == kGateGrad ? 32 : 1];   // 64 bf16, fetched before the wait
        if constexpr (kEpi == kGateGrad) {
          if (g.dh_wide) {   // hidden a multiple of 8: whole 16-byte pieces or none
            const __nv_bfloat16* d = g.dh + (size_t)(live ? row : 0) * g.ldh + f0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint4 w = make_uint4(0, 0, 0, 0);
              if (live && f0 + 8 * i < p.N && !(half && i >= 4))
                w = ld_waited(reinterpret_cast<const uint4*>(d) + i);
              dh[4 * i] = w.x; dh[4 * i + 1] = w.y; dh[4 * i + 2] = w.z; dh[4 * i + 3] = w.w;
            }
          } else {           // rows that start anywhere: a row at a time through the staging
            stage_free(lane);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int c = lane + 32 * i;
              if (half && i) break;
#pragma unroll 8
              for (int r = 0; r < 32; ++r) {
                __nv_bfloat16 v = __float2bfloat16_rn(0.f);
                if (row0 + r < p.M && f0 + c < p.N) v = g.dh[(size_t)(row0 + r) * g.ldh + f0 + c];
                *reinterpret_cast<__nv_bfloat16*>(bounce + stage_piece(r, c / 8) +
                                                  (c % 8) * 2) = v;
              }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 w = *reinterpret_cast<const uint4*>(bounce + stage_piece(lane, i));
              dh[4 * i] = w.x; dh[4 * i + 1] = w.y; dh[4 * i + 2] = w.z; dh[4 * i + 3] = w.w;
            }
            __syncwarp();   // read before the staging is written again
          }
        }
        ok = mbar_wait_warp(&acc_full[buf], aph, kWaitNs);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int out = 0; out < (kEpi == kGateGrad ? 2 : 1); ++out) {   // h; or dG, then dU
          stage_free(lane);
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            if (half && c) break;
            uint32_t G[32], U[32];
            tmem_ld32(tmem + lanes + 256 * buf + 64 * part + c, G);
            if (kEpi == kGate || out == 0)
              tmem_ld32(tmem + lanes + 256 * buf + kTileN / 2 + 64 * part + c, U);
            tmem_ld_wait_regs(G);
            if (kEpi == kGate || out == 0) tmem_ld_wait_regs(U);
            if ((c == 32 || half) && (kEpi == kGate || out == 1)) release();
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float x = __uint_as_float(G[i]);
              if constexpr (kEpi == kGate) {
                v[i] = gate_act(x, g.act) * __uint_as_float(U[i]);
              } else {
                const uint32_t d2 = dh[(c + i) >> 1];
                const float d = __uint_as_float((i & 1) ? d2 & 0xffff0000u : d2 << 16);
                float dG, dU;
                gate_grad(d, x, __uint_as_float(U[i]), g.act, dG, dU);
                v[i] = out == 0 ? dG : dU;
              }
            }
            if constexpr (kNarrow) {   // 32 features leave at a time, each from its half
              uint8_t* own = bounce + c / 32 * (kBounce / 2);
              stage_put<__nv_bfloat16, 64>(own, lane, 0, v);
              stage_out<__nv_bfloat16, 64>(own, lane, p, out, row0, f0 + c);
            } else {
              stage_put<__nv_bfloat16>(bounce, lane, c, v);
            }
          }
          if constexpr (!kNarrow) stage_out<__nv_bfloat16>(bounce, lane, p, out, row0, f0);
        }
        advance();
      }
    }
    stage_free(lane);   // this warp's stores have left shared memory
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

// The outputs c[0], c[1] = out[0], out[1], [M][N] with ldc elements a row:
// TMA stores where rows start on 16 bytes, plain ones elsewhere.  (Parts of K
// write [k_parts][part_rows][N], whose rows past M no one reads; their rows
// have to start on 16 bytes.)
inline bool output_maps(Problem& p, bool f32, int tile_n) {
  if (p.k_parts > 1) f32 = true;
  const int64_t pitch = p.ldc * (f32 ? 4 : 2);
  p.c_tma = pitch % 16 == 0;
  EncodeFn enc = encoder();
  if (!enc) return false;
  for (int i = 0; p.c_tma && i < 2; ++i) {
    if (i == 1 && p.out[1] == p.out[0]) {
      p.c[1] = p.c[0];
      break;
    }
    memset(&p.c[i], 0, sizeof p.c[i]);
    cuuint64_t dims[2] = {(cuuint64_t)p.N,
                          (cuuint64_t)(p.k_parts > 1 ? (int64_t)p.k_parts * p.part_rows : p.M)};
    cuuint64_t strides[1] = {(cuuint64_t)pitch};
    cuuint32_t box[2] = {f32 || tile_n == 192 ? 32u : 64u, 32};
    cuuint32_t es[2] = {1, 1};
    if (enc(&p.c[i], f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            p.out[i], dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            tile_n == 192 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

// Tiles of rows in a group: as many as keep their operand rows (256 x pitch
// bytes each) within 32 MB of the 126 MB L2, from 8, where the tiles in
// flight (76) are about square, to 32 (32768 x 2048 -> 2 x 6144 bf16: 830 us
// with 8, 800 with 32, 855 with 64).
inline int32_t group_rows(int64_t pitch) {
  const int64_t n = (32 << 20) / (256 * pitch);
  return n < 8 ? 8 : n > 32 ? 32 : (int32_t)n;
}

// Whether the gated product's tiles have 192 columns and not 256: a round of
// them takes 5/6 of the time (they read the rows of A for fewer columns), so
// where that many rounds take less.  (2048 -> 2 x 6144, us with 192 and 256:
// 256 tokens 14.3 and 15.5, 512 21.0 and 24.0, 4096, where this says 256, 117
// and 109; 1000 tokens, 1032 -> 2 x 2731: 16.7 and 18.8.)
inline bool narrow_gated(int64_t tokens, int32_t features, int sms) {
  const int64_t pairs = sms / 2, mt = (tokens + 255) / 256;
  const int64_t wide = mt * (((int64_t)features + 127) / 128);
  const int64_t narrow = mt * (((int64_t)features + 95) / 96);
  return 5 * ((narrow + pairs - 1) / pairs) < 6 * ((wide + pairs - 1) / pairs);
}

// The same for 128 columns of an 8-bit product, where a round takes 3/5 of the
// time: 500 to 550 cycles a K block, of them 256 for its products, with four
// accumulators on their way.  (us with 128 and 256: 2048 -> 4608, 512 tokens 8.0
// and 10.0, 1280 16.6 and 18.4; 4096 -> 2048, 1024 tokens 11.9 and 15.9;
// 1024 -> 4608, 300 tokens 5.9 and 7.0; 1552 -> 2005, 3001 tokens 18.7 and 20.1.)
inline bool narrow_fp8(int64_t mt, int32_t n, int sms) {
  const int64_t pairs = sms / 2;
  const int64_t wide = mt * (((int64_t)n + 255) / 256), narrow = mt * (((int64_t)n + 127) / 128);
  return 3 * ((narrow + pairs - 1) / pairs) < 5 * ((wide + pairs - 1) / pairs);
}

template <bool kFp8, int kEpi, int kTileN = 256>
cudaError_t launch_pair(PairArgs& g, int sms, cudaStream_t st) {
  constexpr uint32_t kSmem = Shape<kFp8>::kSmem;
  auto kern = pair_gemm_kernel<kFp8, kEpi, kTileN>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  int64_t tiles = 0;
  int32_t length[2] = {0, 1};   // K blocks of a tile, and about what its end costs
  for (int i = 0; i < g.problems; ++i) {
    if (!output_maps(g.p[i], kEpi == kStoreF32, kTileN)) return cudaErrorUnknown;
    tiles += tiles_of(g.p[i]);
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    g.tiles[i] = (int32_t)tiles_of(g.p[i]);
    length[i] = g.p[i].k_blocks / g.p[i].k_parts + 5;
  }
  g.ahead = length[0] / length[1];
  if (g.ahead > 1 << 20) g.ahead = 1 << 20;
  const int64_t pairs = sms / 2;
  e = launch(true, kern, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), kPairThreads,
                       kSmem, 0, st, g);
  count_launches(1);
  return e;
}

}  // namespace gemm
}  // namespace gdn
