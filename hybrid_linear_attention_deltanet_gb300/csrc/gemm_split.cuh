// Matrix products of few tokens on the tensor cores, the K axis split over a
// thread-block cluster.
//
// With few tokens the weights are all there is to read, so they take the
// MMA's 128 rows and the tokens its columns: a CTA multiplies 128 rows of the
// weights (gated: 64 of Wg and 64 of Wu, the same features) by kNB tokens
// over its share of K, and the CTAs of a cluster, one share each, add their
// fp32 partial products through each other's shared memory, in a fixed order.
// One launch, whose CTAs hold all of the weights' bytes in flight that their
// stages allow.
//
// Roles: the first 4 or 8 warps take accumulators out, then one fetches and
// one multiplies.  8-bit operands: every K block of 128 is an accumulator of
// its own, scaled (a token's scale times the weight block's) into fp32
// registers; with 32 columns or more that takes 8 warps, half the columns
// each (64 tokens, 2048 -> 4608: 5.4 us, 5.9 with 4; 256 tokens, 4096 -> 2048: 8.6
// and 9.6).
// Waits are bounded as in gemm_pair.cuh.
//
// Bound by HBM, then by the launch's own chain.  One token against 2 x 6144 x
// 2048 bf16 (50 MB): 10.1 us a call among others, 5.0 TB/s; against 4608 x 2048
// e4m3 (9.4 MB): 4.4 us, of which an empty launch of this shape takes 1.6 and
// its tensor memory 0.6.
#pragma once

#include "gemm_pair.cuh"

namespace gdn {
namespace gemm {

struct SplitArgs {
  CUtensorMap w[2], x;   // weights (gated: Wg, Wu), tokens
  int32_t k_blocks;      // of 128 bytes
  int32_t tokens, n;     // n: rows of the weights (gated: features)
  int32_t act;
  void* out;             // [tokens][ld]
  void* out2;            // kGateGrad: dU beside dG in out
  int64_t ld;
  const __nv_bfloat16* dh;   // kGateGrad: [tokens][n]
  const float* sx;       // 8-bit: [tokens][k_blocks]
  const float* sw;       //        [ceil(n / 128)][k_blocks]
  unsigned* status;
};

constexpr uint32_t kSplitAlone = 120 * 1024;   // shared memory that keeps a CTA alone on its SM
constexpr int kSplitScaleBytes = 65536;   // most of a CTA's staged scales

template <bool kFp8, int kNB>
struct SplitShape {
  static constexpr int kEpi = kFp8 && kNB >= 32 ? 8 : 4;     // warps that take accumulators out
  static constexpr int kCols = kNB / (kEpi / 4);             // columns of each
  static constexpr int kThreads = 32 * (kEpi + 2);
  static constexpr uint32_t kStage = kOperand + kNB * 128;
  static constexpr int kStages = kNB <= 16 ? 5 : 4;
  static constexpr int kAcc = kFp8 ? 4 : 1;   // accumulators in tensor memory
  static constexpr uint32_t kTmem = kAcc * kNB < 32 ? 32 : kAcc * kNB;
  static constexpr uint32_t kSmem = kStages * kStage + 1024;   // and the scales, a call's own
  static_assert(kNB * 128 * 4 <= kStages * kStage, "the partial products reuse the stages");
};

// Four columns of a row, those past `valid` left out; whole rows start on four.
template <typename T>
__device__ __forceinline__ void store4(T* out, const float (&v)[4], int valid, bool whole) {
  if (whole && valid >= 4) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(out) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    else
      *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < valid) st_out(out + i, v[i]);
  }
}

template <bool kFp8, int kEpi, int kNB, typename T>
__global__ void __launch_bounds__(SplitShape<kFp8, kNB>::kThreads, 2)
    split_gemm_kernel(const __grid_constant__ SplitArgs g) {
  using S = SplitShape<kFp8, kNB>;
  constexpr bool kGated = kEpi >= kGate;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align_smem_1024(smem_raw);
  float* scales = reinterpret_cast<float*>(sm + S::kStages * S::kStage);   // [K block][kNB]
  float* part = reinterpret_cast<float*>(sm);                              // [kNB][128]
  __shared__ uint64_t full[S::kStages], empty[S::kStages], acc_full[S::kAcc], acc_empty[S::kAcc];
  __shared__ uint32_t tmem_base;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rank = blockIdx.x, split = gridDim.x;   // the cluster spans x
  const int kb0 = (int)((int64_t)g.k_blocks * rank / split);
  const int kbs = (int)((int64_t)g.k_blocks * (rank + 1) / split) - kb0;
  const int rows = kGated ? 64 : 128;
  const int f0 = blockIdx.y * rows, t0 = blockIdx.z * kNB;
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < S::kAcc; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], S::kEpi);
    }
    fence_barrier_init();
  }
  if (warp == S::kEpi + 1) tmem_alloc(&tmem_base, S::kTmem);
  if (warp == S::kEpi && lane == 0) {
    prefetch_tensormap(&g.w[0]);
    prefetch_tensormap(&g.x);
    if (kGated) prefetch_tensormap(&g.w[1]);
    // the weights' way from HBM to L2 need not wait for the grid before (L2
    // holds what memory holds, also where that grid still writes): a layer of
    // one token's six launches 27.6 -> 25.8 us
    for (int i = 0; i < kbs && i < S::kStages; ++i) {
      const int k = (kb0 + i) * (kFp8 ? 128 : 64);
      prefetch_l2_2d(&g.w[0], k, f0);
      if (kGated) prefetch_l2_2d(&g.w[1], k, f0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_release_next();
  grid_wait();
  const uint32_t tmem = tmem_base;
  bool ok = true;

  if (warp == S::kEpi) {
    // ---------------------------------------------------------- fetch
    const bool lead = elect_one();
    int st = 0;
    uint32_t ph = 0;
    for (int i = 0; i < kbs; ++i) {
      ok = mbar_wait_warp(&empty[st], ph ^ 1u, kWaitNs);
      if (!ok) break;
      if (lead) {
        uint8_t* W = sm + st * S::kStage;
        const int k = (kb0 + i) * (kFp8 ? 128 : 64);
        mbar_arrive_expect_tx(&full[st], S::kStage);
        if (kGated) {
          tma_load_2d(W, &g.w[0], k, f0, &full[st]);
          tma_load_2d(W + 8192, &g.w[1], k, f0, &full[st]);
        } else {
          tma_load_2d(W, &g.w[0], k, f0, &full[st]);
        }
        tma_load_2d(W + kOperand, &g.x, k, t0, &full[st]);
      }
      __syncwarp();
      if (++st == S::kStages) {
        st = 0;
        ph ^= 1u;
      }
    }
  } else if (warp == S::kEpi + 1) {
    // -------------------------------------------------------- multiply
    const bool lead = elect_one();
    const uint64_t w0 = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);
    constexpr uint32_t idesc = kFp8 ? idesc_e4m3(128, kNB) : idesc_bf16(128, kNB, 0, 0);
    int st = 0, buf = 0;
    uint32_t ph = 0, aph = 0;
    for (int i = 0; i < kbs; ++i) {
      if (kFp8) {
        ok = mbar_wait_warp(&acc_empty[buf], aph ^ 1u, kWaitNs);
        if (!ok) break;
      }
      ok = mbar_wait_warp(&full[st], ph, kWaitNs);
      if (!ok) break;
      tc_fence_after();
      if (lead) {
        const uint64_t wd = w0 + (uint64_t)(st * (S::kStage >> 4)), xd = wd + (kOperand >> 4);
        const uint32_t d = tmem + kNB * buf;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (kFp8) mma_f8(d, wd + 2 * j, xd + 2 * j, idesc, j != 0);
          else mma_bf16(d, wd + 2 * j, xd + 2 * j, idesc, (i | j) != 0);
        }
        mma_commit(&empty[st]);
        if (kFp8 || i + 1 == kbs) mma_commit(&acc_full[buf]);
      }
      __syncwarp();
      if (kFp8 && ++buf == S::kAcc) {
        buf = 0;
        aph ^= 1u;
      }
      if (++st == S::kStages) {
        st = 0;
        ph ^= 1u;
      }
    }
  } else {
    // ------------------------------------- accumulators out of tensor memory
    constexpr int kCols = S::kCols;
    const int row = 32 * (warp & 3) + lane, col0 = kCols * (warp >> 2);
    const uint32_t src = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + col0;
    float acc[kCols];
    if constexpr (kFp8) {
      const float* sw = g.sw + (size_t)(f0 / 128) * g.k_blocks + kb0;
      for (int e = tid; e < kbs * kNB; e += 32 * S::kEpi) {
        const int c = e / kbs, i = e - c * kbs;   // consecutive threads: one token's blocks
        scales[i * kNB + c] =
            t0 + c < g.tokens
                ? ld_waited(g.sx + (size_t)(t0 + c) * g.k_blocks + kb0 + i) * ld_waited(sw + i)
                : 0.f;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * S::kEpi) : "memory");   // these warps
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
      int buf = 0;
      uint32_t aph = 0;
      for (int i = 0; i < kbs; ++i) {
        ok = mbar_wait_warp(&acc_full[buf], aph, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const float4* s4 = reinterpret_cast<const float4*>(scales + i * kNB + col0);
        uint32_t r[2][16];   // two 16-column pieces in turn: one arrives while one is added
        tmem_ld16(src + kNB * buf, r[0]);
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          uint32_t(&x)[16] = r[(c / 16) & 1];
          tmem_ld_wait_regs(x);
          if (c + 16 < kCols) {
            tmem_ld16(src + kNB * buf + c + 16, r[(c / 16 + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float4 s = s4[c / 4 + v];
            acc[c + 4 * v] = fmaf(__uint_as_float(x[4 * v]), s.x, acc[c + 4 * v]);
            acc[c + 4 * v + 1] = fmaf(__uint_as_float(x[4 * v + 1]), s.y, acc[c + 4 * v + 1]);
            acc[c + 4 * v + 2] = fmaf(__uint_as_float(x[4 * v + 2]), s.z, acc[c + 4 * v + 2]);
            acc[c + 4 * v + 3] = fmaf(__uint_as_float(x[4 * v + 3]), s.w, acc[c + 4 * v + 3]);
          }
        }
        if (++buf == S::kAcc) {
          buf = 0;
          aph ^= 1u;
        }
      }
    } else {
      ok = mbar_wait_warp(&acc_full[0], 0, kWaitNs);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        uint32_t r[16];
        tmem_ld16(src + c, r);
        tmem_ld_wait_regs(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c + i] = __uint_as_float(r[i]);
      }
      tc_fence_before();
    }
    // the last accumulator is complete, so are all products and copies: the
    // stages are free
    if (ok) {
#pragma unroll
      for (int c = 0; c < kCols; ++c) part[(col0 + c) * 128 + row] = acc[c];
    }
  }
  if (!ok) {
    flag_status(g.status, GDN_ERR_TIMEOUT);
    const uint64_t from = globaltimer_ns();
    while (globaltimer_ns() - from < 5000000ull) __nanosleep(1000);
  }
  __syncwarp();
  cluster_sync_all();
  if (warp < S::kEpi) {
    // four rows a lane: a column of the tile is 32 lanes (gated: 16, G and U
    // 64 rows apart); the columns are dealt to the cluster's CTAs in turn
    const uint32_t p0 = smem_u32(part);
    uint32_t base[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < split) asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base[s]) : "r"(p0), "r"(s));
    constexpr int kLanes = kGated ? 16 : 32, kSlots = 32 * S::kEpi / kLanes;
    const int cols = g.tokens - t0 < kNB ? g.tokens - t0 : kNB;
    const int row = 4 * (tid % kLanes), f = f0 + row;
    if (f < g.n) {
#pragma unroll 2
      for (int c = rank + split * (tid / kLanes); c < cols; c += split * kSlots) {
        const uint32_t o = (uint32_t)(c * 128 + row) * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < split) {
            const float4 a = ld_shared_cluster4(base[s] + o);
            v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
            if (kGated) {
              const float4 b = ld_shared_cluster4(base[s] + o + 256);
              u[0] += b.x; u[1] += b.y; u[2] += b.z; u[3] += b.w;
            }
          }
        const int64_t at = (int64_t)(t0 + c) * g.ld + f;
        if constexpr (kEpi == kGate) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = gate_act(v[i], g.act) * u[i];
        } else if constexpr (kEpi == kGateGrad) {
          const __nv_bfloat16* dh = g.dh + (int64_t)(t0 + c) * g.n + f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            gate_grad(f + i < g.n ? __bfloat162float(dh[i]) : 0.f, v[i], u[i], g.act, v[i], u[i]);
          store4((T*)g.out2 + at, u, g.n - f, g.ld % 4 == 0);
        }
        store4((T*)g.out + at, v, g.n - f, g.ld % 4 == 0);
      }
    }
  }
  __syncwarp();
  cluster_sync_all();   // no CTA leaves while another may read its partial products
  if (warp == S::kEpi + 1) tmem_dealloc(tmem, S::kTmem);
}

// How a call takes the split form: columns a CTA, CTAs a cluster and whether
// each gets an SM to itself; columns 0: the pair form.
//
// Up to 64 tokens are one tile of columns; more take tiles of 64 while those
// are `most` (the pair form's fewer, longer chains of K blocks would leave most
// SMs idle): one CTA an SM, of 8 bits half of that, where K can be split.  K is
// split (at least four blocks each) while the CTAs are within one an SM, and
// each is then kept alone there: else the scheduler puts two on some SMs and
// none on others.  Tiles that leave no room for a split so take two CTAs an SM
// if K is long.  (us, pair / split.  8 bits: 2048 -> 4608, 16 tokens 7.0 / 4.0,
// 128 tokens 7.1 / 6.4, 192 tokens, 108 tiles, 7.1 / 7.9; 4096 -> 1000, 300
// tokens, 11.1 / 6.9, with two CTAs an SM 7.5; 4096 -> 2048, 256 tokens 10.8 /
// 8.2, 512 tokens, 128 tiles, 11.0 / 11.3.  Gated: 2048 -> 6144, 64 tokens 14.0 /
// 11.2, 128 tokens, 192 tiles, 14.0 / 15.7; 2048 -> 4096, 128 tokens, 128 tiles,
// 12.0 / 10.8; 1000 -> 1000, 200 tokens, 8.9 / 6.6.  Clusters of eight CTAs alone
// on their SMs do not find room side by side: 6.1 against 3.6.)
struct SplitPlan {
  int columns, split;
  bool alone;
};
inline SplitPlan plan_split(int64_t tokens, int64_t row_tiles, int k_blocks, int sms,
                            int most) {
  const int nb = tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64;
  const int64_t units = row_tiles * ((tokens + nb - 1) / nb);
  if (row_tiles > 65535 || (tokens > 64 && units > most)) return {0, 0, false};
  const auto split = [&](int64_t ctas) {
    int64_t s = ctas / units;
    if (s > k_blocks / 4) s = k_blocks / 4;
    return s < 1 ? 1 : s > 8 ? 8 : (int)s;
  };
  int s = split(sms);
  if (s == 1 && k_blocks >= 16) s = split(2 * (int64_t)sms);
  return {nb, s, units * s <= sms && s < 8};
}

template <bool kFp8, int kEpi, int kNB, typename T>
cudaError_t launch_split_nb(const SplitArgs& g, unsigned split, bool alone, cudaStream_t st) {
  using S = SplitShape<kFp8, kNB>;
  constexpr bool kGated = kEpi >= kGate;
  auto kern = split_gemm_kernel<kFp8, kEpi, kNB, T>;
  uint32_t smem = S::kSmem + (kFp8 ? (uint32_t)((g.k_blocks + split - 1) / split) * kNB * 4 : 0);
  if (alone && smem < kSplitAlone) smem = kSplitAlone;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(S::kSmem + kSplitScaleBytes));
  if (e != cudaSuccess) return e;
  const unsigned ny = (unsigned)((g.n + (kGated ? 63 : 127)) / (kGated ? 64 : 128));
  const unsigned nz = (unsigned)((g.tokens + kNB - 1) / kNB);
  e = launch(true, kern, dim3(split, ny, nz), S::kThreads, smem, split, st, g);
  count_launches(1);
  return e;
}

template <bool kFp8, int kEpi, typename T>
cudaError_t launch_split(const SplitArgs& g, const SplitPlan& plan, cudaStream_t st) {
  const unsigned split = (unsigned)plan.split;
  switch (plan.columns) {
    case 16: return launch_split_nb<kFp8, kEpi, 16, T>(g, split, plan.alone, st);
    case 32: return launch_split_nb<kFp8, kEpi, 32, T>(g, split, plan.alone, st);
    default: return launch_split_nb<kFp8, kEpi, 64, T>(g, split, plan.alone, st);
  }
}

}  // namespace gemm
}  // namespace gdn
