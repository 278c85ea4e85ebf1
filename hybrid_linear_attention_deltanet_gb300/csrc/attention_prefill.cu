// Causal attention over whole sequences (contract: include/gdn.h):
//
//   S = scale Q K^T, lse_i = log sum_j exp S_ij, O = exp(S - lse) V
//
// in one pass over the keys: with m_i >= every S_ij seen so far less a bounded
// amount, l_i = sum_j exp(S_ij - m_i) and O_i = sum_j exp(S_ij - m_i) v_j are
// multiplied by exp(old m - new m) where a row's maximum grows by more than 8
// (in powers of two), which after a row's first keys hardly happens.
//
// Bound by the tensor cores (4 d flops a pair of query and key) and, next to
// that, by the exponentials.  A CTA holds two tiles of 128 packed rows.  Their
// scores (128 x 128 fp32) and outputs fill tensor memory; while one tile's eight
// warps' half takes the exponentials of its scores, the tensor cores work on
// the other tile:
//   multiply warp:  P0 V(j-1), Q0 K(j)^T, P1 V(j-1), Q1 K(j)^T, ...
// The probabilities go back to tensor memory as bf16, over the scores that they
// came from, and are the A operand of the second product there.
#include "attention_tc.cuh"

namespace gdn {
namespace {

using namespace attn;
using namespace sm100;

// two warpgroups of softmax; a third with a warp to multiply and one to load
constexpr int kThreads = 384;
constexpr uint32_t kTileBytes = 16384;   // 128 rows x 64 columns bf16
constexpr float kGrow = 8.f;         // a row's probabilities stay below 2^8

struct FwdArgs {
  CUtensorMap q, k, v;
  Seqs s;
  __nv_bfloat16* out;
  float* lse;
  float c;                 // scale log2 e
  int32_t q_heads, per;    // per: queries of a 128-row tile
  unsigned* status;
};

template <int D>
struct Fwd {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTile = kHalves * kTileBytes;     // of Q, K or V
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr uint32_t kSmem = 2 * kTile + kStages * kTile + 1024;
  static constexpr uint32_t kS = 0, kO = 256;                 // tensor-memory columns, + tile * 128
};

// 128 rows x 64 columns a half, K-major: 16 columns a step
__device__ __forceinline__ uint32_t kstep(int s) { return (s >> 2) * kTileBytes + (s & 3) * 32; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ FwdArgs a) {
  using C = Fwd<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align_smem_1024(smem_raw);
  __shared__ uint64_t q_full, kv_full[C::kStages], kv_empty[C::kStages], s_full[2], p_half[2],
      p_full[2], o_full[2];
  __shared__ uint32_t tmem_base;
  __shared__ int64_t scratch[kThreads + 6];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const Seqs& sq = a.s;
  const int head = blockIdx.x % sq.kv_heads;
  Seq seq;
  if (!locate<kThreads>(sq, blockIdx.x / sq.kv_heads, 2 * a.per, false, true, scratch, a.status, seq))
    return;
  if (tid == 0) {
    mbar_init(&q_full, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    fence_barrier_init();
  }
  if (warp == 8) tmem_alloc(&tmem_base, 512);
  if (warp == 9 && lane == 0) {
    prefetch_tensormap(&a.q);
    prefetch_tensormap(&a.k);
    prefetch_tensormap(&a.v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;

  // a tile's first query, its queries, and its blocks of 128 keys
  const int32_t shift = seq.lk - seq.lq;
  int32_t first[2], rows[2], blocks[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    first[w] = seq.tile * 2 * a.per + w * a.per;
    const int32_t left = seq.lq - first[w];
    rows[w] = left < 0 ? 0 : left < a.per ? left : a.per;
    const int32_t seen = rows[w] ? first[w] + rows[w] + shift : 0;   // keys that the last row sees
    blocks[w] = seen > 0 ? (seen + kRows - 1) / kRows : 0;
  }
  const int32_t most = blocks[1] > blocks[0] ? blocks[1] : blocks[0];
  bool ok = true;

  // 384 threads launch with 168 registers each, 64512 in all, which is 256 x 216
  // + 128 x 72: a softmax thread holds a row's 128 scores
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 9) {
    // ------------------------------------------------------------- load
    const bool lead = elect_one();
    if (lead && most > 0) {
      const uint32_t box = (uint32_t)(a.per * sq.group) * 128 * C::kHalves;
      mbar_arrive_expect_tx(&q_full, 2 * box);
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
          tma_load_3d(sm + w * C::kTile + h * kTileBytes, &a.q, 64 * h, head * sq.group,
                      (int32_t)(seq.q0 + first[w]), &q_full);
    }
    int st = 0;
    uint32_t ph = 0;
    for (int32_t j = 0; ok && j < most; ++j) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        ok = ok && mbar_wait_warp(&kv_empty[st], ph ^ 1u, kWaitNs);
        if (ok && lead) {
          uint8_t* to = sm + (2 + st) * C::kTile;
          mbar_arrive_expect_tx(&kv_full[st], C::kTile);
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(to + h * kTileBytes, x ? &a.v : &a.k, 64 * h, head,
                        (int32_t)(seq.k0 + (int64_t)j * kRows), &kv_full[st]);
        }
        __syncwarp();
        if (++st == C::kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 8) {
    // --------------------------------------------------------- multiply
    const bool lead = elect_one();
    const uint32_t base = smem_u32(sm);
    constexpr uint32_t kScores = idesc_bf16(128, 128, 0, 0), kOut = idesc_bf16(128, D, 0, 1);
    const uint64_t qd = smem_desc(base, 16, 1024, kSwizzle128B);
    const uint64_t kd = smem_desc(base + 2 * C::kTile, 16, 1024, kSwizzle128B);
    const uint64_t vd = smem_desc(base + 2 * C::kTile, kTileBytes, 1024, kSwizzle128B);
    if (most > 0) ok = mbar_wait_warp(&q_full, 0, kWaitNs);
    // step j: P V of block j - 1, then Q K^T of block j; a block's K is loaded
    // one stage before its V
    for (int32_t j = 0; ok && j <= most; ++j) {
      const int k_st = (int)((2 * (int64_t)j) % C::kStages);
      const int v_st = (int)((2 * (int64_t)j - 1 + C::kStages) % C::kStages);
      if (j < most) ok = mbar_wait_warp(&kv_full[k_st], (uint32_t)((2 * (int64_t)j / C::kStages) & 1), kWaitNs);
      if (ok && j > 0) {
        ok = mbar_wait_warp(&kv_full[v_st], (uint32_t)(((2 * (int64_t)j - 1) / C::kStages) & 1), kWaitNs);
        // values behind the sequence's last one are another's: a product
        // with a zero probability has to be zero
        const int64_t valid = seq.lk - (int64_t)(j - 1) * kRows;
        if (ok && valid < kRows) {
          for (int h = 0; h < C::kHalves; ++h) {
            uint4* z = reinterpret_cast<uint4*>(sm + (2 + v_st) * C::kTile + h * kTileBytes);
            for (int i = (int)valid * 8 + lane; i < kRows * 8; i += 32) z[i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t s_at = tmem + C::kS + 128 * w, o_at = tmem + C::kO + 128 * w;
        if (ok && j > 0 && j <= blocks[w]) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && mbar_wait_warp(half ? &p_full[w] : &p_half[w], (uint32_t)((j - 1) & 1), kWaitNs);
            tc_fence_after();
            if (ok && lead)
#pragma unroll
              for (int s = 4 * half; s < 4 * half + 4; ++s)
                mma_bf16_ts(o_at, s_at + 8 * s, vd + (uint64_t)((v_st * C::kTile + s * 2048) >> 4), kOut,
                            j > 1 || s > 0);
          }
          if (ok && lead && j == blocks[w]) mma_commit(&o_full[w]);
        }
        if (ok && lead && j < blocks[w]) {
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            mma_bf16(s_at, qd + (uint64_t)((w * C::kTile + kstep(s)) >> 4),
                     kd + (uint64_t)((k_st * C::kTile + kstep(s)) >> 4), kScores, s > 0);
          mma_commit(&s_full[w]);
        }
        __syncwarp();
      }
      if (ok && lead) {
        if (j > 0) mma_commit(&kv_empty[v_st]);
        if (j < most) mma_commit(&kv_empty[k_st]);
      }
      __syncwarp();
    }
  }
  } else {
    // ---------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int w = warp >> 2;
    const int row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // 32 lanes, in the address's upper half
    const uint32_t s_at = tmem + lanes + C::kS + 128 * w, o_at = tmem + lanes + C::kO + 128 * w;
    const int32_t n = blocks[w];
    const int qi = row / sq.group;                         // the row's query in its tile
    const bool live = qi < rows[w];
    // the last key that the row sees
    const int32_t last = first[w] + qi + shift;
    const float c = a.c;
    float m = 0.f, l = 0.f;
    for (int32_t j = 0; j < n; ++j) {
      ok = mbar_wait_warp(&s_full[w], (uint32_t)(j & 1), kWaitNs);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld_wait_regs(s[i]);
      // keys that the tile's first row does not see are in the block?
      const int32_t k0 = j * kRows;
      if (k0 + kRows - 1 > first[w] + shift) {
        const int32_t see = last - k0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (32 * i + x > see) s[i][x] = 0xff800000u;   // -inf
      }
      float mx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mx[i] = __uint_as_float(s[i][0]);
#pragma unroll
        for (int x = 1; x < 31; x += 2)
          mx[i] = fmaxf(mx[i], fmaxf(__uint_as_float(s[i][x]), __uint_as_float(s[i][x + 1])));
        mx[i] = fmaxf(mx[i], __uint_as_float(s[i][31]));
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
      if (j == 0) {
        m = top == -INFINITY ? 0.f : top;
      } else if (__any_sync(0xffffffffu, top > m + kGrow)) {
        // (the scores' commit covers the products before them: O is at rest)
        // a row's bits depend on no other row of its warp: the others get a factor of 1
        const bool grows = top > m + kGrow;
        const float f = grows ? ex2_sfu(m - top) : 1.f;
        l *= f;
        m = grows ? top : m;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(o_at + 32 * i, o);
          tmem_ld_wait_regs(o);
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
          tmem_st32(o_at + 32 * i, o);
        }
      }
      const F2 cc = f2(c, c), mm = f2(-m, -m);
      F2 sum[2] = {f2(l, 0.f), f2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t p[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          float lo, hi;
          f2_split(f2_fma(f2(__uint_as_float(s[i][2 * x]), __uint_as_float(s[i][2 * x + 1])), cc, mm),
                   lo, hi);
          lo = ex2_sfu(lo);
          hi = ex2_sfu(hi);
          sum[x & 1] = f2_add(sum[x & 1], f2(lo, hi));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[x]) : "f"(hi), "f"(lo));
        }
        tmem_st16(s_at + 16 * i, p);
        if (i & 1) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(i == 1 ? &p_half[w] : &p_full[w]);
        }
      }
      float x0, x1;
      f2_split(f2_add(sum[0], sum[1]), x0, x1);
      l = x0 + x1;
    }
    // the row's results
    if (ok && n > 0) ok = mbar_wait_warp(&o_full[w], 0, kWaitNs);
    tc_fence_after();
    if (ok && rows[w] > 0) {
      const int64_t r = (seq.q0 + first[w] + qi) * a.q_heads + (int64_t)head * sq.group + row % sq.group;
      const bool none = n == 0 || l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(o_at + 32 * i, o);
          tmem_ld_wait_regs(o);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t y[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float lo = none ? 0.f : __uint_as_float(o[8 * x + 2 * z]) * inv;
            const float hi = none ? 0.f : __uint_as_float(o[8 * x + 2 * z + 1]) * inv;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y[z]) : "f"(hi), "f"(lo));
          }
          if (live)
            *reinterpret_cast<uint4*>(a.out + r * D + 32 * i + 8 * x) =
                make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      if (live) a.lse[r] = none ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  }
  if (!ok) {
    // copies and products in flight end within microseconds; give them longer
    flag_status(a.status, GDN_ERR_TIMEOUT);
    const uint64_t from = globaltimer_ns();
    while (globaltimer_ns() - from < 5000000ull) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

int prefill(const void* q, const void* k, const void* v, const int32_t* cu_q, const int32_t* cu_k,
            float scale, void* out, float* lse, const Shape& s, cudaStream_t st) {
  if (const int rc = check_shape(s, cu_q, cu_k, scale)) return rc;
  const int64_t tq = s.tq(), tk = s.tk();
  if (tq > 0 && (!q || !out || !lse)) return GDN_ERR_INVALID_ARG;
  if (tk > 0 && (!k || !v)) return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(cu_k, 4))
    return GDN_ERR_ALIGNMENT;
  const size_t cu_bytes = ((size_t)s.batch + 1) * 4;
  const Span ins[] = {span_of(q, s.q_bytes()), span_of(k, s.k_bytes(s.k_stride)),
                      span_of(v, s.k_bytes(s.v_stride)), span_of(cu_q, cu_bytes),
                      span_of(cu_k, cu_bytes)};
  const Span outs[] = {span_of(out, s.rows() * s.d * 2), span_of(lse, s.rows() * 4)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  if (tq == 0) return GDN_OK;
  FwdArgs a;
  memset(&a, 0, sizeof a);
  a.status = status_ptr();
  if (!a.status) return GDN_ERR_CUDA;
  const int32_t group = s.q_heads / s.kv_heads;
  a.s = {cu_q, cu_k, s.batch, s.seqlen_q, s.seqlen_k, group, s.kv_heads};
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.c = scale * kLog2e;
  a.q_heads = s.q_heads;
  a.per = kRows / group;
  const void* kk = tk ? k : q;   // (no keys: nothing is loaded through these)
  if (!heads_map(&a.q, q, tq, s.q_heads, s.d, s.q_stride, group, a.per) ||
      !heads_map(&a.k, kk, tk, s.kv_heads, s.d, tk ? s.k_stride : (int64_t)s.kv_heads * s.d, 1, kRows) ||
      !heads_map(&a.v, tk ? v : q, tk, s.kv_heads, s.d, tk ? s.v_stride : (int64_t)s.kv_heads * s.d, 1, kRows))
    return GDN_ERR_CUDA;
  // packed: an upper bound, sum_n ceil(len_n / per) <= T / per + N
  const int64_t per = 2 * a.per;
  const int64_t tiles = s.packed ? tq / per + s.batch : (s.seqlen_q + per - 1) / per * s.batch;
  const int64_t grid = tiles * s.kv_heads;
  if (grid > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  cudaError_t e;
  auto run = [&](auto shape, auto kern) {
    using C = decltype(shape);
    e = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e == cudaSuccess) e = launch(false, kern, dim3((unsigned)grid), kThreads, C::kSmem, 0, st, a);
  };
  if (s.d == 128) run(Fwd<128>{}, prefill_kernel<128>);
  else run(Fwd<64>{}, prefill_kernel<64>);
  count_launches(1);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" int gdn_attention_prefill(const void* q, const void* k, const void* v,
                                     const int32_t* cu_q, const int32_t* cu_k, float scale,
                                     void* out, float* lse, int32_t batch, int64_t seqlen_q,
                                     int64_t seqlen_k, int32_t q_heads, int32_t kv_heads,
                                     int32_t d, int64_t q_stride, int64_t k_stride,
                                     int64_t v_stride, gdn_stream_t stream) {
  const attn::Shape s = {batch, seqlen_q, seqlen_k, q_heads, kv_heads, d, q_stride, k_stride,
                         v_stride, cu_q != nullptr};
  return prefill(q, k, v, cu_q, cu_k, scale, out, lse, s, (cudaStream_t)stream);
}
