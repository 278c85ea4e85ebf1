// Gradients of the causal attention over whole sequences (contract:
// include/gdn.h):
//
//   P_ij = exp(s_ij - lse_i), D_i = dout_i . out_i, dS_ij = P_ij (dout_i . v_j - D_i)
//   dV = P^T dO, dK = scale dS^T Q, dQ = scale dS K
//
// P is computed again from lse, so that no pass before it keeps anything of the
// size of P.  One kernel holds a tile of keys and goes over the queries that
// see it (S^T, dP^T, dV, dK), one a tile of queries and goes over its keys (S,
// dP, dQ): seven products where five would do, but every sum is one tensor-
// memory accumulator with one order, and nothing is added in memory.  Both are
// bound by the tensor cores; two warps issue, in an order such that the
// cores work on the next tile's scores while P and dS of this one are made:
//   keys:     dV(i-1), S(i) | dK(i-1), dP(i) | ...
//   queries:  dP(j+1) | dQ(j), S(j+2) | ...
// P and dS go back to tensor memory as bf16, over the scores that they came
// from, and are the A operand there.
//
// 16 query and 4 kv heads of 128: 2 x 8192 tokens 1195 to 1213 us call after call (at the
// 1400 W limit), 1105 to 1135 in a run too short for that limit (580 and 509 in the two kernels); in
// such runs 8192 550, 4096 179; heads of 64: 2 x 8192 874.  What holds the products
// back is shared memory: S and dP read two operands of 4 KB per 64 cycles, all that
// it gives, the tiles come in through it, and so do the keys' kernel's statistics.
// Tried and slower (8192 tokens): in the queries' kernel dP(j + 1) as soon as dP(j) is in
// registers 580, Q and dO in tensor memory with one buffer of scores 610, the next
// scores in registers before dS is reported 606.  One kernel that adds dQ in memory
// would save two products in seven, but not keep the sums' order.
#include "attention_tc.cuh"

namespace gdn {
namespace {

using namespace attn;
using namespace sm100;

constexpr int kThreads = 384;   // two warpgroups for P and dS; a third with the issuing warps
constexpr uint32_t kHalfTile = 16384;   // 128 rows x 64 columns bf16

struct BwdArgs {
  CUtensorMap q, k, v, dout;
  Seqs s;
  const float *nlse, *nd;      // [kv_heads][T_q][group]: -lse log2 e and -D
  __nv_bfloat16 *dq, *dk, *dv;
  float c, scale;              // scale log2 e, scale
  int64_t tq;
  int32_t q_heads, per;        // per: queries of a 128-row tile
  // the order of the jobs, longest first (nullptr: that of the sequences)
  const int32_t* count[2];     // [tiles of keys, of queries]
  const Job* jobs[2];
  // parts of a key tile's queries, and their sums of dV and dK, [jobs][parts][2][128][D];
  // parts of a query tile's keys, and their sums of dQ, [jobs][parts][128][D]
  int32_t parts, q_parts;
  float *part, *q_part;
  unsigned* status;
};

// ------------------------------------------------------------ row sums
struct RowArgs {
  const __nv_bfloat16 *out, *dout;
  const float* lse;
  float *nlse, *nd;
  int64_t tq;
  int32_t q_heads, group;
};
// D / 8 lanes a row, 16 bytes of each tensor a lane; bound by HBM.
template <int D>
__global__ void __launch_bounds__(256) rows_kernel(RowArgs a) {
  grid_wait();
  grid_release_next();   // (the next kernels read the sequences before they wait)
  constexpr int kLanes = D / 8;
  const int64_t r = ((int64_t)blockIdx.x * 256 + threadIdx.x) / kLanes;
  const int l = threadIdx.x % kLanes;
  const bool on = r < a.tq * a.q_heads;
  float sum = 0.f;
  if (on) {
    const uint4 x = *reinterpret_cast<const uint4*>(a.out + r * D + l * 8);
    const uint4 y = *reinterpret_cast<const uint4*>(a.dout + r * D + l * 8);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), sum);
      sum = fmaf(__uint_as_float(xs[i] & 0xffff0000u), __uint_as_float(ys[i] & 0xffff0000u), sum);
    }
  }
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (on && l == 0) {
    const int64_t t = r / a.q_heads;
    const int head = (int)(r - t * a.q_heads), h = head / a.group;
    const int64_t to = ((int64_t)h * a.tq + t) * a.group + head - h * a.group;
    const float lse = a.lse[r];
    // a row that sees no key: P = 2^-inf
    a.nlse[to] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
    a.nd[to] = -sum;
  }
}

// ------------------------------------------------------------ the two loops
// Shared memory: two resident tiles, three slots of the operand that is used
// again a product later (Q; K) and two of the other (dO; V), then the
// statistics and the barriers.  D = 128: 224 KB of tiles.
template <int D>
struct Bwd {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTile = kHalves * kHalfTile;
  static constexpr uint32_t kA = 2 * kTile, kB = 5 * kTile;   // the slots of the two operands
  static constexpr int kNA = 3, kNB = 2;
  static constexpr uint32_t kStats = 7 * kTile;               // [2][2][128] fp32
  static constexpr uint32_t kBars = kStats + 2048;
  static constexpr uint32_t kSmem = kBars + 256;
};
struct Bars {
  uint64_t own, a_full[3], a_empty[3], b_full[2], b_empty[2], s_full[2], dp_full, p_ready,
      ds_ready[2], done, turn[2];
  uint32_t tmem;
};
static_assert(sizeof(Bars) <= 256, "");

__device__ __forceinline__ uint32_t kstep(int s) { return (s >> 2) * kHalfTile + (s & 3) * 32; }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Rows [from, 128) of a tile in shared memory become zeros, by one warp.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int lane) {
#pragma unroll
  for (int h = 0; h < D / 64; ++h) {
    uint4* z = reinterpret_cast<uint4*>(tile + h * kHalfTile);
    for (int i = from * 8 + lane; i < kRows * 8; i += 32) z[i] = make_uint4(0, 0, 0, 0);
  }
}
// This lane's row of an accumulator's columns as bf16 (times f) to memory.
template <int kCols>
__device__ __forceinline__ void store_row(uint32_t at, float f, __nv_bfloat16* to, bool live, bool zero) {
#pragma unroll
  for (int i = 0; i < kCols / 32; ++i) {
    uint32_t o[32];
    if (!zero) {
      tmem_ld32(at + 32 * i, o);
      tmem_ld_wait_regs(o);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t y[4];
#pragma unroll
      for (int z = 0; z < 4; ++z)
        y[z] = zero ? 0u
                    : pack(__uint_as_float(o[8 * x + 2 * z]) * f, __uint_as_float(o[8 * x + 2 * z + 1]) * f);
      if (live) *reinterpret_cast<uint4*>(to + 32 * i + 8 * x) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

// The same row as it is, a part's sum: four columns of all rows together, then the
// next four, so that a warp's store is contiguous (rows one after another took a
// CTA 5 us).
template <int kCols>
__device__ __forceinline__ void store_part(uint32_t at, float* to, int row, bool zero) {
#pragma unroll
  for (int i = 0; i < kCols / 32; ++i) {
    uint32_t o[32];
    if (!zero) {
      tmem_ld32(at + 32 * i, o);
      tmem_ld_wait_regs(o);
    }
#pragma unroll
    for (int x = 0; x < 8; ++x)
      *reinterpret_cast<uint4*>(to + ((8 * i + x) * kRows + row) * 4) =
          zero ? make_uint4(0, 0, 0, 0) : make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
  }
}

// Two elements: 2^(x c + l); (x + d) p; and 64 columns' masks and their way back
// to tensor memory.  (The masks apart, behind a branch: selects in the loops above
// were half of their instructions.)
__device__ __forceinline__ void exp_pair(uint32_t& x0, uint32_t& x1, F2 c, F2 l) {
  float y0, y1;
  f2_split(f2_fma(f2(__uint_as_float(x0), __uint_as_float(x1)), c, l), y0, y1);
  x0 = __float_as_uint(ex2_sfu(y0));
  x1 = __float_as_uint(ex2_sfu(y1));
}
__device__ __forceinline__ void times_less(uint32_t& x0, uint32_t& x1, F2 d, uint32_t p0, uint32_t p1) {
  float y0, y1;
  f2_split(f2_mul(f2_add(f2(__uint_as_float(x0), __uint_as_float(x1)), d),
                  f2(__uint_as_float(p0), __uint_as_float(p1))),
           y0, y1);
  x0 = __float_as_uint(y0);
  x1 = __float_as_uint(y1);
}
__device__ __forceinline__ void keep_columns(uint32_t (&x)[32], int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < lo || i >= hi) x[i] = 0;
}
// (In two terms: what the rounding leaves, rounded, 32 columns further.)
template <bool kTwo>
__device__ __forceinline__ void put_bf16(uint32_t at, const uint32_t (&x)[32]) {
  uint32_t p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) p[i] = pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
  tmem_st16(at, p);
  if constexpr (kTwo) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      p[i] = pack(__uint_as_float(x[2 * i]) - __uint_as_float(p[i] << 16),
                  __uint_as_float(x[2 * i + 1]) - __uint_as_float(p[i] & 0xffff0000u));
    tmem_st16(at + 32, p);
  }
}

// A row's statistic as it stands in L2 (the queries' kernel may start beside the
// keys' one, without waiting for it, but after that has waited for the rows').
__device__ __forceinline__ float ld_stat(const float* p) {
  float v;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

// This CTA's job, from the list or the sequences; sm as locate() wants it.
template <int kN>
__device__ __forceinline__ bool find_job(const BwdArgs& a, bool keys, int64_t* sm, unsigned* status,
                                         Seq& seq, int& head) {
  head = blockIdx.x % a.s.kv_heads;
  const int64_t job = blockIdx.x / a.s.kv_heads;
  const Job* list = a.jobs[keys ? 0 : 1];
  if (!list) return locate<kN>(a.s, job, keys ? kRows : a.per, keys, !keys, sm, status, seq);
  if (job >= (int64_t)ld_relaxed_gpu((const uint32_t*)a.count[keys ? 0 : 1])) return false;
  const uint32_t* x = reinterpret_cast<const uint32_t*>(list + job);
  seq = {(int32_t)ld_relaxed_gpu(x), (int32_t)ld_relaxed_gpu(x + 1), (int32_t)ld_relaxed_gpu(x + 2),
         (int32_t)ld_relaxed_gpu(x + 3), (int32_t)ld_relaxed_gpu(x + 4)};
  return true;
}

// The common part of both kernels: the job's place, barriers, tensor memory.
template <int D>
__device__ __forceinline__ bool begin(const BwdArgs& a, uint8_t* sm, bool keys, Seq& seq, int& head) {
  using C = Bwd<D>;
  Bars& b = *reinterpret_cast<Bars*>(sm + C::kBars);
  const int tid = threadIdx.x, lane = tid & 31;
  // the swizzled tiles' pattern repeats every 1024 bytes (without static shared
  // memory the dynamic part starts on one)
  if (smem_u32(sm) & 1023u) {
    if (tid == 0) flag_status(a.status, GDN_ERR_UNSUPPORTED);
    return false;
  }
  if (!find_job<kThreads>(a, keys, reinterpret_cast<int64_t*>(sm), a.status, seq, head)) return false;
  if (tid == 0) {
    mbar_init(&b.own, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&b.a_full[i], 1);
      mbar_init(&b.a_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.b_full[i], 1);
      mbar_init(&b.b_empty[i], keys ? 2 : 1);
      mbar_init(&b.turn[i], 1);
      mbar_init(&b.ds_ready[i], 8);
      mbar_init(&b.s_full[i], 1);
    }
    mbar_init(&b.dp_full, 1);
    mbar_init(&b.p_ready, 8);
    mbar_init(&b.done, keys ? 2 : 1);
    fence_barrier_init();
  }
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (warp == 8) tmem_alloc(&b.tmem, 512);
  if (warp == 9 && lane == 0) {
    prefetch_tensormap(&a.q);
    prefetch_tensormap(&a.k);
    prefetch_tensormap(&a.v);
    prefetch_tensormap(&a.dout);
  }
  return true;
}
__device__ __forceinline__ void finish(bool ok, uint32_t tmem, unsigned* status) {
  if (!ok) {
    // copies and products in flight end within microseconds; give them longer
    flag_status(status, GDN_ERR_TIMEOUT);
    const uint64_t from = globaltimer_ns();
    while (globaltimer_ns() - from < 5000000ull) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x >> 5 == 8) tmem_dealloc(tmem, 512);
}

// A tile of 128 keys of a kv head: dK and dV.  Rows of all products are keys,
// so P^T and dS^T are A operands as they come; a column is a packed query row,
// whose statistics are read from shared memory.
// kTwo: P and dS as two bf16 terms each.
template <int D, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
keys_kernel(const __grid_constant__ BwdArgs a) {
  using C = Bwd<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  Bars& b = *reinterpret_cast<Bars*>(sm + C::kBars);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  Seq seq;
  int head;
  grid_wait();
  grid_release_next();   // the queries' kernel starts where SMs are left: it needs nothing of this one
  if (!begin<D>(a, sm, true, seq, head)) return;
  const int32_t group = a.s.group, shift = seq.lk - seq.lq;
  const int32_t k0 = seq.tile * kRows;                       // the tile's first key
  const int32_t used = a.per * group;                        // rows of a tile of queries
  // tiles of queries: from that of the first query that sees key k0
  const int32_t sees = k0 - shift > 0 ? k0 - shift : 0;
  const int32_t f0 = sees / a.per, f1 = sees < seq.lq ? (seq.lq + a.per - 1) / a.per : f0;
  // this CTA's part of them
  const int32_t t0 = f0 + (int32_t)((int64_t)(f1 - f0) * blockIdx.y / a.parts);
  const int32_t n = f0 + (int32_t)((int64_t)(f1 - f0) * (blockIdx.y + 1) / a.parts) - t0;
  // rows that no query fills take part in the products with P = dS = 0: zeros,
  // so that the products are
  if (used < kRows && warp < 5)
    zero_rows<D>(sm + (2 + warp) * C::kTile, used, lane);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = b.tmem;
  constexpr uint32_t kS = 0, kDP = 128, kDV = 256, kDK = 256 + D;
  bool ok = true;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 9) {
      // ----------------------------------------------------------- load
      const bool lead = elect_one();
      if (lead && n > 0) {
        mbar_arrive_expect_tx(&b.own, 2 * C::kTile);
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
          tma_load_3d(sm + h * kHalfTile, &a.k, 64 * h, head, (int32_t)(seq.k0 + k0), &b.own);
          tma_load_3d(sm + C::kTile + h * kHalfTile, &a.v, 64 * h, head, (int32_t)(seq.k0 + k0), &b.own);
        }
      }
      for (int32_t i = 0; ok && i < n; ++i) {
        const int32_t t = (int32_t)(seq.q0 + (int64_t)(t0 + i) * a.per);
        const int sa = i % C::kNA, sb = i % C::kNB;
        ok = mbar_wait_warp_cycles(&b.a_empty[sa], (uint32_t)((i / C::kNA) & 1) ^ 1u, kWaitCycles);
        if (ok && lead) {
          mbar_arrive_expect_tx(&b.a_full[sa], (uint32_t)used * 128 * C::kHalves);
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(sm + C::kA + sa * C::kTile + h * kHalfTile, &a.q, 64 * h, head * group, t,
                        &b.a_full[sa]);
        }
        __syncwarp();
        ok = ok && mbar_wait_warp_cycles(&b.b_empty[sb], (uint32_t)((i / C::kNB) & 1) ^ 1u, kWaitCycles);
        if (ok && lead) {
          mbar_arrive_expect_tx(&b.b_full[sb], (uint32_t)used * 128 * C::kHalves);
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(sm + C::kB + sb * C::kTile + h * kHalfTile, &a.dout, 64 * h, head * group, t,
                        &b.b_full[sb]);
        }
        __syncwarp();
      }
    } else if (warp == 8 || warp == 10) {
      // ------------------------------------------------------- multiply
      // One warp dV(i - 1) and S(i), one dK(i - 1) and dP(i), in turns: while one's
      // products run, the other waits for the operands that the first one's last
      // results become.  (All of it by one warp took its waits and commits besides
      // the products.)
      const int w = warp == 10;
      const bool lead = elect_one();
      const uint32_t base = smem_u32(sm);
      constexpr uint32_t kScores = idesc_bf16(128, 128, 0, 0), kGrad = idesc_bf16(128, D, 0, 1);
      // w: K (V) and the slots of Q (dO) for the scores, those of dO (Q) for the gradient
      const uint32_t mine = w ? C::kB : C::kA, other = w ? C::kA : C::kB;
      const uint64_t own = smem_desc(base + w * C::kTile, 16, 1024, kSwizzle128B);
      const uint64_t sd = smem_desc(base + mine, 16, 1024, kSwizzle128B);
      const uint64_t gd = smem_desc(base + other, kHalfTile, 1024, kSwizzle128B);
      const uint32_t s_at = tmem + (w ? kDP : kS), g_at = tmem + (w ? kDK : kDV);
      uint64_t* const s_done = w ? &b.dp_full : &b.s_full[0];
      // queries behind the sequence's last are another's: their rows become zeros
      auto clean = [&](uint32_t slots, int slot, int32_t i) {
        const int64_t rows = ((int64_t)seq.lq - (int64_t)(t0 + i) * a.per) * group;
        if (rows < used) {
          zero_rows<D>(sm + slots + slot * C::kTile, (int)rows, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
      };
      if (n > 0) ok = mbar_wait_warp_cycles(&b.own, 0, kWaitCycles);
      for (int32_t i = 0; ok && i <= n && n > 0; ++i) {
        const int sa = i % C::kNA, sb = i % C::kNB;                   // slots of step i ...
        const int ga = (i + C::kNA - 1) % C::kNA, gb = (i + C::kNB - 1) % C::kNB;   // ... and i - 1
        const int s_slot = w ? sb : sa, g_slot = w ? ga : gb;
        if (i < n) {
          ok = w ? mbar_wait_warp_cycles(&b.b_full[sb], (uint32_t)((i / C::kNB) & 1), kWaitCycles)
                 : mbar_wait_warp_cycles(&b.a_full[sa], (uint32_t)((i / C::kNA) & 1), kWaitCycles);
          if (ok) clean(mine, s_slot, i);
        }
        if (ok && i > 0 && !w) {   // (Q's slot: its scores are done, so it is there)
          ok = mbar_wait_warp_cycles(&b.b_full[gb], (uint32_t)(((i - 1) / C::kNB) & 1), kWaitCycles);
          if (ok) clean(other, gb, i - 1);
        }
        ok = ok && mbar_wait_warp_cycles(&b.turn[w], (uint32_t)(i & 1) ^ (w ? 0u : 1u), kWaitCycles);
        if (ok && i > 0)
          ok = mbar_wait_warp_cycles(w ? &b.ds_ready[0] : &b.p_ready, (uint32_t)((i - 1) & 1), kWaitCycles);
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          if (i > 0) {   // dV += P^T dO, dK += dS^T Q
#pragma unroll
            for (int s = 0; s < 8; ++s)
              mma_bf16_ts(g_at, s_at + (s >> 2) * 64 + (s & 3) * 8,
                          gd + (uint64_t)((g_slot * C::kTile + s * 2048) >> 4), kGrad, i > 1 || s > 0);
            if (kTwo)
#pragma unroll
              for (int s = 0; s < 8; ++s)
                mma_bf16_ts(g_at, s_at + 32 + (s >> 2) * 64 + (s & 3) * 8,
                            gd + (uint64_t)((g_slot * C::kTile + s * 2048) >> 4), kGrad, 1);
            if (w) mma_commit(&b.a_empty[ga]);
            else mma_commit(&b.b_empty[gb]);
          }
          if (i < n) {   // S^T = K Q^T, dP^T = V dO^T
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              mma_bf16(s_at, own + (uint64_t)(kstep(s) >> 4),
                       sd + (uint64_t)((s_slot * C::kTile + kstep(s)) >> 4), kScores, s > 0);
            mma_commit(s_done);
          }
          mbar_arrive(&b.turn[w ^ 1]);
          if (w && i < n) mma_commit(&b.b_empty[sb]);
          if (i == n) mma_commit(&b.done);
        }
        __syncwarp();
      }
    }
  } else {
    // ----------------------------------------------------------- P and dS
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int w = warp >> 2, row = tid & 127;             // the columns' half, the key
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_at = tmem + lanes + kS + 64 * w, dp_at = tmem + lanes + kDP + 64 * w;
    float* stats = reinterpret_cast<float*>(sm + C::kStats) + 128 * w;   // [2 buffers: + 256][64 | 64]
    const int64_t stat0 = ((int64_t)head * a.tq + seq.q0) * group;
    const bool fetch = row < 64;
    // column `row` of this half of tile i: its statistics, 0 where there is none
    auto read = [&](int32_t i, float& x, float& y) {
      const int col = 64 * w + row;
      const int64_t at = (int64_t)(t0 + i) * used + col;
      const bool on = fetch && i < n && col < used && at < (int64_t)seq.lq * group;
      x = on ? ld_stat(a.nlse + stat0 + at) : 0.f;
      y = on ? ld_stat(a.nd + stat0 + at) : 0.f;
    };
    float nl, nd;
    read(0, nl, nd);
    const F2 cc = f2(a.c, a.c);
    int32_t i = 0;
    for (; i < n; ++i) {
      float* st = stats + 256 * (i & 1);
      if (fetch) {
        st[row] = nl;
        st[64 + row] = nd;
      }
      bar_sync(1 + w, 128);
      read(i + 1, nl, nd);
      // the columns that see this key: [lo, hi)
      const int32_t q0 = (t0 + i) * a.per;
      const int64_t lo64 = ((int64_t)k0 + row - shift - q0) * group - 64 * w;
      const int64_t hi64 = ((int64_t)seq.lq - q0) * group;
      const int32_t lo = lo64 < 0 ? 0 : lo64 > 64 ? 64 : (int32_t)lo64;
      const int32_t hi = (hi64 < used ? (int32_t)hi64 : kRows) - 64 * w;   // (behind `used`: zeros)
      const bool masked = (int64_t)k0 + kRows - 1 - shift > q0 || hi64 < used;
      ok = mbar_wait_warp_cycles(&b.s_full[0], (uint32_t)(i & 1), kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      // half of the columns at a time: one half's loads and stores pass while the
      // other is computed (2 x 8192 tokens, heads of 64: 946 -> 864 us; of 128 the same)
      uint32_t s[2][32], g[2][32];
      tmem_ld32(s_at, s[0]);
      tmem_ld_wait_regs(s[0]);
      tmem_ld32(s_at + 32, s[1]);
      if (kTwo) tmem_ld_wait_regs(s[1]);   // (its place is written with the first half)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h) tmem_ld_wait_regs(s[1]);
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(st + 32 * h + x);
          exp_pair(s[h][x], s[h][x + 1], cc, f2(l4.x, l4.y));
          exp_pair(s[h][x + 2], s[h][x + 3], cc, f2(l4.z, l4.w));
        }
        if (masked) keep_columns(s[h], lo - 32 * h, hi - 32 * h);
        put_bf16<kTwo>(s_at + 16 * h, s[h]);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.p_ready);
      ok = mbar_wait_warp_cycles(&b.dp_full, (uint32_t)(i & 1), kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(dp_at, g[0]);
      tmem_ld_wait_regs(g[0]);
      tmem_ld32(dp_at + 32, g[1]);
      if (kTwo) tmem_ld_wait_regs(g[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h) tmem_ld_wait_regs(g[1]);
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const float4 d4 = *reinterpret_cast<const float4*>(st + 64 + 32 * h + x);
          times_less(g[h][x], g[h][x + 1], f2(d4.x, d4.y), s[h][x], s[h][x + 1]);
          times_less(g[h][x + 2], g[h][x + 3], f2(d4.z, d4.w), s[h][x + 2], s[h][x + 3]);
        }
        if (masked) keep_columns(g[h], lo - 32 * h, hi - 32 * h);
        put_bf16<kTwo>(dp_at + 16 * h, g[h]);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.ds_ready[0]);
    }
    // A wait of step i ran out: the warp goes on to meet the others of its warpgroup, whose waits
    // may have ended in time, at the barriers of the steps that are left, or they would wait
    // for ever.  (They get no further than their next waits, as the products want all warps'
    // P and dS.  Asking all of them in every step, bar_agree, took 4 % of the ragged batch.)
    if (!ok)
      while (++i < n) bar_sync(1 + w, 128);
    if (ok && n > 0) ok = mbar_wait_warp_cycles(&b.done, 0, kWaitCycles);
    tc_fence_after();
    if (ok) {
      // one warpgroup dV, the other dK
      const bool live = (int64_t)k0 + row < seq.lk;
      const uint32_t from = tmem + lanes + (w ? kDK : kDV);
      if (a.parts == 1) {
        const int64_t to = ((seq.k0 + k0 + row) * a.s.kv_heads + head) * D;
        store_row<D>(from, w ? a.scale : 1.f, (w ? a.dk : a.dv) + to, live, n == 0);
      } else {
        float* to = a.part + (((int64_t)blockIdx.x * a.parts + blockIdx.y) * 2 + w) * kRows * D;
        store_part<D>(from, to, row, n == 0);
      }
    }
  }
  finish(ok, tmem, a.status);
}

// A tile of packed query rows: dQ.
template <int D, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
queries_kernel(const __grid_constant__ BwdArgs a) {
  using C = Bwd<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  Bars& b = *reinterpret_cast<Bars*>(sm + C::kBars);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  Seq seq;
  int head;
  if (!begin<D>(a, sm, false, seq, head)) {
    grid_wait();   // as below: with no job at all, the keys' kernel may still read the sequences
    return;
  }
  const int32_t group = a.s.group, shift = seq.lk - seq.lq;
  const int32_t used = a.per * group;
  const int32_t first = seq.tile * a.per;                    // the tile's first query
  const int32_t rows = seq.lq - first < a.per ? seq.lq - first : a.per;
  const int32_t seen = first + rows + shift;                 // keys that the last row sees
  const int32_t all = seen > 0 ? (seen + kRows - 1) / kRows : 0;
  // this CTA's part of their blocks
  const int32_t j0 = (int32_t)((int64_t)all * blockIdx.y / a.q_parts);
  const int32_t n = (int32_t)((int64_t)all * (blockIdx.y + 1) / a.q_parts) - j0;
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = b.tmem;
  constexpr uint32_t kS = 0, kDP = 256, kDQ = 384;           // two buffers of scores
  bool ok = true;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 9) {
      // ----------------------------------------------------------- load
      const bool lead = elect_one();
      if (lead && n > 0) {
        mbar_arrive_expect_tx(&b.own, 2 * (uint32_t)used * 128 * C::kHalves);
        const int32_t t = (int32_t)(seq.q0 + first);
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
          tma_load_3d(sm + h * kHalfTile, &a.q, 64 * h, head * group, t, &b.own);
          tma_load_3d(sm + C::kTile + h * kHalfTile, &a.dout, 64 * h, head * group, t, &b.own);
        }
      }
      for (int32_t j = 0; ok && j < n; ++j) {
        const int32_t t = (int32_t)(seq.k0 + (int64_t)(j0 + j) * kRows);
        const int sa = j % C::kNA, sb = j % C::kNB;
        ok = mbar_wait_warp_cycles(&b.a_empty[sa], (uint32_t)((j / C::kNA) & 1) ^ 1u, kWaitCycles);
        if (ok && lead) {
          mbar_arrive_expect_tx(&b.a_full[sa], C::kTile);
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(sm + C::kA + sa * C::kTile + h * kHalfTile, &a.k, 64 * h, head, t, &b.a_full[sa]);
        }
        __syncwarp();
        ok = ok && mbar_wait_warp_cycles(&b.b_empty[sb], (uint32_t)((j / C::kNB) & 1) ^ 1u, kWaitCycles);
        if (ok && lead) {
          mbar_arrive_expect_tx(&b.b_full[sb], C::kTile);
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(sm + C::kB + sb * C::kTile + h * kHalfTile, &a.v, 64 * h, head, t, &b.b_full[sb]);
        }
        __syncwarp();
      }
    } else if (warp == 8 || warp == 10) {
      // ------------------------------------------------------- multiply
      // One warp dP(j + 1), as soon as dS(j) is there; then the other dQ(j) and
      // S(j + 2), while dS(j + 1) is made.  (Two barriers each for dS and for the
      // turn: either may be a step further than this warp, but not two, as S(j + 2)
      // comes from here.)
      const bool lead = elect_one();
      const uint32_t base = smem_u32(sm);
      constexpr uint32_t kScores = idesc_bf16(128, 128, 0, 0), kGrad = idesc_bf16(128, D, 0, 1);
      if (n > 0) ok = mbar_wait_warp_cycles(&b.own, 0, kWaitCycles);
      if (warp == 10) {
        const uint64_t own2 = smem_desc(base + C::kTile, 16, 1024, kSwizzle128B);
        const uint64_t bk = smem_desc(base + C::kB, 16, 1024, kSwizzle128B);
        for (int32_t j = 0; ok && j < n; ++j) {   // dP = dO V^T
          const int sb = j % C::kNB;
          ok = mbar_wait_warp_cycles(&b.b_full[sb], (uint32_t)((j / C::kNB) & 1), kWaitCycles);
          if (ok && j > 0)
            ok = mbar_wait_warp_cycles(&b.ds_ready[(j - 1) & 1], (uint32_t)(((j - 1) >> 1) & 1), kWaitCycles);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              mma_bf16(tmem + kDP, own2 + (uint64_t)(kstep(s) >> 4),
                       bk + (uint64_t)((sb * C::kTile + kstep(s)) >> 4), kScores, s > 0);
            mma_commit(&b.dp_full);
            if (j > 0) mbar_arrive(&b.turn[j & 1]);
            mma_commit(&b.b_empty[sb]);
          }
          __syncwarp();
        }
      } else {
        const uint64_t own = smem_desc(base, 16, 1024, kSwizzle128B);
        const uint64_t ak = smem_desc(base + C::kA, 16, 1024, kSwizzle128B);
        const uint64_t an = smem_desc(base + C::kA, kHalfTile, 1024, kSwizzle128B);
        // step j: dQ(j - 2) += dS K, then S(j) = Q K^T in the buffer of dS(j - 2)
        for (int32_t j = 0; ok && j < n + 2 && n > 0; ++j) {
          const int sa = j % C::kNA, ga = (j + 2 * C::kNA - 2) % C::kNA;
          if (j >= 2) {
            ok = mbar_wait_warp_cycles(&b.ds_ready[j & 1], (uint32_t)(((j - 2) >> 1) & 1), kWaitCycles);
            if (ok && j - 1 < n)   // dP(j - 1) goes first: turn[1] for odd ones, from 1; [0] from 2
              ok = mbar_wait_warp_cycles(&b.turn[(j - 1) & 1], (uint32_t)(((j - 2) >> 1) & 1), kWaitCycles);
            tc_fence_after();
            if (ok && lead) {
#pragma unroll
              for (int s = 0; s < 8; ++s)
                mma_bf16_ts(tmem + kDQ, tmem + kS + 128 * (j & 1) + (s >> 2) * 64 + (s & 3) * 8,
                            an + (uint64_t)((ga * C::kTile + s * 2048) >> 4), kGrad, j > 2 || s > 0);
              if (kTwo)
#pragma unroll
                for (int s = 0; s < 8; ++s)
                  mma_bf16_ts(tmem + kDQ, tmem + kS + 32 + 128 * (j & 1) + (s >> 2) * 64 + (s & 3) * 8,
                              an + (uint64_t)((ga * C::kTile + s * 2048) >> 4), kGrad, 1);
              mma_commit(&b.a_empty[ga]);
              if (j == n + 1) mma_commit(&b.done);
            }
            __syncwarp();
          }
          if (j < n) {
            ok = ok && mbar_wait_warp_cycles(&b.a_full[sa], (uint32_t)((j / C::kNA) & 1), kWaitCycles);
            // keys behind the sequence's last are another's: their rows become
            // zeros, so that the products with dS = 0 are
            const int64_t valid = seq.lk - (int64_t)(j0 + j) * kRows;
            if (ok && valid < kRows) {
              zero_rows<D>(sm + C::kA + sa * C::kTile, (int)valid, lane);
              fence_proxy_async_smem();
            }
            __syncwarp();
            tc_fence_after();
            if (ok && lead) {
#pragma unroll
              for (int s = 0; s < D / 16; ++s)
                mma_bf16(tmem + kS + 128 * (j & 1), own + (uint64_t)(kstep(s) >> 4),
                         ak + (uint64_t)((sa * C::kTile + kstep(s)) >> 4), kScores, s > 0);
              mma_commit(&b.s_full[j & 1]);
            }
            __syncwarp();
          }
        }
      }
    }
  } else {
    // ----------------------------------------------------------- P and dS
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int w = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const int qi = row / group;
    const bool live = qi < rows;
    const int64_t stat = ((int64_t)head * a.tq + seq.q0 + first) * group + row;
    const float nl = live ? ld_stat(a.nlse + stat) : 0.f, nd = live ? ld_stat(a.nd + stat) : 0.f;
    const int32_t last = first + qi + shift;               // the last key that the row sees
    const F2 cc = f2(a.c, a.c), ll = f2(nl, nl), dd = f2(nd, nd);
    for (int32_t j = 0; j < n; ++j) {
      const uint32_t s_at = tmem + lanes + kS + 128 * (j & 1) + 64 * w, dp_at = tmem + lanes + kDP + 64 * w;
      const int32_t k0 = (j0 + j) * kRows;
      const bool masked = k0 + kRows - 1 > first + shift;
      const int32_t see = last - k0 - 64 * w;
      ok = mbar_wait_warp_cycles(&b.s_full[j & 1], (uint32_t)((j >> 1) & 1), kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[2][32];
#pragma unroll
      for (int h = 0; h < 2; ++h) tmem_ld32(s_at + 32 * h, s[h]);
#pragma unroll
      for (int h = 0; h < 2; ++h) tmem_ld_wait_regs(s[h]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < 32; x += 2) exp_pair(s[h][x], s[h][x + 1], cc, ll);
      ok = mbar_wait_warp_cycles(&b.dp_full, (uint32_t)(j & 1), kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      uint32_t g[2][32];
#pragma unroll
      for (int h = 0; h < 2; ++h) tmem_ld32(dp_at + 32 * h, g[h]);
#pragma unroll
      for (int h = 0; h < 2; ++h) tmem_ld_wait_regs(g[h]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < 32; x += 2)
          times_less(g[h][x], g[h][x + 1], dd, s[h][x], s[h][x + 1]);
      if (masked) {
        keep_columns(g[0], 0, see + 1);
        keep_columns(g[1], 0, see - 31);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) put_bf16<kTwo>(s_at + 16 * h, g[h]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.ds_ready[j & 1]);
    }
    if (ok && n > 0) ok = mbar_wait_warp_cycles(&b.done, 0, kWaitCycles);
    tc_fence_after();
    if (ok) {
      // half the columns each
      const int64_t r = (seq.q0 + first + qi) * a.q_heads + (int64_t)head * group + row % group;
      const uint32_t from = tmem + lanes + kDQ + D / 2 * w;
      if (a.q_parts == 1)
        store_row<D / 2>(from, a.scale, a.dq + r * D + D / 2 * w, live, n == 0);
      else
        store_part<D / 2>(from,
                          a.q_part + ((int64_t)blockIdx.x * a.q_parts + blockIdx.y) * kRows * D +
                              D / 2 * w * kRows,
                          row, n == 0);
    }
  }
  finish(ok, tmem, a.status);
  grid_wait();   // the keys' kernel, beside which this one ran, is part of the call
}

__global__ void __launch_bounds__(kListThreads) backward_list_kernel(ListArgs keys, ListArgs queries) {
  grid_wait();
  grid_release_next();
  list_jobs(blockIdx.x ? queries : keys);
}

// The parts of a tile's dV and dK, or dQ, added in their order: 8 columns of a row a
// thread.
template <int D, bool kKeys>
__global__ void __launch_bounds__(kThreads) sum_kernel(const __grid_constant__ BwdArgs a) {
  __shared__ int64_t scratch[kThreads + 6];
  Seq seq;
  int head;
  grid_wait();
  grid_release_next();
  if (!find_job<kThreads>(a, kKeys, scratch, nullptr, seq, head)) return;
  constexpr int kVecs = kRows * D / 8, kTensors = kKeys ? 2 : 1;
  const int group = a.s.group;
  const int64_t first = (int64_t)seq.tile * (kKeys ? kRows : a.per);
  const float* part = kKeys ? a.part : a.q_part;
  const int parts = kKeys ? a.parts : a.q_parts;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < kTensors * kVecs; i += gridDim.y * kThreads) {
    const int row = i % kRows, col = i / kRows % (D / 8) * 8, w = i / kVecs;
    const int64_t t = first + (kKeys ? row : row / group);
    if (t >= (kKeys ? seq.lk : seq.lq) || (!kKeys && row >= a.per * group)) continue;
    const float* from = part + (((int64_t)blockIdx.x * parts * kTensors + w) * D + col) * kRows + row * 4;
    float sum[8] = {};
#pragma unroll 4
    for (int p = 0; p < parts; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 x = ld_waited(reinterpret_cast<const float4*>(
            from + (int64_t)p * kTensors * kRows * D + h * 4 * kRows));
        sum[4 * h] += x.x; sum[4 * h + 1] += x.y; sum[4 * h + 2] += x.z; sum[4 * h + 3] += x.w;
      }
    const float f = kKeys && w == 0 ? 1.f : a.scale;
    __nv_bfloat16* to = kKeys ? (w ? a.dk : a.dv) + ((seq.k0 + t) * a.s.kv_heads + head) * D + col
                              : a.dq + ((seq.q0 + t) * a.q_heads + (int64_t)head * group + row % group) * D + col;
    *reinterpret_cast<uint4*>(to) = make_uint4(pack(sum[0] * f, sum[1] * f), pack(sum[2] * f, sum[3] * f),
                                               pack(sum[4] * f, sum[5] * f), pack(sum[6] * f, sum[7] * f));
  }
}

// Fewer rows than this: P and dS enter their products as two bf16 terms each, which loses
// 2^-16 of them, and a gradient carries its own rounding alone.  With one term each of them
// carries theirs too, as large, together about sqrt(2) times its own (1.39 to 1.43 over 2000
// tokens; in 200 batches of 700 to 12000 rows 1.49 at most, over fewer rows more, as few
// terms need not average).  Both are within the bound of one rounding of P and dS; the
// second terms are three products more than seven, which few rows hide best (16/4 heads of 128, one
// term and two: 17 tokens behind 1183 17.4 and 21.5 us, 300 tokens, above, 25 and 30, 8192 550 and 750).
constexpr int64_t kTwoTerms = 4096;

// How a call is launched, and its scratch.
struct Plan {
  int64_t key_tiles, query_tiles;   // packed: upper bounds, sum_n ceil(len_n / per) <= T / per + N
  bool listed;
  int32_t parts, q_parts;
  size_t stat, key_jobs, query_jobs, part, q_part, bytes;   // statistics, then where the others lie
};
constexpr int kLeastSteps = 6, kMostParts = 16;   // steps of a part, parts of a loop
// Parts of a loop of `iters` steps (about 1.2 us each) for `jobs` of them: as many
// as minimise the longest's time and that of the parts' sums, of `bytes` each, out
// and in again (at about 4 TB/s), where that is not less than what the SMs have to do
// meanwhile anyway.
int32_t parts_of(int64_t jobs, int64_t iters, int sms, int64_t bytes) {
  if (jobs == 0 || iters < 2 * kLeastSteps) return 1;
  const float sums = (float)jobs * (float)bytes * 2.f / 4e6f, loop = (float)iters * 1.2f;
  const float share = (float)jobs * (float)iters * 0.9f / (float)sms;   // of both kernels, us
  int32_t best = 1;
  float least_time = fmaxf(loop, share);
  for (int32_t p = 2; p <= kMostParts && p * kLeastSteps <= iters; ++p) {
    const float t = fmaxf(loop / (float)p, share) + (float)p * sums + 4.f;
    if (t < least_time) {
      least_time = t;
      best = p;
    }
  }
  return best;
}
Plan plan_of(const Shape& s, int sms) {
  const int32_t per = kRows / (s.q_heads / s.kv_heads);
  Plan p = {};
  const int64_t tq = s.tq(), tk = s.tk(), iters = (s.seqlen_q + per - 1) / per,
                blocks = (s.seqlen_k + kRows - 1) / kRows;
  p.key_tiles = s.packed ? tk / kRows + s.batch : blocks * s.batch;
  p.query_tiles = s.packed ? tq / per + s.batch : iters * s.batch;
  if (tk == 0) p.key_tiles = 0;
  const int64_t key_jobs = p.key_tiles * s.kv_heads, query_jobs = p.query_tiles * s.kv_heads;
  p.listed = key_jobs > 2 * sms || query_jobs > 2 * sms;
  const int64_t tile = (int64_t)kRows * s.d * 4;
  // (packed: no sequence is taken to be longer than four average ones)
  const int64_t few = s.packed && s.batch > 4 ? s.batch : 4;
  p.parts = parts_of(key_jobs, s.packed ? iters * 4 / few : iters, sms, 2 * tile);
  p.q_parts = parts_of(query_jobs, s.packed ? blocks * 4 / few : blocks, sms, tile);
  p.stat = align_up(s.rows() * 4, 256);
  p.bytes = 2 * p.stat;
  if (p.listed) {
    p.key_jobs = p.bytes + 256;       // counts before
    p.query_jobs = p.key_jobs + align_up((size_t)p.key_tiles * sizeof(Job), 256);
    p.bytes = p.query_jobs + align_up((size_t)p.query_tiles * sizeof(Job), 256);
  }
  p.part = p.bytes;
  if (p.parts > 1) p.bytes += (size_t)key_jobs * p.parts * 2 * tile;
  p.q_part = p.bytes;
  if (p.q_parts > 1) p.bytes += (size_t)query_jobs * p.q_parts * tile;
  return p;
}

// What gdn_attention_prefill_backward_workspace_size answers: at least plan_of()'s bytes of this
// problem and of every one with no more sequences, queries and keys, so that a workspace for
// the largest serves all.  (plan_of()'s own are no such bound: one sequence of 8192 tokens, 16/4
// heads of 128, has enough jobs without parts, one of 4096 needs 33 MB for their sums.)
// parts_of() makes parts only where a loop is longer than its share of the work, J 0.9 / sms < 1.2
// for J jobs, and no more of them than bring it below that: J p < 4/3 sms + J < 3 sms.
size_t workspace_bound(const Shape& s, int sms) {
  const int32_t per = kRows / (s.q_heads / s.kv_heads);
  const int64_t tq = s.tq(), tk = s.tk();
  const int64_t key_tiles = tk ? tk / kRows + s.batch : 0, query_tiles = tq / per + s.batch;
  const int64_t key_jobs = key_tiles * s.kv_heads, query_jobs = query_tiles * s.kv_heads;
  size_t bytes = 2 * align_up(s.rows() * 4, 256);
  if (key_jobs > 2 * sms || query_jobs > 2 * sms)
    bytes += 256 + align_up((size_t)key_tiles * sizeof(Job), 256) +
             align_up((size_t)query_tiles * sizeof(Job), 256);
  auto sums = [&](int64_t jobs, int64_t tokens, int64_t step, int64_t each) {
    const int64_t most = (tokens + step - 1) / step / kLeastSteps;   // parts of the longest loop
    if (most < 2) return (int64_t)0;
    const int64_t parts = jobs * (most < kMostParts ? most : kMostParts);
    return (parts < 3 * sms ? parts : 3 * sms) * each;
  };
  const int64_t tile = (int64_t)kRows * s.d * 4;
  return bytes + (size_t)sums(key_jobs, tq, per, 2 * tile) + (size_t)sums(query_jobs, tk, kRows, tile);
}

int backward(const void* q, const void* k, const void* v, const void* out, const float* lse,
             const void* dout, const int32_t* cu_q, const int32_t* cu_k, float scale, void* dq,
             void* dk, void* dv, const Shape& s, bool use_ws, void* ws, size_t ws_bytes,
             cudaStream_t st) {
  if (const int rc = check_shape(s, cu_q, cu_k, scale)) return rc;
  const int64_t tq = s.tq(), tk = s.tk();
  if (tq > 0 && (!q || !out || !lse || !dout || !dq)) return GDN_ERR_INVALID_ARG;
  if (tk > 0 && (!k || !v || !dk || !dv)) return GDN_ERR_INVALID_ARG;
  const void* v16[] = {q, k, v, out, dout, dq, dk, dv};
  for (const void* p : v16)
    if (!aligned(p, 16)) return GDN_ERR_ALIGNMENT;
  if (!aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(cu_k, 4)) return GDN_ERR_ALIGNMENT;
  const int sms = sm_count();
  const Plan plan = plan_of(s, sms > 0 ? sms : 152);
  const size_t need = tq ? plan.bytes : 0;
  if (use_ws && need) {
    if (!ws || ws_bytes < need) return GDN_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return GDN_ERR_ALIGNMENT;
  }
  const size_t cu_bytes = ((size_t)s.batch + 1) * 4, io = s.rows() * s.d * 2,
               kio = (size_t)tk * s.kv_heads * s.d * 2;
  const Span ins[] = {span_of(q, s.q_bytes()), span_of(k, s.k_bytes(s.k_stride)),
                      span_of(v, s.k_bytes(s.v_stride)), span_of(cu_q, cu_bytes),
                      span_of(cu_k, cu_bytes), span_of(out, io), span_of(dout, io),
                      span_of(lse, s.rows() * 4)};
  const Span outs[] = {span_of(dq, io), span_of(dk, kio), span_of(dv, kio),
                       span_of(use_ws ? ws : nullptr, need)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  if (tq == 0 && tk == 0 && !s.packed) return GDN_OK;
  BwdArgs a;
  memset(&a, 0, sizeof a);
  a.status = status_ptr();
  if (!a.status || sms < 1) return GDN_ERR_CUDA;
  const int32_t group = s.q_heads / s.kv_heads;
  a.s = {cu_q, cu_k, s.batch, s.seqlen_q, s.seqlen_k, group, s.kv_heads};
  if (tq == 0) {   // keys that no query sees
    cudaError_t e;
    if (s.packed) {
      e = no_queries(a.s, dk, dv, kio, a.status, st);
    } else {
      e = cudaMemsetAsync(dk, 0, kio, st);
      if (e == cudaSuccess) e = cudaMemsetAsync(dv, 0, kio, st);
    }
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
  }
  a.dq = (__nv_bfloat16*)dq;
  a.dk = (__nv_bfloat16*)dk;
  a.dv = (__nv_bfloat16*)dv;
  a.c = scale * kLog2e;
  a.scale = scale;
  a.tq = tq;
  a.q_heads = s.q_heads;
  a.per = kRows / group;
  // (no keys: nothing is loaded through their maps)
  const int64_t width = (int64_t)s.kv_heads * s.d;
  if (!heads_map(&a.q, q, tq, s.q_heads, s.d, s.q_stride, group, a.per) ||
      !heads_map(&a.dout, dout, tq, s.q_heads, s.d, (int64_t)s.q_heads * s.d, group, a.per) ||
      !heads_map(&a.k, tk ? k : q, tk, s.kv_heads, s.d, tk ? s.k_stride : width, 1, kRows) ||
      !heads_map(&a.v, tk ? v : q, tk, s.kv_heads, s.d, tk ? s.v_stride : width, 1, kRows))
    return GDN_ERR_CUDA;
  const int64_t row_ctas = ((int64_t)s.rows() * (s.d / 8) + 255) / 256;
  if (plan.key_tiles * s.kv_heads > 0x7fffffffLL || plan.query_tiles * s.kv_heads > 0x7fffffffLL || row_ctas > 0x7fffffffLL)
    return GDN_ERR_UNSUPPORTED;
  void* scratch = ws;
  if (!use_ws && scratch_alloc(&scratch, need, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
  }
  char* base = (char*)scratch;
  a.nlse = (float*)base;
  a.nd = (float*)(base + plan.stat);
  a.parts = plan.parts;
  a.q_parts = plan.q_parts;
  a.part = (float*)(base + plan.part);
  a.q_part = (float*)(base + plan.q_part);
  cudaError_t e = cudaSuccess;
  if (plan.listed) {
    int32_t* head = (int32_t*)(base + plan.key_jobs - 256);
    auto unit = [](int64_t len, int64_t per) {
      return (int32_t)(((len + per - 1) / per + kLevels - 1) / kLevels);
    };
    const ListArgs keys = {a.s, kRows, unit(s.seqlen_k, kRows) > 0 ? unit(s.seqlen_k, kRows) : 1, true,
                           head, (uint32_t*)head + 1, (Job*)(base + plan.key_jobs), a.status};
    const ListArgs queries = {a.s, a.per, unit(s.seqlen_q, a.per), false,
                              head + 2, (uint32_t*)head + 3, (Job*)(base + plan.query_jobs), a.status};
    a.count[0] = head;
    a.count[1] = head + 2;
    a.jobs[0] = (const Job*)(base + plan.key_jobs);
    a.jobs[1] = (const Job*)(base + plan.query_jobs);
    e = launch(true, backward_list_kernel, dim3(2), kListThreads, 0, 0, st, keys, queries);
    count_launches(1);
  }
  const RowArgs r = {(const __nv_bfloat16*)out, (const __nv_bfloat16*)dout, lse, (float*)a.nlse,
                     (float*)a.nd, tq, s.q_heads, group};
  if (e == cudaSuccess)
    e = launch(true, s.d == 128 ? rows_kernel<128> : rows_kernel<64>, dim3((unsigned)row_ctas), 256, 0, 0,
               st, r);
  auto run = [&](auto shape, auto kern, int64_t tiles, int parts, std::atomic<uint64_t>& on) {
    using C = decltype(shape);
    if (e != cudaSuccess || tiles == 0) return;
    e = allow_smem((const void*)kern, C::kSmem, on);
    if (e == cudaSuccess)
      e = launch(true, kern, dim3((unsigned)(tiles * s.kv_heads), (unsigned)parts), kThreads, C::kSmem,
                 0, st, a);
    count_launches(1);
  };
  static std::atomic<uint64_t> on[8];
  auto both = [&](auto shape, auto keys, auto queries, int i) {
    run(shape, keys, plan.key_tiles, plan.parts, on[i]);
    run(shape, queries, plan.query_tiles, plan.q_parts, on[i + 1]);
  };
  const bool two = (int64_t)s.rows() < kTwoTerms;
  if (s.d == 128 && two) both(Bwd<128>{}, keys_kernel<128, true>, queries_kernel<128, true>, 0);
  else if (s.d == 128) both(Bwd<128>{}, keys_kernel<128, false>, queries_kernel<128, false>, 2);
  else if (two) both(Bwd<64>{}, keys_kernel<64, true>, queries_kernel<64, true>, 4);
  else both(Bwd<64>{}, keys_kernel<64, false>, queries_kernel<64, false>, 6);
  auto join = [&](bool on_, auto kern, int64_t tiles) {
    if (!on_ || e != cudaSuccess) return;
    e = launch(true, kern, dim3((unsigned)(tiles * s.kv_heads), 4), kThreads, 0, 0, st, a);
    count_launches(1);
  };
  join(plan.parts > 1, s.d == 128 ? sum_kernel<128, true> : sum_kernel<64, true>, plan.key_tiles);
  join(plan.q_parts > 1, s.d == 128 ? sum_kernel<128, false> : sum_kernel<64, false>, plan.query_tiles);
  count_launches(1);
  if (e != cudaSuccess) (void)cudaGetLastError();
  const cudaError_t f = use_ws ? cudaSuccess : scratch_free(scratch, st);
  return e == cudaSuccess && f == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_attention_prefill_backward(const void* q, const void* k, const void* v, const void* out,
                                   const float* lse, const void* dout, const int32_t* cu_q,
                                   const int32_t* cu_k, float scale, void* dq, void* dk, void* dv,
                                   int32_t batch, int64_t seqlen_q, int64_t seqlen_k,
                                   int32_t q_heads, int32_t kv_heads, int32_t d, int64_t q_stride,
                                   int64_t k_stride, int64_t v_stride, gdn_stream_t stream) {
  const attn::Shape s = {batch, seqlen_q, seqlen_k, q_heads, kv_heads, d, q_stride, k_stride,
                         v_stride, cu_q != nullptr};
  return backward(q, k, v, out, lse, dout, cu_q, cu_k, scale, dq, dk, dv, s, false, nullptr, 0,
                  (cudaStream_t)stream);
}

size_t gdn_attention_prefill_backward_workspace_size(int32_t batch, int64_t seqlen_q,
                                                     int64_t seqlen_k, int32_t varlen,
                                                     int32_t q_heads, int32_t kv_heads, int32_t d) {
  const int32_t some = 0;
  const int64_t width = (int64_t)q_heads * d;
  const attn::Shape s = {batch, seqlen_q, seqlen_k, q_heads, kv_heads, d, width, width, width,
                         varlen != 0};
  if (attn::check_shape(s, varlen ? &some : nullptr, varlen ? &some : nullptr, 1.f)) return SIZE_MAX;
  const int sms = hostcheck::sm_count();
  return s.tq() ? workspace_bound(s, sms > 0 ? sms : 152) : 0;
}

int gdn_attention_prefill_backward_ws(const void* q, const void* k, const void* v,
                                      const void* out, const float* lse, const void* dout,
                                      const int32_t* cu_q, const int32_t* cu_k, float scale,
                                      void* dq, void* dk, void* dv, int32_t batch,
                                      int64_t seqlen_q, int64_t seqlen_k, int32_t q_heads,
                                      int32_t kv_heads, int32_t d, int64_t q_stride,
                                      int64_t k_stride, int64_t v_stride, void* workspace,
                                      size_t workspace_bytes, gdn_stream_t stream) {
  const attn::Shape s = {batch, seqlen_q, seqlen_k, q_heads, kv_heads, d, q_stride, k_stride,
                         v_stride, cu_q != nullptr};
  return backward(q, k, v, out, lse, dout, cu_q, cu_k, scale, dq, dk, dv, s, true, workspace,
                  workspace_bytes, (cudaStream_t)stream);
}

}  // extern "C"
