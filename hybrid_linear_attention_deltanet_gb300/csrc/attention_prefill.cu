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
// scores (128 x 128 fp32) and outputs fill tensor memory; while four warps take
// the exponentials of one tile's scores, the tensor cores work on the other
// tile, whose products a warp of its own issues, the two warps in turns:
//   P0 V(j-1), Q0 K(j)^T | P1 V(j-1), Q1 K(j)^T | ...
// The probabilities go back to tensor memory as bf16, over the scores that they
// came from, and are the A operand of the second product there.
//
// 16 query and 4 kv heads of 128: 4 x 8192 tokens 690 us call after call (1594 TFLOP/s, at the
// 1400 W limit), 600 to 625 in a run too short for that limit; in such runs 8192 156, 1024 14;
// heads of 64, whose exponentials take as long as their products: 2 x 8192 tokens 245 to 274
// (258 where 251 is now with the probabilities over the scores).
// Tried and slower: a pair of CTAs on one tile of keys (979 us where one CTA with one
// multiplying warp took 736), four warpgroups of exponentials (fewer registers than a
// row's scores).
#include "attention_tc.cuh"

namespace gdn {
namespace {

using namespace attn;
using namespace sm100;

// two warpgroups of softmax; a third with a warp to multiply and one to load
constexpr int kThreads = 384;
constexpr uint32_t kTileBytes = 16384;   // 128 rows x 64 columns bf16
// A row's maximum is replaced where it grows by more than 2^8: the probabilities then reach
// 2^8, and their rounding to bf16, which is relative, has the same bound.  In a call of few
// rows (below kFewRows) it is replaced wherever it grows, so that the largest probability is
// 1, which bf16 holds exactly: a result carries 1.25 instead of 1.26 times its own rounding,
// and that costs nothing there (17 tokens behind 1183 10 us both ways; 300 tokens, above,
// 8.5 -> 8.8, 8192 156 -> 175).
constexpr float kGrow = 8.f;
constexpr int64_t kFewRows = 512;
constexpr float kLowest = -3.402823466e38f;

struct FwdArgs {
  CUtensorMap q, k, v;
  Seqs s;
  __nv_bfloat16* out;
  float* lse;
  float c;                 // scale log2 e
  float grow;
  int32_t q_heads, per;    // per: queries of a 128-row tile
  int32_t tiles;           // of a job: 2, or 1 where there are few
  // kListed: the jobs
  const int32_t* count;
  uint32_t* next;
  const Job* jobs;
  // kParts: what the parts of a job leave for join_kernel, [jobs][parts][256 rows]
  int32_t parts;
  int64_t* dest;           // [jobs][256] the row's place in lse, -1: none
  float2* ml;              // maximum (in powers of two) and sum, 0 where the part saw no key
  float* o;                // [jobs][parts][D / 4][256][4]
  unsigned* status;
};

// How a CTA comes to its work: kOnce, one job each; kParts, blockIdx.y's part of
// a job's keys; kListed, persistent CTAs take the next job of a list.
enum Mode { kOnce, kParts, kListed };

template <int D>
struct Fwd {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTile = kHalves * kTileBytes;     // of Q, K or V
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr uint32_t kSmem = 2 * kTile + kStages * kTile + 1024;
  // Tensor-memory columns: scores, + tile * 128; probabilities and outputs.  Heads of
  // 64 leave room for probabilities of their own: the next block's scores come as
  // soon as this one's are in registers.
  static constexpr bool kEarly = D == 64;
  static constexpr uint32_t kS = 0, kP = kEarly ? 256 : 0, kPStep = kEarly ? 64 : 128;
  static constexpr uint32_t kO = kEarly ? 384 : 256, kOStep = D;
};

// 128 rows x 64 columns a half, K-major: 16 columns a step
__device__ __forceinline__ uint32_t kstep(int s) { return (s >> 2) * kTileBytes + (s & 3) * 32; }

// What every warp derives from a job: its tiles' first queries, their numbers,
// and the blocks of 128 keys [begin, end) that this CTA goes over.
struct Place {
  int64_t q0, k0;
  int32_t lk, shift, first[2], rows[2], blocks[2], begin, most;
  // (indexed by selection: a tile's number is no constant in the softmax warps)
  __device__ __forceinline__ int32_t first_of(int w) const { return w ? first[1] : first[0]; }
  __device__ __forceinline__ int32_t rows_of(int w) const { return w ? rows[1] : rows[0]; }
  __device__ __forceinline__ int32_t blocks_of(int w) const { return w ? blocks[1] : blocks[0]; }
  __device__ __forceinline__ Place(const Seq& s, const FwdArgs& a, int part, int parts) {
    const int per = a.per;
    q0 = s.q0;
    k0 = s.k0;
    lk = s.lk;
    shift = s.lk - s.lq;
    int32_t n[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      first[w] = (s.tile * a.tiles + w) * per;
      const int32_t left = w < a.tiles ? s.lq - first[w] : 0;
      rows[w] = left < 0 ? 0 : left < per ? left : per;
      const int32_t seen = rows[w] ? first[w] + rows[w] + shift : 0;   // keys that the last row sees
      n[w] = seen > 0 ? (seen + kRows - 1) / kRows : 0;
    }
    const int32_t all = n[1] > n[0] ? n[1] : n[0];
    begin = parts > 1 ? (int32_t)((int64_t)all * part / parts) : 0;
    const int32_t end = parts > 1 ? (int32_t)((int64_t)all * (part + 1) / parts) : all;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int32_t e = n[w] < end ? n[w] : end;
      blocks[w] = e > begin ? e - begin : 0;
    }
    most = end - begin;
  }
};

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ FwdArgs a) {
  using C = Fwd<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align_smem_1024(smem_raw);
  __shared__ uint64_t q_full, q_empty, kv_full[C::kStages], kv_empty[C::kStages], s_full[2],
      p_half[2], p_full[2], o_full[2], job_full[2], job_empty[2], turn[2], s_free[2];
  __shared__ uint32_t tmem_base;
  __shared__ int64_t scratch[kMode == kListed ? 1 : kThreads + 6];
  __shared__ Seq slots[2];
  __shared__ int32_t slot_head[2];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const Seqs& sq = a.s;
  if (tid == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 2);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&turn[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&job_full[i], 1);
      mbar_init(&job_empty[i], 10);
    }
    fence_barrier_init();
  }
  if (warp == 8) tmem_alloc(&tmem_base, 512);
  if (warp == 9 && lane == 0) {
    prefetch_tensormap(&a.q);
    prefetch_tensormap(&a.k);
    prefetch_tensormap(&a.v);
  }
  // (behind the allocation: a dependent that took this SM's columns first would wait for this
  // grid's end, and this grid for the columns)
  __syncthreads();
  grid_release_next();
  grid_wait();
  bool here = true;
  if constexpr (kMode != kListed) {
    Seq seq;
    here = locate<kThreads>(sq, blockIdx.x / sq.kv_heads, a.tiles * a.per, false, true, scratch, a.status, seq);
    if (here && tid == 0) {
      slots[0] = seq;
      slot_head[0] = blockIdx.x % sq.kv_heads;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  if (!here) {
    if (warp == 8) tmem_dealloc(tmem, 512);
    if (kMode == kParts && blockIdx.y == 0 && tid < 256) a.dest[(int64_t)blockIdx.x * 256 + tid] = -1;
    return;
  }
  const int part = kMode == kParts ? blockIdx.y : 0, parts = kMode == kParts ? a.parts : 1;
  bool ok = true;

  // The next job for a warp that multiplies or takes exponentials (`n` counts
  // them): false when there is none.  It stays in its slot until release().
  auto take = [&](uint32_t n, Seq& s) {
    if constexpr (kMode != kListed) {
      if (n > 0) return false;
      s = slots[0];
      return true;
    } else {
      ok = mbar_wait_warp_cycles(&job_full[n & 1], (n >> 1) & 1, kWaitCycles);
      if (!ok) return false;
      s = slots[n & 1];
      return s.tile >= 0;
    }
  };
  auto release = [&](uint32_t n) {
    if constexpr (kMode == kListed) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&job_empty[n & 1]);
    }
  };

  // 384 threads launch with 168 registers each, 64512 in all, which is 256 x 216
  // + 128 x 72: a softmax thread holds a row's 128 scores
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 9) {
      // ----------------------------------------------------------- load
      const bool lead = elect_one();
      uint32_t kv = 0, jobs_done = 0;     // loads so far; jobs with keys so far
      for (uint32_t n = 0; ok; ++n) {
        Seq seq;
        int head;
        if constexpr (kMode == kListed) {
          int64_t at = 0;
          if (lane == 0) at = atomicAdd(a.next, 1u);
          at = __shfl_sync(0xffffffffu, at, 0);
          ok = mbar_wait_warp_cycles(&job_empty[n & 1], ((n >> 1) & 1) ^ 1u, kWaitCycles);
          if (!ok) break;
          int32_t count;
          asm volatile("ld.global.s32 %0, [%1];" : "=r"(count) : "l"(a.count));
          const bool more = at < (int64_t)count * sq.kv_heads;
          seq.tile = -1;
          head = 0;
          if (more) {
            const int64_t i = at / sq.kv_heads;
            head = (int)(at - i * sq.kv_heads);
            const uint4 x = ld_waited(reinterpret_cast<const uint4*>(a.jobs + i));
            const int32_t tile = ld_waited(&a.jobs[i].tile);
            seq = {(int32_t)x.x, (int32_t)x.y, (int32_t)x.z, (int32_t)x.w, tile};
          }
          if (lane == 0) {
            slots[n & 1] = seq;
            slot_head[n & 1] = head;
            mbar_arrive(&job_full[n & 1]);
          }
          __syncwarp();
          if (!more) break;
        } else {
          if (!take(n, seq)) break;
          head = slot_head[0];
        }
        const Place pl(seq, a, part, parts);
        if (pl.most == 0) continue;
        ok = mbar_wait_warp_cycles(&q_empty, (jobs_done & 1) ^ 1u, kWaitCycles);
        if (!ok) break;
        ++jobs_done;
        if (lead) {
          const uint32_t box = (uint32_t)(a.per * sq.group) * 128 * C::kHalves;
          const int tiles = pl.rows[1] > 0 ? 2 : 1;
          mbar_arrive_expect_tx(&q_full, tiles * box);
          for (int w = 0; w < tiles; ++w)
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_3d(sm + w * C::kTile + h * kTileBytes, &a.q, 64 * h, head * sq.group,
                          (int32_t)(pl.q0 + pl.first_of(w)), &q_full);
        }
        for (int32_t j = 0; ok && j < pl.most; ++j) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t st = kv % C::kStages;
            ok = ok && mbar_wait_warp_cycles(&kv_empty[st], ((kv / C::kStages) & 1) ^ 1u, kWaitCycles);
            if (ok && lead) {
              uint8_t* to = sm + (2 + st) * C::kTile;
              mbar_arrive_expect_tx(&kv_full[st], C::kTile);
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h)
                tma_load_3d(to + h * kTileBytes, x ? &a.v : &a.k, 64 * h, head,
                            (int32_t)(pl.k0 + (int64_t)(pl.begin + j) * kRows), &kv_full[st]);
            }
            __syncwarp();
            ++kv;
          }
        }
      }
    } else if (warp == 8 || warp == 10) {
      // ------------------------------------------------------- multiply
      // A warp for each tile: waiting and issuing for both took one warp 3200
      // cycles a block, half as long again as the products.  They take turns, so that
      // one tile's products run while the other's probabilities are made; left to
      // themselves both wait for these at the same time.
      const int w = warp == 10;
      const bool lead = elect_one();
      const uint32_t base = smem_u32(sm);
      constexpr uint32_t kScores = idesc_bf16(128, 128, 0, 0), kOut = idesc_bf16(128, D, 0, 1);
      const uint64_t qd = smem_desc(base + w * C::kTile, 16, 1024, kSwizzle128B);
      const uint64_t kd = smem_desc(base + 2 * C::kTile, 16, 1024, kSwizzle128B);
      const uint64_t vd = smem_desc(base + 2 * C::kTile, kTileBytes, 1024, kSwizzle128B);
      const uint32_t s_at = tmem + C::kS + 128 * w, o_at = tmem + C::kO + C::kOStep * w;
      const uint32_t p_at = tmem + C::kP + C::kPStep * w;
      uint32_t kv = 0, jobs_done = 0, steps = 0, probs = 0;   // (probs: the tile's blocks so far)
      uint32_t scored = 0;                                    // (scores of it so far)
      Seq seq;
      for (uint32_t n = 0; ok && take(n, seq); ++n) {
        int32_t most, blocks, last;      // last: keys of the last block
        {
          const Place pl(seq, a, part, parts);
          most = pl.most;
          blocks = pl.blocks_of(w);
          const int64_t valid = pl.lk - (int64_t)(pl.begin + most - 1) * kRows;
          last = valid < kRows ? (int32_t)valid : kRows;
        }
        release(n);
        if (most == 0) continue;
        ok = mbar_wait_warp_cycles(&q_full, jobs_done & 1, kWaitCycles);
        ++jobs_done;
        // step j: P V of block j - 1 and Q K^T of block j, in this order where their
        // probabilities and scores share a place; a block's K is loaded one stage
        // before its V
        for (int32_t j = 0; ok && j <= most; ++j, ++steps) {
          const uint32_t ki = kv + 2 * j, vi = kv + 2 * j - 1;
          const uint32_t k_st = ki % C::kStages, v_st = vi % C::kStages;
          auto values_there = [&] {
            ok = ok && mbar_wait_warp_cycles(&kv_full[v_st], (vi / C::kStages) & 1, kWaitCycles);
            // values behind the sequence's last one are another's: a product
            // with a zero probability has to be zero
            if (ok && j == most && last < kRows) {
              for (int h = 0; h < C::kHalves; ++h) {
                uint4* z = reinterpret_cast<uint4*>(sm + (2 + v_st) * C::kTile + h * kTileBytes);
                for (int i = last * 8 + lane; i < kRows * 8; i += 32) z[i] = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
          };
          auto keys_there = [&] {
            if (j < most)
              ok = ok && mbar_wait_warp_cycles(&kv_full[k_st], (ki / C::kStages) & 1, kWaitCycles);
          };
          auto add_values = [&] {
            if (!ok || j == 0 || j > blocks) return;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && mbar_wait_warp_cycles(half ? &p_full[w] : &p_half[w], probs & 1, kWaitCycles);
              tc_fence_after();
              if (ok && lead)
#pragma unroll
                for (int s = 4 * half; s < 4 * half + 4; ++s)
                  mma_bf16_ts(o_at, p_at + 8 * s, vd + (uint64_t)((v_st * C::kTile + s * 2048) >> 4),
                              kOut, j > 1 || s > 0);
            }
            ++probs;
          };
          auto score_keys = [&] {
            if (!ok || !lead || j >= blocks) return;
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              mma_bf16(s_at, qd + (uint64_t)(kstep(s) >> 4),
                       kd + (uint64_t)((k_st * C::kTile + kstep(s)) >> 4), kScores, s > 0);
            mma_commit(&s_full[w]);
          };
          if constexpr (C::kEarly) {
            keys_there();
            if (ok && j < blocks) {
              if (scored > 0) ok = mbar_wait_warp_cycles(&s_free[w], (scored - 1) & 1, kWaitCycles);
              ++scored;
            }
            score_keys();
            if (ok && lead && j < most) mma_commit(&kv_empty[k_st]);
            if (ok && lead && j + 1 == most) mma_commit(&q_empty);
            if (j > 0) values_there();
            add_values();
            if (ok && lead && j > 0) {
              if (j <= blocks) mma_commit(&o_full[w]);
              mma_commit(&kv_empty[v_st]);
            }
          } else {
            if (j > 0) values_there();
            keys_there();
            ok = ok && mbar_wait_warp_cycles(&turn[w], (steps & 1) ^ (w ? 0u : 1u), kWaitCycles);
            add_values();
            if (ok && lead && j > 0 && j == blocks) mma_commit(&o_full[w]);
            score_keys();
            if (ok && lead) {
              mbar_arrive(&turn[w ^ 1]);
              if (j > 0) mma_commit(&kv_empty[v_st]);
              if (j < most) mma_commit(&kv_empty[k_st]);
              if (j + 1 == most) mma_commit(&q_empty);
            }
          }
          __syncwarp();
        }
        kv += 2 * most;
      }
    }
  } else {
    // ---------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int w = warp >> 2;
    const int row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // 32 lanes, in the address's upper half
    const uint32_t s_at = tmem + lanes + C::kS + 128 * w, o_at = tmem + lanes + C::kO + C::kOStep * w;
    const uint32_t p_at = tmem + lanes + C::kP + C::kPStep * w;
    const int qi = row / sq.group;                         // the row's query in its tile
    const float c = a.c;
    if (kMode == kParts && part == 0) {
      // before any wait: the join writes where this says, also when a wait has run out
      const Place pl(slots[0], a, part, parts);
      const int64_t r = (pl.q0 + pl.first_of(w) + qi) * a.q_heads + (int64_t)slot_head[0] * sq.group +
                        row % sq.group;
      a.dest[(int64_t)blockIdx.x * 256 + 128 * w + row] = qi < pl.rows_of(w) ? r : -1;
    }
    uint32_t scores = 0, outs = 0;       // blocks of this tile so far, and outputs waited for
    Seq seq;
    for (uint32_t job = 0; ok && take(job, seq); ++job) {
      int32_t n, first, begin;
      {
        const Place pl(seq, a, part, parts);
        n = pl.blocks_of(w);
        first = pl.first_of(w) + pl.shift;                   // the last key that the first row sees
        begin = pl.begin;
      }
      float m = 0.f, l = 0.f;
      for (int32_t j = 0; j < n; ++j, ++scores) {
        ok = mbar_wait_warp_cycles(&s_full[w], scores & 1, kWaitCycles);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld_wait_regs(s[i]);
        if constexpr (C::kEarly) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[w]);
        }
        // keys that the tile's first row does not see are in the block?
        const int32_t k0 = (begin + j) * kRows;
        if (k0 + kRows - 1 > first) {
          const int32_t see = first + qi - k0;
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
        if (C::kEarly && j > 0) {
          // the last block's product is done with its probabilities' place, and O at rest
          ok = mbar_wait_warp_cycles(&o_full[w], outs++ & 1, kWaitCycles);
          if (!ok) break;
          tc_fence_after();
        }
        if (j == 0) {
          m = fmaxf(top, kLowest);   // (all -inf: the first finite score replaces it)
        } else if (__any_sync(0xffffffffu, top > m + a.grow)) {
          // (one place for both: the scores' commit covers the products before them)
          // a row's bits depend on no other row of its warp: the others get a factor of 1
          const bool grows = top > m + a.grow;
          const float f = grows ? ex2_sfu(m - top) : 1.f;
          l *= f;
          m = grows ? top : m;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t o[16];
            tmem_ld16(o_at + 16 * i, o);
            tmem_ld_wait_regs(o);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            tmem_st16(o_at + 16 * i, o);
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
          tmem_st16(p_at + 16 * i, p);
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
      // the row's results.  (The next job's first product into O waits for this
      // warpgroup's next probabilities, so these loads come before it.)
      if (ok && n > 0) ok = mbar_wait_warp_cycles(&o_full[w], outs++ & 1, kWaitCycles);
      tc_fence_after();
      if (!ok) break;
      const int slot = kMode == kListed ? job & 1 : 0;
      const Place pl(slots[slot], a, part, parts);       // (again: it took registers)
      const bool live = qi < pl.rows_of(w);
      const int64_t r = (pl.q0 + pl.first_of(w) + qi) * a.q_heads +
                        (int64_t)slot_head[slot] * sq.group + row % sq.group;
      release(job);
      if constexpr (kMode == kParts) {
        const int64_t at = ((int64_t)blockIdx.x * parts + part) * 256 + 128 * w + row;
        if (live) a.ml[at] = make_float2(m, n > 0 ? l : 0.f);
        if (n > 0) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_ld32(o_at + 32 * i, o);
            tmem_ld_wait_regs(o);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              if (live)
                // (four columns of all rows together: a warp's store is contiguous)
                *reinterpret_cast<uint4*>(a.o + (at - 128 * w - row) * D +
                                          ((8 * i + x) * 256 + 128 * w + row) * 4) =
                    make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
        }
      } else {
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

__global__ void __launch_bounds__(kListThreads) prefill_list_kernel(ListArgs a) {
  grid_release_next();
  grid_wait();
  list_jobs(a);
}

// The parts of a job, joined in their order: a lane holds a packed row, a warp an
// eighth of its columns, so that loads and stores are contiguous.
constexpr int kJoinThreads = 256;
constexpr int kMostParts = 32;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) prefill_join_kernel(const __grid_constant__ FwdArgs a) {
  constexpr int kV = D / 32;   // groups of four columns
  __shared__ float2 ml[kMostParts][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = 32 * blockIdx.y + lane;      // blockIdx.y: 32 rows of the job's 256
  grid_release_next();
  grid_wait();
  int64_t r;
  asm volatile("ld.global.s64 %0, [%1];" : "=l"(r) : "l"(a.dest + (int64_t)blockIdx.x * 256 + row));
  const float* o = a.o + (int64_t)blockIdx.x * a.parts * 256 * D + (warp * kV * 256 + row) * 4;
  // (rows that are no one's have unset statistics, which no one uses)
#pragma unroll
  for (int i = 0; i < kMostParts / 8; ++i) {
    const int p = warp + 8 * i;
    if (p < a.parts) {
      const float* from =
          reinterpret_cast<const float*>(a.ml + ((int64_t)blockIdx.x * a.parts + p) * 256 + row);
      ml[p][lane] = make_float2(ld_waited(from), ld_waited(from + 1));
    }
  }
  // (the first four parts' sums are on their way while the statistics arrive)
  float4 x[4][kV];
  auto read = [&](int p0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const int p = p0 + i < a.parts ? p0 + i : p0;
        x[i][v] = ld_waited(reinterpret_cast<const float4*>(o + (int64_t)p * 256 * D + v * 1024));
      }
  };
  read(0);
  __syncthreads();
  if (r < 0) return;
  float top = -INFINITY;
  for (int p = 0; p < a.parts; ++p) top = ml[p][lane].y == 0.f ? top : fmaxf(top, ml[p][lane].x);
  float all = 0.f, acc[kV][4] = {};
  bool some = false;
  for (int p0 = 0; p0 < a.parts; p0 += 4) {
    if (p0) read(p0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p0 + i >= a.parts) break;
      const float2 s = ml[p0 + i][lane];
      if (s.y == 0.f) continue;                // (a part without keys left nothing; a NaN counts)
      const float f = ex2_sfu(s.x - top);
      some = true;
      all += s.y * f;
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        acc[v][0] = fmaf(x[i][v].x, f, acc[v][0]);
        acc[v][1] = fmaf(x[i][v].y, f, acc[v][1]);
        acc[v][2] = fmaf(x[i][v].z, f, acc[v][2]);
        acc[v][3] = fmaf(x[i][v].w, f, acc[v][3]);
      }
    }
  }
  const float inv = some ? 1.f / all : 0.f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    uint32_t y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
          : "=r"(y[i])
          : "f"(acc[v][2 * i + 1] * inv), "f"(acc[v][2 * i] * inv));
    *reinterpret_cast<uint2*>(a.out + r * D + (warp * kV + v) * 4) = make_uint2(y[0], y[1]);
  }
  if (warp == 0) a.lse[r] = some ? (top + log2f(all)) * kLn2 : -INFINITY;
}

// Where the SMs hold two jobs each or more: a part of a job's keys, if that takes
// four blocks (a block is 1.1 to 1.7 us) off the longest: the join costs about as
// much as two.  More jobs than two turns of the SMs: from a list.
Mode mode_of(int64_t jobs, int64_t blocks, int sms, int32_t& parts) {
  parts = 1;
  if (jobs > 2 * (int64_t)sms) return kListed;
  int64_t p = sms / jobs;
  if (p > blocks) p = blocks;
  if (p > kMostParts) p = kMostParts;
  if (p < 2 || blocks - (blocks + p - 1) / p < 4) return kOnce;
  parts = (int32_t)p;
  return kParts;
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
  if (tq == 0 && !s.packed) return GDN_OK;
  FwdArgs a;
  memset(&a, 0, sizeof a);
  a.status = status_ptr();
  const int sms = sm_count();
  if (!a.status || sms < 1) return GDN_ERR_CUDA;
  const int32_t group = s.q_heads / s.kv_heads;
  a.s = {cu_q, cu_k, s.batch, s.seqlen_q, s.seqlen_k, group, s.kv_heads};
  if (tq == 0) {
    const bool done = no_queries(a.s, nullptr, nullptr, 0, a.status, st) == cudaSuccess;
    if (!done) (void)cudaGetLastError();
    return done ? GDN_OK : GDN_ERR_CUDA;
  }
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.c = scale * kLog2e;
  a.grow = (int64_t)s.rows() < kFewRows ? 0.f : kGrow;
  a.q_heads = s.q_heads;
  a.per = kRows / group;
  const void* kk = tk ? k : q;   // (no keys: nothing is loaded through these)
  if (!heads_map(&a.q, q, tq, s.q_heads, s.d, s.q_stride, group, a.per) ||
      !heads_map(&a.k, kk, tk, s.kv_heads, s.d, tk ? s.k_stride : (int64_t)s.kv_heads * s.d, 1, kRows) ||
      !heads_map(&a.v, tk ? v : q, tk, s.kv_heads, s.d, tk ? s.v_stride : (int64_t)s.kv_heads * s.d, 1, kRows))
    return GDN_ERR_CUDA;
  // packed: an upper bound, sum_n ceil(len_n / per) <= T / per + N
  auto tiles_of = [&](int64_t per) {
    return s.packed ? tq / per + s.batch : (s.seqlen_q + per - 1) / per * s.batch;
  };
  const int64_t blocks = (s.seqlen_k + kRows - 1) / kRows;
  // One tile a job or two, whichever takes the longest job less time: a block takes one
  // tile 1.1 us, two 1.7, a join 3.  (1024 tokens, 16/4 heads of 128: one 14.5 us, two in
  // two parts 18.5; 2000 tokens, 4/1: 18.8 in two parts, 16.2 in four.)
  int32_t one_parts, two_parts;
  const int64_t ones = tiles_of(a.per) * s.kv_heads, twos = tiles_of(2 * a.per) * s.kv_heads;
  const Mode one = mode_of(ones, blocks, sms, one_parts), two = mode_of(twos, blocks, sms, two_parts);
  auto takes = [&](int32_t parts, float block) {
    return (float)((blocks + parts - 1) / parts) * block + (parts > 1 ? 3.f : 0.f);
  };
  const bool single = ones <= sms && takes(one_parts, 1.1f) <= takes(two_parts, 1.7f);
  const Mode mode = single ? one : two;
  a.tiles = single ? 1 : 2;
  a.parts = single ? one_parts : two_parts;
  const int64_t per = (int64_t)a.tiles * a.per, tiles = tiles_of(per), jobs = tiles * s.kv_heads;
  if (jobs > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  size_t need = 0, at_jobs = 256, at_ml = 0, at_o = 0;
  if (mode == kListed) need = at_jobs + (size_t)tiles * sizeof(Job);
  if (mode == kParts) {
    at_ml = (size_t)jobs * 256 * sizeof(int64_t);
    at_o = at_ml + (size_t)jobs * a.parts * 256 * sizeof(float2);
    need = at_o + (size_t)jobs * a.parts * 256 * s.d * 4;
  }
  void* scratch = nullptr;
  if (need && scratch_alloc(&scratch, need, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
  }
  cudaError_t e = cudaSuccess;
  dim3 grid((unsigned)jobs);
  if (mode == kListed) {
    a.count = (const int32_t*)scratch;
    a.next = (uint32_t*)scratch + 1;
    a.jobs = (const Job*)((char*)scratch + at_jobs);
    const int64_t longest = (s.seqlen_q + per - 1) / per;
    const ListArgs list = {a.s, (int32_t)per, (int32_t)((longest + kLevels - 1) / kLevels), false,
                           (int32_t*)scratch, a.next, (Job*)((char*)scratch + at_jobs), a.status};
    e = launch(true, prefill_list_kernel, dim3(1), kListThreads, 0, 0, st, list);
    count_launches(1);
    grid = dim3((unsigned)sms);
  } else if (mode == kParts) {
    a.dest = (int64_t*)scratch;
    a.ml = (float2*)((char*)scratch + at_ml);
    a.o = (float*)((char*)scratch + at_o);
    grid.y = (unsigned)a.parts;
  }
  auto run = [&](auto shape, auto kern, std::atomic<uint64_t>& on) {
    using C = decltype(shape);
    if (e == cudaSuccess) e = allow_smem((const void*)kern, C::kSmem, on);
    if (e == cudaSuccess) e = launch(true, kern, grid, kThreads, C::kSmem, 0, st, a);
  };
  static std::atomic<uint64_t> on[6];
  if (s.d == 128) {
    if (mode == kListed) run(Fwd<128>{}, prefill_kernel<128, kListed>, on[0]);
    else if (mode == kParts) run(Fwd<128>{}, prefill_kernel<128, kParts>, on[1]);
    else run(Fwd<128>{}, prefill_kernel<128, kOnce>, on[2]);
  } else {
    if (mode == kListed) run(Fwd<64>{}, prefill_kernel<64, kListed>, on[3]);
    else if (mode == kParts) run(Fwd<64>{}, prefill_kernel<64, kParts>, on[4]);
    else run(Fwd<64>{}, prefill_kernel<64, kOnce>, on[5]);
  }
  count_launches(1);
  if (mode == kParts && e == cudaSuccess) {
    e = launch(true, s.d == 128 ? prefill_join_kernel<128> : prefill_join_kernel<64>,
               dim3((unsigned)jobs, 8), kJoinThreads, 0, 0, st, a);
    count_launches(1);
  }
  if (e != cudaSuccess) (void)cudaGetLastError();
  const cudaError_t f = scratch_free(scratch, st);
  return e == cudaSuccess && f == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
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
