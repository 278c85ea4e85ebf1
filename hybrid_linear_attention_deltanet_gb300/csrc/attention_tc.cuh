// What the tensor-core kernels of the attention over prompts share: where a
// tile of queries or keys lies, its tensor maps, its shared-memory images.
//
// The queries of a kv head's group are packed into the rows of a tile: row r
// is query r / group, head r % group, and a 128-row tile holds the largest
// whole number of queries, so that a group's heads read a key once and sum its
// gradients in one accumulator.
#pragma once

#include <string.h>

#include "gdn_internal.cuh"
#include "hostcheck.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace attn {

using namespace hostcheck;

constexpr long long kWaitCycles = 4000000000ll;   // about two seconds
constexpr int kRows = 128;           // of a tile: queries x group, or keys
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same, true where all of them say so: warps whose waits run out one by one leave together.
// One that leaves says false at the barrier at which the others, whose waits ended in time,
// meet next, and they leave there; a barrier without an answer would hold them for ever.
__device__ __forceinline__ bool bar_agree(int id, int threads, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n bar.red.and.pred q, %1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(id), "r"(threads), "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// The call's sequences; dense batches are cu == nullptr.
struct Seqs {
  const int32_t *cu_q, *cu_k;
  int32_t n;
  int64_t len_q, len_k;        // dense: of each; packed: of all
  int32_t group, kv_heads;
};
// One sequence: its first query and key, their numbers.
struct Seq {
  int64_t q0, k0;
  int32_t lq, lk;
  int32_t tile;                // the tile's number in the sequence, -1: none
};

// The sequence and the tile of job `job` (of one kv head), tiles of `per` tokens of
// the queries (or keys); the last tile of a sequence first where `down`, as it
// sees the most keys.  Every thread of the CTA calls it; sm holds kThreads + 6
// words.  false: no such job, or malformed sequences (the first CTA says so).
template <int kThreads>
__device__ bool locate(const Seqs& s, int64_t job, int per, bool keys, bool down, int64_t* sm,
                       unsigned* status, Seq& out) {
  if (!s.cu_q) {
    // all sequences' last tiles, then all the tiles before them
    const int64_t len = keys ? s.len_k : s.len_q, tiles = (len + per - 1) / per;
    const int64_t t = job / s.n, i = job - t * s.n;
    if (t >= tiles) return false;
    out = {i * s.len_q, i * s.len_k, (int32_t)s.len_q, (int32_t)s.len_k,
           (int32_t)(down ? tiles - 1 - t : t)};
    return true;
  }
  const int tid = threadIdx.x;
  if (s.n <= 32) {
    // a lane for each sequence, in every warp: no barriers
    const int lane = tid & 31;
    const bool mine = lane < s.n;
    const int32_t a = mine ? s.cu_q[lane] : 0, b = mine ? s.cu_k[lane] : 0;
    const int32_t lq = mine ? s.cu_q[lane + 1] - a : 0, lk = mine ? s.cu_k[lane + 1] - b : 0;
    bool bad = a < 0 || b < 0 || lq < 0 || lk < 0 || (lane == 0 && (a != 0 || b != 0)) ||
               (lane == s.n - 1 && (a + (int64_t)lq != s.len_q || b + (int64_t)lk != s.len_k));
    if (__any_sync(0xffffffffu, bad)) {
      if (tid == 0 && blockIdx.x == 0) flag_status(status, GDN_ERR_BAD_SEQLENS);
      return false;
    }
    const int64_t t = ((int64_t)(keys ? lk : lq) + per - 1) / per;
    int64_t end = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    const unsigned here = __ballot_sync(0xffffffffu, job < end);
    if (!here) return false;
    const int l = __ffs(here) - 1;
    const int64_t at = job - (__shfl_sync(0xffffffffu, end, l) - __shfl_sync(0xffffffffu, t, l));
    const int64_t of = __shfl_sync(0xffffffffu, t, l);
    out = {__shfl_sync(0xffffffffu, a, l), __shfl_sync(0xffffffffu, b, l),
           __shfl_sync(0xffffffffu, lq, l), __shfl_sync(0xffffffffu, lk, l),
           (int32_t)(down ? of - 1 - at : at)};
    return true;
  }
  const int64_t chunk = ((int64_t)s.n + kThreads - 1) / kThreads;
  const int64_t i0 = tid * chunk, i1 = i0 + chunk < s.n ? i0 + chunk : s.n;
  int64_t mine = 0;
  bool bad = tid == 0 && (s.cu_q[0] != 0 || s.cu_k[0] != 0 || s.cu_q[s.n] != s.len_q ||
                          s.cu_k[s.n] != s.len_k);
  for (int64_t i = i0; i < i1; ++i) {
    const int32_t lq = s.cu_q[i + 1] - s.cu_q[i], lk = s.cu_k[i + 1] - s.cu_k[i];
    bad |= lq < 0 || lk < 0 || s.cu_q[i] < 0 || s.cu_k[i] < 0;
    mine += ((int64_t)(keys ? lk : lq) + per - 1) / per;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0 && blockIdx.x == 0) flag_status(status, GDN_ERR_BAD_SEQLENS);
    return false;
  }
  // exclusive prefix of the threads' tiles
  sm[1 + tid] = mine;
  if (tid == 0) sm[0] = 0;
  __syncthreads();
  if (tid < 32) {
    int64_t carry = 0;
    for (int b = 0; b < kThreads; b += 32) {
      int64_t x = sm[1 + b + tid];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (tid >= o) x += y;
      }
      sm[1 + b + tid] = x + carry;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  if (job >= sm[kThreads]) return false;
  Seq& found = *reinterpret_cast<Seq*>(sm + kThreads + 2);
  static_assert(sizeof(Seq) <= 32, "");
  if (job >= sm[tid] && job < sm[tid + 1]) {
    int64_t left = job - sm[tid];
    for (int64_t i = i0; i < i1; ++i) {
      const int32_t a = s.cu_q[i], b = s.cu_k[i];
      const int32_t lq = s.cu_q[i + 1] - a, lk = s.cu_k[i + 1] - b;
      const int64_t t = ((int64_t)(keys ? lk : lq) + per - 1) / per;
      if (left < t) {
        found = {a, b, lq, lk, (int32_t)(down ? t - 1 - left : left)};
        break;
      }
      left -= t;
    }
  }
  __syncthreads();
  out = found;
  return true;
}

// ------------------------------------------------------------- job lists
// Where a call has more jobs than the GPU has SMs, one CTA lists them first,
// those that see the most tiles first whatever their sequence, and persistent
// CTAs take the next one when they are done with one.  (Sequence by sequence
// the long jobs of the last sequence start late; and a persistent CTA loads its
// next job while the last one ends.)  The order among jobs of equal length, that
// of atomics, does not matter: jobs share nothing.
struct Job {
  int32_t q0, k0, lq, lk, tile, unused[3];
};
constexpr int kListThreads = 1024;
constexpr int kLevels = 2048;     // lengths told apart, in `unit` tiles
struct ListArgs {
  Seqs s;
  int32_t per, unit;     // tokens of a tile; tiles of a level
  bool keys;             // tiles of keys: the first ones see the most
  int32_t* count;        // jobs of a kv head, 0 for malformed sequences
  uint32_t* next;        // the CTAs' place in the list
  Job* jobs;
  unsigned* status;
};
// Are packed sequences malformed?  A thread's share of the answer, `threads` of them in all.
__device__ __forceinline__ bool malformed(const Seqs& s, int tid, int threads) {
  bool bad = tid == 0 && (s.cu_q[0] != 0 || s.cu_k[0] != 0 || s.cu_q[s.n] != s.len_q ||
                          s.cu_k[s.n] != s.len_k);
  for (int i = tid; i < s.n; i += threads)
    bad |= s.cu_q[i] < 0 || s.cu_k[i] < 0 || s.cu_q[i + 1] < s.cu_q[i] || s.cu_k[i + 1] < s.cu_k[i];
  return bad;
}
inline __device__ void list_jobs(const ListArgs& a) {
  __shared__ int32_t level[kLevels];
  __shared__ int32_t warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Seqs& s = a.s;
  const bool bad = s.cu_q && malformed(s, tid, kListThreads);
  for (int i = tid; i < kLevels; i += kListThreads) level[i] = 0;
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      *a.count = 0;
      *a.next = 0;
      flag_status(a.status, GDN_ERR_BAD_SEQLENS);
    }
    return;
  }
  auto seq = [&](int i) {
    Job j = {};
    if (s.cu_q) {
      j.q0 = s.cu_q[i];
      j.k0 = s.cu_k[i];
      j.lq = s.cu_q[i + 1] - j.q0;
      j.lk = s.cu_k[i + 1] - j.k0;
    } else {
      j.lq = (int32_t)s.len_q;
      j.lk = (int32_t)s.len_k;
      j.q0 = (int32_t)(i * s.len_q);
      j.k0 = (int32_t)(i * s.len_k);
    }
    return j;
  };
  // a tile's level: the longest job is level 0
  auto level_of = [&](int64_t t, int64_t tiles) {
    const int64_t longer = (a.keys ? tiles - 1 - t : t) / a.unit;
    return (int)(kLevels - 1 - (longer < kLevels ? longer : kLevels - 1));
  };
  // a warp takes a sequence, its lanes the tiles
  for (int i = warp; i < s.n; i += kListThreads / 32) {
    const Job j = seq(i);
    const int64_t tiles = ((int64_t)(a.keys ? j.lk : j.lq) + a.per - 1) / a.per;
    for (int64_t t = lane; t < tiles; t += 32) atomicAdd(&level[level_of(t, tiles)], 1);
  }
  __syncthreads();
  // where each level begins
  int32_t sum = 0;
  int32_t mine[kLevels / kListThreads];
#pragma unroll
  for (int i = 0; i < kLevels / kListThreads; ++i) {
    mine[i] = sum;
    sum += level[tid * (kLevels / kListThreads) + i];
  }
  int32_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int32_t w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  const int32_t before = (warp ? warp_sum[warp - 1] : 0) + x - sum;
#pragma unroll
  for (int i = 0; i < kLevels / kListThreads; ++i)
    level[tid * (kLevels / kListThreads) + i] = before + mine[i];
  if (tid == 0) {
    *a.count = warp_sum[31];
    *a.next = 0;
  }
  __syncthreads();
  for (int i = warp; i < s.n; i += kListThreads / 32) {
    Job j = seq(i);
    const int64_t tiles = ((int64_t)(a.keys ? j.lk : j.lq) + a.per - 1) / a.per;
    for (int64_t t = lane; t < tiles; t += 32) {
      j.tile = (int32_t)t;
      a.jobs[atomicAdd(&level[level_of(t, tiles)], 1)] = j;
    }
  }
}

// Packed sequences without any query: their check, and zeros for the n 16-byte vectors at
// each of x and y (keys' gradients; n 0 without).
static __global__ void __launch_bounds__(kListThreads)
no_queries_kernel(Seqs s, uint4* x, uint4* y, int64_t n, unsigned* status) {
  grid_release_next();
  grid_wait();
  if (__syncthreads_or(malformed(s, threadIdx.x, kListThreads))) {
    if (threadIdx.x == 0) flag_status(status, GDN_ERR_BAD_SEQLENS);
    return;
  }
  for (int64_t i = (int64_t)blockIdx.x * kListThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kListThreads)
    x[i] = y[i] = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------- host side
inline cudaError_t no_queries(const Seqs& s, void* x, void* y, size_t bytes, unsigned* status,
                              cudaStream_t st) {
  const int64_t n = (int64_t)(bytes / 16), ctas = (n + kListThreads - 1) / kListThreads;
  count_launches(1);
  return launch(true, no_queries_kernel, dim3((unsigned)(ctas < 1 ? 1 : ctas < 256 ? ctas : 256)),
                kListThreads, 0, 0, st, s, (uint4*)x, (uint4*)y, n, status);
}
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
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
// x [tokens][heads][d] bf16, tokens `stride` elements apart, read in boxes of 64
// columns x box_heads heads x box_tokens tokens with the 128-byte swizzle; what
// lies past the last token reads as zeros.
inline bool heads_map(CUtensorMap* m, const void* x, int64_t tokens, int32_t heads, int32_t d,
                      int64_t stride, uint32_t box_heads, uint32_t box_tokens) {
  EncodeFn enc = encoder();
  if (!enc) return false;
  memset(m, 0, sizeof *m);
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)(tokens > 0 ? tokens : 1)};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, box_heads, box_tokens};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// x [rows][d] bf16, contiguous, read in boxes of 64 columns x box_rows rows.
inline bool heads_map(CUtensorMap* m, const void* x, int64_t rows, int32_t d, uint32_t box_rows) {
  EncodeFn enc = encoder();
  if (!enc) return false;
  memset(m, 0, sizeof *m);
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(x), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Its product with log2 e is finite too.
inline bool scale_ok(float scale) { return scale > 0.f && scale <= 0x1p127f; }

// The checks that the prompt kernels share: sizes, strides, alignment.
struct Shape {
  int32_t batch;
  int64_t seqlen_q, seqlen_k;
  int32_t q_heads, kv_heads, d;
  int64_t q_stride, k_stride, v_stride;
  bool packed;
  int64_t tq() const { return packed ? seqlen_q : batch * seqlen_q; }
  int64_t tk() const { return packed ? seqlen_k : batch * seqlen_k; }
  size_t q_bytes() const { return tq() ? (size_t)((tq() - 1) * q_stride + q_heads * d) * 2 : 0; }
  size_t k_bytes(int64_t stride) const {
    return tk() ? (size_t)((tk() - 1) * stride + kv_heads * d) * 2 : 0;
  }
  size_t rows() const { return (size_t)tq() * q_heads; }      // of out and lse
};
inline int check_shape(const Shape& s, const int32_t* cu_q, const int32_t* cu_k, float scale) {
  if (s.batch < 1 || s.seqlen_q < 0 || s.seqlen_k < 0 || s.q_heads < 1 || s.kv_heads < 1)
    return GDN_ERR_INVALID_ARG;
  if ((cu_q == nullptr) != (cu_k == nullptr)) return GDN_ERR_INVALID_ARG;
  if (!scale_ok(scale)) return GDN_ERR_INVALID_ARG;
  if ((s.d != 64 && s.d != 128) || s.q_heads % s.kv_heads || s.q_heads / s.kv_heads > kRows)
    return GDN_ERR_UNSUPPORTED;
  // 32-bit token coordinates, with room for a tile; sequences counted in 32 bits
  if (s.seqlen_q > kLongestAxis || s.seqlen_k > kLongestAxis || s.tq() > kLongestAxis ||
      s.tk() > kLongestAxis || (int64_t)s.q_heads * s.d > kLongestAxis)
    return GDN_ERR_UNSUPPORTED;
  const int64_t wq = (int64_t)s.q_heads * s.d, wk = (int64_t)s.kv_heads * s.d;
  if (s.q_stride < wq || s.k_stride < wk || s.v_stride < wk) return GDN_ERR_INVALID_ARG;
  if (s.q_stride > kLongestAxis || s.k_stride > kLongestAxis || s.v_stride > kLongestAxis)
    return GDN_ERR_UNSUPPORTED;
  if (s.q_stride % 8 || s.k_stride % 8 || s.v_stride % 8) return GDN_ERR_ALIGNMENT;
  return GDN_OK;
}

}  // namespace attn
}  // namespace gdn
