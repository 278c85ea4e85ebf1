// The pages of the attention layers' cache: reserving, appending, gathering, freeing,
// forking, compacting (contracts: include/gdn.h).
//
// The integers (tables, lengths, reference counts) stay on the device and are
// changed there, so that a decoding loop never waits for the host and can be
// captured.  Everything about them is decided by one CTA, which takes pages in
// the order of their numbers: a scan of the reference counts, 4096 a step (a
// step is one load, two warp scans and two barriers, about 1 us), that ends as
// soon as it has found enough.  The kernels are short and come in chains (free,
// reserve; free, fork), so they are programmatic dependents: each waits for the
// one before it first, but is on the GPU by then.  (append_kernel for
// single tokens is not: it is over before the attribute has cost the host its 1.5 us.)
// Copies are split over the GPU, 64 KB a CTA, 16 bytes a lane; they are bound by HBM.
//
// (free, reserve and append of 4 prompts of up to 8192 tokens into 8 bits, 4 kv heads of
// 128: 12.4 us, of which 7 are the append's 37 MB; 256 tokens' append 2.6; free and fork
// of 3 rows 11.2, of 72 16.3, 7 layers; compacting 256 pages of 8 bits 8.5, 922 pages of
// 7 layers 245.)
#include <cuda_fp16.h>

#include "fp8_codes.cuh"
#include "gdn_internal.cuh"
#include "hostcheck.cuh"
#include "kv_cache.cuh"

namespace gdn {
namespace {

using namespace hostcheck;

constexpr int kPlan = 1024;   // threads of the CTA that decides
constexpr int kCopy = 256;

struct ScanMem {
  int64_t warp[32];
  int64_t total;
};
// Exclusive prefix of x over the CTA (all kPlan threads), and the sum of all.
__device__ __forceinline__ int64_t scan(int64_t x, ScanMem& sm, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += t;
  }
  __syncthreads();   // the last call's readers are done
  if (lane == 31) sm.warp[warp] = y;
  __syncthreads();
  if (warp == 0) {
    int64_t w = sm.warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    if (lane == 31) sm.total = w;
    sm.warp[lane] = w;
  }
  __syncthreads();
  total = sm.total;
  return (warp ? sm.warp[warp - 1] : 0) + y - x;
}

// The reference counts of pages [p, p + 4), 1 behind the last.
__device__ __forceinline__ int4 counts_at(const int32_t* refs, int32_t pages, int64_t p) {
  if (p + 4 <= pages) return *reinterpret_cast<const int4*>(refs + p);
  int4 r = make_int4(1, 1, 1, 1);
  if (p < pages) r.x = refs[p];
  if (p + 1 < pages) r.y = refs[p + 1];
  if (p + 2 < pages) r.z = refs[p + 2];
  return r;
}
// The first `want` free pages to list, in order; how many there are (at most want).
// `near` are this thread's counts of the first step, read while the CTA found out
// what it wants.
__device__ int64_t find_free(const int32_t* refs, int32_t pages, int64_t want, int32_t* list,
                             int4 near, ScanMem& sm) {
  int64_t found = 0;
  for (int64_t base = 0; base < pages && found < want; base += 4 * kPlan) {
    const int64_t p = base + 4 * (int64_t)threadIdx.x;
    const int4 t = base == 0 ? near : counts_at(refs, pages, p);
    const int32_t r[4] = {t.x, t.y, t.z, t.w};
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n += r[i] == 0;
    int64_t step;
    int64_t at = found + scan(n, sm, step);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r[i] == 0) {
        if (at < want) list[at] = (int32_t)(p + i);
        ++at;
      }
    found += step;
  }
  __syncthreads();   // the list is there for the CTA
  return found < want ? found : want;
}
constexpr int kNear = 2048;   // pages whose list stays in shared memory

// ------------------------------------------------------------- reserving
__global__ void __launch_bounds__(kPlan)
reserve_kernel(gdn_kv_cache c, const int32_t* counts, int32_t* start, int32_t* list,
               unsigned* status) {
  __shared__ ScanMem sm;
  __shared__ int32_t near_list[kNear];
  const int lane = threadIdx.x & 31;
  grid_release_next();
  grid_wait();
  const int4 near = counts_at(c.refs, c.pages, 4 * (int64_t)threadIdx.x);
  // pages a row holds and will hold; what is asked of it in bad: 1 out of range, 2 no room
  auto ask = [&](int row, int64_t& old, int64_t& now, int64_t& len) {
    if (row >= c.rows) {
      old = now = len = 0;
      return 0;
    }
    len = c.lengths[row];
    const int64_t n = counts[row];
    old = now = (len + c.page - 1) / c.page;
    if (len < 0 || old > c.max_pages || n < 0) {
      old = now = 0;
      return 1;
    }
    const int64_t to = (len + n + c.page - 1) / c.page;
    if (to > c.max_pages) return 2;
    now = to;
    return 0;
  };
  int64_t want = 0, step, old, now, len, first;
  int bad = 0;
  const bool one = c.rows <= kPlan;   // then what the first round found is kept
  for (int base = 0; base < c.rows; base += kPlan) {
    bad = ask(base + threadIdx.x, old, now, len);
    first = scan(now - old, sm, step);
    want += step;
  }
  if (want > c.pages) want = c.pages;
  if (want <= kNear) list = near_list;
  const int64_t found = want ? find_free(c.refs, c.pages, want, list, near, sm) : 0;
  int64_t before = 0;
  for (int base = 0; base < c.rows; base += kPlan) {
    const int row = base + threadIdx.x;
    if (!one) {
      bad = ask(row, old, now, len);
      first = before + scan(now - old, sm, step);
      before += step;
    }
    const int64_t need = now - old;
    const bool ok = bad == 0 && (need == 0 || first + need <= found);
    if (row < c.rows) {
      start[row] = ok ? (int32_t)len : -1;
      if (ok) c.lengths[row] = (int32_t)(len + counts[row]);
      else flag_status(status, bad == 1 ? GDN_ERR_BAD_CACHE : GDN_ERR_CACHE_FULL);
    }
    // the warp writes its rows' new pages, row by row
    unsigned takers = __ballot_sync(0xffffffffu, ok && need > 0 && row < c.rows);
    while (takers) {
      const int l = __ffs(takers) - 1;
      takers &= takers - 1;
      const int64_t n = __shfl_sync(0xffffffffu, need, l), f = __shfl_sync(0xffffffffu, first, l),
                    o = __shfl_sync(0xffffffffu, old, l);
      const int64_t r = __shfl_sync(0xffffffffu, (int64_t)row, l);
      for (int64_t i = lane; i < n; i += 32) {
        const int32_t p = list[f + i];
        c.table[r * c.max_pages + o + i] = p;
        c.refs[p] = 1;
      }
    }
  }
}

// ------------------------------------------------------------- appending
struct AppendArgs {
  gdn_kv_cache c;
  const __nv_bfloat16 *k, *v;
  const int32_t *start, *cu;
  int64_t tokens, k_stride, v_stride;
  int32_t layer, page_log2;
  unsigned* status;
};

// The row of packed token t and its number there; false: outside every sequence.
__device__ __forceinline__ bool find_row(const int32_t* cu, int32_t rows, int64_t t, int64_t& row,
                                         int64_t& i) {
  int lo = 0, hi = rows - 1;   // last row with cu[row] <= t
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (ld_waited(cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  row = lo;
  i = t - ld_waited(cu + lo);
  return i >= 0 && t < ld_waited(cu + lo + 1);
}
// The first element of head h of position pos of a row, -1 where its page is none.
__device__ __forceinline__ int64_t element_of(const gdn_kv_cache& c, int32_t layer, int32_t page_log2,
                                              int64_t row, int64_t pos, int h) {
  const int64_t n = pos >> page_log2;
  int32_t p = -1;
  if (n < c.max_pages) p = ld_waited(c.table + row * c.max_pages + n);
  if (p < 0 || p >= c.pages) return -1;
  return ((((int64_t)layer * c.pages + p) * c.kv_heads + h) << page_log2) + (pos & (c.page - 1));
}

// d / 16 lanes hold one head of one token, 32 bytes of its key and of its value
// each.  A decoding step's few tokens are bound by the chain of small loads
// (sequence, start, page) that their places take, prompts by HBM and, in 8 bits, by
// instructions as much (64-bit divisions, and 16 bytes a lane, made them half as
// long again).
template <int D, bool kFp8>
__global__ void __launch_bounds__(kCopy) append_kernel(AppendArgs a) {
  constexpr int kLanes = D / 16;
  grid_release_next();
  grid_wait();
  const gdn_kv_cache& c = a.c;
  const int64_t units = a.tokens * c.kv_heads;
  const int64_t unit = ((int64_t)blockIdx.x * kCopy + threadIdx.x) / kLanes;
  const int l = threadIdx.x % kLanes;
  const bool there = unit < units;
  const int64_t t = units >> 32 ? unit / c.kv_heads : (int64_t)((uint32_t)unit / (uint32_t)c.kv_heads);
  const int h = (int)(unit - t * c.kv_heads);
  uint4 x[2][2] = {};
  if (there) {
    const uint4* k = reinterpret_cast<const uint4*>(a.k + t * a.k_stride + h * D + l * 16);
    const uint4* v = reinterpret_cast<const uint4*>(a.v + t * a.v_stride + h * D + l * 16);
    x[0][0] = ld_waited(k);
    x[0][1] = ld_waited(k + 1);
    x[1][0] = ld_waited(v);
    x[1][1] = ld_waited(v + 1);
  }
  // the token's row and place
  int64_t at = -1;   // first element of its head in the pool, -1: nowhere
  if (there) {
    int64_t row = t, i = 0;
    bool ok = true;
    if (a.cu) {
      ok = find_row(a.cu, c.rows, t, row, i);
      if (!ok) flag_status(a.status, GDN_ERR_BAD_SEQLENS);
    }
    const int64_t s = ok ? ld_waited(a.start + row) : -1;
    const int64_t len = ok ? ld_waited(c.lengths + row) : 0;
    if (ok && s >= 0 && s + i < len) {
      at = element_of(c, a.layer, a.page_log2, row, s + i, h);
      if (at < 0) flag_status(a.status, GDN_ERR_BAD_CACHE);
    } else if (ok && s < -1) {
      flag_status(a.status, GDN_ERR_BAD_CACHE);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    void* pool = i ? c.v : c.k;
    if constexpr (!kFp8) {
      if (at >= 0) {
        uint4* to = reinterpret_cast<uint4*>((__nv_bfloat16*)pool + at * D + l * 16);
        to[0] = x[i][0];
        to[1] = x[i][1];
      }
    } else {
      float f[2][8];
      float m = kTiny;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t w[4] = {x[i][j].x, x[i][j].y, x[i][j].z, x[i][j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[j][2 * k] = __uint_as_float(w[k] << 16);
          f[j][2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
        m = max_nan(m, amax8(f[j]));
      }
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (at >= 0) {
        const uint2 q0 = quantise8_bf16(f[0], m), q1 = quantise8_bf16(f[1], m);
        *reinterpret_cast<uint4*>((uint8_t*)pool + at * D + l * 16) = make_uint4(q0.x, q0.y, q1.x, q1.y);
        if (l == 0) (i ? c.v_scale : c.k_scale)[at] = scale_of(m);
      }
    }
  }
}

// ------------------------------------------------------------- gathering
struct GatherArgs {
  gdn_kv_cache c;
  __nv_bfloat16 *k, *v;
  const int32_t* cu;
  int64_t tokens;
  int32_t layer, page_log2;
  unsigned* status;
};

// Two e4m3 codes (w's lower half) as fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_half(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(w));
  return r;
}
// The way back, split as the append is: a token's 16 columns of a head a lane.  A code
// times its scale is an fp32 product, rounded to bf16.  Bound by HBM: 32 rows of 4096 tokens, 4 kv
// heads of 128, 80 us (6.7 TB/s), from 8 bits 69 (5.9); one of 1183 tokens 2.9.
template <int D, bool kFp8>
__global__ void __launch_bounds__(kCopy) gather_kernel(GatherArgs a) {
  constexpr int kLanes = D / 16;
  grid_release_next();
  grid_wait();
  const gdn_kv_cache& c = a.c;
  const int64_t unit = ((int64_t)blockIdx.x * kCopy + threadIdx.x) / kLanes;
  const int l = threadIdx.x % kLanes;
  if (unit >= a.tokens * c.kv_heads) return;
  const int64_t t = unit >> 32 ? unit / c.kv_heads : (int64_t)((uint32_t)unit / (uint32_t)c.kv_heads);
  const int h = (int)(unit - t * c.kv_heads);
  int64_t row, i;
  if (!find_row(a.cu, c.rows, t, row, i)) {
    flag_status(a.status, GDN_ERR_BAD_SEQLENS);
    return;
  }
  int64_t at = -1;   // (what the row does not hold becomes zeros: k and v may be new memory)
  if (i >= ld_waited(c.lengths + row)) {
    flag_status(a.status, GDN_ERR_BAD_SEQLENS);
  } else {
    at = element_of(c, a.layer, a.page_log2, row, i, h);
    if (at < 0) flag_status(a.status, GDN_ERR_BAD_CACHE);
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    uint4* to = reinterpret_cast<uint4*>((x ? a.v : a.k) + unit * D + l * 16);
    if (at < 0) {
      to[0] = to[1] = make_uint4(0, 0, 0, 0);
    } else if constexpr (!kFp8) {
      const uint4* from =
          reinterpret_cast<const uint4*>((const __nv_bfloat16*)(x ? c.v : c.k) + at * D + l * 16);
      const uint4 y0 = ld_waited(from), y1 = ld_waited(from + 1);
      to[0] = y0;
      to[1] = y1;
    } else {
      const uint4 q = ld_waited(
          reinterpret_cast<const uint4*>((const uint8_t*)(x ? c.v : c.k) + at * D + l * 16));
      const float f = ld_waited((x ? c.v_scale : c.k_scale) + at);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      uint32_t y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t half = e4m3x2_to_half(j & 1 ? w[j >> 1] >> 16 : w[j >> 1]);
        const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&half));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y[j]) : "f"(z.y * f), "f"(z.x * f));
      }
      to[0] = make_uint4(y[0], y[1], y[2], y[3]);
      to[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

// --------------------------------------------------------------- freeing
__global__ void __launch_bounds__(128)
free_kernel(gdn_kv_cache c, const int32_t* rows, unsigned* status) {
  __shared__ int32_t len;
  grid_release_next();
  grid_wait();
  const int32_t r = rows[blockIdx.x];
  if (r < 0 || r >= c.rows) {
    if (threadIdx.x == 0) flag_status(status, GDN_ERR_BAD_CACHE);
    return;
  }
  // of the CTAs that name a row, the first empties it
  if (threadIdx.x == 0) len = atomicExch(c.lengths + r, 0);
  __syncthreads();
  // (entries behind the last page are -1: of a row of bad length all are gone through, or the
  // pages that it holds would never be free again)
  const int64_t pages = ((int64_t)len + c.page - 1) / c.page;
  const bool bad = len < 0 || pages > c.max_pages;
  const int64_t held = bad ? c.max_pages : pages;
  if (bad && threadIdx.x == 0) flag_status(status, GDN_ERR_BAD_CACHE);
  for (int64_t i = threadIdx.x; i < held; i += blockDim.x) {
    int32_t* e = c.table + (int64_t)r * c.max_pages + i;
    const int32_t p = *e;
    *e = -1;
    if (p >= 0 && p < c.pages) atomicSub(c.refs + p, 1);
    else if (!bad) flag_status(status, GDN_ERR_BAD_CACHE);
  }
}

// --------------------------------------------------------------- copying
// n 16-byte vectors from src to dst by the CTA, four a thread in flight; where
// they lie is the caller's to say.
template <typename F>
__device__ __forceinline__ void copy_vectors(const uint4* src, uint4* dst, int64_t n, F&& place) {
  constexpr int kFly = 8;
  for (int64_t i = threadIdx.x; i < n; i += kFly * kCopy) {
    uint4 x[kFly];
    int64_t p[kFly];
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      p[j] = i + j * kCopy < n ? place(i + j * kCopy) : -1;
      if (p[j] >= 0) x[j] = ld_waited(src + p[j]);
    }
#pragma unroll
    for (int j = 0; j < kFly; ++j)
      if (p[j] >= 0) dst[p[j]] = x[j];
  }
}

// --------------------------------------------------------------- forking
constexpr int32_t kSkip = -1, kNoSource = -3;
struct Pair {
  int32_t len, page, old;   // tokens of the row (negative: the pair is skipped), the new page and the one
                            // that it copies, or -1
};

// The rows' lengths are read before any is changed.  Which of the pairs that name a dst is
// valid is decided by marking its length (0) with i - n < 0: the smallest pair wins whatever
// the order.  The second kernel's CTAs copy.
__global__ void __launch_bounds__(kPlan)
fork_plan_kernel(gdn_kv_cache c, const int32_t* src, const int32_t* dst, int32_t n, Pair* plan,
                 int32_t* list, unsigned* status) {
  __shared__ ScanMem sm;
  __shared__ int32_t near_list[kNear];
  grid_release_next();
  grid_wait();
  const int4 near = counts_at(c.refs, c.pages, 4 * (int64_t)threadIdx.x);
  // a pair's tokens: kSkip where a number is out of range or dst not empty, kNoSource where
  // src's length is bad
  auto read = [&](int i) {
    const int32_t s = src[i], d = dst[i];
    if (s < 0 || s >= c.rows || d < 0 || d >= c.rows || c.lengths[d] != 0) return kSkip;
    const int32_t t = c.lengths[s];
    return t < 0 || t > c.max_pages * c.page ? kNoSource : t;
  };
  const bool one = n <= kPlan;   // then what a thread finds is kept in registers
  int32_t own = kSkip;
  for (int i = threadIdx.x; i < n; i += kPlan) {
    own = read(i);
    if (!one) plan[i].len = own;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan)
    if ((one ? own : plan[i].len) != kSkip) atomicMin(c.lengths + dst[i], i - n);
  __syncthreads();
  // the same, kSkip where an earlier pair names dst; and the page that it copies, or -1
  auto tokens = [&](int i, int32_t& old) {
    old = -1;
    if (i >= n) return kSkip;
    const int32_t t = one ? own : plan[i].len;
    if (t == kSkip || __ldcg(c.lengths + dst[i]) != i - n) return kSkip;
    if (t > 0 && t % c.page) old = c.table[(int64_t)src[i] * c.max_pages + t / c.page];
    return t;
  };
  int64_t want = 0, step, at = 0;
  int32_t t = 0, old = -1;
  for (int base = 0; base < n; base += kPlan) {
    t = tokens(base + threadIdx.x, old);
    at = scan(t > 0 && t % c.page != 0, sm, step);
    want += step;
  }
  if (want <= kNear) list = near_list;
  const int64_t found = want ? find_free(c.refs, c.pages, want, list, near, sm) : 0;
  int64_t before = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + threadIdx.x;
    if (!one) {
      t = tokens(i, old);
      at = before + scan(t > 0 && t % c.page != 0, sm, step);
      before += step;
    }
    const bool need = t > 0 && t % c.page != 0;
    if (i >= n) continue;
    if (t < 0) flag_status(status, GDN_ERR_BAD_CACHE);
    Pair p = {t, -1, -1};
    if (need) {
      if (at < found) {
        p.page = list[at];
        p.old = old;
        c.refs[p.page] = 1;
      } else {
        p.len = -2;   // no page: the mark is taken off
        flag_status(status, GDN_ERR_CACHE_FULL);
      }
    }
    plan[i] = p;
    // the marks become lengths, once no thread reads any more
    if (one && t != kSkip) c.lengths[dst[i]] = p.len > 0 ? p.len : 0;
  }
  if (one) return;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int32_t len = plan[i].len;
    if (len != kSkip) c.lengths[dst[i]] = len > 0 ? len : 0;
  }
}

// blockIdx.x: the pair; y = 0: the table; y = 1 + 2 layer + (0: keys, 1: values)
template <bool kFp8>
__global__ void __launch_bounds__(kCopy)
fork_copy_kernel(gdn_kv_cache c, const int32_t* src, const int32_t* dst, const Pair* plan,
                 unsigned* status) {
  grid_release_next();
  grid_wait();
  const int i = blockIdx.x;
  const int32_t len = ld_waited(&plan[i].len), fresh = ld_waited(&plan[i].page),
                old = ld_waited(&plan[i].old);
  if (len <= 0) return;
  const int32_t* from = c.table + (int64_t)src[i] * c.max_pages;
  const int32_t full = len / c.page, tail = len % c.page;
  if (blockIdx.y == 0) {
    int32_t* to = c.table + (int64_t)dst[i] * c.max_pages;
    for (int32_t j = threadIdx.x; j < full; j += kCopy) {
      const int32_t p = ld_waited(from + j);
      to[j] = p;
      if (p >= 0 && p < c.pages) atomicAdd(c.refs + p, 1);
      else flag_status(status, GDN_ERR_BAD_CACHE);
    }
    if (tail && threadIdx.x == 0) to[full] = fresh;
    return;
  }
  if (!tail) return;
  const int layer = (blockIdx.y - 1) >> 1;
  const bool values = (blockIdx.y - 1) & 1;
  // the two pages; a head is `page` tokens further than the one before, and its
  // first `tail` tokens are copied
  const int64_t heads = (int64_t)c.kv_heads * c.page;
  const int64_t a = ((int64_t)layer * c.pages + old) * heads;
  const int64_t b = ((int64_t)layer * c.pages + fresh) * heads;
  const int vecs = c.d * (kFp8 ? 1 : 2) / 16;   // of a token
  uint4* pool = (uint4*)(values ? c.v : c.k);
  const int mine = tail * vecs, whole = c.page * vecs;
  auto place = [&](int64_t x) {
    const int h = (int)x / mine;
    return (int64_t)h * whole + (int)x - h * mine;
  };
  const bool none = old < 0 || old >= c.pages;   // then zeros: the new page holds what another row left
  if (none) {
    if (threadIdx.x == 0) flag_status(status, GDN_ERR_BAD_CACHE);
    for (int64_t x = threadIdx.x; x < (int64_t)c.kv_heads * mine; x += kCopy)
      pool[b * vecs + place(x)] = make_uint4(0, 0, 0, 0);
  } else {
    copy_vectors(pool + a * vecs, pool + b * vecs, (int64_t)c.kv_heads * mine, place);
  }
  if constexpr (kFp8) {
    float* scale = values ? c.v_scale : c.k_scale;
    for (int x = threadIdx.x; x < c.kv_heads * tail; x += kCopy) {
      const int h = x / tail, t = x - h * tail;
      scale[b + h * c.page + t] = none ? 0.f : ld_waited(scale + a + h * c.page + t);
    }
  }
}

// ------------------------------------------------------------ compacting
// order[new] = old and number[old] = new (-1: free) of the live pages, *count
// how many, or -1 where `into` has not the room.
__global__ void __launch_bounds__(kPlan)
compact_plan_kernel(gdn_kv_cache c, gdn_kv_cache into, int32_t* count, int32_t* order,
                    int32_t* number, unsigned* status) {
  __shared__ ScanMem sm;
  grid_release_next();
  grid_wait();
  int64_t live = 0, step;
  for (int64_t base = 0; base < c.pages; base += 4 * kPlan) {
    const int64_t p = base + 4 * (int64_t)threadIdx.x;
    int n = 0;
    bool on[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      on[i] = p + i < c.pages && c.refs[p + i] > 0;
      n += on[i];
    }
    int64_t at = live + scan(n, sm, step);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p + i < c.pages) number[p + i] = on[i] ? (int32_t)at : -1;
      if (on[i] && at < into.pages) order[at] = (int32_t)(p + i);
      at += on[i];
    }
    live += step;
  }
  const bool fits = live <= into.pages;
  if (threadIdx.x == 0) {
    *count = fits ? (int32_t)live : -1;
    if (!fits) flag_status(status, GDN_ERR_CACHE_FULL);
  }
  __syncthreads();
  if (!fits) return;
  for (int64_t p = threadIdx.x; p < into.pages; p += kPlan)
    into.refs[p] = p < live ? c.refs[order[p]] : 0;
}

// The first c.rows CTAs write a row's table and length, the others copy a page
// of one layer's keys or values each.
template <bool kFp8>
__global__ void __launch_bounds__(kCopy)
compact_copy_kernel(gdn_kv_cache c, gdn_kv_cache into, const int32_t* count, const int32_t* order,
                    const int32_t* number, int64_t jobs, unsigned* status) {
  grid_release_next();
  grid_wait();
  const int32_t live = ld_waited(count);
  if (live < 0) return;
  const int64_t per = (int64_t)c.kv_heads * c.page;
  const int vecs = c.d * (kFp8 ? 1 : 2) / 16;
  for (int64_t b = blockIdx.x; b < c.rows + jobs; b += gridDim.x) {
    if (b < c.rows) {
      const int64_t len = c.lengths[b], held = (len + c.page - 1) / c.page;
      const bool ok = len >= 0 && held <= c.max_pages;
      if (threadIdx.x == 0) {
        into.lengths[b] = ok ? (int32_t)len : 0;
        if (!ok) flag_status(status, GDN_ERR_BAD_CACHE);
      }
      for (int32_t i = threadIdx.x; i < into.max_pages; i += kCopy) {
        int32_t p = -1;
        if (ok && i < held) {
          const int32_t old = c.table[b * c.max_pages + i];
          if (old >= 0 && old < c.pages) p = ld_waited(number + old);
          if (p < 0) flag_status(status, GDN_ERR_BAD_CACHE);
        }
        into.table[b * into.max_pages + i] = p;
      }
      continue;
    }
    // page, then layer, then keys or values
    const int64_t j = b - c.rows, lv = 2 * (int64_t)c.layers;
    const int64_t to = j / lv;
    const int layer = (int)((j - to * lv) >> 1);
    const bool values = (j - to * lv) & 1;
    if (to >= live) return;   // (all later jobs are further pages)
    const int64_t x = ((int64_t)layer * c.pages + ld_waited(order + to)) * per;
    const int64_t y = ((int64_t)layer * into.pages + to) * per;
    copy_vectors((const uint4*)(values ? c.v : c.k) + x * vecs,
                 (uint4*)(values ? into.v : into.k) + y * vecs, per * vecs,
                 [](int64_t i) { return i; });
    if constexpr (kFp8)
      copy_vectors((const uint4*)((values ? c.v_scale : c.k_scale) + x),
                   (uint4*)((values ? into.v_scale : into.k_scale) + y), per / 4,
                   [](int64_t i) { return i; });
  }
}

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

int finish(cudaError_t e, void* scratch, cudaStream_t st) {
  if (e != cudaSuccess) (void)cudaGetLastError();
  const cudaError_t f = scratch_free(scratch, st);
  return e == cudaSuccess && f == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_cache_reserve(const gdn_kv_cache* cache, const int32_t* counts, int32_t* start,
                      gdn_stream_t stream) {
  if (const int rc = kv::check_cache(cache)) return rc;
  if (!counts || !start) return GDN_ERR_INVALID_ARG;
  if (!aligned(counts, 4) || !aligned(start, 4)) return GDN_ERR_ALIGNMENT;
  const gdn_kv_cache c = *cache;
  const kv::Spans own = kv::spans_of(c);
  const Span outs[] = {own.s[0], own.s[1], own.s[2], own.s[3], own.s[4], own.s[5], own.s[6],
                       span_of(start, (size_t)c.rows * 4)};
  const Span ins[] = {span_of(counts, (size_t)c.rows * 4)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  const cudaStream_t st = (cudaStream_t)stream;
  unsigned* status = status_ptr();
  void* list = nullptr;
  const int64_t most = least(c.pages, (int64_t)c.rows * c.max_pages);
  if (!status || scratch_alloc(&list, (size_t)most * 4, st) != cudaSuccess) return GDN_ERR_CUDA;
  count_launches(1);
  return finish(launch(true, reserve_kernel, dim3(1), kPlan, 0, 0, st, c, counts, start,
                       (int32_t*)list, status),
                list, st);
}

int gdn_cache_append(const gdn_kv_cache* cache, int32_t layer, const void* k, const void* v,
                     const int32_t* start, const int32_t* cu_seqlens, int64_t tokens,
                     int64_t k_stride, int64_t v_stride, gdn_stream_t stream) {
  if (const int rc = kv::check_cache(cache)) return rc;
  const gdn_kv_cache c = *cache;
  const int64_t width = (int64_t)c.kv_heads * c.d;
  if (layer < 0 || layer >= c.layers || tokens < 0 || !start) return GDN_ERR_INVALID_ARG;
  if (!cu_seqlens && tokens != c.rows) return GDN_ERR_INVALID_ARG;
  if (tokens > 0 && (!k || !v)) return GDN_ERR_INVALID_ARG;
  if (k_stride < width || v_stride < width || tokens > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4) || !aligned(cu_seqlens, 4) ||
      k_stride % 8 || v_stride % 8)
    return GDN_ERR_ALIGNMENT;
  if (tokens == 0) return GDN_OK;
  const kv::Spans own = kv::spans_of(c);
  const Span ins[] = {span_of(k, (size_t)((tokens - 1) * k_stride + width) * 2),
                      span_of(v, (size_t)((tokens - 1) * v_stride + width) * 2),
                      span_of(start, (size_t)c.rows * 4),
                      span_of(cu_seqlens, (size_t)(c.rows + 1) * 4)};
  if (any_overlap(ins, own.s)) return GDN_ERR_INVALID_ARG;
  AppendArgs a = {c, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, start, cu_seqlens, tokens,
                  k_stride, v_stride, layer, kv::log2_of(c.page), status_ptr()};
  if (!a.status) return GDN_ERR_CUDA;
  const int64_t ctas = (tokens * c.kv_heads * (c.d / 16) + kCopy - 1) / kCopy;
  if (ctas > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  const bool fp8 = c.dtype == GDN_E4M3;
  auto* kern = c.d == 128 ? (fp8 ? append_kernel<128, true> : append_kernel<128, false>)
                          : (fp8 ? append_kernel<64, true> : append_kernel<64, false>);
  count_launches(1);
  return launch(cu_seqlens != nullptr, kern, dim3((unsigned)ctas), kCopy, 0, 0, (cudaStream_t)stream, a) ==
                 cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

int gdn_cache_gather(const gdn_kv_cache* cache, int32_t layer, const int32_t* cu_seqlens,
                     int64_t tokens, void* k, void* v, gdn_stream_t stream) {
  if (const int rc = kv::check_cache(cache)) return rc;
  const gdn_kv_cache c = *cache;
  if (layer < 0 || layer >= c.layers || tokens < 0 || tokens > 0x7fffffffLL || !cu_seqlens)
    return GDN_ERR_INVALID_ARG;
  if (tokens > 0 && (!k || !v)) return GDN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_seqlens, 4)) return GDN_ERR_ALIGNMENT;
  if (tokens == 0) return GDN_OK;
  const size_t bytes = (size_t)tokens * c.kv_heads * c.d * 2;
  const kv::Spans own = kv::spans_of(c);
  const Span ins[] = {own.s[0], own.s[1], own.s[2], own.s[3], own.s[4], own.s[5], own.s[6],
                      span_of(cu_seqlens, (size_t)(c.rows + 1) * 4)};
  const Span outs[] = {span_of(k, bytes), span_of(v, bytes)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  const GatherArgs a = {c, (__nv_bfloat16*)k, (__nv_bfloat16*)v, cu_seqlens, tokens, layer,
                        kv::log2_of(c.page), status_ptr()};
  if (!a.status) return GDN_ERR_CUDA;
  const int64_t ctas = (tokens * c.kv_heads * (c.d / 16) + kCopy - 1) / kCopy;
  if (ctas > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  const bool fp8 = c.dtype == GDN_E4M3;
  auto* kern = c.d == 128 ? (fp8 ? gather_kernel<128, true> : gather_kernel<128, false>)
                          : (fp8 ? gather_kernel<64, true> : gather_kernel<64, false>);
  count_launches(1);
  return launch(true, kern, dim3((unsigned)ctas), kCopy, 0, 0, (cudaStream_t)stream, a) ==
                 cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

int gdn_cache_free(const gdn_kv_cache* cache, const int32_t* rows, int32_t n,
                   gdn_stream_t stream) {
  if (const int rc = kv::check_cache(cache)) return rc;
  if (n < 0 || (n > 0 && !rows)) return GDN_ERR_INVALID_ARG;
  if (!aligned(rows, 4)) return GDN_ERR_ALIGNMENT;
  if (n == 0) return GDN_OK;
  const kv::Spans own = kv::spans_of(*cache);
  const Span ins[] = {span_of(rows, (size_t)n * 4)};
  if (any_overlap(ins, own.s)) return GDN_ERR_INVALID_ARG;
  unsigned* status = status_ptr();
  if (!status) return GDN_ERR_CUDA;
  count_launches(1);
  return launch(true, free_kernel, dim3((unsigned)n), 128, 0, 0, (cudaStream_t)stream, *cache,
                rows, status) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

int gdn_cache_fork(const gdn_kv_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                   gdn_stream_t stream) {
  if (const int rc = kv::check_cache(cache)) return rc;
  if (n < 0 || (n > 0 && (!src || !dst))) return GDN_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4)) return GDN_ERR_ALIGNMENT;
  const gdn_kv_cache c = *cache;
  if (c.layers > 32767 || (int64_t)c.kv_heads * c.page * c.d > 0x7fffffffLL)
    return GDN_ERR_UNSUPPORTED;
  if (n == 0) return GDN_OK;
  const kv::Spans own = kv::spans_of(c);
  const Span ins[] = {span_of(src, (size_t)n * 4), span_of(dst, (size_t)n * 4)};
  if (any_overlap(ins, own.s)) return GDN_ERR_INVALID_ARG;
  const cudaStream_t st = (cudaStream_t)stream;
  unsigned* status = status_ptr();
  void* scratch = nullptr;
  const size_t plan_bytes = align_up((size_t)n * sizeof(Pair), 256);
  if (!status || scratch_alloc(&scratch, plan_bytes + (size_t)n * 4, st) != cudaSuccess)
    return GDN_ERR_CUDA;
  Pair* plan = (Pair*)scratch;
  cudaError_t e = launch(true, fork_plan_kernel, dim3(1), kPlan, 0, 0, st, c, src, dst, n, plan,
                         (int32_t*)((char*)scratch + plan_bytes), status);
  if (e == cudaSuccess)
    e = launch(true, c.dtype == GDN_E4M3 ? fork_copy_kernel<true> : fork_copy_kernel<false>,
               dim3((unsigned)n, 1 + 2 * c.layers), kCopy, 0, 0, st, c, src, dst,
               (const Pair*)plan, status);
  count_launches(2);
  return finish(e, scratch, st);
}

int gdn_cache_compact(const gdn_kv_cache* cache, const gdn_kv_cache* into, gdn_stream_t stream) {
  if (const int rc = kv::check_cache(cache)) return rc;
  if (const int rc = kv::check_cache(into)) return rc;
  const gdn_kv_cache c = *cache, d = *into;
  if (c.layers != d.layers || c.kv_heads != d.kv_heads || c.page != d.page || c.d != d.d ||
      c.dtype != d.dtype || c.rows != d.rows || d.max_pages < c.max_pages)
    return GDN_ERR_INVALID_ARG;
  const kv::Spans a = kv::spans_of(c), b = kv::spans_of(d);
  if (any_overlap(a.s, b.s)) return GDN_ERR_INVALID_ARG;
  const cudaStream_t st = (cudaStream_t)stream;
  unsigned* status = status_ptr();
  void* scratch = nullptr;
  const size_t order_bytes = align_up((size_t)d.pages * 4, 256);
  if (!status ||
      scratch_alloc(&scratch, 256 + order_bytes + (size_t)c.pages * 4, st) != cudaSuccess)
    return GDN_ERR_CUDA;
  int32_t* count = (int32_t*)scratch;
  int32_t* order = (int32_t*)((char*)scratch + 256);
  int32_t* number = (int32_t*)((char*)order + order_bytes);
  cudaError_t e = launch(true, compact_plan_kernel, dim3(1), kPlan, 0, 0, st, c, d, count, order,
                         number, status);
  const int64_t jobs = 2 * (int64_t)c.layers * least(c.pages, d.pages);
  if (e == cudaSuccess)
    e = launch(true, c.dtype == GDN_E4M3 ? compact_copy_kernel<true> : compact_copy_kernel<false>,
               dim3((unsigned)least(c.rows + jobs, 1 << 30)), kCopy, 0, 0, st, c, d,
               (const int32_t*)count, (const int32_t*)order, (const int32_t*)number, jobs, status);
  count_launches(2);
  return finish(e, scratch, st);
}

}  // extern "C"
