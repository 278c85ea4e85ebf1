// Attention of one new token a row over the paged cache (contract:
// include/gdn.h):
//
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q . k_j,  m = max_j s_j
//
// Every key and value is used once by each of a group's query heads, so the
// cache's bytes through HBM bound it, whatever the rows' lengths.  The tiles of
// all rows and kv heads (64 tokens of 256 bytes, 128 of fewer) form one list, with a slot
// for each (row, head)'s end; CTA c of n takes the c-th n-th of it.  One warp walks the CTA's part and has TMA bring the tiles, page by
// page, into a ring; four warps take a quarter of a tile each, with softmax
// statistics of their own.  (With the loads' addresses computed by all threads
// these took more instructions than the attention: heads of 64 ran at 3.8 TB/s,
// 8 bits at 1.4 to 3.)  The heads of a group (up to 16, then in parts) are the rows
// of the matrix instructions: with one token there is nothing else to fill them.
// Where a (row, head) ends, the warps' sums are joined; one that is cut over
// several CTAs is joined from their partial sums by a second kernel, in the order
// of the CTAs.
//
// 16 query and 4 kv heads of 128: 256 rows of up to 8192 tokens 314 us (6.7 TB/s), in
// 8 bits 195 (5.6; widening the codes); of up to 512 tokens 33 and 29; one row of 32768
// tokens in 8 bits 17 us, of which the bytes are 5.  Heads of 64 in 8 bits: 3.8 TB/s, a
// tile's 128 tokens of 64 bytes being too little for the steps that follow one another
// in it.  Tiles of 64 tokens in 8 bits: 18.9 us for the one row, 9 % more for 256.
#include "attention_tc.cuh"
#include "gdn_internal.cuh"
#include "hostcheck.cuh"
#include "kv_cache.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

using namespace hostcheck;
using namespace sm100;

constexpr int kWarps = 4;                       // that compute
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kHeads = 16;          // rows of a matrix instruction
constexpr int kSms = 152;
constexpr int kCtas = 2 * kSms;     // two resident ones an SM
constexpr int kJoinThreads = 256;
constexpr float kLog2e = 1.44269504088896341f;
constexpr long long kWaitCycles = 4000000000ll;   // about two seconds

template <int D, bool kFp8>
struct Shape {
  static constexpr int kRow = D * (kFp8 ? 1 : 2);           // bytes of a token's head
  static constexpr int kTile = kRow == 256 ? 64 : 128;      // tokens
  static constexpr int kSub = kRow < 128 ? kRow : 128;      // bytes of a row of an image
  static constexpr int kHalves = kRow / kSub;               // images side by side
  static constexpr uint32_t kImage = kTile * kSub;
  static constexpr uint32_t kPool = kHalves * kImage;       // of keys or values
  static constexpr uint32_t kScales = kFp8 ? kTile * 4 : 0;
  static constexpr uint32_t kQ = 2 * kPool;                 // where the queries lie
  static constexpr uint32_t kQBytes = kHeads * D * 2;
  static constexpr uint32_t kScaleAt = kQ + kQBytes;
  static constexpr uint32_t kStage = kScaleAt + (kFp8 ? 1024 : 0);
  static constexpr int kStages = kRow == 64 ? 5 : 3;
  static constexpr int kPitch = D + 8;                      // floats of a row of the join
  static constexpr uint32_t kSmall = kStages * kStage;      // where Small lies
  static constexpr uint32_t kSmem = kSmall + 1024;
  static_assert(kWarps * kHeads * kPitch * 4 <= kStage, "the join uses a consumed stage");
  static_assert(2 * kScales <= 1024 && kStage % 1024 == 0, "");
};

// One tile of the list.
struct Tile {
  int32_t row, hh, at, n, len;   // row, its (kv head, part of the group), tile, tiles, tokens
};
// (8 bits, heads of 128: two CTAs' shared memory is all of an SM's but 2.5 KB, so
// there is no static part, and the dynamic one starts on 1024 bytes.)
struct Small {
  uint64_t full[5], empty[5];
  Tile meta[5];
  float ml[kWarps][kHeads][3];   // a warp's maximum and sum, 8 bits: and its weights' maximum
};
static_assert(sizeof(Small) <= 1024, "");

// What is left of a cut (row, head)'s parts: slot 2c of CTA c if the part
// continues one, 2c + 1 if it begins one.
struct Work {
  int4* cut;          // [CTAs] the cut (row, kv head and part of the group) that begins in it, and its
                      // parts (0: none does)
  float* ml;          // [slots][16][2] maximum (of scores in powers of two), sum
  float* o;           // [slots][16][D]
};
struct Args {
  CUtensorMap q, k, v;
  __nv_bfloat16* out;
  gdn_kv_cache c;
  int32_t layer, q_heads, group, parts, items_per_row, page_log2;
  float scale_log2;
  Work w;
  unsigned* status;
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 x 8 += 16 x 16 times 16 x 8, bf16 or (kHalf) fp16 operands
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kHalf)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four e4m3 codes as fp16, two a register (exact: 4 exponent bits in 5, 3 in 10).
__device__ __forceinline__ void e4m3_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
      " cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// base-2 logarithm by the special-function unit (2^-22 absolute near 1)
__device__ __forceinline__ float lg2_sfu(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte of 16-byte chunk `c` of row `r` in TMA's swizzled image of rows of 128 or
// 64 bytes: eight consecutive rows' chunks of one column lie in different bank
// groups.
template <int kSub>
__device__ __forceinline__ uint32_t image(int r, int c) {
  return (uint32_t)(r * kSub + ((c ^ (kSub == 128 ? r & 7 : (r >> 1) & 3)) << 4));
}
// Chunk `c` of row `r` where rows are cut into images of kSub bytes, kRows rows each.
template <int kSub, int kRows>
__device__ __forceinline__ uint32_t place(int r, int c) {
  constexpr int kPer = kSub / 16;
  return (uint32_t)(c / kPer * kRows * kSub) + image<kSub>(r, c % kPer);
}

// The first tile of CTA i of n.
__device__ __forceinline__ int64_t begin_of(int64_t total, int64_t i, int64_t n) {
  const uint64_t x = (uint64_t)total * (uint64_t)i;
  return x >> 32 ? (int64_t)(x / (uint64_t)n) : (int64_t)((uint32_t)x / (uint32_t)n);
}
// The CTA of n that has tile t.
__device__ __forceinline__ int64_t owner_of(int64_t total, int64_t t, int64_t n) {
  const uint64_t x = (uint64_t)(t + 1) * (uint64_t)n - 1;
  return x >> 32 ? (int64_t)(x / (uint64_t)total) : (int64_t)((uint32_t)x / (uint32_t)total);
}

// tokens of a row, 0 where its length is out of range
__device__ __forceinline__ int32_t row_tokens(const gdn_kv_cache& c, int64_t row, unsigned* status) {
  if (row >= c.rows) return 0;
  const int32_t n = c.lengths[row];
  if (n >= 0 && n <= c.max_pages * c.page) return n;
  flag_status(status, GDN_ERR_BAD_CACHE);
  return 0;
}

// Slots of the list that a (row, head) of n tiles takes: one more than its tiles, for its
// end and beginning (the join of its warps' sums, the next one's first tile) cost about a
// tile.  (By tiles alone, 256 rows of up to 512 tokens: the CTAs with short rows ran 33 us where
// the median one ran 25, 38 us in all instead of 29.)
__device__ __forceinline__ int32_t slots_of(int32_t n) { return n > 0 ? n + 1 : 0; }

// Zeros for the rows without tokens, by one warp of every CTA.
template <int D>
__device__ __forceinline__ void zero_empty_rows(const Args& a, int lane) {
  for (int64_t r = blockIdx.x; r < a.c.rows; r += gridDim.x) {
    if (row_tokens(a.c, r, nullptr) > 0) continue;
    uint4* to = reinterpret_cast<uint4*>(a.out + r * a.q_heads * D);
    for (int64_t i = lane; i < (int64_t)a.q_heads * D / 8; i += 32) to[i] = make_uint4(0, 0, 0, 0);
  }
}

// Zeros in the place of a stage's tokens [from, from + n), by one warp.
template <typename S, bool kFp8>
__device__ __forceinline__ void zero_tokens(uint8_t* base, int from, int n, int lane) {
  for (int half = 0; half < 2 * S::kHalves; ++half) {      // of the keys, then of the values
    uint4* z = reinterpret_cast<uint4*>(base + half * S::kImage + from * S::kSub);
    for (int i = lane; i < n * S::kSub / 16; i += 32) z[i] = make_uint4(0, 0, 0, 0);
  }
  if constexpr (kFp8)
    for (int i = lane; i < 2 * n; i += 32)
      *reinterpret_cast<float*>(base + S::kScaleAt + (i < n ? 0 : S::kScales) +
                                (from + (i < n ? i : i - n)) * 4) = 0.f;
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, 2) decode_kernel(const __grid_constant__ Args a) {
  using S = Shape<D, kFp8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Small& small = *reinterpret_cast<Small*>(smem + S::kSmall);
  uint64_t* full = small.full;
  uint64_t* empty = small.empty;
  Tile* meta = small.meta;
  auto& ml = small.ml;
  // (in the stages, before anything is loaded)
  int64_t* sums = reinterpret_cast<int64_t*>(smem);
  int64_t* warp_sums = sums + kThreads + 1;
  int64_t* where = warp_sums + kWarps + 1;
  int32_t* lens = reinterpret_cast<int32_t*>(where + 2);   // a thread's only row, with few rows
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const gdn_kv_cache& c = a.c;
  const int HH = a.items_per_row;
  grid_release_next();
  if (smem_u32(smem) & 1023u) {
    grid_wait();
    if (tid == 0) {
      flag_status(a.status, GDN_ERR_UNSUPPORTED);
      a.w.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    fence_barrier_init();
  }
  if (tid == kThreads - 1) {
    prefetch_tensormap(&a.q);
    prefetch_tensormap(&a.k);
    prefetch_tensormap(&a.v);
  }

  grid_wait();
  // the list's length, and where this CTA's part begins
  const int64_t per = ((int64_t)c.rows + kThreads - 1) / kThreads;
  const int64_t r0 = tid * per, r1 = r0 + per < c.rows ? r0 + per : c.rows;
  const bool few = per == 1;
  int64_t mine = 0;
  if (few) {
    const int32_t n = row_tokens(c, tid, a.status);
    lens[tid] = n;
    mine = slots_of((n + S::kTile - 1) / S::kTile);
  } else {
    for (int64_t r = r0; r < r1; ++r)
      mine += slots_of((row_tokens(c, r, a.status) + S::kTile - 1) / S::kTile);
  }
  {
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += warp_sums[w];
    sums[tid + 1] = x;
    if (tid == 0) sums[0] = 0;
    __syncthreads();
  }
  const int64_t total = sums[kThreads] * HH;
  // (the table that fits the GPU's memory bounds total below 2^50: 64 bits do)
  const int64_t ctas = total < gridDim.x ? total : gridDim.x;   // none has no slot
  if (blockIdx.x >= ctas) {
    if (tid == 0) a.w.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (warp == kWarps) zero_empty_rows<D>(a, lane);
    return;
  }
  int64_t lo = begin_of(total, blockIdx.x, ctas);
  const int64_t hi = begin_of(total, blockIdx.x + 1, ctas);
  if (lo >= sums[tid] * HH && lo < sums[tid + 1] * HH) {
    int64_t left = lo - sums[tid] * HH;
    if (few) {
      where[0] = tid;
      where[1] = left;
    }
    for (int64_t r = few ? r1 : r0; r < r1; ++r) {
      const int64_t n = (int64_t)slots_of((row_tokens(c, r, nullptr) + S::kTile - 1) / S::kTile) * HH;
      if (left < n) {
        where[0] = r;
        where[1] = left;
        break;
      }
      left -= n;
    }
  }
  __syncthreads();
  const int64_t row0 = where[0], in_row = where[1];
  const int32_t len0 = few ? lens[row0] : row_tokens(c, row0, nullptr);
  const int32_t len1 = few && row0 + 1 < kThreads ? lens[row0 + 1] : row_tokens(c, row0 + 1, nullptr);
  fence_proxy_async_smem();
  __syncthreads();
  bool ok = true;
  // the first tile, if the first slot is not a (row, head)'s last, which has none
  const int32_t slots0 = slots_of((len0 + S::kTile - 1) / S::kTile);
  const int32_t hh0 = (int32_t)(in_row / slots0), at0 = (int32_t)(in_row - (int64_t)hh0 * slots0);
  const bool skip = at0 == slots0 - 1;
  if (skip) ++lo;

  if (warp == kWarps) {
    // --------------------------------------------------------------- load
    const bool lead = elect_one();
    const int lg = a.page_log2;
    const int box = c.page < S::kTile ? c.page : S::kTile;   // tokens of one copy
    constexpr int kIds = S::kTile / 16;                      // copies of a tile at most
    Tile t;
    t.row = (int32_t)row0;
    t.len = len0;
    int32_t next_len = len1;
    t.n = (t.len + S::kTile - 1) / S::kTile;
    t.hh = hh0;
    t.at = at0;
    // on to the next tile of the list: true where another (row, head) begins
    auto advance = [&]() {
      if (++t.at < t.n) return false;
      t.at = 0;
      if (++t.hh == HH) {
        t.hh = 0;
        do {
          ++t.row;
          t.len = next_len;
          t.n = (t.len + S::kTile - 1) / S::kTile;
          next_len = row_tokens(c, (int64_t)t.row + 1, nullptr);
        } while (t.n == 0 && t.row < c.rows);
      }
      return true;
    };
    if (skip) {
      t.at = t.n - 1;
      advance();
    }
    // lane i reads the page of the tile's i-th copy, one tile ahead
    auto read_id = [&]() {
      const int64_t pos = (int64_t)t.at * S::kTile + lane * box;
      int32_t id = 0;
      if (lane < kIds && lane * box < S::kTile && pos < t.len)
        id = c.table[(int64_t)t.row * c.max_pages + (pos >> lg)];
      return id;
    };
    int32_t id = lo < hi ? read_id() : 0;
    bool fresh = true;                                       // the first tile of its part
    int64_t step = 1;                                        // slots to the next tile
    int64_t k = 0;
    for (int64_t i = lo; i < hi; i += step, ++k) {
      const int stage = (int)(k % S::kStages);
      const Tile now = t;
      const bool first = fresh;
      const int32_t ids = id;
      fresh = advance();
      step = fresh ? 2 : 1;
      if (i + step < hi) id = read_id();
      ok = mbar_wait_warp_cycles(&empty[stage], (uint32_t)((k / S::kStages) & 1) ^ 1u, kWaitCycles);
      if (!ok) break;
      const int64_t pos = (int64_t)now.at * S::kTile;
      const int64_t tokens = now.len - pos < S::kTile ? now.len - pos : S::kTile;
      const int copies = (int)((tokens + box - 1) / box);
      const int h = now.hh / a.parts, part = now.hh - h * a.parts;
      uint8_t* base = smem + stage * S::kStage;
      const int32_t off = (int32_t)(pos & (c.page - 1));     // (pages longer than a tile)
      auto begin = [&](int from_pages) {
        if (!lead) return;
        meta[stage] = now;
        mbar_arrive_expect_tx(&full[stage], from_pages * box * (2 * S::kRow + (kFp8 ? 8 : 0)) +
                                                (first ? S::kQBytes : 0));
        if (first)
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tma_load_2d(base + S::kQ + x * kHeads * 128, &a.q, 64 * x,
                        now.row * a.q_heads + h * a.group + part * kHeads, &full[stage]);
      };
      auto copy = [&](int x) {
        const int32_t p = __shfl_sync(0xffffffffu, ids, x);
        if (!lead) return;
#pragma unroll
        for (int y = 0; y < S::kHalves; ++y) {
          uint8_t* to = base + y * S::kImage + x * box * S::kSub;
          const int32_t col = y * (S::kSub / (kFp8 ? 1 : 2));
          tma_load_3d(to, &a.k, col, h * c.page + off, a.layer * c.pages + p, &full[stage]);
          tma_load_3d(to + S::kPool, &a.v, col, h * c.page + off, a.layer * c.pages + p, &full[stage]);
        }
        if constexpr (kFp8) {
          const int64_t e = (((int64_t)a.layer * c.pages + p) * c.kv_heads + h) * c.page + off;
          uint8_t* to = base + S::kScaleAt + x * box * 4;
          tma_load_1d(to, c.k_scale + e, box * 4, &full[stage]);
          tma_load_1d(to + S::kScales, c.v_scale + e, box * 4, &full[stage]);
        }
      };
      const bool gone = ids < 0 || ids >= c.pages;
      if (!__any_sync(0xffffffffu, gone)) {
        begin(copies);
        for (int x = 0; x < copies; ++x) copy(x);
      } else {                                               // zeros in the place of pages that are none
        const unsigned none = __ballot_sync(0xffffffffu, gone);
        flag_status(a.status, GDN_ERR_BAD_CACHE);
        for (int x = 0; x < copies; ++x)
          if (none >> x & 1u) zero_tokens<S, kFp8>(base, x * box, box, lane);
        fence_proxy_async_smem();
        __syncwarp();
        begin(copies - __popc(none));
        for (int x = 0; x < copies; ++x)
          if (!(none >> x & 1u)) copy(x);
      }
      __syncwarp();
    }
    zero_empty_rows<D>(a, lane);
  } else {
    // ---------------------------------------------------------- attention
    const int g = lane >> 2, t4 = lane & 3;
    constexpr int kSteps = D / 16;
    constexpr int kTok = S::kTile / kWarps;   // a warp's tokens of a tile
    constexpr int kGroups = kTok / 16;
    // 8 bits: a weight is the probability times the value's scale.  In powers of
    // two its exponent is the score's plus the scale's logarithm; with a running
    // maximum of its own, fp16 holds all weights that matter (the largest is
    // 2^8, what is lost of small ones 2^-33 of that).
    constexpr float kRoom = 8.f;
    uint32_t qa[kSteps][4];
    float o[D / 8][4];
    float m[2], l[2];
    float unit[2];        // scores' factor of rows g and g + 8
    float wm[2];          // 8 bits: the weights' running maxima
    bool start = true;
    int64_t first_of_part = lo, k = 0;
    bool begins = false;         // a (row, head) that is cut begins here
    for (int64_t i = lo, step; i < hi; i += step, ++k) {
      const int stage = (int)(k % S::kStages);
      ok = mbar_wait_warp_cycles(&full[stage], (uint32_t)((k / S::kStages) & 1), kWaitCycles);
      if (!ok) {
        // the others meet where their part ends, which is at this tile or behind it
        attn::bar_agree(2, 32 * kWarps, false);
        break;
      }
      const Tile tile = meta[stage];
      uint8_t* bytes = smem + stage * S::kStage;
      const uint32_t base = smem_u32(bytes);
      if (start) {
        first_of_part = i;
        start = false;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[j][x] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
        unit[0] = unit[1] = a.scale_log2;
        wm[0] = wm[1] = -INFINITY;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if constexpr (!kFp8) {
            // rows 0-7 and 8-15 of the first eight columns, then of the second
            ldmatrix4(qa[s], base + S::kQ + place<128, kHeads>((lane & 7) + ((lane >> 3) & 1) * 8,
                                                               2 * s + (lane >> 4)));
          } else {
            // the order in which four consecutive codes of a key arrive: columns
            // 4t, 4t + 1 in the place of 2t, 2t + 1 and the next two in that of
            // 2t + 8, 2t + 9 (a sum over columns may take them in any order)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t p =
                  base + S::kQ + place<128, kHeads>(g + 8 * x, 2 * s + (t4 >> 1)) + (t4 & 1) * 8;
              asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                           : "=r"(qa[s][x]), "=r"(qa[s][2 + x])
                           : "r"(p));
            }
          }
        }
        if constexpr (kFp8) {
          // queries as fp16, a row times a power of two that puts its largest
          // between 2^8 and 2^9: fp16 holds bf16's digits down to 2^-22 of that,
          // and what it loses below is 2^-33 of it
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
              for (int y = x; y < 4; y += 2) {
                top = max(top, qa[s][y] << 16 & 0x7fffffffu);
                top = max(top, qa[s][y] & 0x7fff0000u);
              }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(8 - exponent), its size kept within fp32's normal numbers
            int e = 8 + 127 - (int)(top >> 23);
            e = top == 0 || top >= 0x7f800000u ? 0 : e > 126 ? 126 : e < -126 ? -126 : e;
            const float f = __uint_as_float((uint32_t)(e + 127) << 23);
            unit[x] *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
              for (int y = x; y < 4; y += 2)
                qa[s][y] = pack_half(__uint_as_float(qa[s][y] << 16) * f,
                                     __uint_as_float(qa[s][y] & 0xffff0000u) * f);
          }
        }
      }
      const int valid = tile.len - tile.at * S::kTile;   // tokens of the tile (or more)
      if (valid < S::kTile) {
        // values behind the last token are whatever the page holds: a product
        // with a zero probability has to be zero
        for (int tok = warp * kTok + lane / (S::kSub / 16); tok < (warp + 1) * kTok;
             tok += 32 / (S::kSub / 16))
          if (tok >= valid)
#pragma unroll
            for (int y = 0; y < S::kHalves; ++y)
              *reinterpret_cast<uint4*>(bytes + S::kPool + y * S::kImage + tok * S::kSub +
                                        lane % (S::kSub / 16) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
      }
      const int tok0 = warp * kTok;
      if (tok0 < valid) {
        // scores of 16 heads and the warp's 16 or 32 tokens
        float s[2 * kGroups][4] = {};
        if constexpr (!kFp8) {
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
              uint32_t b[4];
              ldmatrix4(b, base + place<S::kSub, S::kTile>(tok0 + 16 * i + (lane >> 4) * 8 + (lane & 7),
                                                           2 * k + ((lane >> 3) & 1)));
              mma16816<false>(s[2 * i], qa[k], b[0], b[1]);
              mma16816<false>(s[2 * i + 1], qa[k], b[2], b[3]);
            }
        } else {
#pragma unroll
          for (int k = 0; k < kSteps; k += 2)
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
              uint32_t b[4];
              ldmatrix4(b, base + place<S::kSub, S::kTile>(tok0 + 16 * i + (lane >> 4) * 8 + (lane & 7),
                                                           k + ((lane >> 3) & 1)));
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                uint32_t b0, b1;
                e4m3_to_half(b[x], b0, b1);
                mma16816<true>(s[2 * i + (x >> 1)], qa[k + (x & 1)], b0, b1);
              }
            }
        }
        float vs[2 * kGroups][2];
#pragma unroll
        for (int n = 0; n < 2 * kGroups; ++n) {
          const int col = tok0 + n * 8 + 2 * t4;
          const bool v0 = col < valid, v1 = col + 1 < valid;
          float k0 = 1.f, k1 = 1.f;
          if constexpr (kFp8) {
            const float2 ks = *reinterpret_cast<const float2*>(bytes + S::kScaleAt + col * 4);
            const float2 v2 = *reinterpret_cast<const float2*>(bytes + S::kScaleAt + S::kScales + col * 4);
            k0 = ks.x;
            k1 = ks.y;
            vs[n][0] = lg2_sfu(v2.x);
            vs[n][1] = lg2_sfu(v2.y);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            s[n][2 * x] = v0 ? s[n][2 * x] * (kFp8 ? unit[x] * k0 : unit[x]) : -INFINITY;
            s[n][2 * x + 1] = v1 ? s[n][2 * x + 1] * (kFp8 ? unit[x] * k1 : unit[x]) : -INFINITY;
          }
        }
        // running maximum and sum of rows g and g + 8; 8 bits: the weights' too, whose
        // exponents are the scores' plus the scales' (behind the last token the
        // scale may be anything)
        float top[2][2];
        bool grew = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = -INFINITY, mw = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2 * kGroups; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float v = s[n][2 * x + y];
              mx = fmaxf(mx, v);
              if constexpr (kFp8) mw = fmaxf(mw, v == -INFINITY ? -INFINITY : v + vs[n][y]);
            }
          top[x][0] = mx;
          top[x][1] = mw;
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            top[x][0] = fmaxf(top[x][0], __shfl_xor_sync(0xffffffffu, top[x][0], d));
            if constexpr (kFp8) top[x][1] = fmaxf(top[x][1], __shfl_xor_sync(0xffffffffu, top[x][1], d));
          }
#pragma unroll
        for (int x = 0; x < 2; ++x) grew |= top[x][0] > m[x] || (kFp8 && top[x][1] > wm[x]);
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float f = top[x][0] > m[x] ? ex2_sfu(m[x] - top[x][0]) : 1.f;
            float fo = f;
            l[x] *= f;
            m[x] = fmaxf(m[x], top[x][0]);
            if constexpr (kFp8) {
              fo = top[x][1] > wm[x] ? ex2_sfu(wm[x] - top[x][1]) : 1.f;
              wm[x] = fmaxf(wm[x], top[x][1]);
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
              o[j][2 * x] *= fo;
              o[j][2 * x + 1] *= fo;
            }
          }
        }
        uint32_t p[kGroups][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float z = m[x] == -INFINITY ? 0.f : m[x];
          const float zw = !kFp8 || wm[x] == -INFINITY ? 0.f : kRoom - wm[x];
#pragma unroll
          for (int n = 0; n < 2 * kGroups; ++n) {
            const float s0 = s[n][2 * x], s1 = s[n][2 * x + 1];
            const float p0 = ex2_sfu(s0 - z), p1 = ex2_sfu(s1 - z);
            l[x] += p0 + p1;
            if constexpr (kFp8) {
              const float u0 = s0 == -INFINITY ? -INFINITY : s0 + vs[n][0];
              const float u1 = s1 == -INFINITY ? -INFINITY : s1 + vs[n][1];
              p[n >> 1][2 * (n & 1) + x] = pack_half(ex2_sfu(u0 + zw), ex2_sfu(u1 + zw));
            } else {
              p[n >> 1][2 * (n & 1) + x] = pack_bf16(p0, p1);
            }
          }
        }
        // out of 16 heads, the warp's tokens added
        const uint32_t vb = base + S::kPool;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const int vr = tok0 + 16 * i + ((lane >> 3) & 1) * 8 + (lane & 7);
          if constexpr (!kFp8) {
#pragma unroll
            for (int j = 0; j < D / 8; j += 2) {
              uint32_t b[4];
              ldmatrix4t(b, vb + place<S::kSub, S::kTile>(vr, j + (lane >> 4)));
              mma16816<false>(o[j], p[i], b[0], b[1]);
              mma16816<false>(o[j + 1], p[i], b[2], b[3]);
            }
          } else {
            // a transposed pair of codes is two columns: even ones to o[2j], odd to
            // o[2j + 1], so that a lane ends with four consecutive columns of 16
#pragma unroll
            for (int j = 0; j < D / 16; j += 2) {
              uint32_t b[4];
              ldmatrix4t(b, vb + place<S::kSub, S::kTile>(vr, j + (lane >> 4)));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t e0, d0, e1, d1;
                e4m3_to_half(__byte_perm(b[2 * x], 0, 0x3120), e0, d0);
                e4m3_to_half(__byte_perm(b[2 * x + 1], 0, 0x3120), e1, d1);
                mma16816<true>(o[2 * (j + x)], p[i], e0, e1);
                mma16816<true>(o[2 * (j + x) + 1], p[i], d0, d1);
              }
            }
          }
        }
      }
      const bool item_ends = tile.at == tile.n - 1;
      step = item_ends ? 2 : 1;                          // (behind its last tile a slot without one)
      if (!item_ends && i + 1 < hi) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        continue;
      }

      // the part ends: join the warps' sums, in the consumed stage
      start = true;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        if (t4 == 0) {
          ml[warp][g + 8 * x][0] = m[x];
          ml[warp][g + 8 * x][1] = l[x];
          if constexpr (kFp8) ml[warp][g + 8 * x][2] = wm[x];
        }
      }
      // (the stage's other readers are done at the next barrier but one: every warp's own
      // rows of the join lie behind its tokens' bytes only after this one)
      ok = attn::bar_agree(2, 32 * kWarps, true);
      if (!ok) break;
      const int h = tile.hh / a.parts, part = tile.hh - h * a.parts;
      const int heads = a.group - part * kHeads < kHeads ? a.group - part * kHeads : kHeads;
      float* js = reinterpret_cast<float*>(bytes);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (g + 8 * x >= heads) break;
        float* r = js + (warp * kHeads + g + 8 * x) * S::kPitch;
        if constexpr (!kFp8) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2*>(r + j * 8 + 2 * t4) = make_float2(o[j][2 * x], o[j][2 * x + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
            *reinterpret_cast<float4*>(r + j * 16 + 4 * t4) =
                make_float4(o[2 * j][2 * x], o[2 * j + 1][2 * x], o[2 * j][2 * x + 1],
                            o[2 * j + 1][2 * x + 1]);
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
      const int64_t item_begin = i - tile.at;
      const bool from_begin = first_of_part == item_begin, whole = from_begin && item_ends;
      const int64_t slot = 2 * (int64_t)blockIdx.x + from_begin;
      if (from_begin && !whole) {
        begins = true;
        if (tid == 0)
          a.w.cut[blockIdx.x] = make_int4(
              tile.row, tile.hh, (int)(owner_of(total, item_begin + tile.n - 1, ctas) - blockIdx.x + 1), 0);
      }
#pragma unroll
      for (int v = 0; v < kHeads * D / 4 / (32 * kWarps); ++v) {
        const int e = v * 32 * kWarps + tid, row = e / (D / 4), col = e % (D / 4) * 4;
        if (row >= heads) break;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -INFINITY, all = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][row][0]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(js + (w * kHeads + row) * S::kPitch + col);
          const float mw = ml[w][row][0];
          const float fl = mw == -INFINITY ? 0.f : ex2_sfu(mw - top);
          float f = fl;
          if constexpr (kFp8) {
            const float ww = ml[w][row][2];
            f = mw == -INFINITY || ww == -INFINITY ? 0.f : ex2_sfu(ww - kRoom - top);
          }
          sum.x = fmaf(y.x, f, sum.x); sum.y = fmaf(y.y, f, sum.y);
          sum.z = fmaf(y.z, f, sum.z); sum.w = fmaf(y.w, f, sum.w);
          all += mw == -INFINITY ? 0.f : ml[w][row][1] * fl;
        }
        // (a warp whose scores were all NaN kept the maximum -inf: its sum is NaN)
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          if (isnan(ml[w][row][1])) all = ml[w][row][1];
        if (whole) {
          const float inv = 1.f / all;
          const int64_t to =
              ((int64_t)tile.row * a.q_heads + (int64_t)h * a.group + part * kHeads + row) * D + col;
          *reinterpret_cast<uint2*>(a.out + to) =
              make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
        } else {
          *reinterpret_cast<float4*>(a.w.o + (slot * kHeads + row) * D + col) = sum;
          if (col == 0) {
            a.w.ml[(slot * kHeads + row) * 2] = top;
            a.w.ml[(slot * kHeads + row) * 2 + 1] = all;
          }
        }
      }
      // TMA writes the stage next; ml is written again only by warps that all
      // others have passed here for
      fence_proxy_async_smem();
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
      if (lane == 0) mbar_arrive(&empty[stage]);
    }
    if (tid == 0 && !begins) a.w.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  if (!ok) {
    // copies in flight end within microseconds; give them longer
    flag_status(a.status, GDN_ERR_TIMEOUT);
    const uint64_t from = globaltimer_ns();
    while (globaltimer_ns() - from < 5000000ull) __nanosleep(1000);
  }
}

// The cut (row, head)s: blockIdx.x's is the one that begins in that CTA of the kernel before,
// if one does; a CTA takes one of its query heads, its warps every eighth part, then the
// warps' sums in order.  (Every load of a step in flight at once: parts one after another
// took 11 us for the 76 of a row of 32768 tokens.)
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Args a) {
  constexpr int kN = kJoinThreads / 32, kV = D / 32;
  __shared__ float sm[kN][D + 2], weight[kCtas], sum[kCtas];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_release_next();
  grid_wait();
  const int first = blockIdx.x, r = blockIdx.y;
  const uint4 cut = ld_waited(reinterpret_cast<const uint4*>(a.w.cut + first));
  const int row = (int)cut.x, hh = (int)cut.y, parts = (int)cut.z;
  const int h = hh / a.parts, part = hh - h * a.parts, in = part * kHeads + r;
  if (parts == 0 || in >= a.group) return;
  __nv_bfloat16* out = a.out + ((int64_t)row * a.q_heads + (int64_t)h * a.group + in) * D;
  auto slot = [&](int p) { return (int64_t)((2 * (first + p) + (p == 0)) * kHeads + r); };
  // the parts' maxima and sums, then every part's factor; a warp's first four
  // parts are on their way by then
  float x[4][kV];
  auto read = [&](int p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* src = a.w.o + slot(p + i * kN) * D + lane * kV;
      if (p + i * kN >= parts) continue;
      if constexpr (kV == 4) {
        const float4 t = ld_waited(reinterpret_cast<const float4*>(src));
        x[i][0] = t.x; x[i][1] = t.y; x[i][2] = t.z; x[i][3] = t.w;
      } else {
        x[i][0] = ld_waited(src);
        x[i][1] = ld_waited(src + 1);
      }
    }
  };
  read(warp);
  float m = -INFINITY;
  for (int p = threadIdx.x; p < parts; p += kJoinThreads) {
    const float mp = ld_waited(a.w.ml + slot(p) * 2);
    weight[p] = mp;
    sum[p] = ld_waited(a.w.ml + slot(p) * 2 + 1);
    m = fmaxf(m, mp);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sm[warp][D] = m;
  __syncthreads();
  m = sm[0][D];
#pragma unroll
  for (int w = 1; w < kN; ++w) m = fmaxf(m, sm[w][D]);
  float l = 0.f;
  for (int p = threadIdx.x; p < parts; p += kJoinThreads) {
    const float mp = weight[p], lp = sum[p];
    // (scores that are all NaN leave the maximum -inf and a NaN sum)
    const float f = mp == -INFINITY ? (isnan(lp) ? 1.f : 0.f) : ex2_sfu(mp - m);
    weight[p] = f;
    l += lp * f;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) sm[warp][D + 1] = l;
  __syncthreads();
  // a warp adds every eighth part, four in flight
  float o[kV] = {};
  for (int p = warp; p < parts; p += 4 * kN) {
    if (p != warp) read(p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p + i * kN < parts) {
        const float f = weight[p + i * kN];
#pragma unroll
        for (int j = 0; j < kV; ++j) o[j] = f == 0.f ? o[j] : fmaf(x[i][j], f, o[j]);
      }
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) sm[warp][lane * kV + i] = o[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float all = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < kN; ++w) {
      all += sm[w][D + 1];
      x += sm[w][threadIdx.x];
    }
    out[threadIdx.x] = __float2bfloat16_rn(x / all);
  }
}

struct Layout {
  size_t cut, ml, o, bytes;
};
Layout layout_of(int32_t d) {
  const size_t slots = 2 * (size_t)kCtas;
  Layout l;
  l.cut = 0;
  l.ml = align_up(kCtas * sizeof(int4), 256);
  l.o = l.ml + slots * kHeads * 2 * 4;
  l.bytes = l.o + slots * kHeads * d * 4;
  return l;
}
int heads_check(int32_t rows, int32_t q_heads, int32_t kv_heads, int32_t d) {
  if (rows < 1 || q_heads < 1 || kv_heads < 1) return GDN_ERR_INVALID_ARG;
  if (q_heads % kv_heads || q_heads / kv_heads > 128 || !kv::dim_ok(d)) return GDN_ERR_UNSUPPORTED;
  if ((int64_t)rows * q_heads > kLongestAxis) return GDN_ERR_UNSUPPORTED;   // 32-bit coordinates
  return GDN_OK;
}

// A pool of keys or values as [layers * pages][kv heads * page][row bytes], read in
// boxes of 128 (64) bytes x the smaller of a page and a tile, swizzled.
bool pool_map(CUtensorMap* m, const void* pool, const gdn_kv_cache& c, int32_t row, int32_t tile) {
  attn::EncodeFn enc = attn::encoder();
  if (!enc) return false;
  memset(m, 0, sizeof *m);
  const bool fp8 = c.dtype == GDN_E4M3;
  cuuint64_t dims[3] = {(cuuint64_t)c.d, (cuuint64_t)c.kv_heads * c.page,
                        (cuuint64_t)c.layers * c.pages};
  cuuint64_t strides[2] = {(cuuint64_t)row, (cuuint64_t)row * c.kv_heads * c.page};
  cuuint32_t box[3] = {fp8 ? (cuuint32_t)c.d : 64u, (cuuint32_t)(c.page < tile ? c.page : tile), 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(pool), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int decode(const void* q, const gdn_kv_cache* cache, int32_t layer, int32_t q_heads, float scale,
           void* out, bool use_ws, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (const int rc = kv::check_cache(cache)) return rc;
  const gdn_kv_cache c = *cache;
  if (const int rc = heads_check(c.rows, q_heads, c.kv_heads, c.d)) return rc;
  if ((int64_t)c.layers * c.pages > kLongestAxis || (int64_t)c.kv_heads * c.page > kLongestAxis)
    return GDN_ERR_UNSUPPORTED;
  if (!q || !out || layer < 0 || layer >= c.layers || !attn::scale_ok(scale))
    return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16)) return GDN_ERR_ALIGNMENT;
  const Layout lay = layout_of(c.d);
  if (use_ws) {
    if (!ws || ws_bytes < lay.bytes) return GDN_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return GDN_ERR_ALIGNMENT;
  }
  const size_t io = (size_t)c.rows * q_heads * c.d * 2;
  const kv::Spans own = kv::spans_of(c);
  const Span ins[] = {span_of(q, io), own.s[0], own.s[1], own.s[2], own.s[3],
                      own.s[4],       own.s[5], own.s[6]};
  const Span outs[] = {span_of(out, io), span_of(use_ws ? ws : nullptr, lay.bytes)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  Args a;
  memset(&a, 0, sizeof a);
  a.status = status_ptr();
  if (!a.status) return GDN_ERR_CUDA;
  a.out = (__nv_bfloat16*)out;
  a.c = c;
  a.layer = layer;
  a.q_heads = q_heads;
  a.group = q_heads / c.kv_heads;
  a.parts = (a.group + kHeads - 1) / kHeads;
  a.items_per_row = c.kv_heads * a.parts;
  a.page_log2 = kv::log2_of(c.page);
  a.scale_log2 = scale * kLog2e;
  const bool fp8 = c.dtype == GDN_E4M3;
  const int32_t row = c.d * (fp8 ? 1 : 2), tile = row == 256 ? 64 : 128;
  if (!pool_map(&a.k, c.k, c, row, tile) || !pool_map(&a.v, c.v, c, row, tile) ||
      !attn::heads_map(&a.q, q, (int64_t)c.rows * q_heads, c.d, kHeads))
    return GDN_ERR_CUDA;
  void* scratch = ws;
  if (!use_ws && scratch_alloc(&scratch, lay.bytes, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
  }
  char* p = (char*)scratch;
  a.w.cut = (int4*)(p + lay.cut);
  a.w.ml = (float*)(p + lay.ml);
  a.w.o = (float*)(p + lay.o);
  cudaError_t e;
  static std::atomic<uint64_t> on[4];
  auto run = [&](auto shape, auto kern, std::atomic<uint64_t>& allowed) {
    using S = decltype(shape);
    e = allow_smem((const void*)kern, S::kSmem, allowed);
    if (e == cudaSuccess) e = launch(true, kern, dim3(kCtas), kThreads, S::kSmem, 0, st, a);
  };
  if (c.d == 128)
    fp8 ? run(Shape<128, true>{}, decode_kernel<128, true>, on[0])
        : run(Shape<128, false>{}, decode_kernel<128, false>, on[1]);
  else
    fp8 ? run(Shape<64, true>{}, decode_kernel<64, true>, on[2])
        : run(Shape<64, false>{}, decode_kernel<64, false>, on[3]);
  if (e == cudaSuccess) {
    e = launch(true, c.d == 128 ? join_kernel<128> : join_kernel<64>,
               dim3(kCtas, (unsigned)(a.group < kHeads ? a.group : kHeads)), kJoinThreads, 0, 0, st, a);
  }
  count_launches(2);
  if (e != cudaSuccess) (void)cudaGetLastError();
  const cudaError_t f = use_ws ? cudaSuccess : scratch_free(scratch, st);
  return e == cudaSuccess && f == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_attention_decode_step(const void* q, const gdn_kv_cache* cache, int32_t layer,
                              int32_t q_heads, float scale, void* out, gdn_stream_t stream) {
  return decode(q, cache, layer, q_heads, scale, out, false, nullptr, 0, (cudaStream_t)stream);
}

size_t gdn_attention_decode_step_workspace_size(int32_t rows, int32_t q_heads, int32_t kv_heads,
                                                int32_t d) {
  if (heads_check(rows, q_heads, kv_heads, d)) return SIZE_MAX;
  return layout_of(d).bytes;
}

int gdn_attention_decode_step_ws(const void* q, const gdn_kv_cache* cache, int32_t layer,
                                 int32_t q_heads, float scale, void* out, void* workspace,
                                 size_t workspace_bytes, gdn_stream_t stream) {
  return decode(q, cache, layer, q_heads, scale, out, true, workspace, workspace_bytes,
                (cudaStream_t)stream);
}

}  // extern "C"
