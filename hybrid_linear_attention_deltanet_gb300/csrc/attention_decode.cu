// Attention of one new token a row over the paged cache (contract:
// include/gdn.h):
//
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q . k_j,  m = max_j s_j
//
// Every key and value is used once by each of a group's query heads, so the
// cache's bytes through HBM bound it, whatever the rows' lengths.  The tiles of
// all rows and kv heads (64 tokens; 128 in 8 bits) form one list; CTA c of n
// takes the c-th n-th of it, so that no CTA has more than a tile more than
// another.  A CTA walks its part with three stages of asynchronous 16-byte loads
// (the next tiles' page numbers and lengths a step ahead of them), its four
// warps taking a quarter of a tile each, with softmax statistics of their own.
// The heads of a group (up to 16, then in parts) are the rows of the matrix
// instructions: with one token there is nothing else to fill them, and these
// kernels' products are far from bounding anything.  Where a (row, head) ends,
// the warps' sums are joined; one that is cut over several CTAs is joined from
// their partial sums by a second kernel, in the order of the CTAs.
#include "gdn_internal.cuh"
#include "hostcheck.cuh"
#include "kv_cache.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

using namespace hostcheck;
using sm100::smem_u32;

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kHeads = 16;          // rows of a matrix instruction
constexpr int kSms = 152;
constexpr int kJoinThreads = 256;
constexpr float kLog2e = 1.44269504088896341f;

template <int D, bool kFp8>
struct Shape {
  static constexpr int kTile = kFp8 ? 128 : 64;             // tokens
  static constexpr int kRow = D * (kFp8 ? 1 : 2);           // bytes of a token's head
  static constexpr int kChunks = kRow / 16;
  static constexpr int kPool = kTile * kRow;
  static constexpr int kScales = kFp8 ? kTile * 4 : 0;
  static constexpr int kQ = 2 * kPool + 2 * kScales;        // where the queries lie
  static constexpr int kStage = kQ + kHeads * D * 2;
  static constexpr int kPitch = D + 8;                      // floats of a row of the join
  static constexpr int kSmem = kStages * kStage;
  static_assert(kWarps * kHeads * kPitch * 4 <= kStage, "the join uses a consumed stage");
};

// What is left of a cut (row, head)'s parts: slot 2c of CTA c if the part
// continues one, 2c + 1 if it begins one.
struct Work {
  int64_t total;      // tiles in all
  int64_t* begin;     // [items] first tile of a cut item, ...
  int64_t* end;       // ... and behind its last; 0: the item is not cut
  float* ml;          // [slots][16][2] maximum (of scores in powers of two), sum
  float* o;           // [slots][16][D]
};
struct Args {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  gdn_kv_cache c;
  int32_t layer, q_heads, group, parts, items_per_row, page_log2;
  float scale_log2;
  int64_t* total;     // Work::total in memory
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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
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
// Two e4m3 codes of w, chosen by the permutation that puts each in the upper
// byte of a half, as bf16: the exponent's four bits and the fraction's three
// move to their places, and the product with 2^120 (127 - 7) makes the
// exponent's bias bf16's, subnormal codes included.  Exact; a NaN code becomes
// a number, but then the scale is NaN.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t e4m3_to_bf16(uint32_t w) {
  const uint32_t x = __byte_perm(w, 0, kSel);
  const uint32_t y = ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x7b807b80u));
  return r;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte of 16-byte chunk `c` of row `r` in a swizzled image of rows of kRow bytes:
// eight consecutive rows' chunks of one column lie in different bank groups.
template <int kRow>
__device__ __forceinline__ uint32_t image(int r, int c) {
  return (uint32_t)(r * kRow + ((c ^ (kRow >= 128 ? r & 7 : (r >> 1) & 3)) << 4));
}

// One tile of the list.
struct Tile {
  int32_t row, hh, at, n, len;   // row, its (kv head, part of the group), tile, tiles, tokens
};

// tokens of a row, 0 where its length is out of range
__device__ __forceinline__ int32_t row_tokens(const gdn_kv_cache& c, int64_t row, unsigned* status) {
  if (row >= c.rows) return 0;
  const int32_t n = c.lengths[row];
  if (n >= 0 && n <= c.max_pages * c.page) return n;
  flag_status(status, GDN_ERR_BAD_CACHE);
  return 0;
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 4) decode_kernel(Args a) {
  using S = Shape<D, kFp8>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t sums[kThreads + 1];
  __shared__ int64_t where[2];
  __shared__ Tile meta[kStages];
  __shared__ float ml[kWarps][kHeads][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const gdn_kv_cache& c = a.c;
  const int HH = a.items_per_row;
  grid_release_next();

  // the list's length, and where this CTA's part begins
  const int64_t per = ((int64_t)c.rows + kThreads - 1) / kThreads;
  const int64_t r0 = tid * per, r1 = r0 + per < c.rows ? r0 + per : c.rows;
  int64_t mine = 0;
  for (int64_t r = r0; r < r1; ++r)
    mine += (row_tokens(c, r, a.status) + S::kTile - 1) / S::kTile;
  sums[tid + 1] = mine;
  if (tid == 0) sums[0] = 0;
  __syncthreads();
  for (int o = 1; o < kThreads; o <<= 1) {
    const int64_t t = tid >= o ? sums[tid + 1 - o] : 0;
    __syncthreads();
    sums[tid + 1] += t;
    __syncthreads();
  }
  const int64_t total = sums[kThreads] * HH;
  if (blockIdx.x == 0 && tid == 0) *a.total = total;
  const int64_t ctas = total < gridDim.x ? total : gridDim.x;   // none has no tile
  if (blockIdx.x >= ctas) return;
  const int64_t lo = (int64_t)((unsigned __int128)total * blockIdx.x / ctas);
  const int64_t hi = (int64_t)((unsigned __int128)total * (blockIdx.x + 1) / ctas);
  if (lo >= sums[tid] * HH && lo < sums[tid + 1] * HH) {
    int64_t left = lo - sums[tid] * HH;
    for (int64_t r = r0; r < r1; ++r) {
      const int64_t n = (row_tokens(c, r, nullptr) + S::kTile - 1) / S::kTile * HH;
      if (left < n) {
        where[0] = r;
        where[1] = left;
        break;
      }
      left -= n;
    }
  }
  __syncthreads();
  // the loads' place in the list, with the next row's tokens and the next
  // tile's pages read ahead
  Tile ld;
  ld.row = (int32_t)where[0];
  ld.len = row_tokens(c, ld.row, nullptr);
  ld.n = (ld.len + S::kTile - 1) / S::kTile;
  ld.hh = (int32_t)(where[1] / ld.n);
  ld.at = (int32_t)(where[1] - (int64_t)ld.hh * ld.n);
  int32_t next_len = row_tokens(c, ld.row + 1, nullptr);
  const int page = c.page, lg = a.page_log2;
  constexpr int kIds = S::kTile / 16;   // pages of a tile at most
  int32_t ids[kIds];
  auto read_ids = [&]() {
    const int32_t* t = c.table + (int64_t)ld.row * c.max_pages;
    const int first = (ld.at * S::kTile) >> lg;
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      ids[i] = -1;
      if (i == 0 || (i << lg) < S::kTile)
        if (((int64_t)(first + i) << lg) < ld.len) {
          ids[i] = t[first + i];
          if (ids[i] < 0 || ids[i] >= c.pages) {
            flag_status(a.status, GDN_ERR_BAD_CACHE);
            ids[i] = -1;
          }
        }
    }
  };
  read_ids();
  int64_t left = hi - lo;   // tiles to load
  bool fresh = true;        // the next tile is the first of its part
  const int64_t layer_pages = (int64_t)a.layer * c.pages;

  auto issue = [&](int stage) {
    if (left > 0) {
      const uint32_t base = smem_u32(smem) + stage * S::kStage;
      const int h = ld.hh / a.parts, part = ld.hh - h * a.parts;
      const int64_t pos0 = (int64_t)ld.at * S::kTile;
      constexpr int kRowsStep = kThreads / S::kChunks;   // tokens a round of loads covers
      const int ch = tid % S::kChunks, tr = tid / S::kChunks;
#pragma unroll
      for (int i = 0; i < S::kTile / kRowsStep; ++i) {
        const int tok = i * kRowsStep + tr;
        // (up to 16 tokens from a multiple of their number lie on one page)
        const int at = kRowsStep <= 16 ? i * kRowsStep : tok;
        int32_t id = ids[0];
#pragma unroll
        for (int j = 1; j < kIds; ++j)
          if ((at >> lg) == j) id = ids[j];
        const bool on = pos0 + tok < ld.len && id >= 0;
        const int64_t e =
            ((layer_pages + (on ? id : 0)) * c.kv_heads + h) * page + ((pos0 + tok) & (page - 1));
        const uint32_t to = image<S::kRow>(tok, ch);
        const int64_t off = e * S::kRow + ch * 16;
        cp_async16(base + to, (const uint8_t*)c.k + off, on ? 16 : 0);
        cp_async16(base + S::kPool + to, (const uint8_t*)c.v + off, on ? 16 : 0);
      }
      if constexpr (kFp8) {
        const int tok = tid;   // kTile == kThreads
        int32_t id = ids[0];
#pragma unroll
        for (int j = 1; j < kIds; ++j)
          if ((tok >> lg) == j) id = ids[j];
        const bool on = pos0 + tok < ld.len && id >= 0;
        const int64_t e =
            ((layer_pages + (on ? id : 0)) * c.kv_heads + h) * page + ((pos0 + tok) & (page - 1));
        cp_async4(base + 2 * S::kPool + tok * 4, c.k_scale + e, on ? 4 : 0);
        cp_async4(base + 2 * S::kPool + S::kScales + tok * 4, c.v_scale + e, on ? 4 : 0);
      }
      if (fresh) {
        // the queries of the part's heads, missing ones as zeros
        constexpr int kQChunks = D / 8;
        for (int i = tid; i < kHeads * kQChunks; i += kThreads) {
          const int hr = i / kQChunks, cc = i % kQChunks, head = part * kHeads + hr;
          const bool on = head < a.group;
          const __nv_bfloat16* src =
              a.q + ((int64_t)ld.row * a.q_heads + (int64_t)h * a.group + (on ? head : 0)) * D + cc * 8;
          cp_async16(base + S::kQ + image<D * 2>(hr, cc), src, on ? 16 : 0);
        }
      }
      if (tid == 0) meta[stage] = ld;
      // on to the next tile
      fresh = false;
      --left;
      if (++ld.at == ld.n) {
        ld.at = 0;
        fresh = true;
        if (++ld.hh == HH) {
          ld.hh = 0;
          do {
            ++ld.row;
            ld.len = next_len;
            ld.n = (ld.len + S::kTile - 1) / S::kTile;
            next_len = row_tokens(c, (int64_t)ld.row + 1, nullptr);
          } while (ld.n == 0 && ld.row < c.rows);
        }
      }
      if (left > 0) read_ids();
    }
    cp_async_commit();
  };

  const int g = lane >> 2, t4 = lane & 3;
  constexpr int kSteps = D / 16;
  constexpr int kTok = S::kTile / kWarps;   // a warp's tokens of a tile
  uint32_t qa[kSteps][4];
  float o[D / 8][4];
  float m[2], l[2];
  bool start = true;
  int64_t first_of_part = lo;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  for (int64_t i = lo; i < hi; ++i) {
    const int stage = (int)((i - lo) % kStages);
    cp_async_wait<kStages - 2>();
    __syncthreads();
    issue((int)((i - lo + kStages - 1) % kStages));
    const Tile tile = meta[stage];
    const uint32_t base = smem_u32(smem) + stage * S::kStage;
    if (start) {
      first_of_part = i;
      start = false;
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[j][x] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if constexpr (!kFp8) {
          // rows 0-7 and 8-15 of the first eight columns, then of the second
          ldmatrix4(qa[s], base + S::kQ +
                               image<D * 2>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * s + (lane >> 4)));
        } else {
          // the order in which four consecutive codes of a key arrive: columns
          // 4t, 4t + 1 in the place of 2t, 2t + 1 and the next two in that of
          // 2t + 8, 2t + 9 (a sum over columns may take them in any order)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t p = base + S::kQ + image<D * 2>(g + 8 * x, 2 * s + (t4 >> 1)) + (t4 & 1) * 8;
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(qa[s][x]), "=r"(qa[s][2 + x])
                         : "r"(p));
          }
        }
      }
    }
    const int valid = tile.len - tile.at * S::kTile;   // tokens of the tile (or more)
#pragma unroll
    for (int sub = 0; sub < kTok / 16; ++sub) {
      const int tok0 = warp * kTok + sub * 16;
      if (tok0 >= valid) break;
      // scores of 16 heads and 16 tokens
      float s[2][4] = {};
      if constexpr (!kFp8) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t b[4];
          ldmatrix4(b, base + image<S::kRow>(tok0 + (lane >> 4) * 8 + (lane & 7),
                                             2 * k + ((lane >> 3) & 1)));
          mma16816(s[0], qa[k], b[0], b[1]);
          mma16816(s[1], qa[k], b[2], b[3]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint32_t b[4];
          ldmatrix4(b, base + image<S::kRow>(tok0 + (lane >> 4) * 8 + (lane & 7),
                                             k + ((lane >> 3) & 1)));
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mma16816(s[x >> 1], qa[k + (x & 1)], e4m3_to_bf16<0x1404>(b[x]),
                     e4m3_to_bf16<0x3424>(b[x]));
        }
      }
      float vs[2][2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int col = tok0 + n * 8 + 2 * t4;
        float f0 = a.scale_log2, f1 = a.scale_log2;
        if constexpr (kFp8) {
          const float* sc = reinterpret_cast<const float*>(smem + stage * S::kStage + 2 * S::kPool);
          f0 *= sc[col];
          f1 *= sc[col + 1];
          vs[n][0] = sc[S::kTile + col];
          vs[n][1] = sc[S::kTile + col + 1];
        }
        const bool v0 = col < valid, v1 = col + 1 < valid;
        s[n][0] = v0 ? s[n][0] * f0 : -INFINITY;
        s[n][1] = v1 ? s[n][1] * f1 : -INFINITY;
        s[n][2] = v0 ? s[n][2] * f0 : -INFINITY;
        s[n][3] = v1 ? s[n][3] * f1 : -INFINITY;
      }
      // running maximum and sum of rows g and g + 8
      float sub_m[2];
      bool grew = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        sub_m[x] = fmaxf(m[x], mx);
        grew |= sub_m[x] > m[x];
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float f = sub_m[x] > m[x] ? ex2_sfu(m[x] - sub_m[x]) : 1.f;
          l[x] *= f;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][2 * x] *= f;
            o[j][2 * x + 1] *= f;
          }
          m[x] = sub_m[x];
        }
      }
      uint32_t p[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float z = m[x] == -INFINITY ? 0.f : m[x];
          float p0 = ex2_sfu(s[n][2 * x] - z), p1 = ex2_sfu(s[n][2 * x + 1] - z);
          l[x] += p0 + p1;
          if constexpr (kFp8) {
            p0 *= vs[n][0];
            p1 *= vs[n][1];
          }
          p[2 * n + x] = pack_bf16(p0, p1);
        }
      // out of 16 heads, the warp's tokens added
      const uint32_t vb = base + S::kPool;
      if constexpr (!kFp8) {
#pragma unroll
        for (int j = 0; j < D / 8; j += 2) {
          uint32_t b[4];
          ldmatrix4t(b, vb + image<S::kRow>(tok0 + ((lane >> 3) & 1) * 8 + (lane & 7), j + (lane >> 4)));
          mma16816(o[j], p, b[0], b[1]);
          mma16816(o[j + 1], p, b[2], b[3]);
        }
      } else {
        // a transposed pair of codes is two columns: even ones to o[2j], odd to
        // o[2j + 1], so that a lane ends with four consecutive columns of 16
#pragma unroll
        for (int j = 0; j < D / 16; j += 2) {
          uint32_t b[4];
          ldmatrix4t(b, vb + image<S::kRow>(tok0 + ((lane >> 3) & 1) * 8 + (lane & 7), j + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mma16816(o[2 * (j + x)], p, e4m3_to_bf16<0x2404>(b[2 * x]), e4m3_to_bf16<0x2404>(b[2 * x + 1]));
            mma16816(o[2 * (j + x) + 1], p, e4m3_to_bf16<0x3414>(b[2 * x]),
                     e4m3_to_bf16<0x3414>(b[2 * x + 1]));
          }
        }
      }
    }
    const bool item_ends = tile.at == tile.n - 1;
    if (!item_ends && i + 1 < hi) continue;

    // the part ends: join the warps' sums, in the consumed stage
    start = true;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if (t4 == 0) {
        ml[warp][g + 8 * x][0] = m[x];
        ml[warp][g + 8 * x][1] = l[x];
      }
    }
    __syncthreads();
    float* js = reinterpret_cast<float*>(smem + stage * S::kStage);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][g + 8 * x][0]);
      const float f = m[x] == -INFINITY ? 0.f : ex2_sfu(m[x] - top);
      float* r = js + (warp * kHeads + g + 8 * x) * S::kPitch;
      if constexpr (!kFp8) {
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          *reinterpret_cast<float2*>(r + j * 8 + 2 * t4) =
              make_float2(o[j][2 * x] * f, o[j][2 * x + 1] * f);
      } else {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          *reinterpret_cast<float4*>(r + j * 16 + 4 * t4) =
              make_float4(o[2 * j][2 * x] * f, o[2 * j + 1][2 * x] * f, o[2 * j][2 * x + 1] * f,
                          o[2 * j + 1][2 * x + 1] * f);
      }
    }
    __syncthreads();
    const int h = tile.hh / a.parts, part = tile.hh - h * a.parts;
    const int64_t item_begin = i - tile.at;
    const bool from_begin = first_of_part == item_begin, whole = from_begin && item_ends;
    const int64_t item = (int64_t)tile.row * HH + tile.hh;
    const int64_t slot = 2 * (int64_t)blockIdx.x + from_begin;
    if (tid == 0 && from_begin) {
      a.w.begin[item] = item_begin;
      a.w.end[item] = whole ? 0 : item_begin + tile.n;
    }
    const int heads = a.group - part * kHeads < kHeads ? a.group - part * kHeads : kHeads;
#pragma unroll
    for (int v = 0; v < kHeads * D / 4 / kThreads; ++v) {
      const int e = v * kThreads + tid, row = e / (D / 4), col = e % (D / 4) * 4;
      if (row >= heads) break;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float top = -INFINITY, all = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][row][0]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(js + (w * kHeads + row) * S::kPitch + col);
        sum.x += y.x; sum.y += y.y; sum.z += y.z; sum.w += y.w;
        const float mw = ml[w][row][0];
        all += mw == -INFINITY ? 0.f : ml[w][row][1] * ex2_sfu(mw - top);
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
  }
}

// The cut (row, head)s: a CTA takes one query head at a time, its warps every
// eighth part, then the warps' sums in order.  Rows without tokens get zeros.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(Args a, int grid) {
  constexpr int kN = kJoinThreads / 32, kV = D / 32;
  __shared__ float sm[kN][D + 2];
  const gdn_kv_cache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_wait();
  int64_t total;
  asm volatile("ld.global.s64 %0, [%1];" : "=l"(total) : "l"(a.total));
  const int64_t ctas = total < grid ? total : grid;
  const int64_t jobs = (int64_t)c.rows * a.q_heads;
  for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int64_t row = job / a.q_heads;
    const int head = (int)(job - row * a.q_heads);
    const int h = head / a.group, in = head - h * a.group, part = in / kHeads, r = in % kHeads;
    __nv_bfloat16* out = a.out + job * D;
    if (row_tokens(c, row, nullptr) == 0) {
      for (int i = threadIdx.x; i < D; i += kJoinThreads) out[i] = __float2bfloat16_rn(0.f);
      continue;
    }
    const int64_t item = row * a.items_per_row + h * a.parts + part;
    int64_t b, e;
    asm volatile("ld.global.s64 %0, [%1];" : "=l"(b) : "l"(a.w.begin + item));
    asm volatile("ld.global.s64 %0, [%1];" : "=l"(e) : "l"(a.w.end + item));
    if (e == 0) continue;
    // the CTA that has tile t: part c of n begins at floor(c total / n)
    auto owner = [&](int64_t t) {
      return (int64_t)(((unsigned __int128)(t + 1) * ctas - 1) / total);
    };
    const int64_t first = owner(b), last = owner(e - 1);
    float m = -INFINITY, l = 0.f, o[kV] = {};
    for (int64_t p = first + warp; p <= last; p += kN) {
      const int64_t slot = 2 * p + (p == first);
      const float mp = ld_waited(a.w.ml + (slot * kHeads + r) * 2);
      const float lp = ld_waited(a.w.ml + (slot * kHeads + r) * 2 + 1);
      const float* src = a.w.o + (slot * kHeads + r) * D + lane * kV;
      float x[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] = ld_waited(src + i);
      const float top = fmaxf(m, mp);
      const float fa = m == -INFINITY ? 0.f : ex2_sfu(m - top);
      const float fb = mp == -INFINITY ? (isnan(lp) ? 1.f : 0.f) : ex2_sfu(mp - top);
      l = l * fa + lp * fb;
#pragma unroll
      for (int i = 0; i < kV; ++i) o[i] = o[i] * fa + x[i] * fb;
      m = top;
    }
    if (lane == 0) {
      sm[warp][D] = m;
      sm[warp][D + 1] = l;
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) sm[warp][lane * kV + i] = o[i];
    __syncthreads();
    if (threadIdx.x < D) {
      float top = -INFINITY, all = 0.f, x = 0.f;
#pragma unroll
      for (int w = 0; w < kN; ++w) top = fmaxf(top, sm[w][D]);
#pragma unroll
      for (int w = 0; w < kN; ++w) {
        const float mw = sm[w][D], lw = sm[w][D + 1];
        const float f = mw == -INFINITY ? (isnan(lw) ? 1.f : 0.f) : ex2_sfu(mw - top);
        all += lw * f;
        x += sm[w][threadIdx.x] * f;
      }
      out[threadIdx.x] = __float2bfloat16_rn(x / all);
    }
    __syncthreads();
  }
}

struct Layout {
  size_t begin, end, ml, o, bytes;
};
int ctas_of(int32_t d) { return kSms * (d == 128 ? 2 : 4); }
Layout layout_of(int32_t rows, int32_t q_heads, int32_t kv_heads, int32_t d) {
  const int32_t group = q_heads / kv_heads, parts = (group + kHeads - 1) / kHeads;
  const size_t items = (size_t)rows * kv_heads * parts, slots = 2 * (size_t)ctas_of(d);
  Layout l;
  l.begin = 256;
  l.end = l.begin + align_up(items * 8, 256);
  l.ml = l.end + align_up(items * 8, 256);
  l.o = l.ml + slots * kHeads * 2 * 4;
  l.bytes = l.o + slots * kHeads * d * 4;
  return l;
}
int heads_check(int32_t rows, int32_t q_heads, int32_t kv_heads, int32_t d) {
  if (rows < 1 || q_heads < 1 || kv_heads < 1) return GDN_ERR_INVALID_ARG;
  if (q_heads % kv_heads || q_heads / kv_heads > 128 || !kv::dim_ok(d)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int decode(const void* q, const gdn_kv_cache* cache, int32_t layer, int32_t q_heads, float scale,
           void* out, bool use_ws, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (const int rc = kv::check_cache(cache)) return rc;
  const gdn_kv_cache c = *cache;
  if (const int rc = heads_check(c.rows, q_heads, c.kv_heads, c.d)) return rc;
  if (!q || !out || layer < 0 || layer >= c.layers || !(scale > 0.f) || scale > 3e38f)
    return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16)) return GDN_ERR_ALIGNMENT;
  const Layout lay = layout_of(c.rows, q_heads, c.kv_heads, c.d);
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
  Args a = {};
  a.status = status_ptr();
  if (!a.status) return GDN_ERR_CUDA;
  void* scratch = ws;
  if (!use_ws && scratch_alloc(&scratch, lay.bytes, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
  }
  a.q = (const __nv_bfloat16*)q;
  a.out = (__nv_bfloat16*)out;
  a.c = c;
  a.layer = layer;
  a.q_heads = q_heads;
  a.group = q_heads / c.kv_heads;
  a.parts = (a.group + kHeads - 1) / kHeads;
  a.items_per_row = c.kv_heads * a.parts;
  while ((1 << a.page_log2) < c.page) ++a.page_log2;
  a.scale_log2 = scale * kLog2e;
  char* p = (char*)scratch;
  a.total = (int64_t*)p;
  a.w.begin = (int64_t*)(p + lay.begin);
  a.w.end = (int64_t*)(p + lay.end);
  a.w.ml = (float*)(p + lay.ml);
  a.w.o = (float*)(p + lay.o);
  const bool fp8 = c.dtype == GDN_E4M3;
  const int ctas = ctas_of(c.d);
  cudaError_t e;
  auto run = [&](auto shape, auto kern) {
    using S = decltype(shape);
    e = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e == cudaSuccess)
      e = launch(false, kern, dim3(ctas), kThreads, S::kSmem, 0, st, a);
  };
  if (c.d == 128)
    fp8 ? run(Shape<128, true>{}, decode_kernel<128, true>)
        : run(Shape<128, false>{}, decode_kernel<128, false>);
  else
    fp8 ? run(Shape<64, true>{}, decode_kernel<64, true>)
        : run(Shape<64, false>{}, decode_kernel<64, false>);
  if (e == cudaSuccess) {
    const int64_t jobs = (int64_t)c.rows * q_heads, most = 8 * kSms;
    e = launch(true, c.d == 128 ? join_kernel<128> : join_kernel<64>,
               dim3((unsigned)(jobs < most ? jobs : most)), kJoinThreads, 0, 0, st, a, ctas);
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
  return layout_of(rows, q_heads, kv_heads, d).bytes;
}

int gdn_attention_decode_step_ws(const void* q, const gdn_kv_cache* cache, int32_t layer,
                                 int32_t q_heads, float scale, void* out, void* workspace,
                                 size_t workspace_bytes, gdn_stream_t stream) {
  return decode(q, cache, layer, q_heads, scale, out, true, workspace, workspace_bytes,
                (cudaStream_t)stream);
}

}  // extern "C"
