// The residual addition with its root-mean-square norm, its gradient, and the
// 8-bit quantisation of rows and weight blocks (contracts: include/gdn.h).
//
//   s = round(x + r);  y = s rs w,  rs = 1 / sqrt(mean_j s_j^2 + eps)
//   8 bits: per row and 128 columns m = max(|y|, 2^-100), scale = m / 448,
//           q = e4m3(y (448 / m))
//   gradient: n = s rs, g = dy w:  dx = (g - n mean_j(g_j n_j)) rs + ds,
//             dw = sum_t dy n
//
// All of it is bound by HBM: nothing is read twice and nothing but the results
// is written.  A row is held in registers by 1, 2, 4 or 8 warps, 8 elements
// (16 bytes of bf16) a lane and vector, so that every load of a row is in
// flight before its first use and the 16 lanes of a half warp hold one
// 128-column block: a block's largest magnitude is four shuffles.
//
// Measured (bf16): 32768 x 2048 with residual and 8-bit output 80 us, 5.9 TB/s
// of a copy's 6.7 (86 us with weights that are bf16 numbers, 105 with weights of 1:
// the more values lie on the middle between two codes, the more are settled); the
// gradient of 8191 x 4096 51.8 us, 5.2 TB/s; one token 1.8 us on the GPU.
#include "fp8_codes.cuh"
#include "gdn_internal.cuh"
#include "hostcheck.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

using namespace hostcheck;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDim = 8 * 8 * 256;   // 8 warps x 8 vectors x 256 columns
constexpr int kFewRows = 304;            // two CTAs an SM of one row each
constexpr int kClusterCtas = 8;

// ------------------------------------------------------- 8 elements of a row
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = a;
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void round(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void round(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

__device__ __forceinline__ void load_w(const float* w, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w));
  const float4 b = __ldg(reinterpret_cast<const float4*>(w) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// x times one factor, or element by element, two at a time (rounded as scalar
// products are).
__device__ __forceinline__ void mul8(const float (&x)[8], float c, float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    f2_split(f2_mul(f2(x[i], x[i + 1]), f2(c, c)), y[i], y[i + 1]);
}
__device__ __forceinline__ void mul8(const float (&x)[8], const float (&c)[8], float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    f2_split(f2_mul(f2(x[i], x[i + 1]), f2(c[i], c[i + 1])), y[i], y[i + 1]);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// Is v (of an e4m3 value's size) within 16 units in its last place of the middle
// between two e4m3 values?  fp32 gets y (448 / m) to about 5, so elsewhere its
// rounding is that of the real number.  tie_gap, of v's low 20 bits, is at most
// kNearTie there.  Below the normal range, 2^-6, the codes are 2^-9 apart, as they
// are from 2^-6 to 2^-5: |v| + 2^-6 is looked at in its place, whose units there
// are 2^-29 and v's errors still less than 5 of them.
constexpr float kLeastNormal = 0x1p-6f;
constexpr uint32_t kNearTie = 0x20u << 12;
__device__ __forceinline__ uint32_t tie_gap(float v) {
  return __float_as_uint(v) * 4096u - (0x7fff0u << 12);
}
__device__ __forceinline__ float on_normal_grid(float v) {
  const float a = fabsf(v);
  float below;   // 1 or 0: one instruction, and one more with the product
  asm("set.lt.f32.f32 %0, %1, %2;" : "=f"(below) : "f"(a), "f"(kLeastNormal));
  return __fmaf_rn(below, kLeastNormal, a);
}
__device__ __forceinline__ bool near_tie(float v) { return tie_gap(on_normal_grid(v)) <= kNearTie; }
// kSmallest: the smallest value tells first whether any is below the normal range
// (32768 x 2048: the fp32 quantisation 54.6 us, 59.1 without; the norm 81.9, 80.1
// without).
template <bool kSmallest>
__device__ __forceinline__ bool any_near_tie(const float (&v)[8]) {
  uint32_t g = 0xffffffffu;
  if constexpr (kSmallest) {
    float least = fabsf(v[0]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g = min(g, tie_gap(v[i]));
      least = fminf(least, fabsf(v[i]));
    }
    if (least >= kLeastNormal) return g <= kNearTie;
    g = 0xffffffffu;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) g = min(g, tie_gap(on_normal_grid(v[i])));
  return g <= kNearTie;
}
// v, which is near the tie t, moved to where 448 p / m lies: on t or beside it.
// p = ph + pl and m = mh + ml, magnitudes; t has 5 significant bits.  The
// products (of 448 / 512 and t / 512, which overflow for no p and m) have
// rounding errors that are exact in fp32 (fma), and the leading parts nearly
// cancel, so the sign of the difference is right.
__device__ __forceinline__ float settle_tie(float v, float ph, float pl, float mh, float ml) {
  constexpr float k448 = kE4m3Max * 0x1p-9f;
  const uint32_t tie_z = (__float_as_uint(on_normal_grid(v)) & ~0xfffffu) | 0x80000u;
  const float z = __uint_as_float(tie_z);
  const float t = fabsf(v) < kLeastNormal ? z - kLeastNormal : z, ts = t * 0x1p-9f;
  const float a = __fmul_rn(k448, ph), b = __fmul_rn(ts, mh);
  const float ae = __fmaf_rn(k448, ph, -a), be = __fmaf_rn(ts, mh, -b);
  const float low = __fmaf_rn(k448, pl, -__fmul_rn(ts, ml));
  const float d = __fadd_rn(__fadd_rn(a, -b), __fadd_rn(__fadd_rn(ae, -be), low));
  const uint32_t tie = __float_as_uint(t);   // at least 2^-10
  return copysignf(__uint_as_float(d > 0.f ? tie + 1 : d < 0.f ? tie - 1 : tie), v);
}

// Sum over the kWPR warps that share a row; every thread of the CTA calls it.
template <int kWPR, int kN>
__device__ __forceinline__ void row_sum(float (&x)[kN], float (*part)[kN]) {
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < kN; ++i) x[i] = warp_sum(x[i]);
  if (kWPR == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < kN; ++i) part[warp][i] = x[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < kWPR; ++j) t += part[warp / kWPR * kWPR + j][i];
    x[i] = t;
  }
}

// CTAs an SM that the registers of kVPL vectors a lane leave room for.
constexpr int forward_ctas(int v) { return v <= 2 ? 4 : v <= 3 ? 3 : v <= 4 ? 2 : 1; }
constexpr int backward_ctas(int v, size_t element) {
  return element == 2 ? (v <= 2 ? 4 : v <= 3 ? 3 : v <= 4 ? 2 : 1) : v <= 2 ? 2 : 1;
}

struct NormArgs {
  const void* x; const void* r; const float* w; float eps;
  void* s; void* y; uint8_t* q; float* scale;
  int64_t rows; int32_t dim, blocks;   // blocks: ceil(dim / 128)
};

// x, r, s and y may be the same memory (each thread reads its elements of a
// row before it writes them), hence no __restrict__.
template <typename T, int kVPL, int kWPR, bool kFp8>
__global__ void __launch_bounds__(kThreads, forward_ctas(kVPL)) residual_norm_kernel(NormArgs a) {
  grid_release_next();   // a product that follows may start its prologue
  __shared__ float part[kWarps][1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * (kWarps / kWPR) + warp / kWPR;
  const bool live = row < a.rows;
  const size_t base = (size_t)(live ? row : 0) * a.dim;
  auto col = [&](int j) { return ((j * kWPR + warp % kWPR) * 32 + lane) * 8; };
  Raw<T> s[kVPL], r[kVPL];
#pragma unroll
  for (int j = 0; j < kVPL; ++j) {
    const int c = col(j);
    s[j].zero();
    if (live && c < a.dim) s[j].load((const T*)a.x + base + c);
  }
  constexpr bool kEarlyW = kVPL <= 2;   // w in flight with the row: one latency, not two
  float w[kEarlyW ? kVPL : 1][8];
  if (kEarlyW)
#pragma unroll
    for (int j = 0; j < kVPL; ++j)
      if (col(j) < a.dim) load_w(a.w + col(j), w[j]);
  if (a.r) {
#pragma unroll
    for (int j = 0; j < kVPL; ++j) {
      const int c = col(j);
      r[j].zero();
      if (live && c < a.dim) r[j].load((const T*)a.r + base + c);
    }
#pragma unroll
    for (int j = 0; j < kVPL; ++j) {
      float f[8], g[8];
      s[j].widen(f);
      r[j].widen(g);
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        f2_split(f2_add(f2(f[i], f[i + 1]), f2(g[i], g[i + 1])), f[i], f[i + 1]);
      s[j].round(f);
    }
  }
  float ss[1] = {0.f};
#pragma unroll
  for (int j = 0; j < kVPL; ++j) {
    float f[8];
    s[j].widen(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[0] = fmaf(f[i], f[i], ss[0]);
  }
  row_sum<kWPR>(ss, part);
  const float rs = rsqrtf(ss[0] / (float)a.dim + a.eps);
#pragma unroll
  for (int j = 0; j < kVPL; ++j) {
    const int c = col(j);
    const bool in = live && c < a.dim;
    if (a.r && in && a.s) s[j].store((T*)a.s + base + c);
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float(&wj)[8] = w[kEarlyW ? j : 0];
    if (in) {
      s[j].widen(f);
      if (!kEarlyW) load_w(a.w + c, wj);
      mul8(f, rs, f);
      mul8(f, wj, f);
    }
    if (!kFp8) {
      if (in) {
        Raw<T> o;
        o.round(f);
        o.store((T*)a.y + base + c);
      }
    } else {
      float m = amax8(f);
#pragma unroll
      for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = max_nan(m, kTiny);
      const float inv = codes_per(m);
      float v[8];
      mul8(f, inv, v);
      if (__any_sync(0xffffffffu, any_near_tie<false>(v) && m > kTiny)) {
        // (one in 120 of these) the root cancels in y / m: the codes are those
        // of 448 s_j w_j / max |s w|, a product being hi + lo exactly
        float fs[8], mh = 0.f, ml = 0.f;
        s[j].widen(fs);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!in) fs[i] = 0.f;
          const float hi = fabsf(__fmul_rn(fs[i], wj[i]));
          const float lo = __fmaf_rn(fabsf(fs[i]), fabsf(wj[i]), -hi);
          if (hi > mh || (hi == mh && lo > ml)) mh = hi, ml = lo;
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) {
          const float hi = __shfl_xor_sync(0xffffffffu, mh, o);
          const float lo = __shfl_xor_sync(0xffffffffu, ml, o);
          if (hi > mh || (hi == mh && lo > ml)) mh = hi, ml = lo;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (near_tie(v[i]) && m > kTiny) {
            const float hi = fabsf(__fmul_rn(fs[i], wj[i]));
            v[i] = settle_tie(v[i], hi, __fmaf_rn(fabsf(fs[i]), fabsf(wj[i]), -hi), mh, ml);
          }
      }
      if (in) {
        *reinterpret_cast<uint2*>(a.q + base + c) = codes8(v);
        if ((lane & 15) == 0)
          a.scale[(size_t)row * a.blocks + c / 128] = scale_of(m);
      }
    }
  }
}

struct NormBwdArgs {
  const void* dy; const void* s; const float* w; const void* ds; float eps;
  void* dx; float* part;   // part: [gridDim.x][dim], or dw
  int64_t rows; int32_t dim;
};

// dx, and each CTA's part of dw over the rows it visits: the rows are dealt
// to a fixed grid, so the sums have a fixed order.  kCluster: the grid is one
// cluster, whose CTAs add their parts through each other's shared memory, in
// order, into dw (few rows: one launch and no scratch).  Rows in flight are what
// it lives from: two vectors a lane leave registers for four CTAs an SM
// (8191 rows of 4096 bf16: 51.9 us, 57.4 with four vectors and two CTAs).
template <typename T, int kVPL, int kWPR, bool kCluster>
__global__ void __launch_bounds__(kThreads, backward_ctas(kVPL, sizeof(T)))
    norm_backward_kernel(NormBwdArgs a) {
  grid_release_next();
  constexpr int kGroups = kWarps / kWPR;
  __shared__ float part[2][kWarps][2];
  __shared__ float acc_s[kGroups > 1 ? kVPL * kWPR * 256 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto col = [&](int j) { return ((j * kWPR + warp % kWPR) * 32 + lane) * 8; };
  float dw[kVPL][8];
#pragma unroll
  for (int j = 0; j < kVPL; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  int flip = 0;   // alternating buffers: one barrier a row
  for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < a.rows;
       r0 += (int64_t)gridDim.x * kGroups, flip ^= 1) {
    const int64_t row = r0 + warp / kWPR;
    const bool live = row < a.rows;
    const size_t base = (size_t)(live ? row : 0) * a.dim;
    Raw<T> s[kVPL], dy[kVPL], ds[kVPL];
#pragma unroll
    for (int j = 0; j < kVPL; ++j) {
      const int c = col(j);
      s[j].zero();
      dy[j].zero();
      ds[j].zero();
      if (live && c < a.dim) {
        s[j].load((const T*)a.s + base + c);
        dy[j].load((const T*)a.dy + base + c);
        if (a.ds) ds[j].load((const T*)a.ds + base + c);
      }
    }
    float t[2] = {0.f, 0.f};   // sum s^2, sum g s
#pragma unroll
    for (int j = 0; j < kVPL; ++j) {
      const int c = col(j);
      if (c < a.dim) {
        float f[8], d[8], w[8];
        s[j].widen(f);
        dy[j].widen(d);
        load_w(a.w + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          t[0] = fmaf(f[i], f[i], t[0]);
          t[1] = fmaf(d[i] * w[i], f[i], t[1]);
        }
      }
    }
    row_sum<kWPR>(t, part[flip]);
    const float rs = rsqrtf(t[0] / (float)a.dim + a.eps);
    const float along = t[1] * rs / (float)a.dim;   // mean(g n)
#pragma unroll
    for (int j = 0; j < kVPL; ++j) {
      const int c = col(j);
      if (live && c < a.dim) {
        float f[8], d[8], w[8], e[8];
        s[j].widen(f);
        dy[j].widen(d);
        ds[j].widen(e);
        load_w(a.w + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = f[i] * rs;
          dw[j][i] = fmaf(d[i], n, dw[j][i]);
          e[i] = fmaf(fmaf(-n, along, d[i] * w[i]), rs, e[i]);
        }
        Raw<T> o;
        o.round(e);
        o.store((T*)a.dx + base + c);
      }
    }
  }
  // the row groups' sums, one group after another
  if (kGroups > 1) {
    for (int g = 0; g < kGroups; ++g) {
      if (warp / kWPR == g) {
#pragma unroll
        for (int j = 0; j < kVPL; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float* p = acc_s + col(j) + i;
            if (g) dw[j][i] += *p;
            *p = dw[j][i];
          }
      }
      __syncthreads();
    }
  }
  extern __shared__ __align__(16) float mine[];   // kCluster: [dim]
  if (warp / kWPR == kGroups - 1) {
#pragma unroll
    for (int j = 0; j < kVPL; ++j) {
      const int c = col(j);
      if (c < a.dim) {
        Raw<float> o;
        o.round(dw[j]);
        o.store(kCluster ? mine + c : a.part + (size_t)blockIdx.x * a.dim + c);
      }
    }
  }
  if constexpr (kCluster) {
    sm100::cluster_sync_all();
    uint32_t base[kCluster ? kClusterCtas : 1];
#pragma unroll
    for (int r = 0; r < kClusterCtas; ++r) base[r] = sm100::mapa_smem(mine, r);
    for (int v = blockIdx.x * kThreads + threadIdx.x; v < a.dim / 4; v += kClusterCtas * kThreads) {
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < kClusterCtas; ++r) {
        const float4 x = sm100::ld_shared_cluster4(base[r] + 16 * v);
        t.x += x.x; t.y += x.y; t.z += x.z; t.w += x.w;
      }
      reinterpret_cast<float4*>(a.part)[v] = t;
    }
    sm100::cluster_sync_all();   // read before any CTA leaves
  }
}

// dw[c] = sum_b part[b][c]: 32 strided runs, each in order, then the runs in
// order.  A programmatic dependent of the kernel above (both for 8191 x 4096:
// 51.7 us against 54.0 launched plainly).
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int n, int dim,
                                                       float* dw) {
  grid_release_next();
  grid_wait();
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (c < dim)
#pragma unroll 8
    for (int b = run; b < n; b += 32) t += ld_waited(part + (size_t)b * dim + c);
  sm[run][lane] = t;
  __syncthreads();
  if (run == 0 && c < dim) {
#pragma unroll
    for (int i = 1; i < 32; ++i) t += sm[i][lane];
    dw[c] = t;
  }
}

// ------------------------------------------------------------ quantisation
struct QuantArgs {
  const void* x; uint8_t* q; float* scale;
  int64_t rows; int32_t cols, blocks;
};

// The codes of 448 x / m in a block whose largest magnitude is m.
template <typename T>
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float m) {
  if constexpr (sizeof(T) == 2) {
    return quantise8_bf16(x, m);
  } else {
    float v[8];
    const float inv = codes_per(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(x[i], inv);
    if (any_near_tie<true>(v)) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (near_tie(v[i])) v[i] = settle_tie(v[i], fabsf(x[i]), 0.f, m, 0.f);
    }
    return codes8(v);
  }
}

// 1 x 128 blocks: a half warp each, kTwo at a time so that both loads are in
// flight.
constexpr int kTwo = 2;
template <typename T>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(QuantArgs a) {
  grid_release_next();
  const int64_t units = a.rows * a.blocks;
  const int64_t u0 = ((int64_t)blockIdx.x * kTwo * kThreads + threadIdx.x) >> 4;
  const int l = threadIdx.x & 15;
  Raw<T> x[kTwo];
  int64_t at[kTwo];   // the elements' place, -1 past the row's end
#pragma unroll
  for (int i = 0; i < kTwo; ++i) {
    const int64_t u = u0 + i * (kThreads / 16);
    const int64_t row = u >> 32 ? u / a.blocks : (uint32_t)u / (uint32_t)a.blocks;
    const int c = (int)(u - row * a.blocks) * 128 + l * 8;
    at[i] = u < units && c < a.cols ? row * a.cols + c : -1;
    x[i].zero();
    if (at[i] >= 0) x[i].load((const T*)a.x + at[i]);
  }
#pragma unroll
  for (int i = 0; i < kTwo; ++i) {
    float f[8];
    x[i].widen(f);
    float m = amax8(f);
#pragma unroll
    for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max_nan(m, kTiny);
    if (at[i] >= 0) {
      *reinterpret_cast<uint2*>(a.q + at[i]) = quantise8<T>(f, m);
      if (l == 0) a.scale[u0 + i * (kThreads / 16)] = scale_of(m);
    }
  }
}

// 128 x 128 blocks: a CTA each, thread t holding vector t % 16 of rows
// t / 16 + 16 i.
template <typename T>
__global__ void __launch_bounds__(kThreads) quant_tiles_kernel(QuantArgs a) {
  grid_release_next();
  __shared__ float wm[kWarps];
  const int64_t r0 = (int64_t)blockIdx.y * 128 + (threadIdx.x >> 4);
  const int c = blockIdx.x * 128 + (threadIdx.x & 15) * 8;
  Raw<T> x[8];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i].zero();
    if (r0 + 16 * i < a.rows && c < a.cols)
      x[i].load((const T*)a.x + (size_t)(r0 + 16 * i) * a.cols + c);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    x[i].widen(f);
    m = max_nan(m, amax8(f));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) wm[threadIdx.x >> 5] = m;
  __syncthreads();
  m = kTiny;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) m = max_nan(m, wm[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + 16 * i < a.rows && c < a.cols) {
      float f[8];
      x[i].widen(f);
      *reinterpret_cast<uint2*>(a.q + (size_t)(r0 + 16 * i) * a.cols + c) = quantise8<T>(f, m);
    }
  }
  if (threadIdx.x == 0)
    a.scale[(size_t)blockIdx.y * a.blocks + blockIdx.x] = scale_of(m);
}

// ---------------------------------------------------------------- launchers
// A register layout for rows of `dim` columns: V vectors a lane, W warps.
template <int kV, int kW>
struct Lay {
  static constexpr int V = kV, W = kW;
};
// The fewest warps that hold a row with at most two vectors a lane, from 4096
// columns eight warps with more.  Forward: three vectors where a third of the
// lanes would idle otherwise (2560 columns: 91 against 109 us for 67 M
// elements; the gradient takes 57.3 us for 34 M either way), and eight warps a
// row where there are fewer rows than warps to run them.
template <bool kForward, typename F>
void with_layout(int dim, int64_t rows, F&& f) {
  const int v = (dim + 255) / 256;   // vectors a lane of one warp would hold
  if constexpr (kForward) {
    if (rows <= kFewRows && v <= 8) return f(Lay<1, 8>{});
    if (rows <= kFewRows && v <= 16) return f(Lay<2, 8>{});
    if (v == 5 || v == 6) return f(Lay<3, 2>{});
    if (v >= 9 && v <= 12) return f(Lay<3, 4>{});
  }
  if (v <= 1) f(Lay<1, 1>{});
  else if (v <= 2) f(Lay<2, 1>{});
  else if (v <= 4) f(Lay<2, 2>{});
  else if (v <= 8) f(Lay<2, 4>{});
  else if (v <= 16) f(Lay<2, 8>{});
  else if (v <= 24) f(Lay<3, 8>{});
  else if (v <= 32) f(Lay<4, 8>{});
  else f(Lay<8, 8>{});
}

size_t es_of(int32_t io) { return io == GDN_BF16 ? 2 : 4; }
bool io_ok(int32_t io) { return io == GDN_BF16 || io == GDN_F32; }

int launch_norm(const NormArgs& a, int32_t io, bool fp8, cudaStream_t st) {
  int rc = GDN_OK;
  with_layout<true>(a.dim, a.rows, [&](auto lay) {
    constexpr int V = decltype(lay)::V, W = decltype(lay)::W;
    const int64_t blocks = (a.rows + kWarps / W - 1) / (kWarps / W);
    if (blocks > 0x7fffffffLL) {
      rc = GDN_ERR_UNSUPPORTED;
      return;
    }
    auto kern = io == GDN_BF16
                    ? (fp8 ? residual_norm_kernel<__nv_bfloat16, V, W, true>
                           : residual_norm_kernel<__nv_bfloat16, V, W, false>)
                    : (fp8 ? residual_norm_kernel<float, V, W, true>
                           : residual_norm_kernel<float, V, W, false>);
    kern<<<(unsigned)blocks, kThreads, 0, st>>>(a);
    count_launches(1);
    if (cudaGetLastError() != cudaSuccess) rc = GDN_ERR_CUDA;
  });
  return rc;
}

int norm_common(const void* x, const void* residual, const float* w, float eps, void* s, void* y,
                void* q, float* scale, int64_t tokens, int32_t dim, int32_t io_dtype, bool fp8,
                cudaStream_t stream) {
  if (tokens < 0 || dim < 1 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (!io_ok(io_dtype) || dim % 8 || dim > kMaxDim) return GDN_ERR_UNSUPPORTED;
  if (tokens == 0) return GDN_OK;
  if (!x || !w || (fp8 ? !q || !scale : !y) || (residual && !s) || (!residual && s))
    return GDN_ERR_INVALID_ARG;
  const void* v16[] = {x, residual, w, s, y};
  for (const void* p : v16)
    if (!aligned(p, 16)) return GDN_ERR_ALIGNMENT;
  if (!aligned(q, 16) || !aligned(scale, 4)) return GDN_ERR_ALIGNMENT;
  const size_t n = (size_t)tokens * dim, bytes = n * es_of(io_dtype);
  const int32_t blocks = (dim + 127) / 128;
  const Span sx = span_of(x, bytes), sr = span_of(residual, bytes), sw = span_of(w, (size_t)dim * 4);
  const Span outs[] = {span_of(s, bytes), span_of(y, bytes), span_of(q, n),
                       span_of(scale, (size_t)tokens * blocks * 4)};
  for (int i = 0; i < 4; ++i) {
    // s and y may be x or residual themselves, nothing else overlaps
    const bool whole = i < 2;
    const void* o = i == 0 ? s : y;
    if (intersect(outs[i], sw) || (intersect(outs[i], sx) && !(whole && o == x)) ||
        (intersect(outs[i], sr) && !(whole && o == residual)))
      return GDN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (intersect(outs[i], outs[j])) return GDN_ERR_INVALID_ARG;
  }
  NormArgs a{x, residual, w, eps, s, y, (uint8_t*)q, scale, tokens, dim, blocks};
  return launch_norm(a, io_dtype, fp8, stream);
}

// How the backward's rows are dealt: to one cluster while each warp group of
// it gets at most four (1024 columns, us a call, one launch / two: 32 rows 6.2
// / 10.3, 64 rows 8.2 / 10.8, 128 rows 10.2 / 11.2), else to `grid` CTAs whose
// parts of dw (a row of `dim` each, in scratch) a second launch adds.
struct BackwardPlan {
  bool cluster;
  int grid;
  size_t bytes;   // of the parts
};
BackwardPlan plan_backward(int64_t tokens, int32_t dim, int32_t io) {
  int groups = 1, ctas = 1;
  with_layout<false>(dim, tokens, [&](auto lay) {
    groups = kWarps / decltype(lay)::W;
    ctas = backward_ctas(decltype(lay)::V, es_of(io));
  });
  if (tokens <= 4 * kClusterCtas * groups && dim <= 8192) return {true, kClusterCtas, 0};
  // one wave of CTAs, of two rows a warp group at least; 152 is the device's
  // SMs, a constant, so that the sums' order is one
  const int64_t rounds = (tokens + groups - 1) / groups, most = 152 * ctas;
  int64_t each = (rounds + most - 1) / most;
  if (each < 2) each = 2;
  const int grid = (int)((rounds + each - 1) / each);
  return {false, grid, (size_t)grid * dim * 4};
}
bool backward_shape_ok(int64_t tokens, int32_t dim, int32_t io) {
  return tokens >= 0 && dim >= 1 && io_ok(io) && dim % 8 == 0 && dim <= kMaxDim;
}

int backward_common(const void* dy, const void* s, const float* w, const void* ds, float eps,
                    void* dx, float* dw, int64_t tokens, int32_t dim, int32_t io_dtype,
                    bool use_ws, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (tokens < 0 || dim < 1 || !(eps >= 0.f) || !dw || !w) return GDN_ERR_INVALID_ARG;
  if (!backward_shape_ok(tokens, dim, io_dtype)) return GDN_ERR_UNSUPPORTED;
  if (tokens > 0 && (!dy || !s || !dx)) return GDN_ERR_INVALID_ARG;
  const void* v16[] = {dy, s, w, ds, dx, dw};
  for (const void* p : v16)
    if (!aligned(p, 16)) return GDN_ERR_ALIGNMENT;
  const size_t bytes = (size_t)tokens * dim * es_of(io_dtype);
  const BackwardPlan plan = plan_backward(tokens, dim, io_dtype);
  const size_t need = plan.bytes;
  if (use_ws && need) {
    if (!ws || ws_bytes < need) return GDN_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return GDN_ERR_ALIGNMENT;
  }
  const Span ins[] = {span_of(dy, bytes), span_of(s, bytes), span_of(w, (size_t)dim * 4),
                      span_of(ds, bytes)};
  const Span outs[] = {span_of(dx, bytes), span_of(dw, (size_t)dim * 4),
                       span_of(use_ws ? ws : nullptr, need)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  if (tokens == 0)
    return cudaMemsetAsync(dw, 0, (size_t)dim * 4, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
  void* part = plan.cluster ? dw : ws;
  const bool own = need && !use_ws;
  if (own && scratch_alloc(&part, need, stream) != cudaSuccess) return GDN_ERR_CUDA;
  const NormBwdArgs a{dy, s, w, ds, eps, dx, (float*)part, tokens, dim};
  cudaError_t e = cudaSuccess;
  with_layout<false>(dim, tokens, [&](auto lay) {
    constexpr int V = decltype(lay)::V, W = decltype(lay)::W;
    if constexpr (V <= 4) {
      if (plan.cluster) {
        auto kern = io_dtype == GDN_BF16 ? norm_backward_kernel<__nv_bfloat16, V, W, true>
                                         : norm_backward_kernel<float, V, W, true>;
        e = launch(false, kern, dim3(plan.grid), kThreads, (size_t)dim * 4, kClusterCtas, stream,
                   a);
        return;
      }
    }
    auto kern = io_dtype == GDN_BF16 ? norm_backward_kernel<__nv_bfloat16, V, W, false>
                                     : norm_backward_kernel<float, V, W, false>;
    kern<<<plan.grid, kThreads, 0, stream>>>(a);
    e = cudaGetLastError();
  });
  if (e == cudaSuccess && !plan.cluster)
    e = launch(true, norm_dw_kernel, dim3((dim + 31) / 32), 1024, 0, 0, stream,
               (const float*)part, plan.grid, (int)dim, dw);
  count_launches(plan.cluster ? 1 : 2);
  if (own && scratch_free(part, stream) != cudaSuccess) return GDN_ERR_CUDA;
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_residual_norm(const void* x, const void* residual, const float* w, float eps, void* s,
                      void* y, int64_t tokens, int32_t dim, int32_t io_dtype,
                      gdn_stream_t stream) {
  return norm_common(x, residual, w, eps, s, y, nullptr, nullptr, tokens, dim, io_dtype, false,
                     (cudaStream_t)stream);
}

int gdn_residual_norm_fp8(const void* x, const void* residual, const float* w, float eps, void* s,
                          void* q, float* scale, int64_t tokens, int32_t dim, int32_t io_dtype,
                          gdn_stream_t stream) {
  return norm_common(x, residual, w, eps, s, nullptr, q, scale, tokens, dim, io_dtype, true,
                     (cudaStream_t)stream);
}

size_t gdn_residual_norm_backward_workspace_size(int64_t tokens, int32_t dim, int32_t io_dtype) {
  if (!backward_shape_ok(tokens, dim, io_dtype)) return SIZE_MAX;
  return plan_backward(tokens, dim, io_dtype).bytes;
}

int gdn_residual_norm_backward(const void* dy, const void* s, const float* w, const void* ds,
                               float eps, void* dx, float* dw, int64_t tokens, int32_t dim,
                               int32_t io_dtype, gdn_stream_t stream) {
  return gdn::backward_common(dy, s, w, ds, eps, dx, dw, tokens, dim, io_dtype, false, nullptr, 0,
                              (cudaStream_t)stream);
}

int gdn_residual_norm_backward_ws(const void* dy, const void* s, const float* w, const void* ds,
                                  float eps, void* dx, float* dw, int64_t tokens, int32_t dim,
                                  int32_t io_dtype, void* workspace, size_t workspace_bytes,
                                  gdn_stream_t stream) {
  return gdn::backward_common(dy, s, w, ds, eps, dx, dw, tokens, dim, io_dtype, true, workspace,
                              workspace_bytes, (cudaStream_t)stream);
}

int gdn_quantize_fp8(const void* x, void* q, float* scale, int64_t rows, int32_t cols,
                     int32_t block_rows, int32_t io_dtype, gdn_stream_t stream_) {
  cudaStream_t stream = (cudaStream_t)stream_;
  if (rows < 0 || cols < 1) return GDN_ERR_INVALID_ARG;
  if (!io_ok(io_dtype) || cols % 8 || cols > kLongestAxis ||
      (block_rows != 1 && block_rows != 128))
    return GDN_ERR_UNSUPPORTED;
  if (rows == 0) return GDN_OK;
  if (!x || !q || !scale) return GDN_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return GDN_ERR_ALIGNMENT;
  const int32_t blocks = (cols + 127) / 128;
  const int64_t row_blocks = (rows + block_rows - 1) / block_rows;
  const Span ins[] = {span_of(x, (size_t)rows * cols * es_of(io_dtype))};
  const Span outs[] = {span_of(q, (size_t)rows * cols),
                       span_of(scale, (size_t)row_blocks * blocks * 4)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  QuantArgs a{x, (uint8_t*)q, scale, rows, cols, blocks};
  if (block_rows == 1) {
    const int64_t grid = (rows * blocks + 16 * kTwo - 1) / (16 * kTwo);
    if (grid > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    auto kern = io_dtype == GDN_BF16 ? quant_rows_kernel<__nv_bfloat16> : quant_rows_kernel<float>;
    kern<<<(unsigned)grid, kThreads, 0, stream>>>(a);
  } else {
    if (row_blocks > 65535) return GDN_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, (unsigned)row_blocks);
    auto kern = io_dtype == GDN_BF16 ? quant_tiles_kernel<__nv_bfloat16> : quant_tiles_kernel<float>;
    kern<<<grid, kThreads, 0, stream>>>(a);
  }
  count_launches(1);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
