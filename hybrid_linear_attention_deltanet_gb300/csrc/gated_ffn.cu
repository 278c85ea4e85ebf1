// The gated feed-forward projections and their gradients (contracts:
// include/gdn.h):
//
//   G = x Wg^T, U = x Wu^T, h = act(G) U
//   dU = dh act(G), dG = dh U act'(G)
//   dx = dG Wg + dU Wu, dWg = dG^T x, dWu = dU^T x
//
// Forward: one product (gemm_pair.cuh) whose 256 columns are the same 128
// features of Wg and Wu, so that G and U of a feature meet in one thread and
// only h is written.
//
// Backward: G and U are recomputed (4 of its 12 tokens x dim x hidden
// operations) instead of kept from the forward pass, whose 4 bytes a token
// and feature they would cost; that product's epilogue takes dh and writes
// dG and dU as bf16, the type their products with x, Wg and Wu take (their
// fp32 sums round once more to the bf16 results).  One second launch then
// has the tiles of dx (K runs over dG then dU) and of both weight gradients
// (rows over dG^T then dU^T), the longer K first, so that the short tiles
// fill the end of the grid.  Where a product's tiles are few and their K is
// long, K is cut into parts, whose fp32 sums a third launch adds in order.
#include <utility>

#include "gemm_split.cuh"
#include "hostcheck.cuh"

namespace gdn {
namespace {

using namespace hostcheck;

// [tokens][pitch] of dG and of dU; the pitch keeps rows on 32 bytes
int64_t grad_pitch(int32_t hidden) { return ((int64_t)hidden + 15) / 16 * 16; }
size_t grad_bytes(int64_t tokens, int32_t hidden) {
  return align_up((size_t)tokens * grad_pitch(hidden) * 2, 256);
}

// Parts of K of the second launch's two products: those with the shortest
// estimate of that launch and the sums' together.  The pair count is that of
// the device; a constant, so that a workspace's size needs no device.
constexpr int kPairs = 76;
struct Parts {
  int dx, dw;                     // parts of K
  int64_t dx_rows, dw_rows;       // rows of a part
  size_t dx_off, dw_off, bytes;   // of the fp32 parts in the scratch, after dG and dU
};
struct Work {
  int64_t tiles, blocks;   // of one product: tiles, and K blocks of a tile (with its end, as 5)
};
// K blocks of the longest pair, as gemm_pair.cuh deals the tiles out.
int64_t longest(Work a, Work b) {
  if (a.blocks < b.blocks) std::swap(a, b);
  const int64_t sum = a.tiles + b.tiles, pairs = sum < kPairs ? sum : kPairs;
  const int64_t r = a.tiles % pairs, n = a.tiles / pairs, spared = pairs - r;
  const int64_t ahead = a.blocks / b.blocks, rest = b.tiles - ahead * spared;
  int64_t few = (b.tiles + spared - 1) / spared, many = 0;   // short tiles of either kind of pair
  if (rest > 0) {
    few = ahead + rest / pairs + (rest % pairs > 0);
    many = rest / pairs + (rest % pairs > spared);
  }
  const int64_t x = n * a.blocks + few * b.blocks, y = (n + 1) * a.blocks + many * b.blocks;
  return r && y > x ? y : x;
}
Parts plan_parts(int64_t tokens, int32_t dim, int32_t hidden) {
  const int64_t dt = ((int64_t)dim + 255) / 256, tx = (tokens + 255) / 256 * dt;
  const int64_t tw = 2 * (((int64_t)hidden + 255) / 256) * dt;
  const int64_t kx = 2 * (((int64_t)hidden + 63) / 64), kw = (tokens + 63) / 64;
  Parts p;
  p.dx = p.dw = 1;
  p.dx_rows = (tokens + 255) / 256 * 256;
  p.dw_rows = ((int64_t)hidden + 255) / 256 * 256;
  // a part costs its fp32 tiles' way out and back (256 KB each: 0.1 us, a
  // third of a K block) and the sums one launch (4.5 us, the host's share included)
  static constexpr int kTry[] = {1, 2, 3, 4, 6, 8};
  int64_t best = INT64_MAX;
  for (int a : kTry)
    for (int b : kTry) {
      if ((a > 1 && (kx < 4 * a || tx * a > 4 * kPairs)) ||
          (b > 1 && (kw < 4 * b || tw * b > 4 * kPairs)))
        continue;
      const int64_t sums = (a > 1 ? tx * a : 0) + (b > 1 ? tw * b : 0);
      const int64_t cost = 3 * longest({tx * a, kx / a + 5}, {tw * b, kw / b + 5}) +
                           (sums ? 45 + sums : 0);
      if (cost < best) {
        best = cost;
        p.dx = a;
        p.dw = b;
      }
    }
  p.dx_off = 2 * grad_bytes(tokens, hidden);
  p.dw_off = p.dx_off + (p.dx > 1 ? align_up((size_t)p.dx * p.dx_rows * dim * 4, 256) : 0);
  p.bytes = p.dw_off + (p.dw > 1 ? align_up(2 * (size_t)p.dw * p.dw_rows * dim * 4, 256) : 0);
  return p;
}

// out = the parts' sum, in order, as bf16.
struct SumArgs {
  const float* part[3];
  __nv_bfloat16* out[3];
  int64_t vecs[3];     // elements / 8
  int64_t stride[3];   // elements of a part
  int32_t parts[3];
};
__global__ void __launch_bounds__(256) sum_parts_kernel(const __grid_constant__ SumArgs a) {
  grid_release_next();
  grid_wait();
  const int64_t all = a.vecs[0] + a.vecs[1] + a.vecs[2];
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all;
       i += (int64_t)gridDim.x * 256) {
    const int w = i < a.vecs[0] ? 0 : i < a.vecs[0] + a.vecs[1] ? 1 : 2;
    const int64_t e = 8 * (i - (w > 0 ? a.vecs[0] : 0) - (w > 1 ? a.vecs[1] : 0));
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = 0; p < a.parts[w]; ++p) {
      const float4* f = reinterpret_cast<const float4*>(a.part[w] + p * a.stride[w] + e);
      const float4 x = ld_waited(f), y = ld_waited(f + 1);
      v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    *reinterpret_cast<uint4*>(a.out[w] + e) =
        make_uint4(gemm::pack2(v[0], v[1]), gemm::pack2(v[2], v[3]), gemm::pack2(v[4], v[5]),
                   gemm::pack2(v[6], v[7]));
  }
}

int shape_check(int64_t tokens, int32_t dim, int32_t hidden, int32_t act, int32_t io) {
  if (tokens < 0 || dim < 1 || hidden < 1) return GDN_ERR_INVALID_ARG;
  // (a tile of the projections has two columns for each feature)
  if (io != GDN_BF16 || dim % 8 || tokens > kLongestAxis || dim > kLongestAxis ||
      hidden > kLongestAxis / 2 ||
      (act != GDN_GATE_SILU && act != GDN_GATE_SIGMOID))
    return GDN_ERR_UNSUPPORTED;
  const int64_t mt = (tokens + 255) / 256, ft = (hidden + 127) / 128, dt = (dim + 255) / 256;
  if (mt * ft > 0x3fffffffLL || mt * dt > 0x3fffffffLL || (ft + 1) * dt > 0x3fffffffLL)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// The product with both projections, x [tokens][dim] against Wg and Wu.
template <int kEpi>
cudaError_t projections(gemm::PairArgs& g, const void* x, const void* wg, const void* wu,
                        int64_t tokens, int32_t dim, int32_t hidden, int sms,
                        cudaStream_t stream) {
  const bool narrow = gemm::narrow_gated(tokens, hidden, sms);
  const int32_t features = narrow ? 96 : 128;   // of each projection a tile
  gemm::Problem& p = g.p[0];
  p.m_half = p.m_tiles = (int32_t)((tokens + 255) / 256);
  p.n_tiles = (hidden + features - 1) / features;
  p.k_half = p.k_blocks = (dim + 63) / 64;
  p.k_parts = 1;
  p.M = (int32_t)tokens;
  p.N = hidden;
  g.problems = 1;
  g.group_m = gemm::group_rows((int64_t)dim * 2);
  if (!gemm::matrix_map(&p.a[0], x, false, dim, tokens, (int64_t)dim * 2, 128) ||
      !gemm::matrix_map(&p.b[0], wg, false, dim, hidden, (int64_t)dim * 2, features) ||
      !gemm::matrix_map(&p.b[1], wu, false, dim, hidden, (int64_t)dim * 2, features))
    return cudaErrorUnknown;
  p.a[1] = p.a[0];
  return narrow ? gemm::launch_pair<false, kEpi, 192>(g, sms, stream)
                : gemm::launch_pair<false, kEpi>(g, sms, stream);
}

// The same for few tokens (gemm_split.cuh).
gemm::SplitPlan plan_projections(int64_t tokens, int32_t dim, int32_t hidden, int sms) {
  return gemm::plan_split(tokens, ((int64_t)hidden + 63) / 64, (dim + 63) / 64, sms, sms);
}
bool split_projections(gemm::SplitArgs& a, const gemm::SplitPlan& plan, const void* x,
                       const void* wg, const void* wu, int32_t act, int64_t tokens, int32_t dim,
                       int32_t hidden) {
  memset(&a, 0, sizeof a);
  a.k_blocks = (dim + 63) / 64;
  a.tokens = (int32_t)tokens;
  a.n = hidden;
  a.act = act;
  const int64_t pitch = (int64_t)dim * 2;
  return gemm::matrix_map(&a.w[0], wg, false, dim, hidden, pitch, 64) &&
         gemm::matrix_map(&a.w[1], wu, false, dim, hidden, pitch, 64) &&
         gemm::matrix_map(&a.x, x, false, dim, tokens, pitch, (uint32_t)plan.columns);
}

int ffn_forward(const void* x, const void* wg, const void* wu, int32_t act, void* h,
                int64_t tokens, int32_t dim, int32_t hidden, int32_t io, cudaStream_t stream) {
  if (const int rc = shape_check(tokens, dim, hidden, act, io)) return rc;
  if (tokens == 0) return GDN_OK;
  if (!x || !wg || !wu || !h) return GDN_ERR_INVALID_ARG;
  const void* v16[] = {x, wg, wu, h};
  for (const void* p : v16)
    if (!aligned(p, 16)) return GDN_ERR_ALIGNMENT;
  const size_t wb = (size_t)hidden * dim * 2;
  const Span ins[] = {span_of(x, (size_t)tokens * dim * 2), span_of(wg, wb), span_of(wu, wb)};
  const Span outs[] = {span_of(h, (size_t)tokens * hidden * 2)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  const int sms = sm_count();
  unsigned* status = status_ptr();
  if (sms < 2 || !status) return GDN_ERR_CUDA;
  const gemm::SplitPlan plan = plan_projections(tokens, dim, hidden, sms);
  if (plan.columns) {
    gemm::SplitArgs a;
    if (!split_projections(a, plan, x, wg, wu, act, tokens, dim, hidden)) return GDN_ERR_CUDA;
    a.out = h;
    a.ld = hidden;
    a.status = status;
    return gemm::launch_split<false, gemm::kGate, __nv_bfloat16>(a, plan, stream) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
  }
  gemm::PairArgs g;
  memset(&g, 0, sizeof g);
  g.status = status;
  g.act = act;
  g.p[0].out[0] = g.p[0].out[1] = h;
  g.p[0].ldc = hidden;
  const cudaError_t e =
      projections<gemm::kGate>(g, x, wg, wu, tokens, dim, hidden, sms, stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

cudaError_t launch_backward(const void* x, const void* wg, const void* wu, const void* dh,
                            int32_t act, void* dx, void* dwg, void* dwu, void* scratch,
                            int64_t tokens, int32_t dim, int32_t hidden, int sms,
                            unsigned* status, cudaStream_t stream) {
  const int64_t pitch = grad_pitch(hidden);
  void* dG = scratch;
  void* dU = (char*)scratch + grad_bytes(tokens, hidden);
  cudaError_t e;
  gemm::PairArgs g;
  const gemm::SplitPlan plan = plan_projections(tokens, dim, hidden, sms);
  if (plan.columns) {
    gemm::SplitArgs a;
    if (!split_projections(a, plan, x, wg, wu, act, tokens, dim, hidden)) return cudaErrorUnknown;
    a.out = dG;
    a.out2 = dU;
    a.ld = pitch;
    a.dh = (const __nv_bfloat16*)dh;
    a.status = status;
    e = gemm::launch_split<false, gemm::kGateGrad, __nv_bfloat16>(a, plan, stream);
  } else {
    memset(&g, 0, sizeof g);
    g.status = status;
    g.act = act;
    g.p[0].out[0] = dG;
    g.p[0].out[1] = dU;
    g.p[0].ldc = pitch;
    g.dh = (const __nv_bfloat16*)dh;
    g.ldh = hidden;
    g.dh_wide = hidden % 8 == 0;
    e = projections<gemm::kGateGrad>(g, x, wg, wu, tokens, dim, hidden, sms, stream);
  }
  if (e != cudaSuccess) return e;

  memset(&g, 0, sizeof g);
  g.status = status;
  g.problems = 2;
  g.group_m = 8;   // either operand is read once for the tiles in flight, which are about square
  const int32_t kx = (hidden + 63) / 64, kw = (int32_t)((tokens + 63) / 64);
  const Parts parts = plan_parts(tokens, dim, hidden);
  const int ix = 2 * kx / parts.dx >= kw / parts.dw ? 0 : 1;   // the longer tiles first
  float* dx_parts = (float*)((char*)scratch + parts.dx_off);
  float* dw_parts = (float*)((char*)scratch + parts.dw_off);
  gemm::Problem& px = g.p[ix];
  px.m_half = px.m_tiles = (int32_t)((tokens + 255) / 256);
  px.n_tiles = (dim + 255) / 256;
  px.k_half = kx;
  px.k_blocks = 2 * kx;
  px.b_mn = 1;
  px.M = (int32_t)tokens;
  px.N = dim;
  px.k_parts = parts.dx;
  px.part_rows = (int32_t)parts.dx_rows;
  px.out[0] = px.out[1] = parts.dx > 1 ? dx_parts : dx;
  px.ldc = dim;
  gemm::Problem& pw = g.p[1 - ix];
  pw.m_half = (hidden + 255) / 256;
  pw.m_tiles = 2 * pw.m_half;
  pw.n_tiles = (dim + 255) / 256;
  pw.k_half = pw.k_blocks = kw;
  pw.a_mn = pw.b_mn = 1;
  pw.M = hidden;
  pw.N = dim;
  pw.k_parts = parts.dw;
  pw.part_rows = (int32_t)parts.dw_rows;
  const int64_t dw_half = (int64_t)parts.dw * parts.dw_rows * dim;
  pw.out[0] = parts.dw > 1 ? dw_parts : dwg;
  pw.out[1] = parts.dw > 1 ? dw_parts + dw_half : dwu;
  pw.ldc = dim;
  const int64_t gp = pitch * 2, dp = (int64_t)dim * 2;
  if (!gemm::matrix_map(&px.a[0], dG, false, hidden, tokens, gp, 128) ||
      !gemm::matrix_map(&px.a[1], dU, false, hidden, tokens, gp, 128) ||
      !gemm::matrix_map(&px.b[0], wg, false, dim, hidden, dp, 64) ||
      !gemm::matrix_map(&px.b[1], wu, false, dim, hidden, dp, 64) ||
      !gemm::matrix_map(&pw.a[0], dG, false, hidden, tokens, gp, 64) ||
      !gemm::matrix_map(&pw.a[1], dU, false, hidden, tokens, gp, 64) ||
      !gemm::matrix_map(&pw.b[0], x, false, dim, tokens, dp, 64))
    return cudaErrorUnknown;
  pw.b[1] = pw.b[0];
  e = gemm::launch_pair<false, gemm::kStore>(g, sms, stream);
  if (e != cudaSuccess || (parts.dx == 1 && parts.dw == 1)) return e;
  SumArgs a;
  memset(&a, 0, sizeof a);
  if (parts.dx > 1) {
    a.part[0] = dx_parts;
    a.out[0] = (__nv_bfloat16*)dx;
    a.vecs[0] = tokens * dim / 8;
    a.stride[0] = parts.dx_rows * dim;
    a.parts[0] = parts.dx;
  }
  for (int i = 1; parts.dw > 1 && i < 3; ++i) {
    a.part[i] = dw_parts + (i - 1) * dw_half;
    a.out[i] = (__nv_bfloat16*)(i == 1 ? dwg : dwu);
    a.vecs[i] = (int64_t)hidden * dim / 8;
    a.stride[i] = parts.dw_rows * dim;
    a.parts[i] = parts.dw;
  }
  const int64_t blocks = (a.vecs[0] + a.vecs[1] + a.vecs[2] + 255) / 256, most = 8 * (int64_t)sms;
  e = launch(true, sum_parts_kernel, dim3((unsigned)(blocks < most ? blocks : most)), 256, 0, 0,
                       stream, a);
  count_launches(1);
  return e;
}

int ffn_backward(const void* x, const void* wg, const void* wu, const void* dh, int32_t act,
                 void* dx, void* dwg, void* dwu, int64_t tokens, int32_t dim, int32_t hidden,
                 int32_t io, bool use_ws, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (const int rc = shape_check(tokens, dim, hidden, act, io)) return rc;
  if (!wg || !wu || !dwg || !dwu || (tokens > 0 && (!x || !dh || !dx)))
    return GDN_ERR_INVALID_ARG;
  const void* v16[] = {x, wg, wu, dh, dx, dwg, dwu};
  for (const void* p : v16)
    if (!aligned(p, 16)) return GDN_ERR_ALIGNMENT;
  const size_t need = plan_parts(tokens, dim, hidden).bytes;
  if (use_ws && need) {
    if (!ws || ws_bytes < need) return GDN_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return GDN_ERR_ALIGNMENT;
  }
  const size_t wb = (size_t)hidden * dim * 2, xb = (size_t)tokens * dim * 2;
  const Span ins[] = {span_of(x, xb), span_of(wg, wb), span_of(wu, wb),
                      span_of(dh, (size_t)tokens * hidden * 2)};
  const Span outs[] = {span_of(dx, xb), span_of(dwg, wb), span_of(dwu, wb),
                       span_of(use_ws ? ws : nullptr, need)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  if (tokens == 0)
    return cudaMemsetAsync(dwg, 0, wb, stream) == cudaSuccess &&
                   cudaMemsetAsync(dwu, 0, wb, stream) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
  const int sms = sm_count();
  unsigned* status = status_ptr();
  if (sms < 2 || !status) return GDN_ERR_CUDA;
  void* scratch = ws;
  if (!use_ws && scratch_alloc(&scratch, need, stream) != cudaSuccess) return GDN_ERR_CUDA;
  const cudaError_t e = launch_backward(x, wg, wu, dh, act, dx, dwg, dwu, scratch, tokens, dim,
                                        hidden, sms, status, stream);
  const cudaError_t ef = use_ws ? cudaSuccess : scratch_free(scratch, stream);
  return e == cudaSuccess && ef == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_gated_ffn(const void* x, const void* w_gate, const void* w_up, int32_t act, void* h,
                  int64_t tokens, int32_t dim, int32_t hidden, int32_t io_dtype,
                  gdn_stream_t stream) {
  return ffn_forward(x, w_gate, w_up, act, h, tokens, dim, hidden, io_dtype,
                     (cudaStream_t)stream);
}

size_t gdn_gated_ffn_backward_workspace_size(int64_t tokens, int32_t dim, int32_t hidden,
                                             int32_t io_dtype) {
  if (shape_check(tokens, dim, hidden, GDN_GATE_SILU, io_dtype)) return SIZE_MAX;
  return plan_parts(tokens, dim, hidden).bytes;
}

int gdn_gated_ffn_backward(const void* x, const void* w_gate, const void* w_up, const void* dh,
                           int32_t act, void* dx, void* dw_gate, void* dw_up, int64_t tokens,
                           int32_t dim, int32_t hidden, int32_t io_dtype, gdn_stream_t stream) {
  return ffn_backward(x, w_gate, w_up, dh, act, dx, dw_gate, dw_up, tokens, dim, hidden, io_dtype,
                      false, nullptr, 0, (cudaStream_t)stream);
}

int gdn_gated_ffn_backward_ws(const void* x, const void* w_gate, const void* w_up, const void* dh,
                              int32_t act, void* dx, void* dw_gate, void* dw_up, int64_t tokens,
                              int32_t dim, int32_t hidden, int32_t io_dtype, void* workspace,
                              size_t workspace_bytes, gdn_stream_t stream) {
  return ffn_backward(x, w_gate, w_up, dh, act, dx, dw_gate, dw_up, tokens, dim, hidden, io_dtype,
                      true, workspace, workspace_bytes, (cudaStream_t)stream);
}

}  // extern "C"
