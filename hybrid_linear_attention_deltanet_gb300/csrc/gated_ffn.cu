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
// fill the end of the grid.
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

int shape_check(int64_t tokens, int32_t dim, int32_t hidden, int32_t act, int32_t io) {
  if (tokens < 0 || dim < 1 || hidden < 1) return GDN_ERR_INVALID_ARG;
  if (io != GDN_BF16 || dim % 8 || tokens > 0x7fffff00LL || hidden > 0x7fffff00 ||
      (act != GDN_GATE_SILU && act != GDN_GATE_SIGMOID))
    return GDN_ERR_UNSUPPORTED;
  const int64_t mt = (tokens + 255) / 256, ft = (hidden + 127) / 128, dt = (dim + 255) / 256;
  if (mt * ft > 0x3fffffffLL || mt * dt > 0x3fffffffLL || (ft + 1) * dt > 0x3fffffffLL)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// The product with both projections, x [tokens][dim] against Wg and Wu.
bool projections(gemm::PairArgs& g, const void* x, const void* wg, const void* wu, int64_t tokens,
                 int32_t dim, int32_t hidden) {
  gemm::Problem& p = g.p[0];
  p.m_half = p.m_tiles = (int32_t)((tokens + 255) / 256);
  p.n_tiles = (hidden + 127) / 128;
  p.k_half = p.k_blocks = (dim + 63) / 64;
  p.M = (int32_t)tokens;
  p.N = hidden;
  g.problems = 1;
  g.group_m = gemm::group_rows((int64_t)dim * 2);
  if (!gemm::matrix_map(&p.a[0], x, false, dim, tokens, (int64_t)dim * 2, 128) ||
      !gemm::matrix_map(&p.b[0], wg, false, dim, hidden, (int64_t)dim * 2, 128) ||
      !gemm::matrix_map(&p.b[1], wu, false, dim, hidden, (int64_t)dim * 2, 128))
    return false;
  p.a[1] = p.a[0];
  return true;
}

// Few tokens: the split form, two CTAs an SM to keep the weights coming
// (2048 -> 6144, us, split form / pair form: 1 token 11.1 / 20, 64 tokens
// 12.6 / 17, 128 tokens 14.8 / 17, 256 tokens 19.4 / 16.5).
bool takes_split(int64_t tokens, int32_t hidden) {
  return tokens <= 128 && (hidden + 63) / 64 <= 65535;
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
  if (takes_split(tokens, hidden)) {
    gemm::SplitArgs a;
    memset(&a, 0, sizeof a);
    const int nb = tokens <= 16 ? 16 : tokens <= 32 ? 32 : tokens <= 64 ? 64 : 128;
    a.k_blocks = (dim + 63) / 64;
    a.tokens = (int32_t)tokens;
    a.n = hidden;
    a.act = act;
    a.out = h;
    a.status = status;
    if (!gemm::matrix_map(&a.w[0], wg, false, dim, hidden, (int64_t)dim * 2, 64) ||
        !gemm::matrix_map(&a.w[1], wu, false, dim, hidden, (int64_t)dim * 2, 64) ||
        !gemm::matrix_map(&a.x, x, false, dim, tokens, (int64_t)dim * 2, nb))
      return GDN_ERR_CUDA;
    const int split = gemm::split_of((hidden + 63) / 64, a.k_blocks, 2 * sms, 8);
    return gemm::launch_split<false, true, __nv_bfloat16>(a, nb, split, stream) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
  }
  gemm::PairArgs g;
  memset(&g, 0, sizeof g);
  g.status = status;
  if (!projections(g, x, wg, wu, tokens, dim, hidden)) return GDN_ERR_CUDA;
  g.act = act;
  g.p[0].out[0] = g.p[0].out[1] = h;
  g.p[0].ldc = hidden;
  return gemm::launch_pair<false, gemm::kGate>(g, sms, stream) == cudaSuccess ? GDN_OK
                                                                              : GDN_ERR_CUDA;
}

cudaError_t launch_backward(const void* x, const void* wg, const void* wu, const void* dh,
                            int32_t act, void* dx, void* dwg, void* dwu, void* scratch,
                            int64_t tokens, int32_t dim, int32_t hidden, int sms,
                            unsigned* status, cudaStream_t stream) {
  const int64_t pitch = grad_pitch(hidden);
  void* dG = scratch;
  void* dU = (char*)scratch + grad_bytes(tokens, hidden);
  gemm::PairArgs g;
  memset(&g, 0, sizeof g);
  g.status = status;
  g.act = act;
  if (!projections(g, x, wg, wu, tokens, dim, hidden)) return cudaErrorUnknown;
  g.p[0].out[0] = dG;
  g.p[0].out[1] = dU;
  g.p[0].ldc = pitch;
  g.dh = (const __nv_bfloat16*)dh;
  g.ldh = hidden;
  g.dh_wide = hidden % 8 == 0;
  cudaError_t e = gemm::launch_pair<false, gemm::kGateGrad>(g, sms, stream);
  if (e != cudaSuccess) return e;

  memset(&g, 0, sizeof g);
  g.status = status;
  g.problems = 2;
  g.group_m = 8;   // either operand is read once for the tiles in flight, which are about square
  const int32_t kx = (hidden + 63) / 64, kw = (int32_t)((tokens + 63) / 64);
  const int ix = 2 * kx >= kw ? 0 : 1;
  gemm::Problem& px = g.p[ix];
  px.m_half = px.m_tiles = (int32_t)((tokens + 255) / 256);
  px.n_tiles = (dim + 255) / 256;
  px.k_half = kx;
  px.k_blocks = 2 * kx;
  px.b_mn = 1;
  px.M = (int32_t)tokens;
  px.N = dim;
  px.out[0] = px.out[1] = dx;
  px.ldc = dim;
  gemm::Problem& pw = g.p[1 - ix];
  pw.m_half = (hidden + 255) / 256;
  pw.m_tiles = 2 * pw.m_half;
  pw.n_tiles = (dim + 255) / 256;
  pw.k_half = pw.k_blocks = kw;
  pw.a_mn = pw.b_mn = 1;
  pw.M = hidden;
  pw.N = dim;
  pw.out[0] = dwg;
  pw.out[1] = dwu;
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
  return gemm::launch_pair<false, gemm::kStore>(g, sms, stream);
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
  const size_t need = 2 * grad_bytes(tokens, hidden);
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
  return 2 * grad_bytes(tokens, hidden);
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
