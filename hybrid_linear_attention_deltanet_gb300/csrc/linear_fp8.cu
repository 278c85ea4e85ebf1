// Matrix product of e4m3 operands with a scale for every 1 x 128 block of the
// activations and every 128 x 128 block of the weights (contract:
// include/gdn.h):
//
//   out[t][n] = sum_b sx[t][b] sw[n / 128][b] sum_{k in block b} x[t][k] w[n][k]
//
// The inner sums run on the tensor cores (kind::f8f6f4, fp32 accumulation),
// the outer one in fp32 registers (gemm_pair.cuh).
#include "gemm_split.cuh"
#include "hostcheck.cuh"

namespace gdn {
namespace {

using namespace hostcheck;

int linear_common(const void* x, const float* sx, const void* w, const float* sw, void* out,
                  int64_t tokens, int32_t k, int32_t n, int32_t out_dtype, cudaStream_t stream) {
  if (tokens < 0 || k < 1 || n < 1) return GDN_ERR_INVALID_ARG;
  if (k % 16 || (out_dtype != GDN_BF16 && out_dtype != GDN_F32) || tokens > kLongestAxis ||
      k > kLongestAxis || n > kLongestAxis)
    return GDN_ERR_UNSUPPORTED;
  if (tokens == 0) return GDN_OK;
  if (!x || !sx || !w || !sw || !out) return GDN_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(sx, 4) ||
      !aligned(sw, 4))
    return GDN_ERR_ALIGNMENT;
  const int32_t blocks = (k + 127) / 128;
  const size_t es = out_dtype == GDN_BF16 ? 2 : 4;
  const Span ins[] = {span_of(x, (size_t)tokens * k), span_of(sx, (size_t)tokens * blocks * 4),
                      span_of(w, (size_t)n * k),
                      span_of(sw, (size_t)((n + 127) / 128) * blocks * 4)};
  const Span outs[] = {span_of(out, (size_t)tokens * n * es)};
  if (any_overlap(ins, outs)) return GDN_ERR_INVALID_ARG;
  const int sms = sm_count();
  unsigned* status = status_ptr();
  if (sms < 2 || !status) return GDN_ERR_CUDA;
  const gemm::SplitPlan plan =
      gemm::plan_split(tokens, ((int64_t)n + 127) / 128, blocks, sms, sms / 2);
  if (plan.columns && (int64_t)((blocks + plan.split - 1) / plan.split) * plan.columns * 4 <=
                          gemm::kSplitScaleBytes) {
    gemm::SplitArgs a;
    memset(&a, 0, sizeof a);
    a.k_blocks = blocks;
    a.tokens = (int32_t)tokens;
    a.n = n;
    a.out = out;
    a.ld = n;
    a.sx = sx;
    a.sw = sw;
    a.status = status;
    if (!gemm::matrix_map(&a.w[0], w, true, k, n, k, 128) ||
        !gemm::matrix_map(&a.x, x, true, k, tokens, k, plan.columns))
      return GDN_ERR_CUDA;
    const cudaError_t e =
        out_dtype == GDN_BF16
            ? gemm::launch_split<true, gemm::kStore, __nv_bfloat16>(a, plan, stream)
            : gemm::launch_split<true, gemm::kStore, float>(a, plan, stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
  }
  gemm::PairArgs g;
  memset(&g, 0, sizeof g);
  gemm::Problem& p = g.p[0];
  const int64_t mt = (tokens + 255) / 256;
  const bool narrow = gemm::narrow_fp8(mt, n, sms);
  const int32_t columns = narrow ? 128 : 256;
  const int64_t nt = ((int64_t)n + columns - 1) / columns;
  if (mt * nt > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  p.m_half = p.m_tiles = (int32_t)mt;
  p.n_tiles = (int32_t)nt;
  p.k_half = p.k_blocks = blocks;
  p.k_parts = 1;
  p.M = (int32_t)tokens;
  p.N = n;
  p.out[0] = p.out[1] = out;
  p.ldc = n;
  g.problems = 1;
  g.group_m = gemm::group_rows(k);
  g.sa = sx;
  g.sb = sw;
  g.sblocks = blocks;
  g.status = status;
  if (!gemm::matrix_map(&p.a[0], x, true, k, tokens, k, 128) ||
      !gemm::matrix_map(&p.b[0], w, true, k, n, k, columns / 2))
    return GDN_ERR_CUDA;
  p.a[1] = p.a[0];
  p.b[1] = p.b[0];
  const auto go = out_dtype == GDN_BF16
                      ? narrow ? gemm::launch_pair<true, gemm::kStore, 128>
                               : gemm::launch_pair<true, gemm::kStore, 256>
                      : narrow ? gemm::launch_pair<true, gemm::kStoreF32, 128>
                               : gemm::launch_pair<true, gemm::kStoreF32, 256>;
  const cudaError_t e = go(g, sms, stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

extern "C" int gdn_linear_fp8(const void* x, const float* x_scale, const void* w,
                              const float* w_scale, void* out, int64_t tokens, int32_t k,
                              int32_t n, int32_t out_dtype, gdn_stream_t stream) {
  return gdn::linear_common(x, x_scale, w, w_scale, out, tokens, k, n, out_dtype,
                            (cudaStream_t)stream);
}
