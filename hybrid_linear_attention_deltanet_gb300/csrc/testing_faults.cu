// Fault test hook: the library's two kinds of bounded wait -- an mbarrier
// try-wait and a poll of a ready flag in global memory (the handoff between
// the per-chunk workers and the state pass of the fused prefill) -- run on
// something that never completes, so that the wait gives up after its limit,
// records GDN_ERR_TIMEOUT in the device status word and returns.  Nothing
// traps, hangs or faults; the context stays usable.  And warps that meet at barriers
// between such waits, some of which run out.
#include "../../include/gdn_testing.h"
#include "attention_tc.cuh"
#include "gdn_internal.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

using namespace sm100;

// a ready flag that nothing ever sets
__device__ uint32_t g_never_set_flag = 0;

__global__ void bounded_wait_kernel(int32_t which, uint64_t limit_ns, unsigned* status,
                                    uint32_t* flag) {
  __shared__ uint64_t bar;
  if (threadIdx.x != 0) return;
  bool ok = true;
  if (which == 0) {
    mbar_init(&bar, 1);   // expects one arrival, which never comes
    fence_barrier_init();
    ok = mbar_wait(&bar, 0, limit_ns);
  } else {
    const uint64_t t0 = globaltimer_ns();
    ok = false;
    do {
      if (ld_relaxed_gpu(flag) != 0u) {
        fence_acq_rel_gpu();
        ok = true;
        break;
      }
      __nanosleep(64);
    } while (globaltimer_ns() - t0 < limit_ns);
  }
  if (!ok) flag_status(status, GDN_ERR_TIMEOUT);
}

// Four warps in the two forms that the attention kernels have.  asks = false: a barrier, then
// a wait in every step, and a warp whose wait ran out goes on to the barriers that are left
// (the gradients' P and dS); true: a wait in every step, and behind that of every `part`-th
// and of the last a barrier that asks all (the decoding's tiles and parts).
__global__ void __launch_bounds__(128)
group_wait_kernel(bool asks, uint32_t late, int32_t step, int32_t steps, int32_t part,
                  long long limit, int32_t* left, unsigned* status) {
  __shared__ uint64_t bar[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < 4) mbar_init(&bar[threadIdx.x], 1);
  if (threadIdx.x == 0) fence_barrier_init();
  __syncthreads();
  bool ok = true;
  int32_t i = 0;
  int32_t gone = steps;
  for (; i < steps; ++i) {
    if (!asks) attn::bar_sync(1, 128);
    if (lane == 0 && !(i == step && (late >> warp & 1u))) mbar_arrive(&bar[warp]);
    ok = mbar_wait_warp_cycles(&bar[warp], (uint32_t)(i & 1), limit);
    if (!ok && asks) attn::bar_agree(1, 128, false);
    if (ok && asks && (i % part == part - 1 || i + 1 == steps)) ok = attn::bar_agree(1, 128, true);
    if (!ok) {
      gone = i;
      break;
    }
  }
  if (!ok && !asks)
    while (++i < steps) attn::bar_sync(1, 128);
  if (!ok) flag_status(status, GDN_ERR_TIMEOUT);
  if (lane == 0) left[warp] = gone;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" int gdn_testing_bounded_wait(int32_t which, int64_t limit_ns, gdn_stream_t stream) {
  if ((which != 0 && which != 1) || limit_ns < 0 || limit_ns > 2000000000LL)
    return GDN_ERR_INVALID_ARG;
  unsigned* status = status_ptr();
  uint32_t* flag = nullptr;
  if (!status || cudaGetSymbolAddress((void**)&flag, g_never_set_flag) != cudaSuccess)
    return GDN_ERR_CUDA;
  bounded_wait_kernel<<<1, 32, 0, (cudaStream_t)stream>>>(which, (uint64_t)limit_ns, status,
                                                           flag);
  count_launches(1);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" int gdn_testing_group_wait(int32_t asks, uint32_t late, int32_t step, int32_t steps,
                                      int32_t part, int64_t limit_cycles, int32_t* left,
                                      gdn_stream_t stream) {
  if ((asks != 0 && asks != 1) || late > 15u || step < 0 || steps < 1 || steps > 1000 ||
      part < 1 || limit_cycles < 0 || limit_cycles > 2000000000LL || !left)
    return GDN_ERR_INVALID_ARG;
  unsigned* status = status_ptr();
  if (!status) return GDN_ERR_CUDA;
  group_wait_kernel<<<1, 128, 0, (cudaStream_t)stream>>>(asks != 0, late, step, steps, part,
                                                         limit_cycles, left, status);
  count_launches(1);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
