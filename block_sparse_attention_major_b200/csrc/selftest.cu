// Self-tests of the kernels' bounded waits.
//
// The self-attention's: one warp waits, with the same bounded mbarrier
// wait the attention kernel uses, on a barrier that nothing arrives on. The wait gives up
// after `limit` SM cycles, sets the time-out bit of the error word and returns, so a lost
// arrival surfaces to the caller while the CUDA context stays usable.
//
// The cross attention's: half the warps of a group wait on such a barrier, with the wait of its
// kernels and far fewer tries, the others on one that is complete; then all leave by the vote with
// which the group's warps leave together.
#include "cross.cuh"

namespace bsa {
namespace {

__global__ void __launch_bounds__(32) wait_selftest_kernel(long long limit, uint32_t* err) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_u32(&bar), 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  __syncwarp();
  if (threadIdx.x == 0) ptx::mbar_wait(ptx::smem_u32(&bar), 0, &abort_flag, err, limit);
}

__global__ void __launch_bounds__(256) cross_wait_selftest_kernel(uint32_t* err) {
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ int abort_flag;
  const uint32_t lost = ptx::smem_u32(&bars[0]), done = ptx::smem_u32(&bars[1]);
  if (threadIdx.x == 0) {
    ptx::mbar_init(lost, 1);
    ptx::mbar_init(done, 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::mbar_arrive(done);
  }
  __syncthreads();
  const bool ok = cross::warp_wait<1 << 12>((threadIdx.x >> 5) & 1 ? done : lost, 0, &abort_flag, err);
  if (cross::bar_all(1, 256, ok)) report_error(err, BSA_KERR_BAD_UNIT);
}

}  // namespace

cudaError_t launch_cross_wait_selftest(uint32_t* err, cudaStream_t s) {
  cross_wait_selftest_kernel<<<1, 256, 0, s>>>(err);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_wait_selftest(long long limit_cycles, uint32_t* err, cudaStream_t s) {
  wait_selftest_kernel<<<1, 32, 0, s>>>(limit_cycles, err);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace bsa
