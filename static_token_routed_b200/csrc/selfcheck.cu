// Check of the bounded-wait machinery every kernel relies on: a CTA waits on
// an mbarrier that nothing will ever complete, with the same bounded wait
// the kernels use. The wait must give up after its time limit, raise the
// CTA's abort flag, report DEV_ERR_TIMEOUT in global memory and return, so
// that the launch ends normally and the context stays usable. No trap, no
// fault, no unbounded loop: the only way this kernel ends is the time limit.
// Then the launch that turns a chain's results into NaN when its kernels gave up:
// of two spans, all of them and nothing beside them; before, with the word clear,
// nothing at all.
#include "l3_internal.cuh"
#include "sm100.cuh"

namespace l3 {
namespace {

__global__ void k_wait_never_completes(int *err) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    sm100::mbar_init(&bar, 1);  // one arrival expected; nobody arrives
    abort_flag = 0;
    sm100::fence_mbar_init();
  }
  __syncthreads();
  const sm100::Abort ab{&abort_flag, err};
  if (threadIdx.x == 0 && sm100::mbar_wait(&bar, 0, ab)) atomicOr(err, 1 << 30);  // cannot happen
}

}  // namespace
}  // namespace l3

using namespace l3;

extern "C" l3_status l3_check_bounded_wait(void *stream) {
  set_error("");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  constexpr int N = 9000;  // 16-bit words, of which two spans
  int *err = nullptr;
  L3_CUDA_TRY(cudaMalloc(&err, sizeof(int) + 2 * N));
  uint16_t *words = reinterpret_cast<uint16_t *>(err + 1);
  l3_status st = L3_OK;
  int host = 0;
  uint16_t clear[N], spoilt[N];
  const Spoilt a{words + 3, 2 * (4200 - 3)}, b{words + 4201, 2 * (N - 4 - 4201)};
  cudaError_t e = cudaMemsetAsync(err, 0, sizeof(int) + 2 * N, s);
  if (e == cudaSuccess) st = launch_spoil(err, a, b, s);
  if (e == cudaSuccess && st == L3_OK)
    e = cudaMemcpyAsync(clear, words, 2 * N, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess && st == L3_OK) {
    k_wait_never_completes<<<1, 32, 0, s>>>(err);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && st == L3_OK) st = launch_spoil(err, a, b, s);
  if (e == cudaSuccess && st == L3_OK)
    e = cudaMemcpyAsync(spoilt, words, 2 * N, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess && st == L3_OK) e = cudaMemcpyAsync(&host, err, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  cudaFree(err);
  if (e != cudaSuccess) return cuda_fail(e, "l3_check_bounded_wait");
  if (st != L3_OK) return st;
  for (int i = 0; i < N; ++i) {
    const bool in = (i >= 3 && i < 4200) || (i >= 4201 && i < N - 4);
    if (clear[i] != 0 || spoilt[i] != (in ? 0x7fff : 0)) {
      set_error("results of kernels that gave up were not turned into NaN as they should");
      return L3_ERR_CUDA;
    }
  }
  if (host == DEV_ERR_TIMEOUT) {
    set_error("the bounded wait gave up as it should");
    st = L3_ERR_TIMEOUT;
  } else {
    set_error("the bounded wait did not report its give-up");
    st = L3_ERR_CUDA;
  }
  return st;
}
