// What becomes of the loss's gradients and the update when a wait in their kernels gave
// up: NaN, so that a step that went wrong does not pass for one that went right,
// whoever holds the workspace with the error word. (The loss itself turns into NaN in
// its join.) One launch behind the chain, since the chain's last kernel may be the
// one that gives up: it starts beside that kernel, looks at the word when it has
// ended, and writes only where it is set. About 2 us.
#include "gemm_pair.cuh"

namespace l3 {
namespace {

// 0x7fff is a NaN in bf16 and, twice, in fp32
__device__ void spoil(const Spoilt &s) {
  uint16_t *p = static_cast<uint16_t *>(s.p);
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < s.bytes / 2; i += stride) p[i] = 0x7fff;
}

__global__ void k_spoil(const int *err, Spoilt a, Spoilt b) {
  pairgemm::pdl_wait();
  if (*err == 0) return;
  spoil(a);
  spoil(b);
}

}  // namespace

l3_status launch_spoil(const int *err, const Spoilt &a, const Spoilt &b, cudaStream_t s) {
  LaunchTimer t("spoil", s);
  return pairgemm::launch_link(k_spoil, dim3(16), dim3(256), s, true, err, a, b);
}

}  // namespace l3
