// Shared by the forms of the orthogonalised update (muon.cu: tiles of any matrix;
// muon_small.cu and muon_tiny.cu: a small matrix in one launch): the polynomial, the
// scales of what is stored, the update U and hi + lo pairs.
#pragma once

#include <cuda_fp16.h>

#include "l3_internal.cuh"

namespace l3 {
namespace muon {

constexpr float NS_A = 3.4445f, NS_B = -4.7750f, NS_C = 2.0315f;
// X, A and B are stored times 2^SX, 2^SA and 2^SB. The largest magnitudes:
// the polynomial keeps singular values s in [0, 1.22], so |X_ij| <= s_max
// <= 1.22 (39978 stored), |A_ij| <= 1.5 (24576), and a + b t + c t^2 over t = s^2
// in [0, 1.5] lies in [0.63, 3.4445] (56435), all below fp16's 65504
constexpr int SX = 15, SA = 14, SB = 14;

struct UpdateParams {
  const void *g;  // [batch][rows][cols], fp32 or bf16
  float *mom;     // momentum (fp32) or NULL: U = G
  float mu;
  int nesterov;
  int64_t size;   // rows * cols
  int rows, cols;
  int vec;        // every matrix starts 16-byte aligned in G, M and the output

  // U of a new momentum and its gradient
  __device__ __forceinline__ float update(float m, float grad) const {
    return nesterov ? fmaf(mu, m, grad) : m;
  }
};


// four elements, aligned to their size
__device__ __forceinline__ float4 load_el4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load_el4(const __nv_bfloat16 *p) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.x)),
               b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_el4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store_el4(__nv_bfloat16 *p, float4 v) {
  __nv_bfloat162 b[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
  *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(b);
}
template <class T>
__device__ __forceinline__ float load_el(const T *p) {
  return sizeof(T) == 4 ? *reinterpret_cast<const float *>(p)
                        : __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p));
}
template <class T>
__device__ __forceinline__ void store_el(T *p, float v) {
  if (sizeof(T) == 4)
    *reinterpret_cast<float *>(p) = v;
  else
    *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(v);
}

// U's element i once M holds the new momentum
template <class T, bool MOM>
__device__ __forceinline__ float update_at(const UpdateParams &P, int64_t i) {
  if (!MOM) return load_el(static_cast<const T *>(P.g) + i);
  return P.nesterov ? P.update(P.mom[i], load_el(static_cast<const T *>(P.g) + i)) : P.mom[i];
}

__device__ __forceinline__ void split2(float v, __half &hi, __half &lo) {
  hi = __float2half_rn(v);
  lo = __float2half_rn(v - __half2float(hi));
}
// 2^exp / norm as the product of two floats, neither out of range (a zero norm
// gives zero: a zero update with eps = 0 stays zero)
__device__ __forceinline__ void scale_factors(double norm, int exp, float &f0, float &f1) {
  f0 = f1 = 0.f;
  if (norm == 0.0) return;
  const int k = norm < INFINITY ? ilogb(norm) : 0;
  f1 = ldexpf(1.f, (exp - k) / 2);
  f0 = (float)(ldexp(1.0, k) / norm) * ldexpf(1.f, exp - k - (exp - k) / 2);
}
// two at once, on the packed conversions
__device__ __forceinline__ void split2(float a, float b, __half2 &hi, __half2 &lo) {
  hi = __floats2half2_rn(a, b);
  const float2 f = __half22float2(hi);
  lo = __floats2half2_rn(a - f.x, b - f.y);
}
// eight fp32 values as hi + lo halves, 16 bytes each
__device__ __forceinline__ void pack_pair(const float (&f)[8], uint4 &hi, uint4 &lo) {
  __half2 *h2 = reinterpret_cast<__half2 *>(&hi), *l2 = reinterpret_cast<__half2 *>(&lo);
#pragma unroll
  for (int e = 0; e < 4; ++e) split2(f[2 * e], f[2 * e + 1], h2[e], l2[e]);
}
__device__ __forceinline__ void unpack_pair(uint4 hi, uint4 lo, float (&f)[8]) {
  const __half2 *h2 = reinterpret_cast<const __half2 *>(&hi), *l2 = reinterpret_cast<const __half2 *>(&lo);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = __half22float2(h2[e]), c = __half22float2(l2[e]);
    f[2 * e] = a.x + c.x;
    f[2 * e + 1] = a.y + c.y;
  }
}

struct Target {
  void *out;      // O, or W
  bool fp32;      // its type
  bool keep_w;    // W <- keep W - rate O
  float keep, rate;
};

// whether clusters of `ctas` such CTAs fit the device, asked once (known: 0 before,
// then 1 or -1)
template <class P>
bool clusters_fit(void (*kernel)(P), int ctas, int threads, size_t smem, int &known) {
  if (known == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
    if (!ok) cudaGetLastError();
    known = ok ? 1 : -1;
  }
  return known > 0;
}

// muon_tiny.cu
bool tiny_supported(int64_t m, int steps);
l3_status launch_tiny(const UpdateParams &u, bool g_fp32, int64_t batch, int steps, float eps,
                      const Target &t, int *err, int device, cudaStream_t s);

// muon_small.cu
bool small_always(int64_t m, int64_t n);  // on any device
bool small_supported(int64_t m, int64_t n, int device);
l3_status launch_small(const UpdateParams &u, bool g_fp32, int64_t batch, int steps, float eps,
                       const Target &t, int *err, int device, cudaStream_t s);

}  // namespace muon
}  // namespace l3
