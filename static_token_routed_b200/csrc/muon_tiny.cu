// The whole orthogonalised update of a matrix of few rows in one launch: m <= 32,
// any n, up to 8 steps, a cluster of 1 to 16 CTAs per matrix.
//
// The steps multiply X from the left by polynomials of its own Gram matrix, so
// with A = X X^T of the first X they come down to m x m matrices that commute:
//     B = a I + b A + c A A,   Q <- B Q,   A <- A B B,   and X = Q X_0 at the end.
// X is read once for A and once for Q X_0, nothing between leaves an SM. Rounding
// in the first A grows with the square of what small singular values grow by,
// 11.9-fold a step, so A, B and Q are held in 64 bits, where eight steps leave
// 2^-52 11.9^8 = 9e-8 (more steps take muon_small.cu's way). U's products are
// exact there: the result is off by its own rounding, whatever the spectrum.
//
// The products are the 64-bit matrix instructions (8 x 8 x 4; the tcgen05 ones know
// no such type): a symmetric product's transposed operand is the same registers as
// the other one. Bound by latency (the kernel alone; a call from Python takes 14 us
// of host time): 4 x 1000 takes 6.6 us, 16 x 2000 10.8, 32 x 1000
// 22 (muon_small.cu, with three products of X a step on fewer bits, 72, 78 and
// 77); a step of 32 rows is 4 products of 16 tiles, 512 instructions at about 11
// clocks an SM, 3 us (in one chain a tile or in four), and 8 times that at 64.
// 1024 of 32 x 512, one CTA each: 199 us (clusters of four, which repeat the steps,
// 968; muon_small.cu 982).
#include <algorithm>

#include "muon_common.cuh"
#include "sm100.cuh"

namespace l3 {
namespace {

using namespace sm100;
using namespace muon;

constexpr int THREADS = 256;       // a column of X each
constexpr int PITCH = THREADS + 16;  // of X's rows in shared memory: 16-byte reads of 8 rows apart

struct Params {
  UpdateParams u;
  float eps;
  int m, n, steps;
  int span;  // columns of a CTA
  void *out;  // O, or W
  float keep, rate;
  int *err;
};

constexpr int smem_bytes(int mp) {
  return mp * PITCH * (int)sizeof(float) + 3 * mp * (mp + 4) * (int)sizeof(double);
}

__device__ __forceinline__ void mma_f64(double (&d)[2], double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
               : "+d"(d[0]), "+d"(d[1])
               : "d"(a), "d"(b));
}

// Tiles of the product of two symmetric MP x MP matrices that commute (so that rows
// serve as columns), 8 x 8 each, row-block by row-block over the warps: f(row,
// column, value)
template <int MP, class F>
__device__ __forceinline__ void product(const double *a, const double *b, int warp, int lane, F f) {
  constexpr int RG = MP / 8, WARPS = THREADS / 32, EACH = (RG * RG + WARPS - 1) / WARPS, LD = MP + 4;
  if (RG * RG < WARPS && warp >= RG * RG) return;
  const int i = warp * EACH / RG, j0 = warp * EACH % RG;  // EACH divides RG
  const double *pa = a + (i * 8 + lane / 4) * LD + lane % 4, *pb = b + (j0 * 8 + lane / 4) * LD + lane % 4;
  double d[EACH][2] = {};
#pragma unroll
  for (int k = 0; k < MP; k += 4)
#pragma unroll
    for (int e = 0; e < EACH; ++e) mma_f64(d[e], pa[k], pb[e * 8 * LD + k]);
#pragma unroll
  for (int e = 0; e < EACH; ++e)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      f(i * 8 + lane / 4, (j0 + e) * 8 + lane % 4 * 2 + h, d[e][h]);
}

template <int MP, class TG, bool MOM, class TO, bool KEEP, bool TALL>
__global__ void __launch_bounds__(THREADS) k_muon_tiny(const __grid_constant__ Params P) {
  constexpr int MM = MP * MP, LD = MP + 4;  // LD: no two of 4 x 4 in one bank
  constexpr int RG = MP / 8, TILES = RG * (RG + 1) / 2;
  extern __shared__ uint4 smem[];
  float *x = reinterpret_cast<float *>(smem);  // a block of X's columns; later partial sums
  double *sA = reinterpret_cast<double *>(x + MP * PITCH), *sB = sA + MP * LD, *sQ = sB + MP * LD;
  static_assert(MP * PITCH * sizeof(float) >= 4 * TILES * 64 * sizeof(double), "partial sums of four warps");
  static_assert(MP * PITCH * sizeof(float) >= 2 * MP * LD * sizeof(double), "T and a Q");
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int n_ctas = gridDim.x, rank = (int)cluster_ctarank();
  const int64_t base = (int64_t)blockIdx.y * P.u.size;
  const int m = P.m, begin = rank * P.span, end = min(P.n, begin + P.span);
  if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) *P.err = 0;
  const auto index = [&](int r, int c) -> int64_t {
    return TALL ? base + (int64_t)c * P.u.cols + r : base + (int64_t)r * P.u.cols + c;
  };
  // U's elements at(k), k < MP, that in(k) says are there, else 0; first: the
  // momentum's turn. All loads are on their way before the first store.
  const auto elements = [&](float (&w)[MP], bool first, auto at, auto in) {
    float mom[MOM ? MP : 1];
#pragma unroll
    for (int k = 0; k < MP; ++k) {
      w[k] = in(k) ? load_el(static_cast<const TG *>(P.u.g) + at(k)) : 0.f;
      if (MOM) mom[MOM ? k : 0] = in(k) ? P.u.mom[at(k)] : 0.f;
    }
    if (MOM)
#pragma unroll
      for (int k = 0; k < MP; ++k) {
        float &v = mom[MOM ? k : 0];
        if (first) v = fmaf(P.u.mu, v, w[k]);
        if (first && in(k)) P.u.mom[at(k)] = v;
        w[k] = P.u.update(v, w[k]);
      }
  };
  // A thread's column of the block from c0, of nb columns, in registers and in x,
  // zeros past m and nb. A tall U's block is one run of memory.
  float u[MP];
  const auto load = [&](int c0, int nb, bool first) {
    if (!TALL) {
      elements(u, first, [&](int r) { return index(r, c0 + tid); }, [&](int r) { return r < m && tid < nb; });
#pragma unroll
      for (int r = 0; r < MP; ++r) x[r * PITCH + tid] = u[r];
    } else {
      int r = tid % m, c = tid / m;
      const int dr = THREADS % m, dc = THREADS / m;
      float w[MP];
      elements(w, first, [&](int k) { return index(0, c0) + tid + k * THREADS; },
               [&](int k) { return k < m && tid + k * THREADS < nb * m; });
#pragma unroll
      for (int k = 0; k < MP; ++k) {
        if (k >= m) break;
        x[r * PITCH + c] = w[k];
        r += dr, c += dc;
        if (r >= m) r -= m, ++c;
      }
#pragma unroll
      for (int k = 0; k < MP; ++k)
        if (k >= m) x[k * PITCH + tid] = 0.f;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < MP; ++k) u[k] = x[k * PITCH + tid];
    }
  };

  // U U^T: a warp's 32 columns of each block, then the warps' sums, then the CTAs'
  double acc[TILES][2] = {};
  const int blocks = max(0, (end - begin + THREADS - 1) / THREADS);
  for (int b = 0; b < blocks; ++b) {
    const int c0 = begin + b * THREADS;
    if (b) __syncthreads();
    load(c0, min(THREADS, end - c0), true);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      double a[RG][4];  // row lane / 4 of each 8; four k-steps, whose order is free
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        const float4 v = *reinterpret_cast<const float4 *>(
            &x[(g * 8 + lane / 4) * PITCH + warp * 32 + h * 16 + lane % 4 * 4]);
        a[g][0] = v.x, a[g][1] = v.y, a[g][2] = v.z, a[g][3] = v.w;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0, t = 0; i < RG; ++i)
#pragma unroll
          for (int j = 0; j <= i; ++j, ++t) mma_f64(acc[t], a[i][k], a[j][k]);
    }
  }
  double *part = reinterpret_cast<double *>(x);
#pragma unroll
  for (int w = 4; w >= 1; w /= 2) {
    __syncthreads();
    if (warp >= w && warp < 2 * w)
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        part[(((warp - w) * TILES + t) * 2) * 32 + lane] = acc[t][0];
        part[(((warp - w) * TILES + t) * 2 + 1) * 32 + lane] = acc[t][1];
      }
    __syncthreads();
    if (warp < w)
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        acc[t][0] += part[((warp * TILES + t) * 2) * 32 + lane];
        acc[t][1] += part[((warp * TILES + t) * 2 + 1) * 32 + lane];
      }
  }
  if (warp == 0) {
#pragma unroll
    for (int i = 0, t = 0; i < RG; ++i)
#pragma unroll
      for (int j = 0; j <= i; ++j, ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = i * 8 + lane / 4, c = j * 8 + lane % 4 * 2 + e;
          sB[r * LD + c] = acc[t][e];
          sB[c * LD + r] = acc[t][e];
        }
  }
  __syncthreads();
  if (n_ctas > 1) cluster_sync();
  for (int e = tid; e < MM; e += THREADS) {
    const int at = e / MP * LD + e % MP;
    double sum = 0.0;
    if (n_ctas == 1) {
      sum = sB[at];
    } else {
#pragma unroll 4
      for (int r = 0; r < n_ctas; ++r) {
        double v;
        asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(map_shared_rank(&sB[at], r)) : "memory");
        sum += v;
      }
    }
    sA[at] = sum;
  }
  __syncthreads();
  if (n_ctas > 1) cluster_sync();  // sB has been read by all

  // 1 / norm into A; an infinity or a NaN makes all of its matrix NaN
  double trace = 0.0;
  for (int i = 0; i < m; ++i) trace += sA[i * LD + i];
  const double norm = sqrt(trace) + (double)P.eps;
  const double inv = !(trace < INFINITY) ? (double)__int_as_float(0x7fffffff) : norm > 0.0 ? 1.0 / norm : 0.0;
  __syncthreads();
  // T and one of two Qs lie where X's columns were
  double *sT = reinterpret_cast<double *>(x), *q = sT + MP * LD, *q_next = sQ;
  if (P.steps % 2 == 0) q = sQ, q_next = sT + MP * LD;  // so that the last is sQ
  for (int at = tid; at < MM; at += THREADS) {
    const int i = at / MP, j = at % MP;
    sA[i * LD + j] *= inv * inv;
    q[i * LD + j] = i == j ? inv : 0.0;  // 1 / norm with it
  }
  __syncthreads();
#pragma unroll 1
  for (int step = 1;; ++step) {
    product<MP>(sA, sA, warp, lane, [&](int i, int j, double v) {
      sB[i * LD + j] = fma(2.0315, v, fma(-4.7750, sA[i * LD + j], i == j ? 3.4445 : 0.0));
    });
    __syncthreads();
    product<MP>(sB, q, warp, lane, [&](int i, int j, double v) { q_next[i * LD + j] = v; });
    if (step == P.steps) break;
    product<MP>(sA, sB, warp, lane, [&](int i, int j, double v) { sT[i * LD + j] = v; });
    __syncthreads();
    product<MP>(sT, sB, warp, lane, [&](int i, int j, double v) { sA[i * LD + j] = v; });
    __syncthreads();
    double *was = q;
    q = q_next;
    q_next = was;
  }
  __syncthreads();

  // O = Q U, the last block's columns from registers, through shared memory into
  // the caller's order
  TO *out = static_cast<TO *>(P.out);
  for (int b = blocks - 1; b >= 0; --b) {
    const int c0 = begin + b * THREADS, nb = min(THREADS, end - c0);
    if (b + 1 < blocks) {
      __syncthreads();
      load(c0, nb, false);
    }
    if (TALL) __syncthreads();
    double v[MP];
#pragma unroll
    for (int k = 0; k < MP; ++k) v[k] = u[k];
#pragma unroll 1
    for (int r = 0; r < m; r += 2) {  // two chains (MP is even)
      double s0 = 0.0, s1 = 0.0;
#pragma unroll
      for (int k = 0; k < MP; ++k) {
        s0 = fma(sQ[r * LD + k], v[k], s0);
        s1 = fma(sQ[(r + 1) * LD + k], v[k], s1);
      }
      x[r * PITCH + tid] = (float)s0;
      x[(r + 1) * PITCH + tid] = (float)s1;
    }
    if (TALL) __syncthreads();
    // a thread's elements, eight at a time: its column, or every THREADS-th of the run
    int r = TALL ? tid % m : 0, c = TALL ? tid / m : tid;
    const int dr = TALL ? THREADS % m : 1, dc = TALL ? THREADS / m : 0;
    const int count = TALL ? (nb * m - tid + THREADS - 1) / THREADS : tid < nb ? m : 0;
    TO *to = out + (TALL ? index(0, c0) + tid : index(0, c0 + tid));
    const int64_t stride = TALL ? THREADS : P.u.cols;
    for (int k0 = 0; k0 < count; k0 += 8) {
      float w[8];
      if (KEEP)
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = k0 + k < count ? load_el(to + (k0 + k) * stride) : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k0 + k >= count) break;
        const float o = x[r * PITCH + c];
        store_el(to + (k0 + k) * stride, KEEP ? fmaf(-P.rate, o, P.keep * w[k]) : o);
        r += dr, c += dc;
        if (TALL && r >= m) r -= m, ++c;
      }
    }
  }
}

template <int MP, class TG, bool MOM, class TO, bool KEEP, bool TALL>
l3_status launch_as(const Params &P, int ctas, int64_t batch, int device, cudaStream_t s) {
  const auto kernel = k_muon_tiny<MP, TG, MOM, TO, KEEP, TALL>;
  constexpr int SMEM = smem_bytes(MP);
  static bool attr[64] = {};
  if (!attr[device & 63]) {
    L3_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM));
    L3_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    attr[device & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)batch, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  L3_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, P));
  return L3_OK;
}

template <class TG, bool MOM, class TO, bool KEEP, bool TALL>
l3_status launch_rows(const Params &P, int ctas, int64_t batch, int device, cudaStream_t s) {
  return P.m <= 8    ? launch_as<8, TG, MOM, TO, KEEP, TALL>(P, ctas, batch, device, s)
         : P.m <= 16 ? launch_as<16, TG, MOM, TO, KEEP, TALL>(P, ctas, batch, device, s)
                     : launch_as<32, TG, MOM, TO, KEEP, TALL>(P, ctas, batch, device, s);
}

template <class TG, bool MOM, class TO, bool KEEP>
l3_status launch(const Params &P, int ctas, int64_t batch, int device, cudaStream_t s) {
  return P.u.rows > P.u.cols ? launch_rows<TG, MOM, TO, KEEP, true>(P, ctas, batch, device, s)
                             : launch_rows<TG, MOM, TO, KEEP, false>(P, ctas, batch, device, s);
}

}  // namespace

namespace muon {

bool tiny_supported(int64_t m, int steps) { return m <= 32 && steps <= 8; }

l3_status launch_tiny(const UpdateParams &u, bool g_fp32, int64_t batch, int steps, float eps,
                      const Target &t, int *err, int device, cudaStream_t s) {
  Params P = {};
  P.u = u;
  P.eps = eps;
  P.m = std::min(u.rows, u.cols);
  P.n = std::max(u.rows, u.cols);
  P.steps = steps;
  P.out = t.out;
  P.keep = t.keep;
  P.rate = t.rate;
  P.err = err;
  // A block of columns each, while the cluster and the SMs last: each CTA goes
  // through the steps by itself (16 x 2000: 8 of them 10.7 us, 16 of half a block
  // 12.7; 32 x 4096: 8 of two blocks 35.3, 16 of one 27.2)
  static int known[64] = {};
  const int most = clusters_fit(k_muon_tiny<32, float, false, float, false, false>, 16, THREADS,
                                smem_bytes(32), known[device & 63]) ? 16 : 8;
  int ctas = 1;
  while (ctas < most && ctas * THREADS < P.n && 2 * ctas * batch <= 148) ctas *= 2;
  P.span = (P.n + ctas - 1) / ctas;
  LaunchTimer lt("muon_tiny", s);
  if (t.keep_w)
    return t.fp32 ? launch<float, true, float, true>(P, ctas, batch, device, s)
                  : launch<float, true, __nv_bfloat16, true>(P, ctas, batch, device, s);
  return g_fp32 ? launch<float, false, float, false>(P, ctas, batch, device, s)
                : launch<__nv_bfloat16, false, __nv_bfloat16, false>(P, ctas, batch, device, s);
}

}  // namespace muon
}  // namespace l3
