// The whole orthogonalised update of a small matrix in one launch: m <= 128
// rows of X (up to 32 of them and 8 steps: muon_tiny.cu), n <= 4096 columns (2048
// where the device has no room for clusters of 16), a cluster of 1 to 16 CTAs per
// matrix.
//
// A CTA keeps 256 columns of X as hi + lo fp16 planes in shared memory through
// all steps, in the 128-byte-swizzled layout that serves X both as the K-major
// operand of X X^T and as the MN-major operand of B X. Each CTA's X X^T is a
// partial sum over its columns; the cluster adds them up through distributed
// shared memory (each CTA a slice of rows, then everyone copies the sum), and
// every CTA goes on with the same A: A A on its own tensor core, B in A's
// place, B X on its own columns. Only U is read and O (or M and W) written.
//
// Such a matrix's fifteen products are bound by latency, not by bytes or
// operations: as launches of the tile kernel 64 x 64, 128 x 256 and 128 x 4096 take
// 90, 124 and 188 us, here 37, 66 and 106. A step of 128 x 256 is 16 thousand clocks,
// 9.5 of them MMAs (a 128 x 128 x 16 one about 87), the rest three passes over an
// accumulator; a cluster's exchange of A adds 7 to 10.
#include <algorithm>
#include <type_traits>

#include "muon_common.cuh"
#include "sm100.cuh"

namespace l3 {
namespace {

using namespace sm100;
using namespace muon;

constexpr int ROWS = 128;   // of X, zeros past m
constexpr int SLAB = 256;   // columns of X per CTA
constexpr int THREADS = 512;
constexpr int MAX_CLUSTER = 16;
constexpr int BLOCK = ROWS * 128;                 // 128 rows x 64 halves
constexpr int X_PLANE = SLAB / 64 * BLOCK;        // 64 KB
constexpr int A_PLANE = ROWS / 64 * BLOCK;        // 32 KB
constexpr int OFF_A = 2 * X_PLANE;                // A, then B; also the partial sums, fp32
constexpr int OFF_TAIL = OFF_A + 2 * A_PLANE;

struct Tail {
  uint64_t done;           // a product has completed
  uint64_t drain;
  double part[THREADS / 32];
  double sum[MAX_CLUSTER];  // every CTA's sum of squares
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t SMEM = 1024 + OFF_TAIL + sizeof(Tail);
static_assert(SMEM <= 232448, "shared memory");

// byte offset of half (r, c) of a plane: 64-column blocks, 128-byte rows,
// 16-byte pieces swizzled by the row
__device__ __forceinline__ int at(int r, int c) {
  return (c >> 6) * BLOCK + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4) + (c & 7) * 2;
}

// one thread: D = the products lo hi, hi lo, hi hi over the 16-deep steps k0 .. k1 - 1:
// A K-major planes at a0 (stride ap), B K-major or MN-major at b0
template <bool B_MN>
__device__ __forceinline__ void products(uint32_t d, uint32_t a0, int ap, uint32_t b0, int bp,
                                         int k0, int k1, uint32_t idesc) {
  bool add = false;
#pragma unroll 1
  for (int pr = 0; pr < 3; ++pr) {
    const uint32_t a = a0 + (pr == 0 ? ap : 0), b = b0 + (pr == 1 ? bp : 0);
#pragma unroll 4
    for (int k = k0; k < k1; ++k) {
      const uint32_t ko = (k >> 2) * BLOCK + (k & 3) * 32;
      // MN-major: k is X's row, 16 of them 2 KB apart; 64-column blocks BLOCK apart
      umma_f16(d, sdesc_sw128(a + ko, 16, 1024),
               B_MN ? sdesc_sw128(b + k * 2048, BLOCK, 1024) : sdesc_sw128(b + ko, 16, 1024), idesc,
               add);
      add = true;
    }
  }
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

struct Params {
  UpdateParams u;
  float eps;
  int m, n, steps;
  void *out;  // O, or W
  float keep, rate;
  int *err;
};

// 16-byte piece p (of 32) of row r of the fp32 partial sums
__device__ __forceinline__ int partial_at(int r, int p) { return r * 512 + ((p ^ (r & 31)) << 4); }

// The rank-th of CL groups of the first R rows and columns of the cluster's partial
// sums added up in CTA order, left where this CTA's own partial was. Up to eight
// loads a thread, all on their way at once.
template <int CL, int R>
__device__ __forceinline__ void add_up(uint8_t *sm, int rank, int tid) {
  constexpr int PIECES = R / CL * (R / 4), EACH = (PIECES + THREADS - 1) / THREADS;
  if (EACH * THREADS > PIECES && tid >= PIECES) return;
  float4 w[EACH][CL];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int i = tid + e * THREADS;
    const uint8_t *at = sm + OFF_A + partial_at(rank * (R / CL) + i / (R / 4), i % (R / 4));
#pragma unroll
    for (int r = 0; r < CL; ++r) w[e][r] = ld_cluster4(map_shared_rank(at, r));
  }
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    float4 a = w[e][0];
#pragma unroll
    for (int r = 1; r < CL; ++r) a.x += w[e][r].x, a.y += w[e][r].y, a.z += w[e][r].z, a.w += w[e][r].w;
    const int i = tid + e * THREADS;
    // read by nobody else before the next barrier
    *reinterpret_cast<float4 *>(sm + OFF_A + partial_at(rank * (R / CL) + i / (R / 4), i % (R / 4))) = a;
  }
}

template <class TG, bool MOM, class TO, bool KEEP, bool TALL>
__global__ void __launch_bounds__(THREADS, 1) k_muon_small(const __grid_constant__ Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~uintptr_t(1023));
  Tail *t = reinterpret_cast<Tail *>(sm + OFF_TAIL);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int n_ctas = gridDim.x;  // of the cluster, which is a matrix's grid row
  const int rank = (int)cluster_ctarank();
  const int c0 = rank * SLAB;
  const int64_t base = (int64_t)blockIdx.y * P.u.size;
  if (tid == 0) {
    mbar_init(&t->done, 1);
    mbar_init(&t->drain, 1);
    t->abort_flag = 0;
    fence_mbar_init();
    if (blockIdx.x == 0 && blockIdx.y == 0) *P.err = 0;
  }
  if (warp == 0) {
    tmem_alloc(&t->tmem_base, 512);
    tmem_relinquish();
  }

  // this CTA's part of U: columns c0 .. of X. The momentum is updated once,
  // by the CTA that owns the column.
  const int nc = max(0, min(SLAB, P.n - c0));  // real columns
  const int inner = TALL ? P.m : nc;           // contiguous direction
  const int outer = TALL ? nc : P.m;
  const auto index = [&](int o, int i) -> int64_t {
    return TALL ? base + (int64_t)(c0 + o) * P.u.cols + i : base + (int64_t)o * P.u.cols + c0 + i;
  };
  // A thread's 64 elements, sixteen runs of four, stay in registers from here
  // to the planes, their loads all on the way before the first is used (the
  // momentum's, then the gradient's in two halves). Where rows start aligned
  // for it, a run is four neighbours and one access, else four accesses of
  // which each is coalesced over the warp.
  constexpr int LINE = TALL ? ROWS : SLAB, RUNS = 16, PER_LINE = LINE / 128;
  const bool vec = P.u.vec && P.u.cols % 4 == 0;
  const int lane0 = vec ? lane * 4 : lane, lane_step = vec ? 1 : 32;
  const auto place = [&](int x, int &o, int &i) {  // line and first element of run x
    o = warp + x / PER_LINE * (THREADS / 32);
    i = lane0 + x % PER_LINE * 128;
    return o < outer;
  };
  const auto load = [&](const auto *from, int x) {
    int o, i;
    const bool in = place(x, o, i);
    const auto *p = from + index(o, i);
    if (vec) return in && i < inner ? load_el4(p) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(in && i < inner ? load_el(p) : 0.f, in && i + 32 < inner ? load_el(p + 32) : 0.f,
                       in && i + 64 < inner ? load_el(p + 64) : 0.f,
                       in && i + 96 < inner ? load_el(p + 96) : 0.f);
  };
  alignas(16) float u[4 * RUNS];
  if (MOM)
#pragma unroll
    for (int x = 0; x < RUNS; ++x)
      *reinterpret_cast<float4 *>(u + 4 * x) = load(const_cast<const float *>(P.u.mom), x);
  constexpr int GROUP = MOM ? RUNS / 2 : RUNS;
#pragma unroll
  for (int x0 = 0; x0 < RUNS; x0 += GROUP) {
    float4 g[GROUP];
#pragma unroll
    for (int x = 0; x < GROUP; ++x) g[x] = load(static_cast<const TG *>(P.u.g), x0 + x);
#pragma unroll
    for (int x = 0; x < GROUP; ++x) {
      float *w = u + 4 * (x0 + x);
      if (MOM) {
        const float4 m = make_float4(fmaf(P.u.mu, w[0], g[x].x), fmaf(P.u.mu, w[1], g[x].y),
                                     fmaf(P.u.mu, w[2], g[x].z), fmaf(P.u.mu, w[3], g[x].w));
        int o, i;
        const bool in = place(x0 + x, o, i);
        float *p = P.u.mom + index(o, i);
        if (vec) {
          if (in && i < inner) store_el4(p, m);
        } else {
          if (in && i < inner) p[0] = m.x;
          if (in && i + 32 < inner) p[32] = m.y;
          if (in && i + 64 < inner) p[64] = m.z;
          if (in && i + 96 < inner) p[96] = m.w;
        }
        w[0] = P.u.update(m.x, g[x].x), w[1] = P.u.update(m.y, g[x].y);
        w[2] = P.u.update(m.z, g[x].z), w[3] = P.u.update(m.w, g[x].w);
      } else {
        w[0] = g[x].x, w[1] = g[x].y, w[2] = g[x].z, w[3] = g[x].w;
      }
    }
  }
  // squares in fp32 after a power of two that brings the thread's largest
  // element near one, so that none leaves the range
  float top = 0.f, sq = 0.f;
#pragma unroll
  for (int x = 0; x < 4 * RUNS; ++x) top = fmaxf(top, fabsf(u[x]));
  const int lift = top > 0.f && top < INFINITY ? -ilogbf(top) : 0;
  const float l0 = ldexpf(1.f, lift / 2), l1 = ldexpf(1.f, lift - lift / 2);
#pragma unroll
  for (int x = 0; x < 4 * RUNS; ++x) {
    const float w = u[x] * l0 * l1;
    sq = fmaf(w, w, sq);
  }
  double sum = ldexp((double)sq, -2 * lift);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) t->part[warp] = sum;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // every CTA has started: its shared memory may be written
  if (tid < n_ctas) {
    double s = 0.0;
    for (int w = 0; w < THREADS / 32; ++w) s += t->part[w];
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(map_shared_rank(&t->sum[rank], tid)),
                 "d"(s)
                 : "memory");
  }
  __syncwarp();
  cluster_sync();
  double total = 0.0;
  for (int r = 0; r < n_ctas; ++r) total += t->sum[r];
  const double root = sqrt(total), norm = root + (double)P.eps;
  int e = root > 0.0 && norm > root && norm < INFINITY ? ilogb(norm / root) : 0;
  float inv0, inv1;
  scale_factors(norm, SX + e, inv0, inv1);

  // X as planes, zeros past m and n
#pragma unroll
  for (int x = 0; x < RUNS; ++x) {
    int o, i;
    place(x, o, i);
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = u[4 * x + e] * inv1 * inv0;
    if (!TALL && vec) {
      __half2 hi[2], lo[2];
      split2(f[0], f[1], hi[0], lo[0]);
      split2(f[2], f[3], hi[1], lo[1]);
      *reinterpret_cast<uint2 *>(sm + at(o, i)) = *reinterpret_cast<uint2 *>(hi);
      *reinterpret_cast<uint2 *>(sm + X_PLANE + at(o, i)) = *reinterpret_cast<uint2 *>(lo);
      continue;
    }
    // four neighbours of a tall U lie in four rows of X: started from another
    // one by each lane, a warp's stores spread over all of the swizzled pieces
    const int turn = vec ? lane & 3 : 0;
    if (turn & 1) {
      const float f0 = f[0];
      f[0] = f[1], f[1] = f[2], f[2] = f[3], f[3] = f0;
    }
    if (turn & 2) {
      const float f0 = f[0], f1 = f[1];
      f[0] = f[2], f[1] = f[3], f[2] = f0, f[3] = f1;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int ie = i + (vec ? (e + turn & 3) : 32 * e);
      __half hi, lo;
      split2(f[e], hi, lo);
      const int off = TALL ? at(ie, o) : at(o, ie);
      *reinterpret_cast<__half *>(sm + off) = hi;
      *reinterpret_cast<__half *>(sm + X_PLANE + off) = lo;
    }
  }

  const uint32_t tmem = t->tmem_base, s0 = smem_u32(sm);
  const Abort ab{&t->abort_flag, P.err};
  const uint32_t D_A = tmem, D_X = tmem + 256;  // 128 columns each product of A, 256 of X
  constexpr bool FP32 = sizeof(TO) == 4;
  // a warp reads its lane quarter; four warps share a quarter's columns
  const int q = warp & 3, part = warp >> 2, row = q * 32 + lane;
  const uint32_t lane_off = (uint32_t)(q * 32) << 16;
  // the products' real sizes: 16-deep steps along this CTA's columns and along
  // m, and instruction shapes
  const int ks_x = (nc + 15) / 16, ks_a = (P.m + 15) / 16;
  const uint32_t id_a = idesc_f16(0, 0, ROWS, ks_a * 16), id_x = idesc_f16(0, 1, ROWS, max(ks_x, 1) * 16);
  // Rows and columns of A and B, and rows of X, past the last 16-deep step of m
  // reach nothing that is read. The warps' 32 x 32 of A and B that count, and
  // whether half of the rows hold all of the cluster's sum:
  const bool square = max(q, part) * 32 < ks_a * 16, half = ks_a * 16 <= ROWS / 2;
  uint32_t parity = 0;
  bool ok = true;
  // all threads: what the generic proxy wrote is there for the MMAs, which
  // thread 0 issues (chain(D, first step, end) for the halves of ks steps); then
  // all wait for them. The accumulator drops what does not fit its 24 bits, so an
  // fp32 result's sums are two chains of half the depth, added in registers
  // (131 x 77: 1.9e-6 -> 1.3e-6 off); the second one's columns are free by then.
  const auto run = [&](int ks, uint32_t d0, uint32_t d1, auto chain) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
      if (lane == 0) {
        const int half = FP32 ? (ks + 1) / 2 : ks;
        if (ks) chain(d0, 0, half);
        if (ks > half) chain(d1, half, ks);
        umma_commit(&t->done);
      }
      __syncwarp();  // the other lanes' waits would hold up the issue
    }
    ok = ok && mbar_wait(&t->done, parity, ab);
    __syncwarp();
    parity ^= 1;
    tc_fence_after();
  };
  // 32 columns of the sum
  const auto read = [&](int ks, uint32_t d0, uint32_t d1, uint32_t (&u)[32]) {
    tmem_ld32(d0 + lane_off, u);
    if (FP32 && ks > 1) {
      uint32_t w[32];
      tmem_ld32(d1 + lane_off, w);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) + __uint_as_float(w[i]));
    } else {
      tmem_wait_ld();
    }
  };

#pragma unroll 1
  for (int step = 0; step < P.steps; ++step) {
    // A's partial sum over this CTA's columns
    run(ks_x, D_A, D_A + 128, [&](uint32_t d, int k0, int k1) {
      products<false>(d, s0, X_PLANE, s0, X_PLANE, k0, k1, id_a);
    });
    float v[32];
    if (square) {
      uint32_t u[32];
      read(ks_x, D_A + part * 32, D_A + 128 + part * 32, u);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = ks_x && part * 32 + i < ks_a * 16 ? __uint_as_float(u[i]) : 0.f;
    }
    if (n_ctas > 1) {
      // partials to this CTA's shared memory (B's place: its products are done);
      // CTA r adds up the r-th group of rows in CTA order, leaves the sum where
      // its own partial was, and everyone copies it from there
      if (square)
#pragma unroll
        for (int p = 0; p < 8; ++p)
          *reinterpret_cast<float4 *>(sm + OFF_A + partial_at(row, part * 8 + p)) =
              make_float4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
      __syncwarp();
      cluster_sync();
      const auto sums = [&](auto rows) {
        switch (n_ctas) {
          case 2: add_up<2, rows.value>(sm, rank, tid); break;
          case 4: add_up<4, rows.value>(sm, rank, tid); break;
          case 8: add_up<8, rows.value>(sm, rank, tid); break;
          default: add_up<16, rows.value>(sm, rank, tid);
        }
      };
      if (half)
        sums(std::integral_constant<int, ROWS / 2>{});
      else
        sums(std::integral_constant<int, ROWS>{});
      __syncwarp();
      cluster_sync();
      // a row of sums at a time to a warp: distributed shared memory is as
      // fast as its accesses are contiguous (7 to 12 thousand clocks for 64 KB
      // with a row per lane)
      float4 w[ROWS / (THREADS / 32)];
#pragma unroll
      for (int k = 0; k < ROWS / (THREADS / 32); ++k) {
        const int r = warp + k * (THREADS / 32);
        w[k] = half && k >= ROWS / 2 / (THREADS / 32)
                   ? make_float4(0.f, 0.f, 0.f, 0.f)
                   : ld_cluster4(map_shared_rank(sm + OFF_A + partial_at(r, lane), (half ? 2 * r : r) * n_ctas / ROWS));
      }
      __half2 hi[ROWS / (THREADS / 32)][2], lo[ROWS / (THREADS / 32)][2];
#pragma unroll
      for (int k = 0; k < ROWS / (THREADS / 32); ++k) {
        constexpr float S = 1.f / (1 << (2 * SX - SA));
        split2(w[k].x * S, w[k].y * S, hi[k][0], lo[k][0]);
        split2(w[k].z * S, w[k].w * S, hi[k][1], lo[k][1]);
      }
      __syncwarp();
      cluster_sync();  // all have copied: the place is free for A
#pragma unroll
      for (int k = 0; k < ROWS / (THREADS / 32); ++k) {
        const int off = OFF_A + at(warp + k * (THREADS / 32), lane * 4);
        *reinterpret_cast<uint2 *>(sm + off) = *reinterpret_cast<uint2 *>(hi[k]);
        *reinterpret_cast<uint2 *>(sm + A_PLANE + off) = *reinterpret_cast<uint2 *>(lo[k]);
      }
    } else if (square) {
      // A in hi + lo, stored as an operand
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[p * 8 + i] * exp2f(SA - 2 * SX);
        uint4 hi, lo;
        pack_pair(f, hi, lo);
        const int off = OFF_A + at(row, part * 32 + p * 8);
        *reinterpret_cast<uint4 *>(sm + off) = hi;
        *reinterpret_cast<uint4 *>(sm + A_PLANE + off) = lo;
      }
    }
    // B = a I + b A + c A A, in A's place once the product has read it
    run(ks_a, D_A + 128, D_A, [&](uint32_t d, int k0, int k1) {
      products<false>(d, s0 + OFF_A, A_PLANE, s0 + OFF_A, A_PLANE, k0, k1, id_a);
    });
    const float cb = NS_B * exp2f((float)(SB - SA - 2 * e)), cc = NS_C * exp2f((float)(SB - 2 * SA - 4 * e));
    if (square) {
      uint32_t u[32];
      read(ks_a, D_A + 128 + part * 32, D_A + part * 32, u);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int off = OFF_A + at(row, part * 32 + p * 8);
        float f[8];
        unpack_pair(*reinterpret_cast<uint4 *>(sm + off), *reinterpret_cast<uint4 *>(sm + A_PLANE + off), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = fmaf(__uint_as_float(u[p * 8 + i]), cc, cb * f[i]);
          if (part * 32 + p * 8 + i == row) f[i] += NS_A * exp2f(SB);
        }
        uint4 hi, lo;
        pack_pair(f, hi, lo);
        *reinterpret_cast<uint4 *>(sm + off) = hi;
        *reinterpret_cast<uint4 *>(sm + A_PLANE + off) = lo;
      }
    }
    // X' = B X on this CTA's columns
    run(ks_x ? ks_a : 0, D_X, D_A, [&](uint32_t d, int k0, int k1) {
      products<true>(d, s0 + OFF_A, A_PLANE, s0, X_PLANE, k0, k1, id_x);
    });
    const int e_next = max(e - 2, 0);
    const bool last = step + 1 == P.steps;
    const float scale = exp2f((float)(last ? -SB - SX - e : e_next - e - SB));
#pragma unroll 1
    for (int c = q * 32 < ks_a * 16 ? part * 32 : nc; c < nc; c += 128) {
      uint32_t r[32];
      read(ks_a, D_X + c, D_A + c, r);
      float f[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]) * scale;
      if (!last) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint4 hi, lo;
          float w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = f[p * 8 + i];
          pack_pair(w, hi, lo);
          const int off = at(row, c + p * 8);
          *reinterpret_cast<uint4 *>(sm + off) = hi;
          *reinterpret_cast<uint4 *>(sm + X_PLANE + off) = lo;
        }
      } else if (TALL) {
        // a warp's 32 rows of X are neighbours in the caller's rows
        if (row < P.m) {
          TO *out = static_cast<TO *>(P.out) + base + (int64_t)(c0 + c) * P.u.cols + row;
#pragma unroll
          for (int g = 0; g < 32; g += 16) {
            float w[16];
            if (KEEP)
#pragma unroll
              for (int i = 0; i < 16; ++i)
                w[i] = c + g + i < nc ? load_el(out + (int64_t)(g + i) * P.u.cols) : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + g + i < nc)
                store_el(out + (int64_t)(g + i) * P.u.cols,
                         KEEP ? fmaf(-P.rate, f[g + i], P.keep * w[i]) : f[g + i]);
          }
        }
      } else {
        // X's place is free: the rows in fp32, 16-byte pieces swizzled by the row
#pragma unroll
        for (int p = 0; p < 8; ++p)
          *reinterpret_cast<float4 *>(sm + row * 1024 + (((c / 4 + p) ^ (row & 31)) << 4)) =
              make_float4(f[4 * p], f[4 * p + 1], f[4 * p + 2], f[4 * p + 3]);
      }
    }
    if (last && !TALL) {
      // and from there to the caller's rows, consecutive threads along them,
      // the loads of W of four rows at a time before their use
      __syncthreads();
      for (int r0 = warp; r0 < P.m; r0 += 4 * (THREADS / 32)) {
        TO *out = static_cast<TO *>(P.out) + base + (int64_t)r0 * P.u.cols + c0;
        alignas(16) float w[4 * (SLAB / 128)][4];
#pragma unroll
        for (int k = 0; k < 4 * (SLAB / 128); ++k) {
          const int r = r0 + k / (SLAB / 128) * (THREADS / 32), c = lane0 + k % (SLAB / 128) * 128;
          const TO *p = out + (int64_t)(r - r0) * P.u.cols + c;
          if (!KEEP) continue;
          if (vec)
            *reinterpret_cast<float4 *>(w[k]) =
                r < P.m && c < nc ? load_el4(p) : make_float4(0.f, 0.f, 0.f, 0.f);
          else
#pragma unroll
            for (int x = 0; x < 4; ++x) w[k][x] = r < P.m && c + 32 * x < nc ? load_el(p + 32 * x) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4 * (SLAB / 128); ++k) {
          const int r = r0 + k / (SLAB / 128) * (THREADS / 32), c = lane0 + k % (SLAB / 128) * 128;
          if (r >= P.m || c >= nc) continue;
          alignas(16) float f[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int cx = c + lane_step * x;
            f[x] = *reinterpret_cast<const float *>(sm + r * 1024 + (((cx / 4) ^ (r & 31)) << 4) +
                                                    (cx & 3) * 4);
            if (KEEP) f[x] = fmaf(-P.rate, f[x], P.keep * w[k][x]);
          }
          TO *p = out + (int64_t)(r - r0) * P.u.cols + c;
          if (vec)
            store_el4(p, *reinterpret_cast<float4 *>(f));
          else
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (c + 32 * x < nc) store_el(p + 32 * x, f[x]);
        }
      }
    }
    e = e_next;
  }
  if (!ok && tid == 0) {
    // a product may still be running: wait for it before TMEM goes back
    umma_commit(&t->drain);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(smem_u32(&t->drain), 0) && globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
    }
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  cluster_sync();  // no CTA leaves while another may read its shared memory
  // a wait that gave up, in this CTA or in another of the cluster: NaN in its columns
  if (*const_cast<volatile int *>(P.err)) {
    for (int o = warp; o < outer; o += THREADS / 32)
      for (int i = lane; i < inner; i += 32)
        store_el(static_cast<TO *>(P.out) + index(o, i), __int_as_float(0x7fffffff));
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <class TG, bool MOM, class TO, bool KEEP, bool TALL>
l3_status launch_as(const Params &P, int ctas, int64_t batch, int device, cudaStream_t s) {
  static bool attr[64] = {};
  if (!attr[device & 63]) {
    L3_CUDA_TRY(cudaFuncSetAttribute(k_muon_small<TG, MOM, TO, KEEP, TALL>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM));
    attr[device & 63] = true;
  }
  if (ctas > 8)
    L3_CUDA_TRY(cudaFuncSetAttribute(k_muon_small<TG, MOM, TO, KEEP, TALL>,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
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
  L3_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_muon_small<TG, MOM, TO, KEEP, TALL>, P));
  return L3_OK;
}

template <class TG, bool MOM, class TO, bool KEEP>
l3_status launch(const Params &P, int ctas, int64_t batch, int device, cudaStream_t s) {
  return P.u.rows > P.u.cols ? launch_as<TG, MOM, TO, KEEP, true>(P, ctas, batch, device, s)
                             : launch_as<TG, MOM, TO, KEEP, false>(P, ctas, batch, device, s);
}

}  // namespace

namespace muon {

static bool clusters_of_16(int device) {
  static int known[64] = {};
  return clusters_fit(k_muon_small<float, false, float, false, false>, MAX_CLUSTER, THREADS, SMEM, known[device & 63]);
}

bool small_always(int64_t m, int64_t n) { return m <= ROWS && n <= (int64_t)SLAB * 8; }

bool small_supported(int64_t m, int64_t n, int device) {
  return small_always(m, n) || (m <= ROWS && n <= (int64_t)SLAB * MAX_CLUSTER && clusters_of_16(device));
}

l3_status launch_small(const UpdateParams &u, bool g_fp32, int64_t batch, int steps, float eps,
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
  int ctas = 1;
  while (ctas * SLAB < P.n) ctas *= 2;
  LaunchTimer lt("muon_small", s);
  if (t.keep_w)
    return t.fp32 ? launch<float, true, float, true>(P, ctas, batch, device, s)
                  : launch<float, true, __nv_bfloat16, true>(P, ctas, batch, device, s);
  return g_fp32 ? launch<float, false, float, false>(P, ctas, batch, device, s)
                : launch<__nv_bfloat16, false, __nv_bfloat16, false>(P, ctas, batch, device, s);
}

}  // namespace muon
}  // namespace l3
