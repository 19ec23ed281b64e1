// Orthogonalising a weight matrix's update by Newton-Schulz products, as the
// Muon optimiser does: X = U / (|U|_F + eps), then `steps` times
//     A = X X^T,   X <- a X + (b A + c A^2) X,
// which drives every singular value of U towards 1 (the polynomial
// a s + b s^3 + c s^5 applied to each, s its value after the division). X is
// kept wide, m <= n (a tall U is transposed on the way in and out), so that A
// is the smaller Gram matrix.
//
// Per step three products on the tensor cores: A (m x m, depth n) and
// B = a I + b A + c A A (depth m), of whose symmetric results only the tiles
// that touch or lie below the diagonal exist, and
// X' = B X (depth m; with a I in B no epilogue has to read X).
//
// Precision. Small singular values grow by up to a^5 = 485 in five steps and
// the rounding of the large ones' components with them, so X, A and B are held
// as hi + lo pairs of fp16 (22 bits) and a product keeps hi hi + hi lo + lo hi:
// one fp16 product (11 bits) is 3e-2 off where the leading directions are a
// thousand times the rest, the pairs 6e-6. fp16's narrow range is no limit:
// |X| <= 1.3, |A| <= 1.6 and |B| <= 2.9 elementwise once the norm is divided
// out, so each is stored times a fixed power of two near the top of the range.
// A bf16 result takes the same pairs: with A and B in one part (15 products instead
// of 21) an update is 1e-3 off for noise and 7e-3 where few or equal singular values
// let the roundings add up, which a W that is large beside it hides, but not one
// that starts at zero.
// Where eps is not small beside |U|, X starts below one and V = X 2^e, of norm
// in (1/2, 1], is held in its place: e falls by two a step (V grows by at most
// a < 4) until X itself is, and the polynomial's coefficients take the powers
// of 2^-2e that A's and A^2's scales differ by.
#include "gemm_pair.cuh"
#include "muon_common.cuh"

namespace l3 {
namespace {

using namespace sm100;
using namespace muon;
namespace pg = pairgemm;

struct Head {
  int err;
  int pad[3];
};

constexpr int64_t HEAD_BYTES = 1024;

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

constexpr int NORM_THREADS = 256;

struct Layout {
  int64_t batch, m, n;  // wide form of one matrix
  int64_t mp, np;       // padded to whole k-blocks, zeros
  int64_t norm_blocks;  // partial sums of squares per matrix
  pg::Tiling gram, poly, step;
  size_t head, part, exps, x0, x1, a, b, share, total;

  Layout(int64_t batch_, int64_t rows, int64_t cols)
      : batch(batch_), m(std::min(rows, cols)), n(std::max(rows, cols)) {
    mp = round_up(m, 64);
    np = round_up(n, 64);
    // about 8 K elements a block
    norm_blocks = std::min<int64_t>((m * n + 8191) / 8192, 1184);
    const int64_t tile_rows = (mp + 255) / 256;
    const auto sym_tiles = [&](int tn) {
      const int tiles_n = (int)((mp + tn - 1) / tn);
      int64_t t = 0;
      for (int i = 0; i < tile_rows; ++i)
        t += tn == 256 ? pg::sym_row_tiles<256>(i, tiles_n) : pg::sym_row_tiles<128>(i, tiles_n);
      return t * batch;
    };
    // a partial is written and read as fp32, half of it (the rest mirrors it)
    gram = pg::choose_tiling(sym_tiles, np / pg::BK, 3, batch * mp * mp / 2);
    // one share: m deep, shares would not be repaid for any m and batch
    poly = pg::choose_tiling(sym_tiles, mp / pg::BK, 3, INT64_MAX / 1024);
    step = pg::choose_tiling([&](int tn) { return batch * tile_rows * ((np + tn - 1) / tn); }, mp / pg::BK,
                             3, INT64_MAX / 1024);
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t r = at;
      at += (bytes + 1023) & ~size_t(1023);
      return r;
    };
    head = take(HEAD_BYTES);
    part = take((size_t)batch * norm_blocks * 8);
    exps = take((size_t)batch * 4);
    x0 = take((size_t)2 * batch * mp * np * 2);
    x1 = take((size_t)2 * batch * mp * np * 2);
    a = take((size_t)2 * batch * mp * mp * 2);
    b = take((size_t)2 * batch * mp * mp * 2);
    share = take(gram.splits > 1 ? (size_t)gram.splits * batch * mp * mp * 4 : 0);
    total = at;
  }
};

// ---------------------------------------------------------------------------
// the update U, its norm, and X = U / (|U| + eps)
// ---------------------------------------------------------------------------
// M <- mu M + G, and sums of U's squares (in 64 bits: squares of large
// elements leave fp32's range), one per block; memory-bound
template <class T, bool MOM>
__global__ void __launch_bounds__(NORM_THREADS) k_update_norm(UpdateParams P, Head *head,
                                                              bool clear_err, double *part) {
  pg::pdl_launch();
  const int64_t base = (int64_t)blockIdx.y * P.size;
  if (clear_err && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) head->err = 0;
  double sum = 0.0;
  const int64_t first = blockIdx.x * (int64_t)NORM_THREADS + threadIdx.x;
  const int64_t stride = (int64_t)gridDim.x * NORM_THREADS;
  const int64_t quads = P.vec ? P.size / 4 : 0;
#pragma unroll 4
  for (int64_t i = first; i < quads; i += stride) {
    const float4 gv = load_el4(static_cast<const T *>(P.g) + base + 4 * i);
    float g[4] = {gv.x, gv.y, gv.z, gv.w};
    if (MOM) {
      float4 m = *reinterpret_cast<const float4 *>(P.mom + base + 4 * i);
      m.x = fmaf(P.mu, m.x, g[0]), m.y = fmaf(P.mu, m.y, g[1]);
      m.z = fmaf(P.mu, m.z, g[2]), m.w = fmaf(P.mu, m.w, g[3]);
      *reinterpret_cast<float4 *>(P.mom + base + 4 * i) = m;
      g[0] = P.update(m.x, g[0]), g[1] = P.update(m.y, g[1]);
      g[2] = P.update(m.z, g[2]), g[3] = P.update(m.w, g[3]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum = fma((double)g[e], (double)g[e], sum);
  }
  for (int64_t i = 4 * quads + first; i < P.size; i += stride) {
    if (MOM) P.mom[base + i] = fmaf(P.mu, P.mom[base + i], load_el(static_cast<const T *>(P.g) + base + i));
    const double u = update_at<T, MOM>(P, base + i);
    sum = fma(u, u, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __shared__ double s[NORM_THREADS / 32];
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < NORM_THREADS / 32; ++w) sum += s[w];
    part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
  }
}

// X as hi + lo planes [2][batch][mp][np], zeros in the padding; a 64 x 64
// block of X per thread block, through shared memory where U is tall
template <class T, bool MOM>
__global__ void __launch_bounds__(256) k_normalise(UpdateParams P, const double *part, int n_part,
                                                   float eps, int transpose, int m, int n, int mp,
                                                   int np, __half *x, int64_t plane, int *exps) {
  __shared__ double s_sum[8];
  __shared__ float tile[64][65];
  pg::pdl_launch();
  pg::pdl_wait();
  const int b = blockIdx.z, tid = threadIdx.x;
  const int64_t base = (int64_t)b * P.size;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;  // block of X
  // consecutive threads along U's rows, four neighbours each where those start
  // aligned; all of a thread's loads are on their way while the norm is summed
  const int line = transpose ? c0 : r0, along = transpose ? r0 : c0;
  const int lines = transpose ? n : m, length = transpose ? m : n;
  const bool vec = P.vec && P.cols % 4 == 0;
  const int step = vec ? 1 : 16, first = vec ? tid % 16 * 4 : tid % 16;
  float v[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int o = line + tid / 16 + 16 * k, i = along + first;
    const int64_t at = base + (int64_t)o * P.cols + i;
    const T *g = static_cast<const T *>(P.g) + at;
    if (vec) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (o < lines && i < length) {
        f = load_el4(g);
        if (MOM) {
          const float4 w = load_el4(P.mom + at);
          f = make_float4(P.update(w.x, f.x), P.update(w.y, f.y), P.update(w.z, f.z), P.update(w.w, f.w));
        }
      }
      v[k][0] = f.x, v[k][1] = f.y, v[k][2] = f.z, v[k][3] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[k][e] = o < lines && i + 16 * e < length ? update_at<T, MOM>(P, at + 16 * e) : 0.f;
    }
  }
  double sum = 0.0;
  for (int i = tid; i < n_part; i += 256) sum += part[(int64_t)b * n_part + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (tid % 32 == 0) s_sum[tid / 32] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < 8; ++w) sum += s_sum[w];
  // V = X 2^e with |V| in (1/2, 1]
  const double root = sqrt(sum), norm = root + (double)eps;
  const int e = root > 0.0 && norm > root && norm < INFINITY ? ilogb(norm / root) : 0;
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) exps[b] = e;
  float inv0, inv1;
  scale_factors(norm, SX + e, inv0, inv1);
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int o = tid / 16 + 16 * k, i = first + step * x;
      tile[transpose ? i : o][transpose ? o : i] = v[k][x] * inv1 * inv0;
    }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = tid / 16 + 16 * k, c = tid % 16 * 4;
    __half2 hi[2], lo[2];
    split2(tile[r][c], tile[r][c + 1], hi[0], lo[0]);
    split2(tile[r][c + 2], tile[r][c + 3], hi[1], lo[1]);
    __half *dst = x + ((int64_t)b * mp + r0 + r) * np + c0 + c;
    *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(hi);
    *reinterpret_cast<uint2 *>(dst + plane) = *reinterpret_cast<uint2 *>(lo);
  }
}

// ---------------------------------------------------------------------------
// epilogues
// ---------------------------------------------------------------------------
// e of a matrix after `done` steps (see the top of the file)
__device__ __forceinline__ int exp_at(const int *exps, int b, int done) {
  return max(exps[b] - 2 * done, 0);
}

// The hi (and lo) boxes of a stack's matrices (planes of batch x mp rows) as an
// epilogue warp's operand. A tile's first columns are asked for while its
// products still run, the next ones when the boxes have been copied out.
struct PairIn {
  CUtensorMap map;
  int mp, batch_rows;  // rows of a matrix and of a plane

  __device__ __forceinline__ void fetch(pg::WarpBoxes &box, int b, int m_warp, int col) const {
    box.written();  // what the boxes held is done with
    if (box.lane == 0) box.load<2>(&map, col, b * mp + m_warp, batch_rows);
  }
};

// A warp's 32 x 32 block (thread = row) turned round through its box (16-byte
// pieces swizzled by the row): v[e] becomes row e, column = thread
__device__ __forceinline__ void turn_block(pg::WarpBoxes &box, float (&v)[32]) {
  __syncwarp();  // the last block has been read
#pragma unroll
  for (int p = 0; p < 8; ++p)
    *reinterpret_cast<float4 *>(box.mem + box.lane * 128 + ((p ^ (box.lane & 7)) << 4)) =
        make_float4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 32; ++e)
    v[e] = *reinterpret_cast<const float *>(box.mem + e * 128 + (((box.lane >> 2) ^ (e & 7)) << 4) +
                                            (box.lane & 3) * 4);
}

// eight elements of a warp's row from its boxes
__device__ __forceinline__ void unpack(const pg::WarpBoxes &box, int j, float (&f)[8]) {
  unpack_pair(*box.piece(0, j), *box.piece(1, j), f);
}

// A = X X^T (POLY = false) or B = a I + b A + c A A (POLY = true), both symmetric:
// the blocks right of the diagonal one are not written
template <int TN, bool POLY>
struct EpiSym {
  __half *out;  // two planes of batch x mp x mp
  int64_t plane;
  PairIn a;  // POLY: A
  int mp;
  const int *exps;
  int done;

  // A in (POLY), the result out
  static constexpr int BOX_BYTES = 2 * pg::BOX;
  static constexpr bool LOADS = POLY;
  static constexpr int WARPS = 16;
  static constexpr bool SUMS = true;

  __device__ __forceinline__ void prefetch(pg::WarpBoxes &box, int b, int m_warp, int c0) const {
    if (POLY && m_warp < mp && c0 < mp) a.fetch(box, b, m_warp, c0);
  }
  struct State {
    int b, m_warp, c0;
    float cb, cc;
    __half *o;
  };
  __device__ __forceinline__ State begin(int b, int m, int c0, int) const {
    const int e2 = POLY ? 2 * exp_at(exps, b, done) : 0;
    return State{b, m & ~31, c0, NS_B * exp2f((float)(SB - SA - e2)),
                 NS_C * exp2f((float)(SB - 2 * SA - 2 * e2)), out + (int64_t)b * mp * mp};
  }
  __device__ __forceinline__ void chunk(State &s, pg::WarpBoxes &box, int c, float (&v)[32]) const {
    const int col = s.c0 + c;
    if (s.m_warp >= mp || col >= mp) return;  // the whole warp alike
    if (POLY) {
      if (c > 0) a.fetch(box, s.b, s.m_warp, col);
      box.loaded();  // a give-up: the tile's values are lost, its stores in bounds
    }
    __syncwarp();  // the last columns' boxes have been copied out
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
      if (POLY) unpack(box, j, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[e] = POLY ? fmaf(v[j * 8 + e], s.cc, s.cb * f[e]) : v[j * 8 + e] * exp2f(SA - 2 * SX);
        if (POLY && col + j * 8 + e == s.m_warp + box.lane) f[e] += NS_A * exp2f(SB);
      }
      uint4 hi, lo;
      pack_pair(f, hi, lo);
      *box.piece(0, j) = hi;
      *box.piece(1, j) = lo;
    }
    __syncwarp();
    __half *to = s.o + (int64_t)s.m_warp * mp + col;
    box.copy_out(0, to, mp);
    box.copy_out(1, to + plane, mp);
  }
  __device__ __forceinline__ void end(State &) const {}
};

// A share of A's product, fp32, as the accumulator has it; k_sym_join adds the
// shares up
template <int TN>
struct EpiShare {
  float *out;  // [share][batch][mp][mp]
  int mp;

  static constexpr int BOX_BYTES = pg::BOX;
  static constexpr bool LOADS = false;
  static constexpr int WARPS = 16;
  static constexpr bool SUMS = true;
  __device__ __forceinline__ void prefetch(pg::WarpBoxes &, int, int, int) const {}

  struct State {
    int m_warp, c0;
    float *o;
  };
  __device__ __forceinline__ State begin(int b, int m, int c0, int) const {
    return State{m & ~31, c0, out + ((int64_t)b * mp + (m & ~31)) * mp};
  }
  __device__ __forceinline__ void chunk(State &s, pg::WarpBoxes &box, int c, float (&v)[32]) const {
    if (s.m_warp >= mp || s.c0 + c >= mp) return;  // the whole warp alike
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // sixteen columns fill a box
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float *f = v + h * 16 + j * 4;
        *reinterpret_cast<float4 *>(box.piece(0, j)) = make_float4(f[0], f[1], f[2], f[3]);
      }
      __syncwarp();
      box.copy_out(0, s.o + s.c0 + c + h * 16, 2 * mp);  // ld in 16-bit elements
    }
  }
  __device__ __forceinline__ void end(State &) const {}
};

// The shares of A added up in their order, and A as hi + lo planes: a 64 x 64
// block in or left of the 256-wide diagonal block per thread block. Memory-bound.
__global__ void __launch_bounds__(256) k_sym_join(const float *share, int shares, int64_t batch,
                                                  int mp, __half *out) {
  pg::pdl_launch();
  pg::pdl_wait();
  const int bi = blockIdx.y, bj = blockIdx.x, b = blockIdx.z;
  if (bj / 4 > bi / 4) return;
  const int64_t one = (int64_t)mp * mp, plane = batch * one;
  const int c = threadIdx.x % 16 * 4;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = threadIdx.x / 16 + 16 * k;
    const int64_t at = b * one + (int64_t)(bi * 64 + r) * mp + bj * 64 + c;
    float4 s = *reinterpret_cast<const float4 *>(share + at);
    for (int i = 1; i < shares; ++i) {
      const float4 w = *reinterpret_cast<const float4 *>(share + i * plane + at);
      s.x += w.x, s.y += w.y, s.z += w.z, s.w += w.w;
    }
    float f[4] = {s.x, s.y, s.z, s.w};
    __half2 hi[2], lo[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f[2 * h] *= exp2f(SA - 2 * SX);
      f[2 * h + 1] *= exp2f(SA - 2 * SX);
      split2(f[2 * h], f[2 * h + 1], hi[h], lo[h]);
    }
    *reinterpret_cast<uint2 *>(out + at) = *reinterpret_cast<uint2 *>(hi);
    *reinterpret_cast<uint2 *>(out + plane + at) = *reinterpret_cast<uint2 *>(lo);
  }
}

// X' = B X
template <int TN>
struct EpiStep {
  __half *out;  // planes of batch x mp x cols
  int64_t plane;
  int mp, cols;
  const int *exps;
  int done;

  static constexpr int BOX_BYTES = 2 * pg::BOX;
  static constexpr bool LOADS = false;
  static constexpr int WARPS = 16;
  static constexpr bool SUMS = true;
  __device__ __forceinline__ void prefetch(pg::WarpBoxes &, int, int, int) const {}

  struct State {
    int m_warp, c0;
    float up;
    __half *o;
  };
  __device__ __forceinline__ State begin(int b, int m, int c0, int) const {
    // V' = X' 2^(e of the next step)
    return State{m & ~31, c0,
                 exp2f((float)(exp_at(exps, b, done + 1) - exp_at(exps, b, done) - SB)),
                 out + ((int64_t)b * mp + (m & ~31)) * cols};
  }
  __device__ __forceinline__ void chunk(State &s, pg::WarpBoxes &box, int c, float (&v)[32]) const {
    const int col = s.c0 + c;
    if (s.m_warp >= mp || col >= cols) return;  // the whole warp alike
    __syncwarp();  // the last chunk's boxes have been copied out
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = v[j * 8 + e] * s.up;
      uint4 hi, lo;
      pack_pair(f, hi, lo);
      *box.piece(0, j) = hi;
      *box.piece(1, j) = lo;
    }
    __syncwarp();
    box.copy_out(0, s.o + col, cols);
    box.copy_out(1, s.o + plane + col, cols);
  }
  __device__ __forceinline__ void end(State &) const {}
};

// The last step, in the caller's layout: O = X' (KEEP = false), or the
// weights' update W <- keep W - rate X' (KEEP = true)
template <int TN, class T, bool KEEP>
struct EpiOut {
  T *out;
  int64_t size;
  int m, n;       // X is m x n
  int cols;       // of the caller's matrix
  int transpose;  // which is X^T
  float keep, rate;
  const int *exps;
  int done;

  static constexpr int BOX_BYTES = 32 * 32 * 4;
  static constexpr bool LOADS = false;
  static constexpr int WARPS = 16;
  static constexpr bool SUMS = true;
  __device__ __forceinline__ void prefetch(pg::WarpBoxes &, int, int, int) const {}

  struct State {
    int r, c0;
    float down;
    T *o;
  };
  __device__ __forceinline__ State begin(int b, int r, int c0, int) const {
    return State{r, c0, exp2f((float)(-SB - SX - exp_at(exps, b, done))), out + (int64_t)b * size};
  }
  __device__ __forceinline__ void chunk(State &s, pg::WarpBoxes &box, int c, float (&v)[32]) const {
    const int c1 = s.c0 + c, r0 = s.r & ~31;
    if (r0 >= m || c1 >= n) return;  // the whole warp alike
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] *= s.down;
    // Consecutive threads along the caller's rows. The output X^T has X's rows
    // there, a thread each; otherwise the 32 x 32 block is turned round
    int64_t at = (int64_t)c1 * cols + s.r, step = cols;
    int count = s.r < m ? n - c1 : 0;  // elements of this thread, `step` apart
    if (!transpose) {
      turn_block(box, v);
      at = (int64_t)r0 * cols + c1 + box.lane;
      count = c1 + box.lane < n ? m - r0 : 0;
    }
    T *p = s.o + at;
#pragma unroll
    for (int g = 0; g < 32; g += 16) {
      float w[16];
      if (KEEP)
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = g + e < count ? load_el(p + (g + e) * step) : 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (g + e < count)
          store_el(p + (g + e) * step, KEEP ? fmaf(-rate, v[g + e], keep * w[e]) : v[g + e]);
    }
  }
  __device__ __forceinline__ void end(State &) const {}
};

template <class T, bool MOM>
l3_status launch_prologue(const Layout &L, const UpdateParams &U, char *ws, float eps, bool clear_err,
                          cudaStream_t s) {
  Head *head = reinterpret_cast<Head *>(ws + L.head);
  double *part = reinterpret_cast<double *>(ws + L.part);
  {
    LaunchTimer t("muon_norm", s);  // the chain's first: waits for all that came before
    k_update_norm<T, MOM><<<dim3((unsigned)L.norm_blocks, (unsigned)L.batch), NORM_THREADS, 0, s>>>(
        U, head, clear_err, part);
    L3_CUDA_TRY(cudaGetLastError());
  }
  LaunchTimer t("muon_normalise", s);
  return pg::launch_link(k_normalise<T, MOM>,
                         dim3((unsigned)(L.np / 64), (unsigned)(L.mp / 64), (unsigned)L.batch),
                         dim3(256), s, true, U, part, (int)L.norm_blocks, eps,
                         (int)(U.rows > U.cols), (int)L.m, (int)L.n, (int)L.mp, (int)L.np,
                         reinterpret_cast<__half *>(ws + L.x0), L.batch * L.mp * L.np,
                         reinterpret_cast<int *>(ws + L.exps));
}

struct Chain {
  const Layout &L;
  char *ws;
  int device;
  cudaStream_t s;
  __half *x[2], *a, *bm;
  const int *exps;
  int64_t xr;  // rows of one plane
  bool fp32;   // the result's type
  CUtensorMap x_m[2], x_n[2][2], x_k[2];  // X as M (128 rows), as N, as k rows
  CUtensorMap a_s, a_box, b_s;  // A and B as symmetric operands

  l3_status maps() {
    l3_status st = L3_OK;
    const auto want = [&](l3_status got) {
      if (st == L3_OK) st = got;
    };
    const int64_t rows = 2 * xr;
    for (int i = 0; i < 2; ++i) {
      want(pg::operand_map(&x_m[i], x[i], false, rows, L.np, L.np, false, pg::BM));
      want(pg::operand_map(&x_n[i][0], x[i], false, rows, L.np, L.np, false, 64));
      want(pg::operand_map(&x_n[i][1], x[i], false, rows, L.np, L.np, false, 128));
      want(pg::operand_map(&x_k[i], x[i], false, rows, L.np, L.np, true, 0));
    }
    want(pg::operand_map(&a_s, a, false, rows, L.mp, L.mp, true, 0));
    want(pg::box_map(&a_box, a, false, rows, L.mp, L.mp));
    want(pg::operand_map(&b_s, bm, false, rows, L.mp, L.mp, true, 0));
    return st;
  }

  pg::Args args(int tn, bool sym) const {
    pg::Args P = {};
    P.tiles_m = (int)((L.mp + 255) / 256);
    P.tiles_n = (int)(((sym ? L.mp : L.np) + tn - 1) / tn);
    P.batch = (int)L.batch;
    // rounding grows from step to step: 128 deep in one chain where the result is
    // fp32 (2048 x 4096: 5e-6 off; 512 deep, 2e-5 and 3 % faster), and 64 where
    // few rows let fp32 products be better than that: A and A^2 of up to 1024
    // (1000 x 3000: 5.5e-6 -> 3.4e-6 and 306 -> 326 us; fp32 3.7e-6), X' of up to
    // 512 (with them 400 x 1500: 4.9e-6 -> 2.2e-6, 190 -> 199 us; fp32 2.5e-6)
    P.chunk = !fp32 ? 8 : L.m <= (sym ? 1024 : 512) ? 1 : 2;
    P.sym = sym;
    P.group = 8;
    P.a_batch = P.b_batch = (int)L.mp;
    P.a_plane = P.b_plane = (int)xr;
    P.err = &reinterpret_cast<Head *>(ws + L.head)->err;
    return P;
  }

  template <int TN, bool POLY>
  l3_status sym_product(int cur, int done) {
    pg::Args P = args(TN, true);
    P.nkb = (int)((POLY ? L.mp : L.np) / pg::BK);
    EpiSym<TN, POLY> e{POLY ? bm : a, xr * L.mp, {a_box, (int)L.mp, (int)xr}, (int)L.mp, exps, done};
    const CUtensorMap &mA = POLY ? a_s : x_m[cur], &mB = POLY ? a_s : x_n[cur][TN / 256];
    LaunchTimer t(POLY ? "muon_poly" : "muon_gram", s);
    constexpr pg::Major MAJOR = POLY ? pg::SYMMETRIC : pg::K_MAJOR;
    if constexpr (!POLY) {
      if (L.gram.splits > 1) {
        P.splits = L.gram.splits;
        P.batch *= P.splits;
        const EpiShare<TN> es{reinterpret_cast<float *>(ws + L.share), (int)L.mp};
        const l3_status st = pg::launch<TN, 2, 2, MAJOR, MAJOR>(mA, mB, P, es, device, s);
        if (st != L3_OK) return st;
        const unsigned blocks = (unsigned)(L.mp / 64);
        return pg::launch_link(k_sym_join, dim3(blocks, blocks, (unsigned)L.batch), dim3(256), s, true,
                               es.out, P.splits, L.batch, (int)L.mp, a);
      }
    }
    return pg::launch<TN, 2, 2, MAJOR, MAJOR>(mA, mB, P, e, device, s);
  }
  template <bool POLY>
  l3_status sym_product(int cur, int done) {
    const bool wide = (POLY ? L.poly : L.gram).tn == 256;
    return wide ? sym_product<256, POLY>(cur, done) : sym_product<128, POLY>(cur, done);
  }
  template <int TN, class E>
  l3_status step(int cur, E &e, int done) {
    pg::Args P = args(TN, false);
    P.nkb = (int)(L.mp / pg::BK);
    e.exps = exps;
    e.done = done;
    LaunchTimer t("muon_step", s);
    return pg::launch<TN, 2, 2, pg::SYMMETRIC, pg::MN_MAJOR>(b_s, x_k[cur], P, e, device, s);
  }
  template <int TN, class T, bool KEEP>
  l3_status out(int cur, int done, const Target &t, int64_t rows, int64_t cols) {
    EpiOut<TN, T, KEEP> e{};
    e.out = static_cast<T *>(t.out);
    e.size = rows * cols;
    e.m = (int)L.m;
    e.n = (int)L.n;
    e.cols = (int)cols;
    e.transpose = rows > cols;
    e.keep = t.keep;
    e.rate = t.rate;
    return step<TN>(cur, e, done);
  }
  template <int TN>
  l3_status last(int cur, int done, const Target &t, int64_t rows, int64_t cols) {
    return t.keep_w ? (t.fp32 ? out<TN, float, true>(cur, done, t, rows, cols)
                              : out<TN, __nv_bfloat16, true>(cur, done, t, rows, cols))
                    : (t.fp32 ? out<TN, float, false>(cur, done, t, rows, cols)
                              : out<TN, __nv_bfloat16, false>(cur, done, t, rows, cols));
  }
  template <int TN>
  l3_status inner(int cur, int done) {
    EpiStep<TN> e{};
    e.out = x[cur ^ 1];
    e.plane = xr * L.np;
    e.mp = (int)L.mp;
    e.cols = (int)L.np;
    return step<TN>(cur, e, done);
  }
};

// matrices whose tiles' X, A and B are held at a time: 1 GB of them, one at least.
// That is far more than fills the GPU, and a stack may be larger than what is free
// beside it.
int64_t slice_of(int64_t batch, int64_t rows, int64_t cols) {
  const int64_t one = (int64_t)Layout(1, rows, cols).total;
  return std::min(batch, std::max<int64_t>((int64_t(1) << 30) / one, 1));
}

int64_t workspace_of(int64_t batch, int64_t rows, int64_t cols) {
  // one launch, whatever the steps and the device: the error word alone
  if (small_always(std::min(rows, cols), std::max(rows, cols))) return HEAD_BYTES;
  const int64_t slice = slice_of(batch, rows, cols), rest = batch % slice;
  // fewer matrices may be shared out more
  return (int64_t)std::max(Layout(slice, rows, cols).total, rest ? Layout(rest, rows, cols).total : 0);
}

l3_status newton_schulz(const Layout &L, char *ws, int steps, const Target &t, int64_t rows,
                        int64_t cols, int device, cudaStream_t s) {
  Chain c{L, ws, device, s,
          {reinterpret_cast<__half *>(ws + L.x0), reinterpret_cast<__half *>(ws + L.x1)},
          reinterpret_cast<__half *>(ws + L.a), reinterpret_cast<__half *>(ws + L.b),
          reinterpret_cast<const int *>(ws + L.exps), L.batch * L.mp, t.fp32};
  l3_status st = c.maps();
  const bool wide = L.step.tn == 256;
  for (int i = 0; st == L3_OK && i < steps; ++i) {
    const int cur = i & 1;
    st = c.sym_product<false>(cur, i);
    if (st == L3_OK) st = c.sym_product<true>(cur, i);
    if (st != L3_OK) break;
    if (i + 1 < steps)
      st = wide ? c.inner<256>(cur, i) : c.inner<128>(cur, i);
    else
      st = wide ? c.last<256>(cur, i, t, rows, cols) : c.last<128>(cur, i, t, rows, cols);
  }
  if (st != L3_OK) return st;
  return launch_spoil(&reinterpret_cast<Head *>(ws + L.head)->err,
                      {t.out, L.batch * rows * cols * (t.fp32 ? 4 : 2)}, {nullptr, 0}, s);
}

// The whole update, whichever form it takes: U of a gradient of type T (and a momentum)
// into t
template <class T, bool MOM>
l3_status run(UpdateParams U, Target t, int64_t batch, int steps, float eps, char *ws, int device,
              cudaStream_t s) {
  const int64_t rows = U.rows, cols = U.cols, m = std::min(rows, cols), n = std::max(rows, cols);
  int *err = &reinterpret_cast<Head *>(ws)->err;
  if (tiny_supported(m, steps)) return launch_tiny(U, sizeof(T) == 4, batch, steps, eps, t, err, device, s);
  if (small_supported(m, n, device)) return launch_small(U, sizeof(T) == 4, batch, steps, eps, t, err, device, s);
  const int64_t slice = slice_of(batch, rows, cols);
  for (int64_t b = 0; b < batch; b += slice) {
    const Layout L(std::min(slice, batch - b), rows, cols);
    l3_status st = launch_prologue<T, MOM>(L, U, ws, eps, b == 0, s);
    if (st == L3_OK) st = newton_schulz(L, ws, steps, t, rows, cols, device, s);
    if (st != L3_OK) return st;
    U.g = static_cast<const T *>(U.g) + slice * U.size;
    if (MOM) U.mom += slice * U.size;
    t.out = static_cast<char *>(t.out) + slice * U.size * (t.fp32 ? 4 : 2);
  }
  return L3_OK;
}

struct Pointer {
  const void *p;
  uintptr_t align;
};
// 1 where all are 16-byte aligned and a matrix's elements keep the next one so
int vectors(const Pointer *ptrs, int n, int64_t size) {
  uintptr_t all = 0;
  for (int i = 0; i < n; ++i) all |= reinterpret_cast<uintptr_t>(ptrs[i].p);
  return (all & 15) == 0 && size % 8 == 0;
}

// the sizes that the calls take, before anything is computed from them
l3_status check_sizes(const std::string &name, int64_t batch, int64_t rows, int64_t cols) {
  if (batch < 0 || rows < 0 || cols < 0) {
    set_error(name + ": need batch, rows, cols >= 0");
    return L3_ERR_INVALID_ARG;
  }
  if (rows > 65536 || cols > 65536 || batch > 4096 || 2 * batch * std::min(rows, cols) > (1 << 28)) {
    set_error(name + ": rows and cols are at most 65536, batch at most 4096, and batch times the "
                     "smaller of rows and cols at most 2^27");
    return L3_ERR_UNSUPPORTED;
  }
  return L3_OK;
}

l3_status check(const char *who, int64_t batch, int64_t rows, int64_t cols, int32_t dtype,
                int32_t steps, float eps, const Pointer *ptrs, int n_ptrs, int64_t ws_bytes,
                int *device) {
  const std::string name = who;
  if (dtype != L3_BF16 && dtype != L3_FP32) {
    set_error(name + ": dtype must be L3_BF16 or L3_FP32");
    return L3_ERR_INVALID_ARG;
  }
  if (steps < 1 || steps > 16 || !(eps >= 0.f)) {
    set_error(name + ": need 1 <= steps <= 16 and eps >= 0");
    return L3_ERR_INVALID_ARG;
  }
  const l3_status st = check_sizes(name, batch, rows, cols);
  if (st != L3_OK || batch == 0 || rows == 0 || cols == 0) return st;
  for (int i = 0; i < n_ptrs; ++i) {
    if (!ptrs[i].p) {
      set_error(name + ": a tensor or workspace pointer is NULL");
      return L3_ERR_INVALID_ARG;
    }
    if (reinterpret_cast<uintptr_t>(ptrs[i].p) & (ptrs[i].align - 1)) {
      set_error(name + ": the workspace must be 16-byte aligned, tensors to their elements");
      return L3_ERR_INVALID_ARG;
    }
  }
  const int64_t need = workspace_of(batch, rows, cols);
  if (ws_bytes < need) {
    set_error(name + ": the workspace holds " + std::to_string(ws_bytes) + " bytes, " +
              std::to_string(need) + " are needed");
    return L3_ERR_INVALID_ARG;
  }
  L3_CUDA_TRY(current_device(device));
  return L3_OK;
}

}  // namespace
}  // namespace l3

using namespace l3;

extern "C" {

int64_t l3_muon_workspace(int64_t batch, int64_t rows, int64_t cols) {
  set_error("");
  if (check_sizes("l3_muon_workspace", batch, rows, cols) != L3_OK) return -1;
  if (batch == 0 || rows == 0 || cols == 0) return 0;
  return workspace_of(batch, rows, cols);
}

l3_status l3_orthogonalize(const void *G, int64_t batch, int64_t rows, int64_t cols, int32_t dtype,
                           int32_t steps, float eps, void *O, void *workspace,
                           int64_t workspace_bytes, void *stream) {
  set_error("");
  int device = 0;
  const uintptr_t el = dtype == L3_FP32 ? 4 : 2;
  const Pointer ptrs[] = {{G, el}, {O, el}, {workspace, 16}};
  l3_status st = check("l3_orthogonalize", batch, rows, cols, dtype, steps, eps, ptrs, 3,
                       workspace_bytes, &device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (st != L3_OK) return st;
  if (batch == 0 || rows == 0 || cols == 0) return clear_error_word(workspace, workspace_bytes, s);
  char *ws = static_cast<char *>(workspace);
  UpdateParams U = {};
  U.g = G;
  U.size = rows * cols;
  U.rows = (int)rows;
  U.cols = (int)cols;
  U.vec = vectors(ptrs, 2, U.size);
  const Target t{O, dtype == L3_FP32, false, 0.f, 0.f};
  return dtype == L3_FP32 ? run<float, false>(U, t, batch, steps, eps, ws, device, s)
                          : run<__nv_bfloat16, false>(U, t, batch, steps, eps, ws, device, s);
}

l3_status l3_muon_step(void *W, float *M, const float *G, int64_t batch, int64_t rows,
                       int64_t cols, int32_t dtype, float lr, float momentum, int32_t nesterov,
                       float weight_decay, float scale, int32_t steps, float eps, void *workspace,
                       int64_t workspace_bytes, void *stream) {
  set_error("");
  int device = 0;
  const Pointer ptrs[] = {{W, dtype == L3_FP32 ? 4u : 2u}, {M, 4}, {G, 4}, {workspace, 16}};
  l3_status st = check("l3_muon_step", batch, rows, cols, dtype, steps, eps, ptrs, 4,
                       workspace_bytes, &device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (st != L3_OK) return st;
  if (batch == 0 || rows == 0 || cols == 0) return clear_error_word(workspace, workspace_bytes, s);
  char *ws = static_cast<char *>(workspace);
  UpdateParams U = {};
  U.g = G;
  U.mom = M;
  U.mu = momentum;
  U.nesterov = nesterov;
  U.size = rows * cols;
  U.rows = (int)rows;
  U.cols = (int)cols;
  U.vec = vectors(ptrs, 3, U.size);
  const Target t{W, dtype == L3_FP32, true, 1.f - lr * weight_decay, lr * scale};
  return run<float, true>(U, t, batch, steps, eps, ws, device, s);
}

l3_status l3_workspace_status(const void *workspace, void *stream) {
  set_error("");
  if (!workspace) {
    set_error("workspace is NULL");
    return L3_ERR_INVALID_ARG;
  }
  int32_t err = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  L3_CUDA_TRY(cudaMemcpyAsync(&err, workspace, 4, cudaMemcpyDeviceToHost, s));
  L3_CUDA_TRY(cudaStreamSynchronize(s));
  if (err & DEV_ERR_TIMEOUT) {
    set_error("a bounded device-side wait of the call that used this workspace gave up; its "
              "outputs are incomplete");
    return L3_ERR_TIMEOUT;
  }
  return L3_OK;
}

}  // extern "C"
