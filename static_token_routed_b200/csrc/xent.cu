// Softmax cross entropy of an output projection over a large vocabulary,
// without keeping the logits. With s = x W^T (x [n, d], W [vocab, d]),
//     lse_i = log sum_j exp(s_ij),   loss_i = lse_i - s_i,t_i,
//     G_ij = g_i (exp(s_ij - lse_i) - [j = t_i]),   dx = G W,   dW = G^T x.
//
// Forward: one product on the tensor cores whose epilogue reduces each row of
// a tile to (max, sum of exponentials) over 128 columns, without the target's
// logit, which it picks out; a second kernel joins a row's partials. 8 bytes leave
// the SMs for 128 logits. With S the sum over the others, the loss is
// log1p(S exp(-s_t)): where the target is all but certain, lse - s_t would leave
// the rounding of two numbers a hundred times its size.
// Backward: in pieces of the vocabulary, the logits once more with G as the
// epilogue, then dx += G W_piece and dW_piece = G^T x in one launch, so that the
// many short tiles of one fill the gaps of the other's few long ones (8192 x 180000
// x 2048: 256 tiles of dx alone are 3.5 rounds of 74 pairs of SMs). A piece's G is the only
// array of n rows and many columns, and its size is bounded.
//
// Scoring a few tokens is bound by reading W: up to 128 of them are the product's
// N and W's rows its M, so that a tile's operands are nearly all W's; up to 256
// are read where they lie, without the gather below.
//
// Tokens whose target is negative take no part: the first kernel gathers the
// rows of the others into the workspace, so padding costs nothing and a NaN in
// it reaches no sum. Their count stays on the device; the products read it.
//
// Types. bf16: bf16 operands, fp32 accumulation; G is rounded to bf16, the
// type of the gradients themselves, without the largest weight max|g|, which
// multiplies the fp32 accumulators instead: with equal weights, 1 - p near 1 then
// stays exact. Of the roundings in a row of G the target's alone can weigh as
// much as all others together, and so it can in a column, most of whose tokens
// have other targets. For dx, what it left of that element is kept in fp32 and
// the epilogue adds it times the target's row of W. For dW, G gets a second bf16 part
// in the blocks of 64 tokens x 256 columns that hold a target, and the product takes
// that part in these blocks: at most one a token, and fewer where tokens are frequent
// (8192 tokens x 180000: 4 % of the blocks). Up to 128 tokens, where one wrong guess can weigh as much as a
// target, dW takes it everywhere, and dx from 4 tokens or less. dx and dW are 1.7e-3
// off for it, their own rounding; with one part alone, dx 2.3e-3 (6e-3 from one
// token) and dW up to 2.4e-3. It costs loss and gradients of 8192 x 180000 x 2048 4 %
// (19.5 ms) and 1794 live tokens x 32003 x 1024 12 % (519 us). fp32:
// every operand in three bf16 parts (8 + 8 + 8 bits of the 24), the six
// products of parts down to 2^-16 of the largest kept.
#include "attn_common.cuh"
#include "gemm_pair.cuh"

namespace l3 {
namespace {

using namespace sm100;
namespace pg = pairgemm;

constexpr float LOG2E = 1.4426950408889634f;

// first words of the workspace
struct Head {
  int err;       // DEV_ERR_TIMEOUT
  int n_live;    // tokens that take part
  float g_max;   // the largest |g| over them, 1 where all are zero (backward)
  int pad;
};

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

// Sizes and the workspace's layout, from the arguments alone.
struct Layout {
  int64_t n, vocab, d;
  bool fp32, bwd;
  int planes;            // bf16 parts of a value of x and W
  int g_planes, dx_planes;  // and of G, for dW's product and in dx's
  bool lo_all;           // G's second part everywhere, or where `lo` says
  int lo_ld;             // of `lo`: a byte for each 256 columns x 64 tokens of a piece
  int64_t np, dp;        // rows and columns of the gathered x, padded
  int64_t vc, n_pieces;  // vocabulary columns of a piece
  int64_t n_parts;
  // forward of few bf16 tokens: x in place (direct), and as N of a tile of
  // `turned` columns with W's rows as M (0: not so)
  bool direct;
  int turned;
  pg::Tiling logits;
  pg::TwoTilings back;  // dx's and dW's shares
  int part_cols;         // vocabulary columns behind one (max, sum) partial
  size_t head, idx, tgt, lse, ratio, resid, x, part, tlogit, g, lo, dxacc, dwacc, w, total;

  Layout(int64_t n_, int64_t vocab_, int64_t d_, bool fp32_, bool bwd_)
      : n(n_), vocab(vocab_), d(d_), fp32(fp32_), bwd(bwd_) {
    planes = fp32 ? 3 : 1;
    g_planes = fp32 ? 3 : 2;
    lo_all = fp32 || n <= 128;
    dx_planes = fp32 ? 3 : n <= 4 ? 2 : 1;
    np = round_up(std::max<int64_t>(n, 1), 256);
    dp = round_up(d, 64);
    lo_ld = (int)round_up(np / 64, 16);
    // a piece's G takes at most 512 MB (one tile column at least), and so do
    // the parts of its rows of an fp32 W: large enough that a piece's products
    // fill the GPU many times over, small beside the memory of the model
    const int64_t cap = int64_t(512) << 20;
    int64_t most = round_up(vocab, 256);
    if (bwd) most = std::min(most, std::max<int64_t>(cap / (np * 2 * g_planes) / 256 * 256, 256));
    if (fp32) most = std::min(most, std::max<int64_t>(cap / (dp * 2 * planes) / 256 * 256, 256));
    n_pieces = (vocab + most - 1) / most;
    vc = round_up((vocab + n_pieces - 1) / n_pieces, 256);
    n_pieces = (vocab + vc - 1) / vc;
    // One tile row of tokens needs no gather (256 x 32000 x 1024: 23.3 us, 26.8
    // with it). As N they are worth it while the other form's x tile is mostly
    // padding: 1 token 20.7 us against 30.9, 128 tokens x 180000 x 2048 134
    // against 147, 128 x 32000 x 1024 22.7 either way; 64 columns rather than 128
    // take 20.6 instead of 22.7 us for one token.
    direct = !bwd && !fp32 && n <= 256;
    turned = direct && n <= 128 ? (n <= 64 ? 64 : 128) : 0;
    const int products = fp32 ? 6 : 1;
    logits = pg::choose_tiling([&](int tn) { return np / 256 * ((vc + tn - 1) / tn); }, dp / pg::BK,
                               products, INT64_MAX / 1024);  // one share
    part_cols = turned ? 32 : logits.tn / 2;
    n_parts = (vocab + part_cols - 1) / part_cols;
    back = pg::choose_tilings({np / 256, d, vc / pg::BK, np * d, n_pieces > 1, fp32 ? 6 : dx_planes},
                              {vc / 256, d, np / pg::BK, vc * d, false, fp32 ? 6 : lo_all ? 2 : 1});
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t r = at;
      at += (bytes + 1023) & ~size_t(1023);
      return r;
    };
    head = take(sizeof(Head));
    idx = take(np * 4);
    tgt = take(np * 4);
    lse = take(bwd ? np * 4 : 0);
    ratio = take(bwd ? np * 4 : 0);
    resid = take(bwd && dx_planes == 1 ? np * 4 : 0);
    x = take(direct ? 0 : (size_t)planes * np * dp * 2);
    part = take(bwd ? 0 : (size_t)n_parts * np * 8);
    tlogit = take(bwd ? 0 : np * 4);
    g = take(bwd ? (size_t)g_planes * np * vc * 2 : 0);
    lo = take(bwd && !lo_all ? (size_t)(vc / 256) * lo_ld : 0);
    dxacc = take(bwd && dx_partial() ? (size_t)back.splits1 * np * d * 4 : 0);
    dwacc = take(bwd && back.splits2 > 1 ? (size_t)back.splits2 * vc * d * 4 : 0);
    w = take(fp32 ? (size_t)planes * vc * dp * 2 : 0);
    total = at;
  }
  bool dx_partial() const { return n_pieces > 1 || back.splits1 > 1; }
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// v as the sum of three bf16 values, 8 significant bits each
__device__ __forceinline__ void split3(float v, __nv_bfloat16 (&p)[3]) {
  p[0] = __float2bfloat16_rn(v);
  const float r = v - __bfloat162float(p[0]);
  p[1] = __float2bfloat16_rn(r);
  p[2] = __float2bfloat16_rn(r - __bfloat162float(p[1]));
}

// ---------------------------------------------------------------------------
// gather of the tokens that take part
// ---------------------------------------------------------------------------
struct GatherParams {
  const void *x;
  const int32_t *targets;
  const float *lse, *dloss;  // backward
  int n, vocab, d, dp, np;
  int chunk;  // tokens per block, at most 256
  Head *head;
  int32_t *idx, *tgt;
  float *lse_c, *ratio;  // backward
  __nv_bfloat16 *xg;     // planes x np x dp
  float *loss, *lse_out; // forward: values of the tokens left out
  void *dx;              // backward: rows of the tokens left out
};

constexpr int GATHER_THREADS = 512;

// Each block counts the live tokens before its chunk and in all, so that one launch
// orders the rows without atomics. Up to some 10^5 tokens the copy of x bounds it, read
// once and written once (65536 x 1024 bf16: 60 us forward, 113 backward, where the
// blocks read the weights too). Every block reads all targets, from L2: that
// grows with the square of n and bounds the largest calls (2^20 x 1024: 1.8 and 4.4 ms,
// of which the copy is 0.7).
template <bool FP32, bool BWD>
__global__ void __launch_bounds__(GATHER_THREADS) k_xent_gather(GatherParams P) {
  pg::pdl_launch();
  __shared__ int s_before, s_total;
  __shared__ int s_gmax;  // bits of a non-negative float: ordered as integers
  __shared__ int s_pos[256], s_warp[8];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int t0 = blockIdx.x * P.chunk;
  if (tid == 0) {
    s_before = s_total = 0;
    s_gmax = 0;
  }
  __syncthreads();
  int before = 0, total = 0, gm = 0;
#pragma unroll 8
  for (int i = tid; i < P.n; i += GATHER_THREADS) {
    const int t = P.targets[i];
    const bool live = t >= 0 && t < P.vocab;
    total += live;
    before += live && i < t0;
    if (BWD && live) {
      // the largest finite weight: a NaN or infinite one reaches its own row
      // of G, and no other
      const int g = __float_as_int(fabsf(P.dloss[i]));
      if (g < 0x7f800000) gm = max(gm, g);
    }
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (BWD) gm = __reduce_max_sync(0xffffffffu, gm);
  if (lane == 0) {
    atomicAdd(&s_before, before);
    atomicAdd(&s_total, total);
    if (BWD) atomicMax(&s_gmax, gm);
  }
  const int n_chunk = min(P.chunk, P.n - t0);
  int t = -1;
  bool live = false;
  unsigned mask = 0;
  if (warp < 8) {
    if (tid < n_chunk) t = P.targets[t0 + tid];
    live = t >= 0 && t < P.vocab;
    mask = __ballot_sync(0xffffffffu, live);
    if (lane == 0) s_warp[warp] = __popc(mask);
  }
  __syncthreads();
  const float g_max = s_gmax ? __int_as_float(s_gmax) : 1.f;
  if (warp < 8) {
    int pos = s_before + __popc(mask & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) pos += s_warp[w];
    s_pos[tid] = live ? pos : -1;
    if (live) {
      P.idx[pos] = t0 + tid;
      P.tgt[pos] = t;
      if (BWD) {
        P.lse_c[pos] = P.lse[t0 + tid];
        P.ratio[pos] = P.dloss[t0 + tid] / g_max;
      }
    } else if (!BWD && tid < n_chunk) {
      // a target past the vocabulary is a mistake: its loss says so
      const float v = t >= P.vocab ? __int_as_float(0x7fffffff) : 0.f;
      P.loss[t0 + tid] = v;
      P.lse_out[t0 + tid] = v;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    P.head->err = 0;
    P.head->n_live = s_total;
    P.head->g_max = g_max;
  }
  __syncthreads();
  constexpr int WARPS = GATHER_THREADS / 32;
  const int64_t plane = (int64_t)P.np * P.dp;
  for (int j = warp; j < n_chunk; j += WARPS) {
    const int pos = s_pos[j];
    const int64_t tok = t0 + j;
    if (pos < 0) {
      if (BWD) {
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<char *>(P.dx) +
                                               tok * P.d * (FP32 ? 4 : 2));
        for (int c = lane; c < P.d / (FP32 ? 4 : 8); c += 32) out[c] = make_uint4(0, 0, 0, 0);
      }
      continue;
    }
    __nv_bfloat16 *dst = P.xg + (int64_t)pos * P.dp;
    if (FP32) {
      const float *src = static_cast<const float *>(P.x) + tok * P.d;
      for (int c = lane * 4; c < P.dp; c += 128) {
        const float4 v = c < P.d ? *reinterpret_cast<const float4 *>(src + c)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
        __nv_bfloat16 a[4][3];
        split3(v.x, a[0]);
        split3(v.y, a[1]);
        split3(v.z, a[2]);
        split3(v.w, a[3]);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          __nv_bfloat162 o[2] = {{a[0][p], a[1][p]}, {a[2][p], a[3][p]}};
          *reinterpret_cast<uint2 *>(dst + p * plane + c) = *reinterpret_cast<uint2 *>(o);
        }
      }
    } else {
      const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(P.x) + tok * P.d;
      for (int c = lane * 8; c < P.dp; c += 256)
        *reinterpret_cast<uint4 *>(dst + c) =
            c < P.d ? *reinterpret_cast<const uint4 *>(src + c) : make_uint4(0, 0, 0, 0);
    }
  }
  // Rows past the live tokens: a product over the tokens (dW) reads them to
  // the end of its last k-block, where they have to be zeros; elsewhere they
  // reach only results of their own, which are dropped.
  if (!BWD) return;
  const int end = max(64, (s_total + 63) / 64 * 64);
  for (int r = s_total + blockIdx.x; r < end; r += gridDim.x) {
    for (int p = 0; p < (FP32 ? 3 : 1); ++p)
      for (int c = tid * 8; c < P.dp; c += GATHER_THREADS * 8)
        *reinterpret_cast<uint4 *>(P.xg + p * plane + (int64_t)r * P.dp + c) =
            make_uint4(0, 0, 0, 0);
  }
}

// rows v0 .. of an fp32 W as three bf16 planes of vc x dp, zeros past the
// vocabulary and past d; bound by its traffic (10 bytes an element)
__global__ void k_split_w(const float *W, int64_t v0, int64_t vocab, int d, int dp, int64_t vc,
                          __nv_bfloat16 *out) {
  pg::pdl_launch();
  pg::pdl_wait();
  const int per_row = dp / 4;
  const int64_t total = vc * per_row, plane = vc * dp;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / per_row;
    const int c = (int)(i - r * per_row) * 4;
    const float4 v = c < d && v0 + r < vocab
                         ? *reinterpret_cast<const float4 *>(W + (v0 + r) * d + c)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    __nv_bfloat16 a[4][3];
    split3(v.x, a[0]);
    split3(v.y, a[1]);
    split3(v.z, a[2]);
    split3(v.w, a[3]);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      __nv_bfloat162 o[2] = {{a[0][p], a[1][p]}, {a[2][p], a[3][p]}};
      *reinterpret_cast<uint2 *>(out + p * plane + r * dp + c) = *reinterpret_cast<uint2 *>(o);
    }
  }
}

// ---------------------------------------------------------------------------
// epilogues of the products
// ---------------------------------------------------------------------------
// (max, sum of exp(s - max)) of a row over the warp's half of a tile, but for the
// target's logit, which is stored where it is among them
struct EpiStats {
  const int32_t *tgt;
  float2 *part;  // [n_parts][np]
  float *tlogit;
  int64_t np;
  int v0, vocab;
  int n;  // > 0: that many rows, all live (x in place)
  int part_cols;

  static constexpr int BOX_BYTES = 0;
  static constexpr bool LOADS = false;
  static constexpr int WARPS = 8;
  static constexpr bool SUMS = true;
  __device__ __forceinline__ void prefetch(pg::WarpBoxes &, int, int, int) const {}

  struct State {
    int m, nv, te, slot;
    float mx, sum;
  };
  __device__ __forceinline__ State begin(int, int m, int c0, int n_live) const {
    const int col0 = v0 + c0;
    const bool live = m < (n ? n : n_live);
    // nv: columns of this warp inside the vocabulary (none for a dead row)
    return State{m, live ? vocab - col0 : 0, live ? tgt[m] - col0 : -1, col0 / part_cols, -INFINITY, 0.f};
  }
  __device__ __forceinline__ void chunk(State &s, pg::WarpBoxes &, int c, float (&v)[32]) const {
    if (c + 32 > s.nv) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (c + e >= s.nv) v[e] = -INFINITY;
    }
    if (s.te >= c && s.te < c + 32) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (s.te == c + e) {
          tlogit[s.m] = v[e];
          v[e] = -INFINITY;
        }
    }
    float cm = s.mx;
#pragma unroll
    for (int e = 0; e < 32; ++e) cm = fmaxf(cm, v[e]);
    // a row of -inf so far has no finite reference. The difference first: a
    // rounded max * log2 e would be off by 2^-24 of the logit, not of the difference
    const float ref = cm == -INFINITY ? 0.f : cm;
    float s0 = s.sum * ex2((s.mx - ref) * LOG2E), s1 = 0.f;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      s0 += ex2((v[e] - ref) * LOG2E);
      s1 += ex2((v[e + 1] - ref) * LOG2E);
    }
    s.sum = s0 + s1;
    s.mx = cm;
  }
  __device__ __forceinline__ void end(State &s) const {
    if (s.nv > 0) part[(int64_t)s.slot * np + s.m] = make_float2(s.mx, s.sum);
  }
};

// The same with W's rows as the tile's rows and the tokens as its columns: a
// warp's 32 rows are one partial of each token. The reductions over the rows run
// across the warp's lanes, 32 tokens at a time, and leave token t's result in
// lane t.
struct EpiStatsTurned {
  const int32_t *targets;
  float2 *part;  // [n_parts][np]
  float *tlogit;
  int64_t np;
  int n, vocab;

  static constexpr int BOX_BYTES = 0;
  static constexpr bool LOADS = false;
  static constexpr int WARPS = 8;
  static constexpr bool SUMS = true;
  __device__ __forceinline__ void prefetch(pg::WarpBoxes &, int, int, int) const {}

  struct State {
    int m, c0;
  };
  __device__ __forceinline__ State begin(int, int m, int c0, int) const { return State{m, c0}; }
  __device__ __forceinline__ void chunk(State &s, pg::WarpBoxes &box, int c, float (&v)[32]) const {
    if (s.c0 + c >= n || (s.m & ~31) >= vocab) return;  // the whole warp alike
    const int tok = s.c0 + c + box.lane;
    // targets among the warp's rows: in few warps, but there as many as the tokens (a
    // batch may have the same target throughout)
    const int row = tok < n ? targets[tok] - (s.m & ~31) : -1;
    if (__any_sync(0xffffffffu, row >= 0 && row < 32)) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (__shfl_sync(0xffffffffu, row, e) == box.lane) {
          tlogit[s.c0 + c + e] = v[e];
          v[e] = -INFINITY;
        }
    }
    float w[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) w[e] = v[e] = s.m < vocab ? v[e] : -INFINITY;
    const float mx = attn::warp_transpose_reduce<false>(w, box.lane);
    // a row of -inf has no finite reference
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = ex2((v[e] - __shfl_sync(0xffffffffu, ref, e)) * LOG2E);
    const float sum = attn::warp_transpose_reduce<true>(v, box.lane);
    if (tok < n) part[(int64_t)(s.m / 32) * np + tok] = make_float2(mx, sum);
  }
  __device__ __forceinline__ void end(State &) const {}
};

// G = (exp(s - lse) - [column is the target]) g / g_max in bf16 parts; zeros
// past the live tokens and past the vocabulary
template <int PLANES>
struct EpiGrad {
  CUtensorMap out;  // planes x np rows, vc columns
  const int32_t *tgt;
  const float *lse, *ratio;
  int np, v0, vocab;
  float *resid;  // what the target's element lost to the first part, or NULL
  // not NULL: a byte [256 columns][64 tokens] that says whether the block holds a
  // target, and the second part only where it does
  uint8_t *lo;
  int lo_ld;

  static constexpr int BOX_BYTES = 2 * pg::BOX;  // in turn, a plane's 32 columns each
  static constexpr bool LOADS = false;
  static constexpr int WARPS = 8;
  static constexpr bool SUMS = true;
  __device__ __forceinline__ void prefetch(pg::WarpBoxes &, int, int, int) const {}

  struct State {
    int nv, te, m, c0;
    float lse, rt;
    bool parts;  // more than the first
  };
  __device__ __forceinline__ State begin(int, int m, int c0, int n_live) const {
    const bool live = m < n_live;
    const int t = live ? tgt[m] - v0 : -1;
    bool parts = PLANES > 1;
    if (PLANES == 2 && lo) {
      // the block's other 32 tokens are another warp's, which comes to the same answer
      const int t2 = (m ^ 32) < n_live ? tgt[m ^ 32] - v0 : -1, block = c0 >> 8;
      parts = __any_sync(0xffffffffu, (t >= 0 && t >> 8 == block) || (t2 >= 0 && t2 >> 8 == block));
      if ((m & 31) == 0) lo[(int64_t)block * lo_ld + (m >> 6)] = parts;
    }
    return State{live ? vocab - (v0 + c0) : 0, live ? t - c0 : -1, m, c0,
                 live ? lse[m] : 0.f, live ? ratio[m] : 0.f, parts};
  }
  __device__ __forceinline__ void chunk(State &s, pg::WarpBoxes &box, int c, float (&v)[32]) const {
    // a row's target is in few of its columns, and few tiles end inside their columns
    const bool hit = s.te >= c && s.te < c + 32;
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = ex2((v[e] - s.lse) * LOG2E);
    if (hit) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (s.te == c + e) v[e] -= 1.f;
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] *= s.rt;
    if (c + 32 > s.nv) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (c + e >= s.nv) v[e] = 0.f;
    }
    if (PLANES < 3 && hit && resid) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (s.te == c + e) resid[s.m] = v[e] - __bfloat162float(__float2bfloat16_rn(v[e]));
    }
#pragma unroll
    for (int p = 0; p < PLANES; ++p) {
      const int b = (s.parts ? c / 32 * PLANES + p : c / 32) & 1;
      box.stores_read<1>();  // this box's last store
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 o;
        __nv_bfloat162 *o2 = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
        for (int e = 0; e < 4; ++e) o2[e] = __floats2bfloat162_rn(v[j * 8 + 2 * e], v[j * 8 + 2 * e + 1]);
        *box.piece(b, j) = o;
      }
      box.written();
      if (box.lane == 0) {
        box.store(b, &out, s.c0 + c, p * np + (s.m & ~31));
        box.commit();
      }
      if (!s.parts) break;
      if (p + 1 < PLANES) {  // what the next part has to hold
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] -= __bfloat162float(__float2bfloat16_rn(v[e]));
      }
    }
  }
  __device__ __forceinline__ void end(State &) const {}
};

__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint4 o;
  __nv_bfloat162 *o2 = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
  for (int e = 0; e < 4; ++e) o2[e] = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
  *reinterpret_cast<uint4 *>(p) = o;
}

// What a finished dx from one part of G still lacks: resid[m] times the target's
// row of W (resid NULL: nothing)
struct Lost {
  const float *resid;
  const int32_t *tgt;
  const __nv_bfloat16 *w;
};

// A gradient's rows: dx (row m of the live tokens, in the caller's row idx[m])
// or a piece of dW. Either finished here, times g_max, or as an fp32 partial
// (a share of the depth, or the sum of the pieces so far) that k_sum_rows joins.
template <class T>
struct EpiRows {
  const int32_t *idx;  // dx
  const Head *head;
  T *out;       // the finished rows, or NULL:
  float *acc;   // [share][slice rows][d]
  int64_t slice;
  int rows, d;  // rows of dW's piece
  int add;      // onto what acc holds
  Lost lost;

  static constexpr int BOX_BYTES = 0;
  static constexpr bool LOADS = false;
  static constexpr int WARPS = 8;
  static constexpr bool SUMS = sizeof(T) == 4;
  __device__ __forceinline__ void prefetch(pg::WarpBoxes &, int, int, int) const {}

  struct State {
    bool live;
    int c0;
    float gm;
    T *out;
    float *acc;
    float r;
    const __nv_bfloat16 *w;
  };
  __device__ __forceinline__ State begin(int share, int m, int c0, int n_live) const {
    const bool live = m < (idx ? n_live : rows);
    const int64_t row = !live ? 0 : out && idx ? idx[m] : m;
    const bool lost_any = sizeof(T) == 2 && out && lost.resid && live;
    return State{live, c0, out ? head->g_max : 1.f, out ? out + row * d : nullptr,
                 out ? nullptr : acc + share * slice + row * d, lost_any ? lost.resid[m] : 0.f,
                 lost_any ? lost.w + (int64_t)lost.tgt[m] * d : nullptr};
  }
  __device__ __forceinline__ void chunk(State &s, pg::WarpBoxes &, int c, float (&v)[32]) const {
    if (!s.live) return;
    uint4 w[4];  // on their way together
    if (sizeof(T) == 2 && s.w)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = s.c0 + c + j * 8;
        if (col < d) w[j] = __ldg(reinterpret_cast<const uint4 *>(s.w + col));
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = s.c0 + c + j * 8;
      if (sizeof(T) == 2 && s.w && col < d) {
        const __nv_bfloat162 *w2 = reinterpret_cast<const __nv_bfloat162 *>(&w[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __bfloat1622float2(w2[e]);
          v[j * 8 + 2 * e] = fmaf(s.r, f.x, v[j * 8 + 2 * e]);
          v[j * 8 + 2 * e + 1] = fmaf(s.r, f.y, v[j * 8 + 2 * e + 1]);
        }
      }
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = v[j * 8 + e] * s.gm;
      // d is a multiple of 16 (bf16) or 4 (fp32): the last four may be absent
      const bool lo = col < d, hi = col + 4 < d;
      if (out) {
        if (hi)
          store8(s.out + col, f);
        else if (sizeof(T) == 4 && lo)
          *reinterpret_cast<float4 *>(s.out + col) = make_float4(f[0], f[1], f[2], f[3]);
        continue;
      }
      if (add) {
        if (lo) {
          const float4 a = *reinterpret_cast<const float4 *>(s.acc + col);
          f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
        }
        if (hi) {
          const float4 a = *reinterpret_cast<const float4 *>(s.acc + col + 4);
          f[4] += a.x, f[5] += a.y, f[6] += a.z, f[7] += a.w;
        }
      }
      if (lo) *reinterpret_cast<float4 *>(s.acc + col) = make_float4(f[0], f[1], f[2], f[3]);
      if (hi) *reinterpret_cast<float4 *>(s.acc + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
  __device__ __forceinline__ void end(State &) const {}
};

// A finished piece of a bf16 dW through boxes, whose stores fill whole sectors
// and end at dW's last row and column: with few tokens the rows are all that
// dW costs (32000 x 1024 from 256 tokens: its launch 50 -> 35 us)
struct EpiDwBoxes {
  CUtensorMap out;  // the piece's rows
  const Head *head;
  int rows, d;

  static constexpr int BOX_BYTES = 2 * pg::BOX;
  static constexpr bool LOADS = false;
  static constexpr int WARPS = 8;
  static constexpr bool SUMS = false;
  __device__ __forceinline__ void prefetch(pg::WarpBoxes &, int, int, int) const {}

  struct State {
    int m_warp, c0;
    float gm;
  };
  __device__ __forceinline__ State begin(int, int m, int c0, int) const {
    return State{m & ~31, c0, head->g_max};
  }
  __device__ __forceinline__ void chunk(State &s, pg::WarpBoxes &box, int c, float (&v)[32]) const {
    if (s.m_warp >= rows || s.c0 + c >= d) return;  // the whole warp alike
    const int b = c / 32 & 1;
    box.stores_read<1>();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 o;
      __nv_bfloat162 *o2 = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o2[e] = __floats2bfloat162_rn(v[j * 8 + 2 * e] * s.gm, v[j * 8 + 2 * e + 1] * s.gm);
      *box.piece(b, j) = o;
    }
    box.written();
    if (box.lane == 0) {
      box.store(b, &out, s.c0 + c, s.m_warp);
      box.commit();
    }
  }
  __device__ __forceinline__ void end(State &) const {}
};

// out[row] = g_max times the sum of the shares' partials, in share order;
// memory-bound. Two such sums share a launch: the first `blocks` blocks run `a`,
// the others `b`.
template <class T>
struct SumRows {
  const float *acc;  // [shares][slice]
  int64_t slice;
  int shares;
  const int32_t *idx;  // the row in `out`, of the live ones; NULL: all `rows`
  int rows;
  T *out;
  Lost lost;
};

template <class T>
__global__ void k_sum_rows(SumRows<T> a, SumRows<T> b, int blocks, const Head *head, int d) {
  pg::pdl_launch();
  pg::pdl_wait();
  const bool second = (int)blockIdx.x >= blocks;
  const SumRows<T> P = second ? b : a;
  const int block = second ? blockIdx.x - blocks : blockIdx.x;
  const int grid = second ? gridDim.x - blocks : blocks;
  const int n = P.idx ? head->n_live : P.rows, per_row = d / 4;
  const float gm = head->g_max;
  for (int64_t i = block * (int64_t)blockDim.x + threadIdx.x; i < (int64_t)n * per_row;
       i += (int64_t)grid * blockDim.x) {
    const int64_t r = i / per_row;
    const int c = (int)(i - r * per_row) * 4;
    float4 v = *reinterpret_cast<const float4 *>(P.acc + r * d + c);
    for (int s = 1; s < P.shares; ++s) {
      const float4 w = *reinterpret_cast<const float4 *>(P.acc + s * P.slice + r * d + c);
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    if (sizeof(T) == 2 && P.lost.resid) {
      const uint2 w = *reinterpret_cast<const uint2 *>(P.lost.w + (int64_t)P.lost.tgt[r] * d + c);
      const float2 w0 = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(&w)[0]);
      const float2 w1 = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(&w)[1]);
      const float e = P.lost.resid[r];
      v.x = fmaf(e, w0.x, v.x), v.y = fmaf(e, w0.y, v.y);
      v.z = fmaf(e, w1.x, v.z), v.w = fmaf(e, w1.y, v.w);
    }
    v.x *= gm, v.y *= gm, v.z *= gm, v.w *= gm;
    T *o = P.out + (P.idx ? (int64_t)P.idx[r] : r) * d + c;
    if (sizeof(T) == 4) {
      *reinterpret_cast<float4 *>(o) = v;
    } else {
      __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
      *reinterpret_cast<uint2 *>(o) = *reinterpret_cast<uint2 *>(h);
    }
  }
}

struct JoinParams {
  const float2 *part;
  int64_t np;
  int n_parts;
  const float *tlogit;
  const int32_t *idx;      // NULL: rows in place, `targets` tells which are out
  const int32_t *targets;
  int n, vocab;
  const Head *head;
  float *loss, *lse;
};

// Joins a row's partials: 32 rows a block, 32 threads a row, and CL blocks (a
// cluster) a row where there are few rows: each joins every CL-th group of
// partials, the first one the blocks' results.
template <int CL>
__global__ void __launch_bounds__(1024) k_xent_join(JoinParams P) {
  __shared__ float2 s[32][33];
  __shared__ float2 joined[32];
  pg::pdl_wait();
  const int n_live = P.idx ? P.head->n_live : P.n;
  const int rank = CL > 1 ? blockIdx.x % CL : 0, r0 = blockIdx.x / CL * 32;
  const int r = r0 + threadIdx.x, y = threadIdx.y;
  if (r0 >= n_live) return;  // the whole cluster alike
  float mx = -INFINITY, sum = 0.f;
  auto join = [&](float2 v) {
    const float m = fmaxf(mx, v.x);
    const float ref = m == -INFINITY ? 0.f : m;
    sum = sum * ex2((mx - ref) * LOG2E) + v.y * ex2((v.x - ref) * LOG2E);
    mx = m;
  };
  if (r < n_live)
#pragma unroll 4
    for (int p = y * CL + rank; p < P.n_parts; p += 32 * CL) join(P.part[(int64_t)p * P.np + r]);
  s[y][threadIdx.x] = make_float2(mx, sum);
  __syncthreads();
  // thread x of the first warp holds its row's result of this block
  if (y == 0) {
    for (int p = 1; p < 32; ++p) join(s[p][threadIdx.x]);
    joined[threadIdx.x] = make_float2(mx, sum);
  }
  if (CL > 1) {
    __syncwarp();
    cluster_sync();
  }
  if (rank == 0 && y == 0 && r < n_live) {
    for (int c = 1; c < CL; ++c) {
      const uint32_t at = map_shared_rank(&joined[threadIdx.x], c);
      join(make_float2(ld_shared_cluster_f32(at), ld_shared_cluster_f32(at + 4)));
    }
    const float nan = __int_as_float(0x7fffffff);
    const int live_t = P.idx ? 0 : P.targets[r];
    const bool live = live_t >= 0 && live_t < P.vocab;
    // the others' sum, and the target beside it
    const float st = live ? P.tlogit[r] : 0.f, top = fmaxf(mx, st), above = top - st;
    const float others = sum * expf(mx - top);
    float lse = top + logf(others + expf(-above));
    float loss = above < 30.f ? log1pf(others * expf(above)) : above + logf(others + expf(-above));
    // a wait that gave up left rows unwritten: say so in every loss
    if (P.head->err) loss = lse = nan;
    if (!live) loss = lse = live_t < 0 ? 0.f : nan;
    const int at = P.idx ? P.idx[r] : r;
    P.lse[at] = lse;
    P.loss[at] = loss;
  }
  if (CL > 1) cluster_sync();  // the first block has read the others' shared memory
}

struct Pointer {
  const void *p;
  uintptr_t align;
};

// the sizes that the calls take, before anything is computed from them
l3_status check_sizes(int64_t n, int64_t vocab, int64_t d, int32_t dtype) {
  if (n < 0 || vocab < 1 || d < 1 || (dtype != L3_BF16 && dtype != L3_FP32)) {
    set_error("cross entropy: need n >= 0, vocab >= 1, d >= 1 and dtype L3_BF16 or L3_FP32");
    return L3_ERR_INVALID_ARG;
  }
  if (d % (dtype == L3_BF16 ? 16 : 4) || d > 16384 || n > (1 << 20) || vocab > (1 << 24)) {
    set_error("cross entropy: d must be a multiple of 16 (bf16) or 4 (fp32) and at most 16384, "
              "n at most 2^20, vocab at most 2^24");
    return L3_ERR_UNSUPPORTED;
  }
  return L3_OK;
}

l3_status check(const Pointer *ptrs, int n_ptrs, int64_t n, int64_t vocab, int64_t d,
                int32_t dtype, int64_t ws_bytes, bool bwd, int *device) {
  const l3_status st = check_sizes(n, vocab, d, dtype);
  if (st != L3_OK || (n == 0 && !bwd)) return st;
  for (int i = 0; i < n_ptrs; ++i) {
    if (!ptrs[i].p) {
      set_error("cross entropy: a tensor or workspace pointer is NULL");
      return L3_ERR_INVALID_ARG;
    }
    if (reinterpret_cast<uintptr_t>(ptrs[i].p) & (ptrs[i].align - 1)) {
      set_error("cross entropy: x, W, dx, dW and the workspace must be 16-byte aligned, the "
                "vectors 4-byte aligned");
      return L3_ERR_INVALID_ARG;
    }
  }
  const Layout L(n, vocab, d, dtype == L3_FP32, bwd);
  if (ws_bytes < (int64_t)L.total) {
    set_error("cross entropy: the workspace holds " + std::to_string(ws_bytes) + " bytes, " +
              std::to_string(L.total) + " are needed");
    return L3_ERR_INVALID_ARG;
  }
  L3_CUDA_TRY(current_device(device));
  return L3_OK;
}

template <bool FP32, bool BWD>
l3_status launch_gather(const GatherParams &G, cudaStream_t s) {
  const unsigned blocks = (unsigned)((G.n + G.chunk - 1) / G.chunk);
  LaunchTimer t("xent_gather", s);
  k_xent_gather<FP32, BWD><<<blocks, GATHER_THREADS, 0, s>>>(G);
  L3_CUDA_TRY(cudaGetLastError());
  return L3_OK;
}

// k-blocks of the logits' chains. The losses are fp32: short chains (bf16 operands
// 2048 deep in one chain leave the loss 1.7e-6 off; 256-deep ones cost 12 % of the
// forward pass, 512-deep ones 2 %). Few tokens, whose tiles wait for W, can have
// shorter ones: a sure token's loss is 2.6e-6 off at worst with 256-deep chains, 1.3e-6
// with 128-deep ones (64 x 32000 x 1024: 20.8 and 22.8 us; 1 token 20.8 both).
// The backward pass takes the same chains: in others, a logit drifts away from the
// lse that holds it, and exp(s - lse) - 1 with it (one chain 4096 deep, logits near
// 100: 1.5e-3). It costs the gradients of 8192 tokens x 180000 x 2048 2.5 %.
int logits_chunk(const Layout &L) { return L.fp32 ? 1 : L.n <= 32 ? 2 : L.n <= 128 ? 4 : 8; }

// x W_piece^T with the given epilogue
template <int PLANES, class Epi>
l3_status launch_logits(const Layout &L, char *ws, const void *x, const void *W, int64_t v0,
                        const Epi &epi, const char *name, int device, cudaStream_t s) {
  CUtensorMap mA, mB;
  l3_status st;
  const int64_t rows = std::min(L.vc, L.vocab - v0);
  st = L.direct ? pg::operand_map(&mA, x, true, L.n, L.d, L.d, false, pg::BM)
                : pg::operand_map(&mA, ws + L.x, true, L.planes * L.np, L.dp, L.dp, false, pg::BM);
  if (st != L3_OK) return st;
  st = L.fp32 ? pg::operand_map(&mB, ws + L.w, true, L.planes * L.vc, L.dp, L.dp, false, L.logits.tn / 2)
              : pg::operand_map(&mB, W, true, L.vocab, L.d, L.d, false, L.logits.tn / 2);
  if (st != L3_OK) return st;
  const Head *head = reinterpret_cast<const Head *>(ws + L.head);
  pg::Args P = {};
  P.tiles_m = (int)(L.np / 256);
  P.tiles_n = (int)((rows + L.logits.tn - 1) / L.logits.tn);
  P.batch = 1;
  P.nkb = (int)(L.dp / pg::BK);
  P.dyn = L.direct ? nullptr : &head->n_live;
  P.dyn_rows = !L.direct;
  P.clear_err = L.direct;
  P.chunk = logits_chunk(L);
  P.group = 16;  // 16 tile rows of x beside a few of W's columns: both stay in L2
  P.bf16 = 1;
  P.b_off = (int)(L.fp32 ? 0 : v0);
  P.a_plane = (int)L.np;
  P.b_plane = (int)L.vc;
  P.err = &const_cast<Head *>(head)->err;
  LaunchTimer t(name, s);
  // in place, it is the chain's first
  return L.logits.tn == 256
             ? pg::launch<256, PLANES, PLANES, pg::K_MAJOR, pg::K_MAJOR>(mA, mB, P, epi, device, s, !L.direct)
             : pg::launch<128, PLANES, PLANES, pg::K_MAJOR, pg::K_MAJOR>(mA, mB, P, epi, device, s, !L.direct);
}

// W x^T of few tokens: W's rows are M, the tokens N
template <int T>
l3_status launch_turned(const Layout &L, Head *head, const void *x, const void *W,
                        const EpiStatsTurned &epi, int device, cudaStream_t s) {
  CUtensorMap mA, mB;
  l3_status st;
  if ((st = pg::operand_map(&mA, W, true, L.vocab, L.d, L.d, false, pg::BM)) != L3_OK) return st;
  if ((st = pg::operand_map(&mB, x, true, L.n, L.d, L.d, false, T / 2)) != L3_OK) return st;
  pg::Args P = {};
  P.tiles_m = (int)((L.vocab + 255) / 256);
  P.tiles_n = P.batch = P.group = 1;
  P.nkb = (int)(L.dp / pg::BK);
  P.chunk = logits_chunk(L);
  P.bf16 = 1;
  P.clear_err = 1;
  P.err = &head->err;
  LaunchTimer t("xent_logits", s);
  return pg::launch<T, 1, 1, pg::K_MAJOR, pg::K_MAJOR>(mA, mB, P, epi, device, s, false);
}

l3_status split_w(const Layout &L, char *ws, const void *W, int64_t v0, int device, cudaStream_t s) {
  if (!L.fp32) return L3_OK;
  LaunchTimer t("xent_split_w", s);
  const int64_t work = (L.vc * (L.dp / 4) + 255) / 256;
  return pg::launch_link(k_split_w, dim3((unsigned)std::min<int64_t>(work, sm_count(device) * 8)),
                         dim3(256), s, true, static_cast<const float *>(W), v0, L.vocab, (int)L.d,
                         (int)L.dp, L.vc, reinterpret_cast<__nv_bfloat16 *>(ws + L.w));
}

int chunk_of(int64_t n) { return n <= 2048 ? 16 : n <= 8192 ? 32 : n <= 65536 ? 128 : 256; }

// dx and a piece of dW
template <int PA, int PB, class Dx, class Dw>
l3_status launch_gradients(Dx dx, Dw dw, const Layout &L, int device, cudaStream_t s) {
  dx.P.batch = dx.P.splits = L.back.splits1;
  dw.P.batch = dw.P.splits = L.back.splits2;
  dx.P.tiles_n = dw.P.tiles_n = (int)((L.d + L.back.tn - 1) / L.back.tn);
  LaunchTimer t("xent_gradients", s);
  return L.back.tn == 256 ? pg::launch_problems<256, PA, PB, true>(dx, dw, device, s, true)
                          : pg::launch_problems<128, PA, PB, true>(dx, dw, device, s, true);
}

// one sum, or two (out NULL: none)
template <class T>
l3_status sum_rows(const SumRows<T> &a, const SumRows<T> &b, const Head *head, int64_t d,
                   int device, cudaStream_t s) {
  if (!a.out && !b.out) return L3_OK;
  const auto blocks = [&](const SumRows<T> &w) {
    return !w.out ? 0 : (int)std::min<int64_t>((w.rows * (d / 4) + 255) / 256, sm_count(device) * 8);
  };
  LaunchTimer t("xent_sum_rows", s);
  return pg::launch_link(k_sum_rows<T>, dim3((unsigned)(blocks(a) + blocks(b))), dim3(256), s, true,
                         a, b, blocks(a), head, (int)d);
}

template <class T>
l3_status backward(const Layout &L, char *ws, const void *x, const void *W, const int32_t *targets,
                   const float *lse, const float *dloss, void *dx, void *dW, int device,
                   cudaStream_t s) {
  constexpr bool FP32 = sizeof(T) == 4;
  constexpr int PLANES = FP32 ? 3 : 1, GP = FP32 ? 3 : 2;  // parts of x and W, and of G
  Head *head = reinterpret_cast<Head *>(ws + L.head);
  GatherParams G = {};
  G.x = x;
  G.targets = targets;
  G.lse = lse;
  G.dloss = dloss;
  G.n = (int)L.n;
  G.vocab = (int)L.vocab;
  G.d = (int)L.d;
  G.dp = (int)L.dp;
  G.np = (int)L.np;
  G.chunk = chunk_of(L.n);
  G.head = head;
  G.idx = reinterpret_cast<int32_t *>(ws + L.idx);
  G.tgt = reinterpret_cast<int32_t *>(ws + L.tgt);
  G.lse_c = reinterpret_cast<float *>(ws + L.lse);
  G.ratio = reinterpret_cast<float *>(ws + L.ratio);
  G.xg = reinterpret_cast<__nv_bfloat16 *>(ws + L.x);
  G.dx = dx;
  l3_status st = launch_gather<FP32, true>(G, s);
  __nv_bfloat16 *g = reinterpret_cast<__nv_bfloat16 *>(ws + L.g);
  float *resid = L.dx_planes == 1 ? reinterpret_cast<float *>(ws + L.resid) : nullptr;
  const Lost lost{resid, G.tgt, static_cast<const __nv_bfloat16 *>(W)};
  for (int64_t i = 0; st == L3_OK && i < L.n_pieces; ++i) {
    const int64_t v0 = i * L.vc;
    const int64_t rows = std::min(L.vc, L.vocab - v0);
    if ((st = split_w(L, ws, W, v0, device, s)) != L3_OK) return st;
    uint8_t *lo = L.lo_all ? nullptr : reinterpret_cast<uint8_t *>(ws + L.lo);
    EpiGrad<GP> eg{{}, G.tgt, G.lse_c, G.ratio, (int)L.np, (int)v0, (int)L.vocab, resid, lo, L.lo_ld};
    if ((st = pg::box_map(&eg.out, g, true, GP * L.np, L.vc, L.vc)) != L3_OK) return st;
    if ((st = launch_logits<PLANES>(L, ws, x, W, v0, eg, "xent_grad_logits", device, s)) != L3_OK) return st;
    // dx += G W: G K-major, W MN-major (its rows are k)
    pg::Problem<pg::K_MAJOR, pg::MN_MAJOR, EpiRows<T>> px{};
    if ((st = pg::operand_map(&px.mA, g, true, GP * L.np, L.vc, L.vc, false, pg::BM)) != L3_OK)
      return st;
    st = FP32 ? pg::operand_map(&px.mB, ws + L.w, true, L.planes * L.vc, L.dp, L.dp, true, 0)
              : pg::operand_map(&px.mB, W, true, L.vocab, L.d, L.d, true, 0);
    if (st != L3_OK) return st;
    pg::Args &P = px.P;
    P.tiles_m = (int)(L.np / 256);
    P.nkb = (int)((rows + pg::BK - 1) / pg::BK);
    P.dyn = &head->n_live;
    P.dyn_rows = 1;
    P.chunk = FP32 ? 1 : 0;  // a bf16 result's own rounding is far larger
    P.group = 8;
    P.bf16 = 1;
    P.b_off = (int)(FP32 ? 0 : v0);
    P.a_plane = (int)L.np;
    P.b_plane = (int)L.vc;
    P.a_hi = L.dx_planes == 1;
    P.err = &head->err;
    px.epi.idx = G.idx;
    px.epi.head = head;
    px.epi.out = L.dx_partial() ? nullptr : static_cast<T *>(dx);
    px.epi.acc = reinterpret_cast<float *>(ws + L.dxacc);
    px.epi.slice = L.np * L.d;
    px.epi.d = (int)L.d;
    px.epi.add = i > 0;
    px.epi.lost = lost;
    // dW = G^T x: both MN-major (their rows are the tokens)
    EpiRows<T> ew{};
    ew.head = head;
    ew.out = L.back.splits2 > 1 ? nullptr : static_cast<T *>(dW) + v0 * L.d;
    ew.acc = reinterpret_cast<float *>(ws + L.dwacc);
    ew.slice = L.vc * L.d;
    ew.rows = (int)rows;
    ew.d = (int)L.d;
    const auto dw_problem = [&](auto &p) {
      p.P = P;
      p.P.tiles_m = (int)((rows + 255) / 256);
      p.P.nkb = (int)(L.np / pg::BK);
      p.P.dyn_rows = 0;
      p.P.a_hi = 0;
      p.P.a_lo = lo;
      p.P.a_lo_ld = L.lo_ld;
      p.P.dyn_k = 1;
      p.P.b_off = 0;
      p.P.b_plane = (int)L.np;
      const l3_status r = pg::operand_map(&p.mA, g, true, GP * L.np, L.vc, L.vc, true, 0);
      return r != L3_OK ? r
                        : pg::operand_map(&p.mB, ws + L.x, true, L.planes * L.np, L.dp, L.dp, true, 0);
    };
    const auto run = [&](auto &pw) {
      const l3_status r = dw_problem(pw);
      return r != L3_OK ? r : launch_gradients<GP, PLANES>(px, pw, L, device, s);
    };
    bool boxes = false;
    if constexpr (!FP32) {
      if (ew.out) {
        boxes = true;
        pg::Problem<pg::MN_MAJOR, pg::MN_MAJOR, EpiDwBoxes> pw{{}, {}, {}, {{}, head, ew.rows, ew.d}};
        st = pg::box_map(&pw.epi.out, ew.out, true, rows, L.d, L.d);
        if (st == L3_OK) st = run(pw);
      }
    }
    if (!boxes) {
      pg::Problem<pg::MN_MAJOR, pg::MN_MAJOR, EpiRows<T>> pw{{}, {}, {}, ew};
      st = run(pw);
    }
    if (st != L3_OK) return st;
    // the piece's dW, and after the last piece dx
    SumRows<T> sw{}, sx{};
    if (!ew.out)
      sw = SumRows<T>{ew.acc, ew.slice, L.back.splits2, nullptr, (int)rows, static_cast<T *>(dW) + v0 * L.d};
    if (L.dx_partial() && i + 1 == L.n_pieces)
      sx = SumRows<T>{px.epi.acc, px.epi.slice, L.back.splits1, G.idx, (int)L.n, static_cast<T *>(dx), lost};
    st = sum_rows(sw, sx, head, L.d, device, s);
  }
  if (st != L3_OK) return st;
  const int64_t row = L.d * (int64_t)sizeof(T);
  return launch_spoil(&head->err, {dx, L.n * row}, {dW, L.vocab * row}, s);
}

}  // namespace
}  // namespace l3

using namespace l3;

extern "C" {

int64_t l3_xent_workspace(int64_t n, int64_t vocab, int64_t d, int32_t dtype, int32_t backward) {
  set_error("");
  if (check_sizes(n, vocab, d, dtype) != L3_OK) return -1;
  return (int64_t)Layout(n, vocab, d, dtype == L3_FP32, backward != 0).total;
}

l3_status l3_xent_forward(const void *x, const void *W, const int32_t *targets, int64_t n,
                          int64_t vocab, int64_t d, int32_t dtype, float *loss, float *lse,
                          void *workspace, int64_t workspace_bytes, void *stream) {
  set_error("");
  int device = 0;
  const Pointer ptrs[] = {{x, 16}, {W, 16}, {workspace, 16}, {targets, 4}, {loss, 4}, {lse, 4}};
  l3_status st = check(ptrs, 6, n, vocab, d, dtype, workspace_bytes, false, &device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (st != L3_OK) return st;
  if (n == 0) return clear_error_word(workspace, workspace_bytes, s);
  const Layout L(n, vocab, d, dtype == L3_FP32, false);
  char *ws = static_cast<char *>(workspace);
  Head *head = reinterpret_cast<Head *>(ws + L.head);
  JoinParams J = {};
  J.part = reinterpret_cast<float2 *>(ws + L.part);
  J.np = L.np;
  J.n_parts = (int)L.n_parts;
  J.targets = targets;
  J.n = (int)n;
  J.vocab = (int)vocab;
  J.tlogit = reinterpret_cast<float *>(ws + L.tlogit);
  J.head = head;
  J.loss = loss;
  J.lse = lse;
  float2 *part = reinterpret_cast<float2 *>(ws + L.part);
  float *tlogit = reinterpret_cast<float *>(ws + L.tlogit);
  if (L.turned) {
    const EpiStatsTurned e{targets, part, tlogit, L.np, (int)n, (int)vocab};
    st = L.turned == 64 ? launch_turned<64>(L, head, x, W, e, device, s)
                        : launch_turned<128>(L, head, x, W, e, device, s);
  } else {
    EpiStats es{targets, part, tlogit, L.np, 0, (int)vocab, (int)n, L.part_cols};
    if (!L.direct) {
      GatherParams G = {};
      G.x = x;
      G.targets = targets;
      G.n = (int)n;
      G.vocab = (int)vocab;
      G.d = (int)d;
      G.dp = (int)L.dp;
      G.np = (int)L.np;
      G.chunk = chunk_of(n);
      G.head = head;
      G.idx = reinterpret_cast<int32_t *>(ws + L.idx);
      G.tgt = reinterpret_cast<int32_t *>(ws + L.tgt);
      G.xg = reinterpret_cast<__nv_bfloat16 *>(ws + L.x);
      G.loss = loss;
      G.lse_out = lse;
      J.idx = G.idx;
      es.tgt = G.tgt;
      es.n = 0;
      st = L.fp32 ? launch_gather<true, false>(G, s) : launch_gather<false, false>(G, s);
    }
    for (int64_t i = 0; st == L3_OK && i < L.n_pieces; ++i) {
      es.v0 = (int)(i * L.vc);
      if ((st = split_w(L, ws, W, es.v0, device, s)) != L3_OK) return st;
      st = L.fp32 ? launch_logits<3>(L, ws, x, W, es.v0, es, "xent_logits", device, s)
                  : launch_logits<1>(L, ws, x, W, es.v0, es, "xent_logits", device, s);
    }
  }
  if (st != L3_OK) return st;
  // Eight blocks a row group where there are few groups and many partials. Replayed
  // back to back (d = 512), eight blocks take longer by, in us: one token, 125 partials
  // -0.2, 250 -0.9, 500 -2.2, 1000 -4.7; 256 tokens, 125 partials +0.7, 187 -0.3, 500 -1.5; 512 tokens,
  // 125 partials +0.4, 187 -0.3; 1024 tokens, 500 partials +0.9, 1000 -1.7.
  const int cl = n <= 512 && L.n_parts >= 160 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((n + 31) / 32 * cl));
  cfg.blockDim = dim3(32, 32);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 8;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  LaunchTimer t("xent_join", s);
  if (cl > 1)
    L3_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_xent_join<8>, J));
  else
    L3_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_xent_join<1>, J));
  return L3_OK;
}

l3_status l3_xent_backward(const void *x, const void *W, const int32_t *targets, const float *lse,
                           const float *dloss, int64_t n, int64_t vocab, int64_t d, int32_t dtype,
                           void *dx, void *dW, void *workspace, int64_t workspace_bytes,
                           void *stream) {
  set_error("");
  int device = 0;
  // with no tokens, dW alone is written
  const Pointer ptrs[] = {{dW, 16}, {W, 16}, {workspace, 16}, {x, 16}, {dx, 16}, {targets, 4}, {lse, 4}, {dloss, 4}};
  l3_status st = check(ptrs, n ? 8 : 1, n, vocab, d, dtype, n ? workspace_bytes : INT64_MAX, true,
                       &device);
  if (st != L3_OK) return st;
  const Layout L(n, vocab, d, dtype == L3_FP32, true);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  if (n == 0) {
    L3_CUDA_TRY(cudaMemsetAsync(dW, 0, (size_t)vocab * d * (L.fp32 ? 4 : 2), s));
    return clear_error_word(workspace, workspace_bytes, s);
  }
  return L.fp32 ? backward<float>(L, ws, x, W, targets, lse, dloss, dx, dW, device, s)
                : backward<__nv_bfloat16>(L, ws, x, W, targets, lse, dloss, dx, dW, device, s);
}

}  // extern "C"
