// The tensor-core product that the cross entropy and the orthogonalised
// update are built on: D = A B^T on CTA pairs, each 256 x TN tile handed to an
// epilogue functor in fp32 straight from TMEM.
//
// Two CTAs on neighbouring SMs share a tile (cta_group::2, M = 256): each
// loads its own 128 rows of A and half of B's TN rows with TMA into a ring of
// 64-deep k-blocks, the pair's first CTA issues the MMAs, each CTA's TMEM
// receives its 128 rows, and eight or sixteen epilogue warps drain one accumulator
// while the MMAs fill the others. Persistent: a pair takes every n_pairs-th tile.
//
// Two independent products may share a launch: the tiles of the deeper one come
// first, those of the other fill up the pairs that got fewer of them.
//
// The tensor core's accumulator drops what does not fit its 24 bits instead of
// rounding it, so its error grows with every 16-deep step and always towards
// zero: 4096 deep, 3e-5 of the orthogonalised result. Where the result is wanted
// in fp32, `chunk` k-blocks at a time are accumulated there, and the epilogue
// warps add the chunks up in registers with rounded additions.
//
// Operands are 16-bit and of one type. Either may be K-major (its rows are M
// or N, k contiguous) or MN-major (its rows are k, M or N contiguous), so that
// no product needs a transposed copy; or symmetric, with the 256-wide blocks
// right of the diagonal never written: a k-block from there is read as MN-major
// from its mirror (writing the mirror cost 3.4 us of a 14 us launch, 512 x 512).
// A value held in several 16-bit parts
// (hi + lo, ...) is stored as stacked planes; the ring takes a k-block's planes
// one after the other, and the kept products of parts are issued when all of
// them are there, so that each plane is loaded once for the two or three
// products it enters (2048 x 4096 pairs: 442 instead of 663 MB from L2 in X X^T).
// The smallest products come first, since the accumulator's own rounding is
// relative to its size.
//
// Times in the comments here and in the files that use this compare the forms of one
// choice, measured when it was made: calls back to back on the same inputs. Later steps
// changed the totals: 512 x 512 takes 182 us now, 1000 x 3000 338, 2048 x 4096 864, and 880
// where the inputs change from call to call.
#pragma once

#include <algorithm>
#include <type_traits>

#include "l3_internal.cuh"
#include "sm100.cuh"

namespace l3 {

// 2-D row-major 16-bit tensor map, 128-byte swizzle (gemm_tc.cu)
l3_status make_map_2d16(CUtensorMap *m, const void *base, bool bf16, uint64_t rows, uint64_t cols,
                        uint64_t ld, uint32_t box_cols, uint32_t box_rows, int swizzle_bytes);

namespace pairgemm {

using namespace sm100;

// The cta_group::2 forms, as the layer's own GEMMs use them: arrivals on a
// barrier of either CTA of the pair (default semantics: a cluster-scope release
// would be a full fence per stage), loads counted there (no multicast), the MMA,
// and its completion signalled in both CTAs
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t cluster_addr,
                                                              uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map,
                                                 uint32_t bar_cluster_addr, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar_cluster_addr), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit_pair(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

constexpr int BM = 128;  // rows of A per CTA (TMEM lanes)
constexpr int BK = 64;   // 64 16-bit elements = one 128-byte swizzle row
constexpr int A_BYTES = BM * BK * 2;

struct Args {
  int tiles_m, tiles_n, batch;  // 256-row and TN-column tiles of each matrix of the batch
  int nkb;                      // 64-deep k-blocks
  // > 1: the k-blocks shared out over so many partial results, for products of
  // few tiles; batch counts them all, and a functor's `matrix` is
  // share * matrices + matrix
  int splits;
  int chunk;                    // k-blocks per accumulation; 0: all (Epi::SUMS)
  // a count on the device that bounds the rows (dyn_rows) or the depth (dyn_k)
  // of this launch; at least one tile row and one k-block always run
  const int *dyn;
  int dyn_rows, dyn_k;
  int group;  // tile order: m fastest within groups of this many tile rows
  int sym;    // only the tiles that touch or lie below the diagonal
  // the operands' first rows in their tensor maps, and the rows from one plane
  // and from one matrix of the batch to the next
  int a_off, b_off, a_plane, b_plane, a_batch, b_batch;
  int a_hi;       // of A's two parts (and one of B) only the first
  // not NULL: the second part only in the k-blocks whose byte [tile row][k-block] is set
  const uint8_t *a_lo;
  int a_lo_ld;    // a multiple of 16; rows start 16-byte aligned
  uint32_t bf16;  // 1: bf16 operands, 0: fp16
  int *err;
  int clear_err;  // the chain's first kernel: *err is zeroed (a wait that gives up does so 2 s later)
};

constexpr int MAX_STAGES = 8;

struct Bars {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[8], tempty[8], drain;
  uint64_t in[16];  // an epilogue warp's own loads
  uint32_t tmem_base;
  int abort_flag;
};

// the products of PA-part and PB-part values that are kept (part of A, part of
// B), smallest first, and the part that is done with after each (or -1)
template <int PA, int PB>
struct Products;
template <>
struct Products<1, 1> {
  static constexpr int N = 1;
  __host__ __device__ static constexpr int a(int) { return 0; }
  __host__ __device__ static constexpr int b(int) { return 0; }
  __host__ __device__ static constexpr int frees(int) { return 0; }
};
template <>
struct Products<2, 1> {  // lo hi, hi hi
  static constexpr int N = 2;
  __host__ __device__ static constexpr int a(int i) { return i == 0; }
  __host__ __device__ static constexpr int b(int) { return 0; }
  __host__ __device__ static constexpr int frees(int i) { return i == 0; }
};
template <>
struct Products<2, 2> {  // lo hi, hi lo, hi hi
  static constexpr int N = 3;
  __host__ __device__ static constexpr int a(int i) { return i == 0; }
  __host__ __device__ static constexpr int b(int i) { return i == 1; }
  __host__ __device__ static constexpr int frees(int i) { return i == 1 ? 1 : i == 2 ? 0 : -1; }
};
template <>
struct Products<3, 3> {  // lo hi, hi lo, mid mid, mid hi, hi mid, hi hi
  static constexpr int N = 6;
  __host__ __device__ static constexpr int a(int i) { return i == 0 ? 2 : i == 2 || i == 3; }
  __host__ __device__ static constexpr int b(int i) { return i == 1 ? 2 : i == 2 || i == 4; }
  __host__ __device__ static constexpr int frees(int i) {
    return i == 1 ? 2 : i == 4 ? 1 : i == 5 ? 0 : -1;
  }
};

// Shared memory: the ring takes what the epilogue's boxes leave of 227 KB
template <int TN, class Epi, class Epi2 = Epi>
struct Cfg {
  static constexpr int B_BYTES = TN / 2 * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  // epilogue warps share a TMEM lane quarter's columns, 32 at least each
  static constexpr int WARPS = Epi::WARPS < TN / 8 ? Epi::WARPS : TN / 8;
  static constexpr int SPAN = TN * 4 / WARPS;  // columns of a warp
  static constexpr int THREADS = 64 + 32 * WARPS;
  static constexpr int ACCS = 512 / TN;  // accumulators in TMEM's 512 columns
  static_assert(Epi::WARPS == Epi2::WARPS, "epilogue warps");
  static constexpr int BOX_BYTES = Epi::BOX_BYTES > Epi2::BOX_BYTES ? Epi::BOX_BYTES : Epi2::BOX_BYTES;
  static constexpr int BOXES = WARPS * BOX_BYTES;
  static constexpr int ROOM = 232448 - 1024 - (int)sizeof(Bars) - BOXES;
  static constexpr int STAGES = ROOM / STAGE < MAX_STAGES ? ROOM / STAGE : MAX_STAGES;
  static_assert(STAGES >= 4, "ring too short for a k-block in use and one on its way");
  static constexpr size_t SMEM = 1024 + STAGES * STAGE + BOXES + sizeof(Bars);
};

// An epilogue warp's share of shared memory: boxes of 32 rows x 32 16-bit
// columns (2 KB, 64-byte swizzle: 16-byte piece k of row r lies at piece
// k ^ ((r >> 1) & 3)) that move to and from memory by TMA, so that memory sees
// whole sectors and no thread waits for a load of its own.
constexpr int BOX = 2048;

struct WarpBoxes {
  uint8_t *mem;     // the warp's Epi::BOX_BYTES
  uint64_t *bar;
  uint32_t parity;  // of the next load
  int lane;
  Abort ab;
  bool failed = false;  // a load's wait gave up

  __device__ __forceinline__ uint4 *piece(int box, int k) const {
    return reinterpret_cast<uint4 *>(mem + box * BOX + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4));
  }
  // at most N of the warp's committed groups of stores still read their boxes
  template <int N>
  __device__ __forceinline__ void stores_read() const {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
    __syncwarp();
  }
  // the lanes' writes to the boxes are done: what lane 0 stores next sees them
  __device__ __forceinline__ void written() const {
    fence_proxy_async_smem();
    __syncwarp();
  }
  // the box's 32 x 32 elements to rows of memory (ld elements apart), four lanes
  // a row: whole sectors, and nothing to wait for before the box is used again
  // but the warp itself
  __device__ __forceinline__ void copy_out(int box, void *to, int64_t ld) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + lane / 4, k = lane % 4;
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(to) + r * ld + k * 8) =
          *reinterpret_cast<const uint4 *>(mem + box * BOX + r * 64 + ((k ^ ((r >> 1) & 3)) << 4));
    }
  }
  // lane 0 only
  __device__ __forceinline__ void store(int box, const CUtensorMap *map, int x, int y) const {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
        "r"(smem_u32(mem + box * BOX)), "r"(x), "r"(y)
        : "memory");
  }
  __device__ __forceinline__ void commit() const {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  // lane 0 only: box p from row y + p * plane_rows, p < N
  template <int N>
  __device__ __forceinline__ void load(const CUtensorMap *map, int x, int y, int plane_rows) const {
    mbar_arrive_expect_tx(bar, N * BOX);
#pragma unroll
    for (int p = 0; p < N; ++p) tma_load_2d(mem + p * BOX, map, bar, x, y + p * plane_rows);
  }
  __device__ __forceinline__ void loaded() {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, ab));
    parity ^= 1;
    failed |= !ok;
  }
};

// Programmatic dependent launch: a kernel of a chain may start while the one
// before it drains; nothing of the chain's memory is touched before pdl_wait.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// tiles of row i that touch or lie below the diagonal (tiles 256 x TN)
template <int TN>
__host__ __device__ __forceinline__ int sym_row_tiles(int i, int tiles_n) {
  const int n = (i + 1) * (256 / TN);
  return n < tiles_n ? n : tiles_n;
}

// A product's tiles and depth, once the count on the device is known
struct Shape {
  int tiles_m, per_matrix, n_tiles;
  int nkb, share;  // k-blocks in all and of a tile (a share, where there are some)
  int matrices;

  template <int TN>
  __device__ __forceinline__ static Shape of(const Args &P, int dyn) {
    Shape s;
    s.tiles_m = P.dyn_rows ? min(P.tiles_m, max(1, (dyn + 2 * BM - 1) / (2 * BM))) : P.tiles_m;
    s.nkb = P.dyn_k ? min(P.nkb, max(1, (dyn + BK - 1) / BK)) : P.nkb;
    s.per_matrix = s.tiles_m * P.tiles_n;
    if (P.sym) {
      s.per_matrix = 0;
      for (int i = 0; i < s.tiles_m; ++i) s.per_matrix += sym_row_tiles<TN>(i, P.tiles_n);
    }
    s.n_tiles = s.per_matrix * P.batch;
    s.share = P.splits > 1 ? (s.nkb + P.splits - 1) / P.splits : s.nkb;
    s.matrices = P.splits > 1 ? P.batch / P.splits : P.batch;
    return s;
  }
};

// matrix (share-major), tile row and column of a tile, and its k-blocks
struct Tile {
  int b, mi, ni, k0, k_count;

  template <int TN>
  __device__ __forceinline__ static Tile at(const Args &P, const Shape &s, int t) {
    Tile x;
    x.b = t / s.per_matrix;
    x.k0 = P.splits > 1 ? x.b / s.matrices * s.share : 0;
    x.k_count = max(0, min(s.share, s.nkb - x.k0));
    int r = t - x.b * s.per_matrix;
    if (P.sym) {
      // the longest rows first
      x.mi = s.tiles_m - 1;
      for (int w; r >= (w = sym_row_tiles<TN>(x.mi, P.tiles_n)); --x.mi) r -= w;
      x.ni = r;
      return x;
    }
    const int per_group = P.group * P.tiles_n;
    const int g = r / per_group;
    r -= g * per_group;
    const int rows = min(P.group, s.tiles_m - g * P.group);
    x.ni = r / rows;
    x.mi = g * P.group + (r - x.ni * rows);
    return x;
  }
};

// Which tiles a pair takes. Of one product every n_pairs-th; of two, n1 tiles
// of c1 k-blocks and then n2 of c2 <= c1: the pairs with one tile less of the first
// take c1 / c2 of the second before all go on in turn.
struct Order {
  int pair, n_pairs, n1, n2;
  int rem, extra;  // pairs with one more of the first; tiles that make up for it
  bool swapped;    // the second product is the deeper one

  __device__ __forceinline__ Order(int pair_, int n_pairs_, const Shape &a, const Shape &b, bool two)
      : pair(pair_), n_pairs(n_pairs_) {
    swapped = two && b.share > a.share;
    n1 = swapped ? b.n_tiles : a.n_tiles;
    n2 = !two ? 0 : swapped ? a.n_tiles : b.n_tiles;
    rem = n1 % n_pairs;
    const int c1 = max(a.share, b.share), c2 = max(1, min(a.share, b.share));
    extra = two && rem ? (c1 + c2 / 2) / c2 : 0;
  }
  // the pair's k-th tile: of which product, and its number there
  __device__ __forceinline__ bool nth(int k, int &which, int &t) const {
    const int own = n1 / n_pairs + (pair < rem);
    if (k < own) {
      which = swapped;
      t = pair + k * n_pairs;
      return true;
    }
    int j = k - own;
    which = !swapped;
    const int light = n_pairs - rem;
    if (rem && pair >= rem && j < extra) {
      t = pair - rem + j * light;
      return t < n2;
    }
    if (rem && pair >= rem) j -= extra;
    t = light * extra + pair + j * n_pairs;
    return t < n2;
  }
};

// Which k-blocks of a tile row take A's second part; sixteen bytes at a time, from L2
// (the kernel before wrote them)
struct SecondPart {
  const uint4 *row;
  bool never, always;
  uint4 w;
  int have = -1;

  __device__ __forceinline__ SecondPart(const Args &P, int tile_row)
      : row(reinterpret_cast<const uint4 *>(P.a_lo + (P.a_lo ? (int64_t)tile_row * P.a_lo_ld : 0))),
        never(P.a_hi), always(!P.a_lo) {}
  __device__ __forceinline__ bool at(int kb) {
    if (never || always) return !never;
    if (kb >> 4 != have) w = __ldcg(row + (have = kb >> 4));
    const uint32_t x = kb & 8 ? kb & 4 ? w.w : w.z : kb & 4 ? w.y : w.x;
    return x >> (kb & 3) * 8 & 0xff;
  }
};

// An epilogue functor sees a warp's share of a tile, 32 columns at a time:
//   prefetch(boxes, matrix, row of lane 0, first column c0)   before the tile is done
//   State begin(matrix, row m, first column c0, dynamic count)
//   chunk(State &, boxes, c, float (&v)[32])   columns c0 + c .. c0 + c + 31, c = 0, 32, ...
//   end(State &)
// for thread = row, Cfg::SPAN columns in all. BOX_BYTES: shared memory per warp.
// SUMS: whether the depth may come in chunks (see the top); without it the tile
// is one chain and no warp holds more of it than 32 columns.
// WARPS: eight for tiles that come in long rows, where the warps keep up and a
// row's columns stay together; sixteen where a CTA has a tile or two, whose
// epilogues nothing hides (orthogonalising 512 x 512: 162 us, 170 with eight;
// 2048 x 4096: 756, 748 with eight).
enum Major : int { K_MAJOR = 0, MN_MAJOR = 1, SYMMETRIC = 2 };

// One product: operands, sizes and what becomes of its tiles
template <Major A_, Major B_, class Epi_>
struct Problem {
  using Epi = Epi_;
  static constexpr Major A = A_, B = B_;
  CUtensorMap mA, mB;
  Args P;
  Epi epi;
};

// TWO: P2 is a second product, else it repeats P1's type and is not read
template <int TN, int PA, int PB, bool TWO, class P1, class P2>
__global__ void __launch_bounds__(Cfg<TN, typename P1::Epi, typename P2::Epi>::THREADS, 1)
    k_gemm_pair(const __grid_constant__ P1 p1, const __grid_constant__ P2 p2) {
  using C = Cfg<TN, typename P1::Epi, typename P2::Epi>;
  using Pr = Products<PA, PB>;
  constexpr int PL = PA > PB ? PA : PB;  // ring stages of a k-block
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  Bars *b = reinterpret_cast<Bars *>(ring + STAGES * C::STAGE + C::BOXES);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();  // 0 issues the MMAs
  const int pair_id = blockIdx.x / 2, n_pairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&b->full[s], 2);   // used in CTA 0: one arrival per CTA, plus both CTAs' bytes
      mbar_init(&b->empty[s], 1);  // MMA completion, signalled in both CTAs
    }
    for (int a = 0; a < C::ACCS; ++a) {
      mbar_init(&b->tfull[a], 1);
      mbar_init(&b->tempty[a], 2 * C::WARPS);  // used in CTA 0: every epilogue warp of both CTAs
    }
    for (int w = 0; w < C::WARPS; ++w) mbar_init(&b->in[w], 1);
    mbar_init(&b->drain, 1);
    b->abort_flag = 0;
    if (p1.P.clear_err && blockIdx.x == 0) *p1.P.err = 0;
    fence_mbar_init();
    prefetch_tensormap(&p1.mA);
    prefetch_tensormap(&p1.mB);
    if (TWO) {
      prefetch_tensormap(&p2.mA);
      prefetch_tensormap(&p2.mB);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&b->tmem_base)),
                 "r"(C::ACCS * TN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_launch();
  // whether k-block kb of the operand whose tile begins at m or n lies MN-major
  const auto is_mn = [](Major major, int kb, int at) {
    return major == MN_MAJOR || (major == SYMMETRIC && kb * BK / 256 > at / 256);
  };
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers initialised before any cross-CTA signal
  tc_fence_after();
  // all of the set-up above runs beside the kernel before this one
  pdl_wait();
  const int dyn = p1.P.dyn ? *p1.P.dyn : 0;
  const Shape s1 = Shape::of<TN>(p1.P, dyn);
  const Shape s2 = TWO ? Shape::of<TN>(p2.P, dyn) : s1;
  const Order order(pair_id, n_pairs, s1, s2, TWO);
  // f(problem, shape) of the product a tile belongs to
  const auto of = [&](int which, auto f) {
    if (TWO && which)
      f(p2, s2);
    else
      f(p1, s1);
  };
  const uint32_t tmem = b->tmem_base;
  const Abort ab{&b->abort_flag, p1.P.err};

  if (warp == 0) {
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed_parity[STAGES];
      bool armed[STAGES];
      for (int s = 0; s < STAGES; ++s) armed[s] = false;
      bool ok = true;
      int which, t;
      for (int n = 0; ok && order.nth(n, which, t); ++n) of(which, [&](const auto &pb, const Shape &sh) {
        using PT = std::decay_t<decltype(pb)>;
        constexpr Major A = PT::A, B = PT::B;
        const Args &P = pb.P;
        const Tile x = Tile::at<TN>(P, sh, t);
        const int m0 = x.mi * (2 * BM) + (int)rank * BM;
        const int n0 = x.ni * TN + (int)rank * (TN / 2);
        const int mat = x.b % sh.matrices;
        SecondPart second(P, x.mi);
        for (int kb = x.k0; ok && kb < x.k0 + x.k_count; ++kb) {
          const bool a_mn = is_mn(A, kb, x.mi * 256), b_mn = is_mn(B, kb, x.ni * TN);
          const bool hi = PA > PB && !second.at(kb);
#pragma unroll
          for (int pl = PL - 1; pl >= 0; --pl) {  // in the order that they are done with
            if (hi && pl) continue;
            if (!mbar_wait(&b->empty[stage], phase ^ 1, ab)) {
              ok = false;
              break;
            }
            uint8_t *sa = ring + stage * C::STAGE;
            uint8_t *sb = sa + A_BYTES;
            const int ya = P.a_off + mat * P.a_batch + pl * P.a_plane;
            const int yb = P.b_off + mat * P.b_batch + pl * P.b_plane;
            const uint32_t full0 = map_shared_rank(&b->full[stage], 0);
            mbar_arrive_expect_tx_cluster(full0, (pl < PA ? A_BYTES : 0) + (pl < PB ? C::B_BYTES : 0));
            armed[stage] = true;
            armed_parity[stage] = phase;
            static_assert(B == K_MAJOR || TN >= 128, "a 64-column MN-major box per CTA");
            if (pl >= PA) {
            } else if (A == K_MAJOR) {
              tma_load_2d_pair(sa, &pb.mA, full0, kb * BK, ya + m0);
            } else {  // two boxes of 64 x 64, along m either way
#pragma unroll
              for (int o = 0; o < 128; o += 64)
                tma_load_2d_pair(sa + o * 128, &pb.mA, full0, a_mn ? m0 + o : kb * BK,
                                 ya + (a_mn ? kb * BK : m0 + o));
            }
            if (pl >= PB) {
            } else if (B == K_MAJOR) {
              tma_load_2d_pair(sb, &pb.mB, full0, kb * BK, yb + n0);
            } else {  // TN / 128 boxes of 64 x 64, along n
#pragma unroll
              for (int o = 0; o < TN / 2; o += 64)
                tma_load_2d_pair(sb + o * 128, &pb.mB, full0, b_mn ? n0 + o : kb * BK,
                                 yb + (b_mn ? kb * BK : n0 + o));
            }
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      });
      // after a give-up CTA 0 waits for the phases it armed, which complete
      // only once both CTAs' copies have landed
      if (!ok && rank == 0) {
        for (int s = 0; s < STAGES; ++s)
          if (armed[s]) {
            const uint32_t a = smem_u32(&b->full[s]);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(a, armed_parity[s]) && globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
            }
          }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int job = 0;
      int which, t;
      for (int n = 0; ok && order.nth(n, which, t); ++n) of(which, [&](const auto &pb, const Shape &sh) {
        using PT = std::decay_t<decltype(pb)>;
        constexpr Major A = PT::A, B = PT::B;
        const Tile x = Tile::at<TN>(pb.P, sh, t);
        const int k_count = x.k_count, chunk = PT::Epi::SUMS && pb.P.chunk ? pb.P.chunk : sh.nkb;
        SecondPart second(pb.P, x.mi);
        for (int i0 = 0; ok && i0 < k_count; i0 += chunk, ++job) {
          const int acc = job % C::ACCS;
          // the epilogue has finished with this accumulator's previous chunk
          if (!mbar_wait(&b->tempty[acc], (job / C::ACCS & 1) ^ 1, ab)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + acc * TN;
          const int i1 = min(k_count, i0 + chunk);
          for (int i = i0; ok && i < i1; ++i) {
            const bool hi = PA > PB && !second.at(x.k0 + i);
            uint32_t sa[PL];
            uint64_t *empty[PL];  // by part
#pragma unroll
            for (int pl = PL - 1; pl >= 0; --pl) {
              if (hi && pl) continue;
              if (!mbar_wait(&b->full[stage], phase, ab)) {
                ok = false;
                break;
              }
              sa[pl] = smem_u32(ring + stage * C::STAGE);
              empty[pl] = &b->empty[stage];
              if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
              }
            }
            if (!ok) break;
            tc_fence_after();
            const bool a_mn = is_mn(A, x.k0 + i, x.mi * 256), b_mn = is_mn(B, x.k0 + i, x.ni * TN);
            const uint32_t idesc = idesc_f16(pb.P.bf16, b_mn, 2 * BM, TN) | (a_mn ? 1u << 15 : 0u);
            // a 16-deep step is 32 bytes along a K-major operand's rows, 16
            // rows of 128 bytes down an MN-major one (its 64-wide blocks 8 KB apart)
#pragma unroll
            for (int pr = 0; pr < Pr::N; ++pr) {
              if (hi && Pr::a(pr)) continue;
              const uint32_t at = sa[Pr::a(pr)], bt = sa[Pr::b(pr)] + A_BYTES;
#pragma unroll
              for (int kq = 0; kq < BK / 16; ++kq)
                umma_f16_pair(d,
                              a_mn ? sdesc_sw128(at + kq * 2048, BK * 128, 1024)
                                   : sdesc_sw128(at + kq * 32, 16, 1024),
                              b_mn ? sdesc_sw128(bt + kq * 2048, BK * 128, 1024)
                                   : sdesc_sw128(bt + kq * 32, 16, 1024),
                              idesc, (i - i0) | (hi ? 0 : pr) | kq);
              // the part that no later product reads makes room
              if (Pr::frees(pr) >= 0) umma_commit_pair(empty[Pr::frees(pr)]);
            }
          }
          if (ok) umma_commit_pair(&b->tfull[acc]);
        }
      });
      if (!ok) {
        umma_commit_pair(&b->drain);
        const uint32_t a = smem_u32(&b->drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
        }
      }
    }
  } else {
    // warp % 4 selects the TMEM lane quarter that a warp may read
    constexpr int SPAN = C::SPAN;
    const int q = warp & 3, part = (warp - 2) / 4;
    const uint32_t tempty0 = map_shared_rank(&b->tempty[0], 0);
    int job = 0;
    bool ok = true;
    WarpBoxes box{ring + STAGES * C::STAGE + (warp - 2) * C::BOX_BYTES, &b->in[warp - 2], 0, lane, ab};
    int which, t;
    // two products with the same kind of epilogue run the same code
    const auto of_epi = [&](int w, auto f) {
      if constexpr (std::is_same_v<typename P1::Epi, typename P2::Epi>) {
        f(w ? p2.epi : p1.epi, w ? p2.P : p1.P, w ? s2 : s1);
      } else {
        of(w, [&](const auto &pb, const Shape &sh) { f(pb.epi, pb.P, sh); });
      }
    };
    for (int n = 0; ok && order.nth(n, which, t); ++n)
     of_epi(TWO ? which : 0, [&](const auto &epi, const Args &P, const Shape &sh) {
      constexpr bool SUMS = std::decay_t<decltype(epi)>::SUMS;
      const Tile x = Tile::at<TN>(P, sh, t);
      const int k_count = x.k_count, chunk = SUMS && P.chunk ? P.chunk : sh.nkb;
      const int m_warp = x.mi * (2 * BM) + (int)rank * BM + q * 32, c0 = x.ni * TN + part * SPAN;
      epi.prefetch(box, x.b, m_warp, c0);
      const auto wait = [&] {
        ok = __all_sync(0xffffffffu, mbar_wait(&b->tfull[job % C::ACCS], job / C::ACCS & 1, ab));
        tc_fence_after();
        return ok;
      };
      const auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * (job % C::ACCS));
        ++job;
      };
      const auto read = [&](int c, uint32_t (&v)[32]) {
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + job % C::ACCS * TN + part * SPAN + c, v);
        tmem_wait_ld();
      };
      if constexpr (!SUMS) {
        // one chain: 32 columns at a time, straight from TMEM
        if (k_count && !wait()) return;
        auto st = epi.begin(x.b, m_warp + lane, c0, dyn);
#pragma unroll 1
        for (int c = 0; c < SPAN; c += 32) {
          uint32_t u[32];
          float v[32];
          if (k_count) read(c, u);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = k_count ? __uint_as_float(u[e]) : 0.f;
          if (k_count && c + 32 == SPAN) release();
          epi.chunk(st, box, c, v);
        }
        epi.end(st);
      } else {
        float r[SPAN / 32][32];
        if (k_count == 0) {  // a share past the depth adds nothing
#pragma unroll
          for (int c = 0; c < SPAN / 32; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) r[c][e] = 0.f;
        }
        for (int i0 = 0; i0 < k_count; i0 += chunk) {
          if (!wait()) return;
#pragma unroll
          for (int c = 0; c < SPAN / 32; ++c) {
            uint32_t v[32];
            read(c * 32, v);
            if (i0 == 0) {
#pragma unroll
              for (int e = 0; e < 32; ++e) r[c][e] = __uint_as_float(v[e]);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) r[c][e] += __uint_as_float(v[e]);
            }
          }
          release();
        }
        auto st = epi.begin(x.b, m_warp + lane, c0, dyn);
        // written out: r has to stay in registers
        epi.chunk(st, box, 0, r[0]);
        if constexpr (SPAN >= 64) epi.chunk(st, box, 32, r[1]);
        if constexpr (SPAN == 128) {
          epi.chunk(st, box, 64, r[2]);
          epi.chunk(st, box, 96, r[3]);
        }
        epi.end(st);
      }
    });
    // the boxes' stores are in memory, and a load that a give-up left behind
    // has landed, before the CTA ends
    if (C::BOX_BYTES && lane == 0) {
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      if ((!ok || box.failed) && (P1::Epi::LOADS || P2::Epi::LOADS)) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(box.bar), box.parity) && globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no signal crosses between the CTAs after this
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::ACCS * TN)
                 : "memory");
  }
}

// Tensor map of an operand: `rows` x `cols` elements, K-major boxes of
// `tile_rows` x 64, or boxes of 64 x 64 for MN-major and symmetric ones.
inline l3_status operand_map(CUtensorMap *m, const void *base, bool bf16, int64_t rows,
                             int64_t cols, int64_t ld, bool mn_major, int tile_rows) {
  return make_map_2d16(m, base, bf16, (uint64_t)rows, (uint64_t)cols, (uint64_t)ld, BK,
                       mn_major ? BK : tile_rows, 128);
}

template <int TN>
int64_t count_tiles(const Args &P) {
  int64_t per_matrix = (int64_t)P.tiles_m * P.tiles_n;
  if (P.sym) {
    per_matrix = 0;
    for (int i = 0; i < P.tiles_m; ++i) per_matrix += sym_row_tiles<TN>(i, P.tiles_n);
  }
  return per_matrix * P.batch;
}

template <int TN, int PA, int PB, bool TWO, class P1, class P2>
l3_status launch_problems(const P1 &p1, const P2 &p2, int device, cudaStream_t s, bool pdl) {
  using C = Cfg<TN, typename P1::Epi, typename P2::Epi>;
  const auto kernel = k_gemm_pair<TN, PA, PB, TWO, P1, P2>;
  static bool attr[64] = {};
  if (!attr[device & 63]) {
    L3_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM));
    attr[device & 63] = true;
  }
  const int64_t n_tiles = count_tiles<TN>(p1.P) + (TWO ? count_tiles<TN>(p2.P) : 0);
  const int pairs = (int)std::min<int64_t>(n_tiles, sm_count(device) / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl ? 2 : 1;
  L3_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p1, p2));
  return L3_OK;
}

template <int TN, int PA, int PB, Major A, Major B, class Epi>
l3_status launch(const CUtensorMap &mA, const CUtensorMap &mB, const Args &P, const Epi &epi,
                 int device, cudaStream_t s, bool pdl = true) {
  const Problem<A, B, Epi> p{mA, mB, P, epi};
  return launch_problems<TN, PA, PB, false>(p, p, device, s, pdl);
}

// Tile width and number of shares of a product's depth. Time, in SM clocks: a
// k-block of one part product takes 512 on a 256-column tile and about 300 on a
// 128-column one (whose operands load less densely), a tile 3000 more (fill,
// drain, epilogue), and shares are written and joined at about 3000 bytes a
// clock by a launch of 6000. Measured with and without: orthogonalising 512 x 512
// in 128-column tiles 161 us, in 256-column ones 253 (2048 x 4096: 756, 812);
// 1000 x 3000 with shares 304 us, without 351; the gradients of 256 tokens x
// 32000 x 1024 with shares 70 us, without 130.
struct Tiling {
  int tn, splits;
};
template <class Tiles>  // tn -> number of tiles
Tiling choose_tiling(Tiles tiles_of, int64_t nkb, int products, int64_t out_elements) {
  constexpr int64_t PAIRS = 74;  // of the 148 SMs
  Tiling best{256, 1};
  double best_t = 0;
  for (int tn : {256, 128})
    for (int sp : {1, 2, 3, 4, 5, 6, 8, 12, 16, 24}) {
      if (sp > 1 && sp > nkb) break;
      const int64_t tiles = tiles_of(tn) * sp;
      const int64_t waves = (tiles + PAIRS - 1) / PAIRS, kb = (nkb + sp - 1) / sp;
      double t = (double)waves * (kb * products * (tn == 256 ? 512. : 300.) + 3000.);
      if (sp > 1) t += 6000. + sp * (double)out_elements * 8. / 3000.;
      if (best_t == 0 || t < 0.95 * best_t) {
        best_t = t;
        best = Tiling{tn, sp};
      }
    }
  return best;
}

// The same for two products in one launch, whose tiles together are spread over
// the pairs to within about half of the longest one.
struct TwoTilings {
  int tn, splits1, splits2;
};
struct Work {
  int64_t tiles_m, cols, nkb, out_elements;
  bool partial;  // written as partials whether or not it is shared out
  int products;  // of parts
};
inline TwoTilings choose_tilings(const Work &a, const Work &b) {
  constexpr int PAIRS = 74;
  constexpr int SHARES[] = {1, 2, 3, 4, 5, 6, 8, 12, 16, 24};
  TwoTilings best{256, 1, 1};
  double best_t = 0;
  for (int tn : {256, 128})
    for (int s1 : SHARES)
      for (int s2 : SHARES) {
        if ((s1 > 1 && s1 > a.nkb) || (s2 > 1 && s2 > b.nkb)) continue;
        double total = 0, longest = 0, more = 0;
        for (const auto &[w, sp] : {std::pair(&a, s1), std::pair(&b, s2)}) {
          const int64_t tiles = w->tiles_m * ((w->cols + tn - 1) / tn) * sp;
          const double one = (double)((w->nkb + sp - 1) / sp) * w->products * (tn == 256 ? 512. : 300.) + 3000.;
          total += tiles * one;
          longest = std::max(longest, one);
          if (sp > 1) more += (w->partial ? 0. : 6000.) + sp * (double)w->out_elements * 8. / 3000.;
        }
        const double t = std::max(total / PAIRS + longest / 2, longest) + more;
        if (best_t == 0 || t < 0.95 * best_t) {
          best_t = t;
          best = TwoTilings{tn, s1, s2};
        }
      }
  return best;
}

// map of the boxes that an epilogue moves
inline l3_status box_map(CUtensorMap *m, const void *base, bool bf16, int64_t rows, int64_t cols,
                         int64_t ld) {
  return make_map_2d16(m, base, bf16, (uint64_t)rows, (uint64_t)cols, (uint64_t)ld, 32, 32, 64);
}

// launch of a plain kernel as a link of such a chain
template <class... K, class... A>
l3_status launch_link(void (*kernel)(K...), dim3 grid, dim3 block, cudaStream_t s, bool pdl,
                      A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl ? 1 : 0;
  L3_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, K(args)...));
  return L3_OK;
}

}  // namespace pairgemm
}  // namespace l3
