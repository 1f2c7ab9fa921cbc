// K9: attention of many new tokens over the paged cache on the tcgen05 tensor
// cores. The mathematics, the row order (token by token, the heads of a group
// side by side) and the masks are K8's.
//
// A piece of work is a part of the key tiles of 256 rows of one sequence and key
// head, held as two sub-tiles of 128 rows that take turns: while the tensor pipe
// works on one sub-tile's products, the other's softmax runs. Per 128 keys and
// sub-tile: S = Q K^T into TMEM (both operands from shared memory, fp32), one
// thread per row reads its 128 scores, writes the probabilities back over them as
// packed bf16, and O += P V with P read from TMEM as the A operand and V from
// shared memory as it was loaded (rows = keys, the transposed-B form), so neither
// S nor P touches shared memory. TMEM: two S of 128 columns and two O of D.
//
// One block per SM takes row tiles (key head by key head, the longest of a sequence
// first) from a counter, so that at any time the blocks read the keys and values of
// few heads, close together: the copies' way through L2 is what a scattered order
// loses on (ragged prompts ran 1.8 times longer with the heads side by side). Where
// the tiles are long, whole ones only fill whole waves, and the (row tile, key tile)
// units of the rest (of all when there are fewer tiles than SMs) are dealt evenly
// over the blocks. A block's
// first and last pieces of those may be parts: they leave fp32 partial sums, and the
// last block to arrive adds them in block order. Which block takes a whole tile does
// not touch its result, and the parts are cut by block number, so results do not
// depend on the order of arrival.
//
// Roles (12 warps): 0 takes pieces of work, announces them to the others through a
// two-entry queue and copies K and V tiles by TMA, page by page, into a ring;
// 1 issues the products; 2 and 3 fetch the next piece's Q; 4-7 and 8-11 are the two
// sub-tiles' softmax, which also write the result.
// A row's accumulators are rescaled only when its maximum has grown by more than 8
// (a factor of 256) since the last time: the probabilities stay below 256, exact
// enough in bf16's and fp32's floating formats, and most key tiles need no pass
// over O.
//
// Bound: a key tile costs 4 * 128 * 128 * D multiply-adds on the tensor pipe (2048
// cycles at D = 128) and 2 * 128 * 128 exponentials (2048 cycles of the special-
// function units, which run under the products). What keeps it from the tensor peak
// is the way from a sub-tile's scores to its probabilities (about 2100 cycles: 80 to
// load a row, 450 for its maximum, 1500 for the exponentials) being longer than the
// other sub-tile's products (1350: Q K^T reads both operands from shared memory, at
// its full rate). Measured and left out: a part of the exponentials as polynomials on
// the FMA pipe (1345 -> 1369 .. 1564 us with one pair in eight .. two), and the first
// half of a tile's probabilities handed over early (1345 -> 1401 us).
//
// 4-bit pages: rows and scales arrive as they are by bulk copies; warps 2 and 3 unpack key and
// value tiles as 128 + code and code - 8, which bf16 holds exactly, and put the rows'
// scales beside them. The softmax applies them in fp32: s (q . (128 + c)) +
// (m - 128 s) sum(q) to the scores, p s as the second product's operand and
// sum(p (m + 8 s)) added at the end, as K8 does; neither keys nor values are rounded.
// The codes of a word keep the order in which shifts and masks bring them out; Q's
// rows are stored in that order of d and the result's are put back.
//
// There the softmax, with a scale and an offset for every score and probability, takes
// longer than the products and than unpacking, which alone takes 1.2 us a key tile at
// D = 64 and 2 us at 128. It is time spent waiting, not issue slots: these are used to
// 32 % and the tensor pipe to 11 % (five prompts of 100 to 900 tokens continued over
// 4-bit pages, D = 64, 81 us). Two of the softmax's warps share a scheduler, and a new
// piece's tiles are unpacked only once its Q is in, which waits for the last piece's
// products. The scores go back to TMEM adjusted, in loops over 32 of them: unrolled over
// the tile, waiting for instructions was the largest stall (102 -> 82 us).
// Left out: codes fetched through registers ahead of their use (111 -> 124 us on these
// prompts), and scales as bf16 pairs in shared memory, half the loads and twice the
// conversions (82 -> 91 us).
//
// Slots that no row of the piece sees are not copied (whole pages) or are zeroed
// in V's tile before the product (rows), since 0 * NaN would reach the result;
// their scores are replaced, not added to.
#pragma once

#include "k8_attend.cuh"

namespace fnl {

// 3-D tiled bulk tensor load (value, row of the page, page).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// The products are issued from convergent code under a predicate (`issue`, one lane)
// rather than inside a branch: the descriptors then stay in uniform registers and an
// instruction costs the issuing warp a few cycles instead of the ~90 that kept 64-cycle
// products waiting.
// D[tmem] (+)= A[smem desc] * B[smem desc]^T, bf16, fp32 accumulate.
__device__ __forceinline__ void umma_bf16_if(uint32_t issue, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(issue)
      : "memory");
}
// The same with A in TMEM: bf16, two consecutive k packed in a 32-bit column, row = lane.
__device__ __forceinline__ void umma_bf16_ts_if(uint32_t issue, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(issue)
      : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint32_t issue, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(issue)
      : "memory");
}
// Operand whose rows (128 bytes = 64 values of the M or N dimension, 128-byte
// swizzle) are steps of the k dimension: 8-row groups 1024 bytes apart along k,
// blocks of 64 values `block` bytes apart along M or N.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t block) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(block >> 4) << 16;   // leading byte offset: next 64 values
  d |= static_cast<uint64_t>(1024 >> 4) << 32;    // stride byte offset: next 8 steps of k
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;            // SWIZZLE_128B
  return d;
}
// Warp-collective: 32 lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Three-input maximum.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Bits 0 .. n set (none for n < 0, all from 31 on).
__device__ __forceinline__ uint32_t ones_to(int n) {
  return n < 0 ? 0u : 0xffffffffu >> (31 - min(n, 31));
}

namespace k9 {

constexpr int WARPS = 12;
constexpr int THREADS = WARPS * 32;
constexpr int TILE = 128;              // keys of a tile, rows of a sub-tile
constexpr int ROWS = 2 * TILE;
constexpr int REG_SOFTMAX = 200, REG_OTHER = 96;   // 256 * 200 + 128 * 96 <= 384 * 168, the launch's registers
constexpr uint32_t TMEM_COLS = 512;
constexpr float GROWTH = 8.f;          // rescale when the maximum (base 2) has grown by more
constexpr int kMaxSeqs = 16384;        // the plan's two prefix sums fit the ring
constexpr int CTRL_BYTES = 2048;
constexpr int kPartFloats = ROWS * (128 + 2);   // of one slot: accumulators, maximum, sum

template <int D, int FMT>
struct Cfg {
  static constexpr bool INT4 = FMT == kKvInt4;
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = TILE * D * 2;   // Q sub-tile, K tile, V tile: HALVES blocks of 128 x 64
  static constexpr int HALF_BYTES = TILE * 128;
  static constexpr int STAGES = (INT4 ? 4 : 5) * (D == 128 ? 1 : 2);
  // 4-bit pages: scales of a tile's keys, then of its values, three tiles deep: for keys
  // c, c + 1 the four floats (scale, scale, offset, offset)
  static constexpr int AFFINE_TILE = 2 * TILE * 8, AFFINES = 3;
  static constexpr int AFFINE = INT4 ? AFFINES * AFFINE_TILE : 0;
  // and key or value tiles as they are in the pages, three deep: codes, then scale pairs
  static constexpr int RAW_CODES = TILE * D / 2, RAW_TILE = RAW_CODES + TILE * 4, RAWS = INT4 ? 3 : 0;
  static constexpr int SMEM = 2 * TILE_BYTES + STAGES * TILE_BYTES + AFFINE + RAWS * RAW_TILE + 1024 + CTRL_BYTES;
  static_assert(SMEM <= 227 * 1024, "shared memory of a block");
  static constexpr uint32_t S0 = 0, O0 = 256;       // TMEM columns: S at 0 and 128 (P over it), O at 256 and 256 + D
  static_assert(2 * (kMaxSeqs + 1) * 4 <= STAGES * TILE_BYTES + AFFINE, "prefix sums in the ring");
};

struct Params {
  AttnParams a;
  unsigned* claim;   // whole tiles taken beyond the first wave; blocks that have ended. Both zero between launches
};

// A row tile: 256 rows of a sequence (one key head) and its key tiles, the union
// of what its rows see: tiles that hold sinks, then those from the window on.
struct RowTile {
  int first, n, rows, pos_first;   // the sequence's rows in the batch, its new tokens, rows and first position
  int r0;
  int lo_tile, sink_tiles, n0, n1; // key tiles that the two sub-tiles reach: the first n0, n1 of the list
  k8::Sight sight;
  __device__ __forceinline__ int tiles() const { return max(max(n0, n1), 1); }   // one at least writes the rows
};
__device__ __forceinline__ RowTile row_tile(const AttnParams& p, int b, int j) {
  const KvSeq q = kv_seq(p.kv, b);
  RowTile t;
  t.first = q.first;
  t.n = q.n;
  t.rows = q.n * p.group;
  t.pos_first = q.len - q.n;
  t.r0 = j * ROWS;
  k8::Sight& s = t.sight;
  s.pos0 = t.pos_first + t.r0 / p.group;
  s.last = t.pos_first + (min(t.r0 + ROWS, t.rows) - 1) / p.group;
  s.rows = t.rows;
  s.group = p.group;
  s.len = min(q.len, s.last + 1);
  s.window = p.window;
  s.sinks = p.sinks;
  s.lo = p.window > 0 ? max(0, s.pos0 - p.window + 1) : 0;
  t.lo_tile = s.lo / TILE;
  t.sink_tiles = min((min(p.sinks, max(s.len, 0)) + TILE - 1) / TILE, t.lo_tile);
  auto reach = [&](int first) {
    if (first >= t.rows) return 0;
    const int end = min(q.len, t.pos_first + (min(first + TILE, t.rows) - 1) / p.group + 1);
    return end > 0 ? t.sink_tiles + (end + TILE - 1) / TILE - t.lo_tile : 0;
  };
  t.n0 = reach(t.r0);
  t.n1 = reach(t.r0 + TILE);
  return t;
}
__device__ __forceinline__ int row_tiles(const AttnParams& p, int b) {
  return (kv_seq(p.kv, b).n * p.group + ROWS - 1) / ROWS;
}

// A piece of work: key tiles [t0, t1) of a row tile for one key head; t1 = 0: the end.
// Parts of a tile shared by the blocks c0 .. c1.
struct Piece {
  RowTile t;
  int head, b, t0, t1, c0, c1;
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == t.tiles(); }
};

struct Ctrl {
  uint64_t full[10], empty[10], s_full[2], p_full[2], o_full[2], q_full, q_empty, work_full[2], work_empty[2], join, drain;
  uint64_t a_full[4], a_empty[4], raw_full[3], raw_empty[3];
  uint32_t tmem_base;
  uint32_t armed, armed_parity;   // ring slots with a copy issued, and the parity of each one's last
  int abort_flag;
  int scan[WARPS];
  int found[2];                   // the block's first shared tile, units before it
  int last;                       // this block arrived last at a shared piece
  Piece piece[2];
};
static_assert(sizeof(Ctrl) <= CTRL_BYTES, "the control block");

// Sequence and row tile of tile `idx` of the plan's order, from the prefix sums: all
// row tiles, and late ones, before each sequence.
__device__ __forceinline__ void tile_at(const int* all, const int* late, int B, long long N1, long long idx, int& b, int& j) {
  const bool second = idx >= N1;
  auto before = [&](int i) { return second ? late[i] : all[i] - late[i]; };
  const int r = static_cast<int>((second ? idx - N1 : idx) % before(B));
  int lo = 0, hi = B - 1;
  while (lo < hi) {   // the last sequence whose first tile of the kind is at most r
    const int mid = (lo + hi + 1) >> 1;
    if (before(mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  b = lo;
  j = (second ? late[lo + 1] - late[lo] : all[lo + 1] - all[lo]) - 1 - (r - before(lo));
}

template <int D, int FMT>
__global__ void __launch_bounds__(THREADS, 1)
    k9_prompt(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ Params prm) {
  typedef Cfg<D, FMT> C;
  const AttnParams& p = prm.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * C::TILE_BYTES;
  uint8_t* affine = ring + C::STAGES * C::TILE_BYTES;
  uint8_t* raw = affine + C::AFFINE;
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(raw + C::RAWS * C::RAW_TILE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abortf = &ctrl->abort_flag;
  int* status = p.kv.status;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&ctrl->full[s], C::INT4 ? 2 : 1);   // the unpacking warps, or the TMA copies
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctrl->s_full[s], 1);
      mbar_init(&ctrl->p_full[s], 4);
      mbar_init(&ctrl->o_full[s], 1);
    }
    for (int s = 0; s < C::AFFINES; ++s) {
      mbar_init(&ctrl->a_full[s], 2);
      mbar_init(&ctrl->a_empty[s], 8);
    }
    for (int s = 0; s < C::RAWS; ++s) {
      mbar_init(&ctrl->raw_full[s], 1);
      mbar_init(&ctrl->raw_empty[s], 2);
    }
    mbar_init(&ctrl->q_full, 2);
    mbar_init(&ctrl->q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctrl->work_full[s], 1);
      mbar_init(&ctrl->work_empty[s], 11);   // the warps that read the queue
    }
    mbar_init(&ctrl->join, 8);
    mbar_init(&ctrl->drain, 1);
    ctrl->abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();

  // ---- the plan: prefix sums of the sequences' row tiles, then of the row tiles' key tiles
  int* first_tile = reinterpret_cast<int*>(ring);   // [B + 1] row tiles before each sequence
  auto block_scan = [&](int v, int& total) {        // inclusive scan over the block's threads
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) ctrl->scan[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += ctrl->scan[w];
      all += ctrl->scan[w];
    }
    total = all;
    return x + before;
  };
  const int B = p.kv.B;
  int R = 0;
  for (int i = 0; i < B; i += THREADS) {
    const int b = i + threadIdx.x;
    int total;
    const int x = block_scan(b < B ? row_tiles(p, b) : 0, total);
    if (b < B) first_tile[b + 1] = R + x;
    R += total;
  }
  if (threadIdx.x == 0) first_tile[0] = 0;
  __syncthreads();
  // Tiles in the order they are taken: first, key head by key head and from the longest
  // of a sequence down, those behind a sequence's first `cut` row tiles; then these
  // first ones, key head by key head, about two for every block: causal tiles grow from
  // a sequence's start, so the blocks end on short ones.
  const int G = gridDim.x;
  const int cut = static_cast<int>((2LL * G + static_cast<long long>(p.kv.Hkv) * B - 1) / (static_cast<long long>(p.kv.Hkv) * B));
  int late = 0;   // row tiles (of one key head) of the second kind
  int* late_tile = first_tile + kMaxSeqs + 1;
  for (int i = 0; i < B; i += THREADS) {
    const int b = i + threadIdx.x;
    int total;
    const int x = block_scan(b < B ? min(first_tile[b + 1] - first_tile[b], cut) : 0, total);
    if (b < B) late_tile[b + 1] = late + x;
    late += total;
  }
  if (threadIdx.x == 0) late_tile[0] = 0;
  __syncthreads();
  const int early = R - late;
  const long long N = static_cast<long long>(R) * p.kv.Hkv, N1 = static_cast<long long>(early) * p.kv.Hkv;
  // Of many tiles, whole waves are taken whole and the rest may be shared; of few (one a
  // thread here) all may. They are, in parts of six key tiles at least (a part costs its
  // sums' way through memory, about 8 us, some six key tiles' time), where that ends
  // sooner than whole ones would: with the longest when every block has one at most,
  // else about half of the longest after the even share. Against always sharing what
  // fills no wave, four chunks of 25 tokens and one prompt of 900 over 4-bit pages
  // (D = 128) took 30 and 49 us instead of 41 and 65; five prompts of 172 row tiles, up
  // to 18 key tiles long, 100 instead of 115 as one shared list.
  const long long full = N <= THREADS ? 0 : N / G * G;
  int units_rest = 0, my_tiles = 0;
  const int rest0 = static_cast<int>(N - full);   // <= THREADS (G is below it)
  if (static_cast<int>(threadIdx.x) < rest0) {
    int b, j;
    tile_at(first_tile, late_tile, B, N1, full + threadIdx.x, b, j);
    my_tiles = row_tile(p, b, j).tiles();
  }
  if (threadIdx.x == 0) ctrl->last = 0;
  const int my_end = block_scan(my_tiles, units_rest);
  const int longest_in_warp = __reduce_max_sync(0xffffffffu, my_tiles);
  if (lane == 0 && longest_in_warp > 0) atomicMax(&ctrl->last, longest_in_warp);
  __syncthreads();
  const int shared_by = min(G, max(rest0, units_rest / 6));
  const int longest = ctrl->last;
  const int whole_rest = rest0 <= G ? longest : max(longest, units_rest / G + longest / 2);
  const bool share_rest = rest0 > 0 && units_rest / shared_by + 6 < whole_rest;
  const long long W = share_rest ? full : N;
  const int Gr = share_rest ? shared_by : 0;
  const bool shares = static_cast<int>(blockIdx.x) < Gr;
  const int u0 = shares ? static_cast<int>(static_cast<long long>(blockIdx.x) * units_rest / Gr) : 0;
  const int u1 = shares ? static_cast<int>(static_cast<long long>(blockIdx.x + 1) * units_rest / Gr) : 0;
  if (shares && my_tiles > 0 && my_end > u0 && my_end - my_tiles <= u0) {
    ctrl->found[0] = threadIdx.x;
    ctrl->found[1] = my_end - my_tiles;
  }
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  fence_proxy_async_smem();   // the plan's stores into the ring come before its bulk copies
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;

  // The other roles' side of the queue: the next piece (null when the wait gives up),
  // and its release.
  uint32_t taken = 0;
  auto take = [&]() -> const Piece* {
    const int q = taken & 1;
    if (!warp_wait(&ctrl->work_full[q], (taken >> 1) & 1, abortf, status, kStatusWaitFull, p.wait_ns)) return nullptr;
    return &ctrl->piece[q];
  };
  auto release = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctrl->work_empty[taken & 1]);
    ++taken;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_OTHER));
    const int page = 1 << p.kv.page_shift;
    const int bp = min(page, TILE);                          // keys of one copy
    const int copies = (TILE / bp) * C::HALVES;              // at most 16 lanes
    const int part = lane / C::HALVES, half = lane % C::HALVES;
    int slot = 0;
    uint32_t ph = 0, armed = 0, parity = 0;
    bool withhold = p.stall != 0 && blockIdx.x == 0;
    bool ok = true;
    uint32_t sent = 0;
    // the last tile taken: its kind, head and sequence, row tiles of that kind before the sequence
    int at_kind = 0, at_head = 0, at_b = 0, at_r = 0;
    // Tile `idx` for the whole warp: 32 sequences at a time from the last one on.
    auto find = [&](long long idx, int& head, int& b, int& j) {
      const int kind = idx >= N1;
      const int per = kind ? late : early;
      if (kind) idx -= N1;
      head = static_cast<int>(idx / per);
      const int r = static_cast<int>(idx - static_cast<long long>(head) * per);
      if (kind != at_kind || head != at_head || r < at_r) at_b = at_r = 0;
      at_kind = kind;
      at_head = head;
      while (at_b < B) {
        const int all = at_b + lane < B ? row_tiles(p, at_b + lane) : 0;
        const int mine = kind ? min(all, cut) : max(all - cut, 0);
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const unsigned behind = __ballot_sync(0xffffffffu, at_r + x > r);
        if (behind) {
          const int l = __ffs(behind) - 1;
          const int end = at_r + __shfl_sync(0xffffffffu, x, l), m = __shfl_sync(0xffffffffu, mine, l);
          const int n = __shfl_sync(0xffffffffu, all, l);
          at_b += l;
          at_r = end - m;
          b = at_b;
          j = (kind ? m : n) - 1 - (r - at_r);
          return;
        }
        at_r += __shfl_sync(0xffffffffu, x, 31);
        at_b += 32;
      }
      b = j = at_b = at_r = 0;   // the batch's arrays have changed under the kernel: any tile will do
    };
    // Announces a piece (t1 < 0: to the tile's end) and copies its tiles.
    auto serve = [&](int head, int b, int j, int t0, int t1, int c0, int c1) {
      const int q = sent & 1;
      ok = warp_wait(&ctrl->work_empty[q], ((sent >> 1) & 1) ^ 1u, abortf, status, kStatusWaitEmpty, p.wait_ns);
      if (!ok) return;
      Piece& w = ctrl->piece[q];
      if (lane == 0) {
        if (t1 != 0) w.t = row_tile(p, b, j);
        w.head = head;
        w.b = b;
        w.t0 = t0;
        w.t1 = t1 < 0 ? w.t.tiles() : t1;
        w.c0 = c0;
        w.c1 = c1;
        mbar_arrive(&ctrl->work_full[q]);
      }
      __syncwarp();
      ++sent;
      t1 = w.t1;
      const k8::Sight sight = w.t.sight;
      const int lo_tile = w.t.lo_tile, sink_tiles = w.t.sink_tiles;
      if (C::INT4) {   // whole runs of rows and of their scale pairs, for warps 2 and 3 to unpack
        for (int i = t0; i < t1 && ok; ++i) {
          const int key = (i < sink_tiles ? i : lo_tile + i - sink_tiles) * TILE + lane * bp;
          int id = -1;   // of this lane's run
          if (lane < TILE / bp && key < sight.len && (key + bp > sight.lo || key < sight.sinks)) id = kv_page(p.kv, b, key);
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * bp * (D / 2 + 4);
          const int row = kv_row_in_page(p.kv, head, key);
          for (int kv = 0; kv < 2; ++kv) {
            ok = warp_wait(&ctrl->raw_empty[slot], ph ^ 1u, abortf, status, kStatusWaitEmpty, p.wait_ns);
            if (!ok) break;
            if (withhold) {
              withhold = false;
            } else {
              if (lane == 0) {
                if (bytes) mbar_arrive_expect_tx(&ctrl->raw_full[slot], bytes);
                else mbar_arrive(&ctrl->raw_full[slot]);
              }
              __syncwarp();
              if (id >= 0) {
                const uint32_t dst = smem_u32(raw) + slot * C::RAW_TILE;
                k8::bulk_load_at(dst + lane * bp * (D / 2),
                          (kv ? p.kv.v : p.kv.k) + id * p.kv.page_stride + static_cast<long long>(row) * (D / 2), bp * (D / 2),
                          &ctrl->raw_full[slot]);
                k8::bulk_load_at(dst + C::RAW_CODES + lane * bp * 4, (kv ? p.kv.v_scale : p.kv.k_scale) + id * p.kv.scale_stride + row,
                          bp * 4, &ctrl->raw_full[slot]);
              }
              armed |= 1u << slot;
              parity = (parity & ~(1u << slot)) | (ph << slot);
            }
            if (++slot == C::RAWS) {
              slot = 0;
              ph ^= 1u;
            }
          }
        }
        return;
      }
      for (int i = t0; i < t1 && ok; ++i) {
        const int key = (i < sink_tiles ? i : lo_tile + i - sink_tiles) * TILE + part * bp;
        int id = -1;
        if (lane < copies && key < sight.len && (key + bp > sight.lo || key < sight.sinks)) id = kv_page(p.kv, b, key);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * bp * 128;
        const int row = kv_row_in_page(p.kv, head, key);
        for (int kv = 0; kv < 2; ++kv) {
          ok = warp_wait(&ctrl->empty[slot], ph ^ 1u, abortf, status, kStatusWaitEmpty, p.wait_ns);
          if (!ok) break;
          if (withhold) {
            withhold = false;
          } else {
            if (lane == 0) {
              if (bytes) mbar_arrive_expect_tx(&ctrl->full[slot], bytes);
              else mbar_arrive(&ctrl->full[slot]);
            }
            __syncwarp();
            if (id >= 0)
              tma_load_3d(smem_u32(ring) + slot * C::TILE_BYTES + half * C::HALF_BYTES + part * bp * 128,
                          kv ? &tm_v : &tm_k, &ctrl->full[slot], half * 64, row, id);
            armed |= 1u << slot;
            parity = (parity & ~(1u << slot)) | (ph << slot);
          }
          if (++slot == C::STAGES) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
    };
    int head, b, j;
    for (long long idx = blockIdx.x; ok && idx < W;) {   // whole tiles: the first by block number, then as they come
      find(idx, head, b, j);
      serve(head, b, j, 0, -1, 0, 0);
      unsigned got = 0;
      if (lane == 0) got = atomicAdd(prm.claim, 1u);
      idx = static_cast<long long>(G) + __shfl_sync(0xffffffffu, got, 0);
    }
    if (shares) {
      int tile = ctrl->found[0], base = ctrl->found[1];
      for (int u = u0; ok && u < u1; ++tile) {
        find(W + tile, head, b, j);
        const int n = row_tile(p, b, j).tiles();
        serve(head, b, j, u - base, min(u1 - base, n), unit_owner(base, Gr, units_rest), unit_owner(base + n - 1, Gr, units_rest));
        base += n;
        u = base;
      }
    }
    if (ok) serve(0, 0, 0, 0, 0, 0, 0);   // the end
    if (lane == 0) {
      ctrl->armed = armed;
      ctrl->armed_parity = parity;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_OTHER));
    constexpr uint32_t idesc_qk = idesc_bf16(TILE, TILE);
    constexpr uint32_t idesc_pv = idesc_bf16(TILE, D) | (1u << 16);   // B rows are keys: transposed
    int slot = 0;
    uint32_t ph = 0, pieces = 0, done[2] = {0, 0};   // done: tiles of each sub-tile so far, over all pieces
    auto advance = [&]() {
      if (++slot == C::STAGES) {
        slot = 0;
        ph ^= 1u;
      }
    };
    // descriptors differ in their address field alone (16-byte units)
    const uint64_t kmajor = sw128_desc(0), nmajor = sw128_mn_desc(0, C::HALF_BYTES);
    const uint32_t q16 = smem_u32(smem) >> 4, ring16 = smem_u32(ring) >> 4;
    const uint32_t one = lane == 0;
    auto commit = [&](uint64_t* bar) { umma_commit_if(one, bar); };
    auto qk = [&](int s, int at) {
      const uint64_t q = kmajor + q16 + s * (C::TILE_BYTES >> 4), k = kmajor + ring16 + at * (C::TILE_BYTES >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = ((kk >> 2) * C::HALF_BYTES + (kk & 3) * 32) >> 4;
        umma_bf16_if(one, tmem + C::S0 + s * TILE, q + o, k + o, idesc_qk, kk > 0);
      }
      commit(&ctrl->s_full[s]);
    };
    auto pv = [&](int s, int at, bool first) {
      const uint64_t v = nmajor + ring16 + at * (C::TILE_BYTES >> 4);
      const uint32_t o = tmem + C::O0 + s * D, a = tmem + C::S0 + s * TILE;
#pragma unroll
      for (int kk = 0; kk < TILE / 16; ++kk)
        umma_bf16_ts_if(one, o, a + kk * 8, v + kk * (2048 >> 4), idesc_pv, !first || kk > 0);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
      const bool r = warp_wait(bar, parity & 1u, abortf, status, code, p.wait_ns);
      if (r) tc_fence_after();
      return r;
    };
    bool ok = true;
    while (ok) {
      const Piece* w = take();
      ok = w != nullptr;
      if (!ok || w->t1 == 0) break;
      const int reach[2] = {w->t.n0, w->t.n1};
      const k8::Sight sight = w->t.sight;
      const int t0 = w->t0, t1 = w->t1, lo_tile = w->t.lo_tile, sink_tiles = w->t.sink_tiles;
      release();
      ok = wait(&ctrl->q_full, pieces++, kStatusWaitConv) && wait(&ctrl->full[slot], ph, kStatusWaitFull);
      if (!ok) break;
      for (int s = 0; s < 2; ++s)
        if (t0 < reach[s]) qk(s, slot);
      commit(&ctrl->empty[slot]);
      if (t1 - t0 == 1) commit(&ctrl->q_empty);
      advance();
      for (int i = t0; i < t1 && ok; ++i) {
        // V of tile i at `slot`, K of tile i + 1 behind it
        const int vs = slot;
        ok = wait(&ctrl->full[slot], ph, kStatusWaitFull);
        if (!ok) break;
        const int key = (i < sink_tiles ? i : lo_tile + i - sink_tiles) * TILE;
        if (!C::INT4 && (key + TILE > sight.len || (key < sight.lo && key + TILE > sight.sinks))) {
          // rows of V that nobody sees become zeros (a warp instruction covers 4 rows' halves)
          for (int r = lane >> 3; r < TILE; r += 4)
            if (!sight.any(key + r))
              for (int h = 0; h < C::HALVES; ++h)
                st_shared_v4(smem_u32(ring) + vs * C::TILE_BYTES + h * C::HALF_BYTES + r * 128 + (lane & 7) * 16,
                             make_uint4(0, 0, 0, 0));
          fence_proxy_async_smem();
          __syncwarp();
        }
        advance();
        // (K first: nothing is waited for between a sub-tile's two products)
        const int ks = slot;
        if (i + 1 < t1) ok = wait(&ctrl->full[ks], ph, kStatusWaitFull);
        for (int s = 0; s < 2 && ok; ++s) {
          if (i < reach[s]) {
            ok = wait(&ctrl->p_full[s], done[s], kStatusWaitConv);
            if (!ok) break;
            ++done[s];
            pv(s, vs, i == t0);
            if (i + 1 < t1 && i + 1 < reach[s]) qk(s, ks);
            else commit(&ctrl->o_full[s]);
          }
          if (s == 1) commit(&ctrl->empty[vs]);
        }
        if (ok && i + 1 < t1) {
          commit(&ctrl->empty[ks]);
          if (i + 2 == t1) commit(&ctrl->q_empty);
          advance();
        }
      }
    }
    if (!ok || *abortf) {   // every product issued is done before TMEM is freed
      commit(&ctrl->drain);
      if (lane == 0) k8::drain_wait(&ctrl->drain, 0);
      __syncwarp();
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ Q
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_OTHER));
    constexpr int CH = D / 8, STEP = 64 / CH;   // 16-byte chunks of a row; rows of one turn of the 64 threads
    const int t = threadIdx.x - 64, c = t % CH;
    uint32_t pieces = 0, tiles = 0, ph = 0, raw_ph = 0;
    int slot = 0, raw_slot = 0;
    bool ok = true;
    while (ok) {
      const Piece* w = take();
      ok = w != nullptr;
      if (!ok || w->t1 == 0) break;
      const int t0 = w->t0, t1 = w->t1, lo_tile = w->t.lo_tile, sink_tiles = w->t.sink_tiles;
      const k8::Sight sight = w->t.sight;
      const int r0 = w->t.r0, rows = w->t.rows, first = w->t.first, head0 = w->head * p.group;
      release();
      if (pieces > 0) ok = warp_wait(&ctrl->q_empty, (pieces - 1) & 1u, abortf, status, kStatusWaitEmpty, p.wait_ns);
      if (!ok) break;
      ++pieces;
      // rows t / CH, + STEP, ..: the row's token and head advance without divisions, and
      // the swizzle repeats every 8 rows
      const int row0 = t / CH;
      int hq = (r0 + row0) % p.group;
      const bf16* src = p.q + (static_cast<long long>(head0 + hq) * p.kv.M + first + (r0 + row0) / p.group) * D + c * 8;
      const long long step = (static_cast<long long>(STEP % p.group) * p.kv.M + STEP / p.group) * D;
      const long long wrap = (1 - static_cast<long long>(p.group) * p.kv.M) * D;
      const uint32_t dst = smem_u32(smem) + (c >> 3) * C::HALF_BYTES;
      auto to = [&](int k, int e) {   // shared address of this thread's chunk of row k * 8 + e * STEP + row0
        const int row = k * 8 + e * STEP + row0;
        return dst + (row >= TILE ? C::TILE_BYTES - TILE * 128 : 0) + row * 128 + (((c & 7) ^ ((e * STEP + row0) & 7)) << 4);
      };
      auto advance = [&]() {
        src += step;
        hq += STEP % p.group;
        if (hq >= p.group) {
          hq -= p.group;
          src += wrap;
        }
      };
      if (C::INT4) {   // the d of every eight in the order in which codes come out of a word
        constexpr int AT_ONCE = 16, PER = 8 / STEP;   // loads at a time; of one k
#pragma unroll 1
        for (int k = 0; k < ROWS / 8; k += AT_ONCE / PER) {
          uint4 y[AT_ONCE];
#pragma unroll
          for (int e = 0; e < AT_ONCE; ++e) {
            y[e] = r0 + k * 8 + e * STEP + row0 < rows ? ldg16(src) : make_uint4(0, 0, 0, 0);
            advance();
          }
#pragma unroll
          for (int e = 0; e < AT_ONCE; ++e)
            st_shared_v4(to(k + e / PER, e % PER),
                         make_uint4(__byte_perm(y[e].x, y[e].z, 0x5410), __byte_perm(y[e].x, y[e].z, 0x7632),
                                    __byte_perm(y[e].y, y[e].w, 0x5410), __byte_perm(y[e].y, y[e].w, 0x7632)));
        }
      } else {
#pragma unroll 2
        for (int k = 0; k < ROWS / 8; ++k) {
#pragma unroll
          for (int e = 0; e < 8 / STEP; ++e) {
            const bool in = r0 + k * 8 + e * STEP + row0 < rows;
            k8::cp16(to(k, e), in ? src : p.q, in ? 16 : 0);
            advance();
          }
        }
        k8::cp_commit();
        k8::cp_wait<0>();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->q_full);
      if (C::INT4) {   // the piece's key and value tiles, unpacked into the ring
        // codes: 16 bytes (32 values) a load, D / 32 lanes a row
        constexpr int LR = D / 32, PASS = 64 / LR;   // lanes of a row, rows of a load
        const int lr = t % LR, row0 = t / LR;
        for (int i = t0; i < t1 && ok; ++i, ++tiles) {
          const int key = (i < sink_tiles ? i : lo_tile + i - sink_tiles) * TILE;
          const int at = tiles % C::AFFINES;
          ok = warp_wait(&ctrl->a_empty[at], ((tiles / C::AFFINES) & 1u) ^ 1u, abortf, status, kStatusWaitEmpty, p.wait_ns);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = ok && warp_wait(&ctrl->raw_full[raw_slot], raw_ph, abortf, status, kStatusWaitFull, p.wait_ns) &&
                 warp_wait(&ctrl->empty[slot], ph ^ 1u, abortf, status, kStatusWaitEmpty, p.wait_ns);
            if (!ok) break;
            const uint32_t from = smem_u32(raw) + raw_slot * C::RAW_TILE;
            {
              uint32_t pair[2];
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(pair[0]), "=r"(pair[1]) : "r"(from + C::RAW_CODES + t * 8));
              float v[4];   // scales, offsets
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const bool seen = sight.any(key + 2 * t + e);   // (other slots may hold anything)
                const float sc = seen ? kv_scale_of(pair[e]) : 0.f, lo = seen ? kv_min_of(pair[e]) : 0.f;
                // the scores in base 2; keys enter the product as 128 + code, values as code - 8
                v[e] = kv ? sc : sc * p.scale_log2;
                v[2 + e] = kv ? fmaf(8.f, sc, lo) : fmaf(-128.f, sc, lo) * p.scale_log2;
              }
              float4* a = reinterpret_cast<float4*>(affine + at * C::AFFINE_TILE + kv * (TILE * 8)) + t;
              *a = make_float4(v[0], v[1], v[2], v[3]);
            }
            const uint32_t dst = smem_u32(ring) + slot * C::TILE_BYTES + (lr >> 1) * C::HALF_BYTES + row0 * 128;
            uint4 x[TILE / PASS];
#pragma unroll
            for (int e = 0; e < TILE / PASS; ++e) x[e] = ld_shared_v4(from + (e * 64 + t) * 16);
#pragma unroll
            for (int e = 0; e < TILE / PASS; ++e) {
              const uint32_t words[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {   // a word's codes in the order (0, 4), (1, 5), (2, 6), (3, 7)
                const uint32_t y = words[q];
                const uint4 o = kv ? make_uint4(k8::code_pair8(y), k8::code_pair8(y >> 4), k8::code_pair8(y >> 8), k8::code_pair8(y >> 12))
                                   : make_uint4(k8::code_pair(y), k8::code_pair(y >> 4), k8::code_pair(y >> 8), k8::code_pair(y >> 12));
                st_shared_v4(dst + e * PASS * 128 + (((((lr & 1) << 2) + q) ^ (row0 & 7)) << 4), o);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (kv) mbar_arrive(&ctrl->a_full[at]);
              mbar_arrive(&ctrl->full[slot]);
              mbar_arrive(&ctrl->raw_empty[raw_slot]);
            }
            if (++raw_slot == C::RAWS) {
              raw_slot = 0;
              raw_ph ^= 1u;
            }
            if (++slot == C::STAGES) {
              slot = 0;
              ph ^= 1u;
            }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFTMAX));
    const int s = (warp - 4) >> 2, quarter = warp & 3;
    const int row = s * TILE + quarter * 32 + lane;          // this thread's row of the 256
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + C::S0 + s * TILE, to = tmem + lanes + C::O0 + s * D;
    const float scale = p.scale_log2;
    uint32_t done = 0, outs = 0;   // tiles and pieces of this sub-tile so far
    uint32_t joins = 0, before = 0;   // before: tiles of the earlier pieces
    auto join = [&]() {            // a bounded barrier of the 8 softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->join);
      return warp_wait(&ctrl->join, joins++ & 1u, abortf, status, kStatusWaitDrain, p.wait_ns);
    };
    bool ok = true;
    while (true) {
      const Piece* w = take();
      if (w == nullptr || w->t1 == 0) break;
      const int rows = w->t.rows, r0 = w->t.r0, r = r0 + row;
      const int t0 = w->t0, end = min(w->t1, s ? w->t.n1 : w->t.n0);
      const int rr = max(min(r, rows - 1), 0);   // (rows is 0 only where the arrays change under the kernel)
      const int pos = w->t.pos_first + rr / p.group;
      // the warp's own span of positions, for its masks
      const int w0 = w->t.pos_first + min(r0 + s * TILE + quarter * 32, rows - 1) / p.group;
      const int w1 = w->t.pos_first + min(r0 + s * TILE + quarter * 32 + 31, rows - 1) / p.group;
      const int lo_tile = w->t.lo_tile, sink_tiles = w->t.sink_tiles;
      float qsum = 0.f;        // 4-bit pages: the row's sum of q
      f32x2 corr2 = pk2(0.f, 0.f);   // and sum of p (minimum + 8 scale)
      if (C::INT4) {
        const bf16* src = p.q + (static_cast<long long>(w->head * p.group + rr % p.group) * p.kv.M + w->t.first + rr / p.group) * D;
#pragma unroll 4
        for (int d = 0; d < D; d += 8) {
          float f[8];
          unpack8(ldg16(src + d), f);
          qsum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        }
      }
      const int t1 = w->t1;
      float top = -INFINITY;   // the maximum that the sum and the accumulators are relative to
      f32x2 sum2 = pk2(0.f, 0.f);
      for (int i = t0; i < end && ok; ++i, ++done) {
        ok = warp_wait(&ctrl->s_full[s], done & 1u, abortf, status, kStatusWaitTmemFull, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        const int key = (i < sink_tiles ? i : lo_tile + i - sink_tiles) * TILE;
        // some row of the warp does not see some key
        const bool edge = key + TILE - 1 > w0 || (p.window > 0 && key <= w1 - p.window && key + TILE > p.sinks);
        const int hi = pos - key, lo = p.window > 0 ? hi - p.window : -1, sk = p.sinks - key;
        auto mask = [&](uint32_t* y, int c0) {   // of 32 scores; bit c: key c0 + c is seen (at most hi; above lo, or below sk)
          const uint32_t seen = ones_to(hi - c0) & (~ones_to(lo - c0) | ones_to(sk - 1 - c0));
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(seen >> c & 1u)) y[c] = 0xff800000u;   // -inf
        };
        uint32_t x[TILE];   // bf16 pages: the row's scores
        const uint32_t at = (before + (i - t0)) % C::AFFINES;
        const uint32_t ak = smem_u32(affine) + at * C::AFFINE_TILE;
        float m;
        if (C::INT4) {
          // s (q . (128 + c)) + (m - 128 s) sum(q), in base 2 already. In loops over 32 scores, which go back to TMEM
          // in between: unrolled over the tile, this code does not stay in the instruction cache
          ok = warp_wait(&ctrl->a_full[at], ((before + (i - t0)) / C::AFFINES) & 1u, abortf, status, kStatusWaitConv, p.wait_ns);
          if (!ok) break;
          const f32x2 qs2 = pk2(qsum, qsum);
          m = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < TILE; c0 += 32) {
            uint32_t y[32];
            tmem_ld32(ts + c0, y);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const uint4 a = ld_shared_v4(ak + (c0 + c) * 8);
              const f32x2 z = fma2(pk2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])),
                                   pk2(__uint_as_float(a.x), __uint_as_float(a.y)),
                                   mul2(pk2(__uint_as_float(a.z), __uint_as_float(a.w)), qs2));
              float y0, y1;
              unpk2(z, y0, y1);
              y[c] = __float_as_uint(y0);
              y[c + 1] = __float_as_uint(y1);
            }
            if (edge) mask(y, c0);
            float m2[2] = {m, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; c += 4)
#pragma unroll
              for (int e = 0; e < 2; ++e) m2[e] = max3(m2[e], __uint_as_float(y[c + 2 * e]), __uint_as_float(y[c + 2 * e + 1]));
            m = fmaxf(m2[0], m2[1]);
#pragma unroll
            for (int c = 0; c < 32; c += 16) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = y[c + e];
              tmem_st16(ts + c0 + c, w);
            }
          }
          tmem_st_wait();
        } else {
#pragma unroll
          for (int c = 0; c < TILE; c += 32) tmem_ld32(ts + c, x + c);
          tmem_ld_wait();
          if (edge) {
#pragma unroll
            for (int c0 = 0; c0 < TILE; c0 += 32) mask(x + c0, c0);
          }
          float m4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) m4[c] = fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 4]));
#pragma unroll
          for (int c = 8; c < TILE; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], __uint_as_float(x[c + e]), __uint_as_float(x[c + 4 + e]));
          m = max3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * scale;
        }
        if (__any_sync(0xffffffffu, m > top + GROWTH)) {
          const bool grow = m > top + GROWTH;
          const float f = grow && top != -INFINITY ? k8::ex2(top - m) : 1.f;
          if (grow) top = m;
          float a, c;
          unpk2(sum2, a, c);
          sum2 = pk2(a * f, c * f);
          if (C::INT4) corr2 = mul2(corr2, pk2(f, f));
          if (i > t0 && __any_sync(0xffffffffu, f != 1.f)) {   // (before the first product O holds nothing)
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t o[16];
              tmem_ld16(to + c0, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(to + c0, o);
            }
          }
        }
        const float base = top == -INFINITY ? 0.f : top;
        const f32x2 scale2 = pk2(scale, scale), base2 = pk2(-base, -base);
        f32x2 part2 = pk2(0.f, 0.f);
        if (C::INT4) {
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            uint32_t y[32], w[16];
            tmem_ld32(ts + h * 32, y);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float a, d;
              unpk2(add2(pk2(__uint_as_float(y[2 * c]), __uint_as_float(y[2 * c + 1])), base2), a, d);
              const f32x2 e = pk2(k8::ex2(a), k8::ex2(d));
              if (c & 1) part2 = add2(part2, e);
              else sum2 = add2(sum2, e);
              // p s goes to the product, p (m + 8 s) is added at the end
              const uint4 v = ld_shared_v4(ak + TILE * 8 + (h * 32 + 2 * c) * 8);
              corr2 = fma2(e, pk2(__uint_as_float(v.z), __uint_as_float(v.w)), corr2);
              unpk2(mul2(e, pk2(__uint_as_float(v.x), __uint_as_float(v.y))), a, d);
              w[c] = pack_bf16x2(a, d);
            }
            tmem_st16(ts + h * 16, w);   // (over scores that have been read)
          }
        } else {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const f32x2 z = pk2(__uint_as_float(x[h * 32 + 2 * c]), __uint_as_float(x[h * 32 + 2 * c + 1]));
              float a, d;
              unpk2(fma2(z, scale2, base2), a, d);
              a = k8::ex2(a);
              d = k8::ex2(d);
              if (c & 1) part2 = add2(part2, pk2(a, d));
              else sum2 = add2(sum2, pk2(a, d));
              w[c] = pack_bf16x2(a, d);
            }
            tmem_st16(ts + h * 16, w);
          }
        }
        sum2 = add2(sum2, part2);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->p_full[s]);
        if (C::INT4 && lane == 0) mbar_arrive(&ctrl->a_empty[at]);
      }
      if (C::INT4) {   // tiles that this sub-tile does not reach
        for (int i = max(end, t0); i < t1 && ok; ++i) {
          const uint32_t at = (before + (i - t0)) % C::AFFINES;
          ok = warp_wait(&ctrl->a_full[at], ((before + (i - t0)) / C::AFFINES) & 1u, abortf, status, kStatusWaitConv, p.wait_ns);
          if (ok && lane == 0) mbar_arrive(&ctrl->a_empty[at]);
        }
        before += t1 - t0;
      }
      // ---- the piece's result
      float a, c;
      unpk2(sum2, a, c);
      float sum = a + c;
      unpk2(corr2, a, c);
      const float corr = a + c;
      if (ok && t0 < end) {
        ok = warp_wait(&ctrl->o_full[s], outs & 1u, abortf, status, kStatusWaitTmemFull, p.wait_ns);
        ++outs;
        tc_fence_after();
      }
      const int token = w->t.first + rr / p.group, hq = w->head * p.group + rr % p.group;
      bf16* dst = p.out + (static_cast<long long>(token) * p.Hq + hq) * D;
      auto put = [&](int c0, const float (&o)[16], float inv) {   // 16 values of this thread's row
        float f[8];
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[C::INT4 ? (k >> 1) + 4 * (k & 1) : k] = o[e + k] * inv;   // (4-bit: a word's order of d)
          kv_store(p.kv, dst + c0 + e, pack8(f), p.out, k8::out_bytes(p, D));
        }
      };
      auto put_lse = [&]() {
        if (p.lse)
          kv_store(p.kv, p.lse + static_cast<long long>(hq) * p.kv.M + token,
                   sum != 0.f ? (top + log2f(sum)) * k8::kLn2 : -INFINITY, p.lse, k8::lse_bytes(p));
      };
      const bool whole = w->whole();
      const int c0 = w->c0, c1 = w->c1;
      // slot 2i + 1 for a piece that begins in block i, 2i for one begun before; [D / 4][256] float4, maxima, sums
      auto slot_of = [&](int blk) { return p.part + static_cast<long long>(2 * blk + (blk == c0)) * kPartFloats; };
      if (ok) {
        float* mine_part = whole ? nullptr : slot_of(blockIdx.x);
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += 16) {
          uint32_t o[16];
          float f[16];
          if (t0 < end) {
            tmem_ld16(to + d0, o);
            tmem_ld_wait();
          }
          // (a row without keys, and a sub-tile without tiles, have no accumulators; a sum that is NaN stays one)
#pragma unroll
          for (int e = 0; e < 16; ++e) f[e] = sum != 0.f ? __uint_as_float(o[e]) + (C::INT4 ? corr : 0.f) : 0.f;
          if (r < rows) {
            if (whole) {
              put(d0, f, sum != 0.f ? 1.f / sum : 0.f);
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                kv_store_cg(p.kv, reinterpret_cast<float4*>(mine_part) + ((d0 + e) >> 2) * ROWS + row,
                            make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]), mine_part, kPartFloats * 4);
            }
          }
        }
        if (r < rows) {
          if (whole) {
            put_lse();
          } else {
            kv_store_cg(p.kv, mine_part + ROWS * D + row, top, mine_part, kPartFloats * 4);
            kv_store_cg(p.kv, mine_part + ROWS * D + ROWS + row, sum, mine_part, kPartFloats * 4);
          }
        }
      }
      if (!whole && ok) {   // the 8 warps together: the last block to arrive adds the parts
        __threadfence();
        ok = join();
        if (threadIdx.x == 128)
          ctrl->last = ok && atom_add_acq_rel_gpu(p.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
        ok = ok && join();
        if (ok && ctrl->last) {
          __threadfence();
          if (r < rows) {
            // four parts' loads at a time
            constexpr int AT_ONCE = 4;
            top = -INFINITY;
            for (int k = c0; k <= c1; k += AT_ONCE) {
              float x[AT_ONCE];
#pragma unroll
              for (int e = 0; e < AT_ONCE; ++e) x[e] = __ldcg(slot_of(min(k + e, c1)) + ROWS * D + row);
#pragma unroll
              for (int e = 0; e < AT_ONCE; ++e) top = fmaxf(top, x[e]);
            }
            sum = 0.f;
            for (int k = c0; k <= c1; ++k)
              sum += (top == -INFINITY ? 0.f : k8::ex2(__ldcg(slot_of(k) + ROWS * D + row) - top)) *
                     __ldcg(slot_of(k) + ROWS * D + ROWS + row);
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 16) {
              float acc[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[e] = 0.f;
              for (int k = c0; k <= c1; k += AT_ONCE) {
                float4 y[AT_ONCE][4];
                float f[AT_ONCE];
#pragma unroll
                for (int q = 0; q < AT_ONCE; ++q) {
                  const float* from = slot_of(min(k + q, c1));
                  f[q] = __ldcg(from + ROWS * D + row);
#pragma unroll
                  for (int e = 0; e < 4; ++e) y[q][e] = __ldcg(reinterpret_cast<const float4*>(from) + (d0 / 4 + e) * ROWS + row);
                }
#pragma unroll
                for (int q = 0; q < AT_ONCE; ++q) {
                  const float g = top == -INFINITY || k + q > c1 ? 0.f : k8::ex2(f[q] - top);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    acc[4 * e] = fmaf(g, y[q][e].x, acc[4 * e]);
                    acc[4 * e + 1] = fmaf(g, y[q][e].y, acc[4 * e + 1]);
                    acc[4 * e + 2] = fmaf(g, y[q][e].z, acc[4 * e + 2]);
                    acc[4 * e + 3] = fmaf(g, y[q][e].w, acc[4 * e + 3]);
                  }
                }
              }
              put(d0, acc, sum != 0.f ? 1.f / sum : 0.f);
            }
            put_lse();
          }
          if (threadIdx.x == 128) p.counters[c0] = 0;
        }
      }
      release();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
  if (warp == 0 && *abortf)   // after an abort nobody has waited for the copies in flight
    for (int s = 0; s < (C::INT4 ? C::RAWS : C::STAGES); ++s)
      if (ctrl->armed & (1u << s)) k8::drain_wait(C::INT4 ? &ctrl->raw_full[s] : &ctrl->full[s], (ctrl->armed_parity >> s) & 1);
  if (threadIdx.x == 0 && atomicAdd(prm.claim + 1, 1u) == gridDim.x - 1) prm.claim[0] = prm.claim[1] = 0;   // the last block
}

}  // namespace k9
}  // namespace fnl
