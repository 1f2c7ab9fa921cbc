// K8: attention over the paged cache, softmax(scale q k^T) v with a causal
// mask, a sliding window and first tokens that stay visible.
//
// One pass over the keys with the running maximum and sum of the softmax
// (base 2: the scores carry scale * log2 e). The rows of a sequence and key head
// are its new tokens times the `group` query heads that share that head, token
// by token: row r is token r / group, head r % group. So one query token of a
// grouped model still fills the 16 rows of an m16n8k16 product, and every key
// and value row is read once for all of them.
//
// Two forms of the same arithmetic:
//   split  few rows (a decode step, a few draft tokens). HBM bound: the keys and
//          values are read once, at 2 * rows products per element, far below
//          what the tensor pipe can do, so the register-level mma form is used:
//          scores and probabilities stay in registers and no accumulator makes a
//          round trip through tensor memory. Each warp streams its own keys
//          through its own ring of asynchronous copies and keeps its own softmax
//          state, so the main loop has no block barrier. The (sequence, key head,
//          key tile) units of the whole batch are dealt evenly over the blocks,
//          so ragged lengths cost nothing; a block's first and last pieces may
//          share their rows with other blocks, which leave fp32 partial sums
//          that the last one to arrive adds in block order (results do not
//          depend on the order of arrival).
//   rows   many rows: each warp owns 16 of the block's rows, all warps read the
//          same key tile.
//
// 4-bit pages: a code enters the product as the exact bf16 value 128 + code
// (two bit operations for two codes); the row's scale and minimum are applied to
// the score, s (q . c) + (m - 128 s) sum(q), in fp32. For the values, code - 8
// is formed exactly in bf16 (centred, so that the sum over many keys keeps its
// low bits), p * s is the rounded operand, and sum(p (m + 8 s)) is added at the
// end. Neither keys nor values are ever rounded.
//
// Rounding: the probabilities enter the second product as bf16 (relative error
// 2^-8 at most each, the same size as the output's own rounding); their sum is taken in
// fp32 before that rounding.
//
// Keys that no row may see (behind the sequence's end, before the window) are
// never read: their copies write zeros, so what such slots hold, NaN included,
// cannot reach a result. A row that sees nothing gives 0 (log-sum-exp -inf).
#pragma once

#include "kv_common.cuh"

namespace fnl {

struct AttnParams {
  KvParams kv;
  const bf16* q;      // [Hq][M][D]
  bf16* out;          // [M][Hq * D]
  float* lse;         // [Hq][M], may be null
  int Hq, group;
  float scale_log2;   // scale * log2(e)
  int window, sinks;  // window 0: none
  float* part;        // split form: [2 * blocks][kPartFloats]
  unsigned* counters; // split form: [blocks], zero between launches
};

namespace k8 {

constexpr int kRowsMax = 16;                                   // rows of one piece of the split form
constexpr int kPartFloats = kRowsMax * (128 + 2);              // accumulators, maximum, sum
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two codes at bits 0-3 and 16-19 -> bf16 pair 128 + code
__device__ __forceinline__ uint32_t code_pair(uint32_t w) { return (w & 0x000F000Fu) | 0x43004300u; }
// the same, centred: code - 8 (exact)
__device__ __forceinline__ uint32_t code_pair8(uint32_t w) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(code_pair(w)), "r"(0x43084308u));   // 136
  return r;
}

// Layout of one warp step (split form) or one block tile (rows form) of KEYS
// keys in shared memory.
template <int D, int FMT, int KEYS>
struct Tile {
  // bf16: rows of D values, 16-byte chunks XORed with the row number (ldmatrix
  // reads 8 rows of one chunk). 4-bit: key rows packed; value rows at a pitch
  // whose even rows fall on distinct banks (a lane reads words of rows 2t, 2t+1).
  static constexpr int kKRow = FMT == kKvBf16 ? D * 2 : D / 2;
  static constexpr int kVRow = FMT == kKvBf16 ? D * 2 : (D == 128 ? 80 : 48);
  static constexpr int kV = KEYS * kKRow;
  static constexpr int kKs = kV + KEYS * kVRow;            // 4-bit: scale pairs of the keys, then of the values
  static constexpr int kVs = kKs + (FMT == kKvBf16 ? 0 : KEYS * 4);
  static constexpr int kBytes = kVs + (FMT == kKvBf16 ? 0 : KEYS * 4);
  static constexpr int kChunks = (FMT == kKvBf16 ? D * 2 : D / 2) / 16;   // 16-byte chunks of a row

  static __device__ __forceinline__ uint32_t k_chunk(int row, int c) {
    return FMT == kKvBf16 ? row * kKRow + ((c ^ (row & 7)) << 4) : row * kKRow + (c << 4);
  }
  static __device__ __forceinline__ uint32_t v_chunk(int row, int c) {
    return FMT == kKvBf16 ? kV + row * kVRow + ((c ^ (row & 7)) << 4) : kV + row * kVRow + (c << 4);
  }
};

// What the rows of one piece may see.
struct Sight {
  int pos0;          // position of row 0's token
  int rows, group;
  int len;           // keys of the sequence
  int window, sinks;
  int lo;            // first key of the window of the piece's first token (0 without a window)
  int last;          // position of the last row's token
  __device__ __forceinline__ bool any(int key) const { return key < len && (key >= lo || key < sinks); }
  __device__ __forceinline__ bool sees(int pos, int key) const {
    return key <= pos && (window == 0 || key > pos - window || key < sinks);
  }
  // every row sees every key of [key, key + n)
  __device__ __forceinline__ bool all(int key, int n) const {
    return key + n - 1 <= pos0 && (window == 0 || key > last - window || key + n <= sinks);
  }
};

// Softmax state and accumulators of 16 rows held by one warp (rows g and g + 8
// of each lane's quad), and the step over NT * 8 keys in shared memory.
template <int D, int FMT, int NT>
struct Rows16 {
  static constexpr int kQ = D / 16;
  uint32_t q[kQ][4];
  float o[D / 8][4];
  float m0, m1, l0, l1;
  float qs0, qs1;      // 4-bit: sum of the row's q
  float c0, c1;        // 4-bit: sum of p (minimum + 8 scale)
  int p0, p1;          // positions of the two rows' tokens

  __device__ __forceinline__ void reset() {
    m0 = m1 = -INFINITY;
    l0 = l1 = c0 = c1 = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  // q row pointers of rows g and g + 8 (null: an empty row of zeros)
  __device__ __forceinline__ void load_q(const bf16* r0, const bf16* r1) {
    const int t = threadIdx.x & 3;
    auto pair = [](const bf16* r, int a, int b) -> uint32_t {
      if (!r) return 0u;
      return static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(r) + a)) |
             (static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(r) + b)) << 16);
    };
    if (FMT == kKvBf16) {
#pragma unroll
      for (int s = 0; s < kQ; ++s) {
        const int a = s * 16 + 2 * t;
        q[s][0] = r0 ? __ldg(reinterpret_cast<const uint32_t*>(r0 + a)) : 0u;
        q[s][1] = r1 ? __ldg(reinterpret_cast<const uint32_t*>(r1 + a)) : 0u;
        q[s][2] = r0 ? __ldg(reinterpret_cast<const uint32_t*>(r0 + a + 8)) : 0u;
        q[s][3] = r1 ? __ldg(reinterpret_cast<const uint32_t*>(r1 + a + 8)) : 0u;
      }
    } else {
      // word j of a lane's codes holds d = (D / 4) t + 8 j + 0..7; product step
      // (j, half) pairs codes (0, 4) and (1, 5), or (2, 6) and (3, 7), as they
      // come out of the word by shifts, and q follows that order of d
#pragma unroll
      for (int s = 0; s < kQ; ++s) {
        const int d = (D / 4) * t + 8 * (s >> 1) + 2 * (s & 1);
        q[s][0] = pair(r0, d, d + 4);
        q[s][1] = pair(r1, d, d + 4);
        q[s][2] = pair(r0, d + 1, d + 5);
        q[s][3] = pair(r1, d + 1, d + 5);
      }
      qs0 = qs1 = 0.f;
#pragma unroll
      for (int s = 0; s < kQ; ++s) {
        qs0 += bf_lo(q[s][0]) + bf_hi(q[s][0]) + bf_lo(q[s][2]) + bf_hi(q[s][2]);
        qs1 += bf_lo(q[s][1]) + bf_hi(q[s][1]) + bf_lo(q[s][3]) + bf_hi(q[s][3]);
      }
      qs0 += __shfl_xor_sync(0xffffffffu, qs0, 1);
      qs1 += __shfl_xor_sync(0xffffffffu, qs1, 1);
      qs0 += __shfl_xor_sync(0xffffffffu, qs0, 2);
      qs1 += __shfl_xor_sync(0xffffffffu, qs1, 2);
    }
  }

  // Keys [key, key + 8 NT) whose rows start at row `row` of the tile at `base`.
  template <int KEYS>
  __device__ __forceinline__ void step(uint32_t base, int row, int key, const Sight& sight, float scale_log2) {
    typedef Tile<D, FMT, KEYS> T;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    // ---- scores
    if (FMT == kKvBf16) {
#pragma unroll
      for (int kk = 0; kk < kQ; ++kk) {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t b[4];
          ldsm4(b, base + T::k_chunk(row + n * 8 + ((lane >> 4) << 3) + (lane & 7), kk * 2 + ((lane >> 3) & 1)));
          mma(s[n], q[kk], b[0], b[1]);
          mma(s[n + 1], q[kk], b[2], b[3]);
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t a = base + (row + n * 8 + g) * T::kKRow + t * (D / 8);
        uint32_t w[D / 32];
        if (D == 128) {
          const uint4 x = ld_shared_v4(a);
          w[0] = x.x; w[1] = x.y; w[D / 32 - 2] = x.z; w[D / 32 - 1] = x.w;
        } else {
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          mma(s[n], q[2 * j], code_pair(w[j]), code_pair(w[j] >> 4));
          mma(s[n], q[2 * j + 1], code_pair(w[j] >> 8), code_pair(w[j] >> 12));
        }
      }
    }
    float vs[NT][2], vm[NT][2];   // 4-bit: scale of the value rows, minimum + 8 scale
    if (FMT == kKvInt4) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t x, y;
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(base + T::kKs + (row + n * 8 + 2 * t) * 4));
        const float sx = kv_scale_of(x), sy = kv_scale_of(y);
        const float mx = fmaf(-128.f, sx, kv_min_of(x)), my = fmaf(-128.f, sy, kv_min_of(y));
        s[n][0] = fmaf(sx, s[n][0], mx * qs0);
        s[n][1] = fmaf(sy, s[n][1], my * qs0);
        s[n][2] = fmaf(sx, s[n][2], mx * qs1);
        s[n][3] = fmaf(sy, s[n][3], my * qs1);
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(base + T::kVs + (row + n * 8 + 2 * t) * 4));
        vs[n][0] = kv_scale_of(x);
        vs[n][1] = kv_scale_of(y);
        vm[n][0] = fmaf(8.f, vs[n][0], kv_min_of(x));
        vm[n][1] = fmaf(8.f, vs[n][1], kv_min_of(y));
      }
    }
    // ---- masks, only where some row does not see some key
    if (!sight.all(key, NT * 8)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = key + n * 8 + 2 * t + e;
          if (!sight.sees(p0, j)) s[n][e] = -INFINITY;
          if (!sight.sees(p1, j)) s[n][2 + e] = -INFINITY;
        }
      }
    }
    // ---- running maximum
    float x0 = s[0][0], x1 = s[0][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      x0 = fmaxf(x0, fmaxf(s[n][0], s[n][1]));
      x1 = fmaxf(x1, fmaxf(s[n][2], s[n][3]));
    }
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)) * scale_log2;
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)) * scale_log2;
    if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      const float f0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0), f1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= f0;
      l1 *= f1;
      if (FMT == kKvInt4) {
        c0 *= f0;
        c1 *= f1;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= f0;
        o[i][1] *= f0;
        o[i][2] *= f1;
        o[i][3] *= f1;
      }
    }
    const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
    // ---- probabilities, and the second product
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) {
      uint32_t a[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = 2 * j + h;
        float e0 = ex2(fmaf(s[n][0], scale_log2, -b0)), e1 = ex2(fmaf(s[n][1], scale_log2, -b0));
        float e2 = ex2(fmaf(s[n][2], scale_log2, -b1)), e3 = ex2(fmaf(s[n][3], scale_log2, -b1));
        l0 += e0 + e1;
        l1 += e2 + e3;
        if (FMT == kKvInt4) {
          c0 = fmaf(e0, vm[n][0], fmaf(e1, vm[n][1], c0));
          c1 = fmaf(e2, vm[n][0], fmaf(e3, vm[n][1], c1));
          e0 *= vs[n][0]; e1 *= vs[n][1]; e2 *= vs[n][0]; e3 *= vs[n][1];
        }
        a[2 * h] = pack_bf16x2(e0, e1);
        a[2 * h + 1] = pack_bf16x2(e2, e3);
      }
      if (FMT == kKvBf16) {
#pragma unroll
        for (int i = 0; i < D / 8; i += 2) {
          uint32_t b[4];
          ldsm4t(b, base + T::v_chunk(row + j * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), i + (lane >> 4)));
          mma(o[i], a, b[0], b[1]);
          mma(o[i + 1], a, b[2], b[3]);
        }
      } else {
        const uint32_t v = base + T::kV + (row + j * 16 + 2 * t) * T::kVRow + g * 4;
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint32_t x[4];   // word g + 8 w of the rows 2t, 2t + 1, 2t + 8, 2t + 9
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[0]) : "r"(v + w * 32));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[1]) : "r"(v + w * 32 + T::kVRow));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[2]) : "r"(v + w * 32 + 8 * T::kVRow));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[3]) : "r"(v + w * 32 + 9 * T::kVRow));
          // neighbouring rows side by side: codes i and i of both for i = 0..3, then 4..7
          const uint32_t a0 = __byte_perm(x[0], x[1], 0x5410), a1 = __byte_perm(x[0], x[1], 0x7632);
          const uint32_t d0 = __byte_perm(x[2], x[3], 0x5410), d1 = __byte_perm(x[2], x[3], 0x7632);
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // tile i of word w: column g is d = 8 (g + 8 w) + i
            mma(o[w * 8 + i], a, code_pair8(a0 >> (4 * i)), code_pair8(d0 >> (4 * i)));
            mma(o[w * 8 + 4 + i], a, code_pair8(a1 >> (4 * i)), code_pair8(d1 >> (4 * i)));
          }
        }
      }
    }
  }

  // Sums of the quad's lanes; the 4-bit minimum term joins the accumulators.
  __device__ __forceinline__ void finish() {
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (FMT == kKvInt4) {
      c0 += __shfl_xor_sync(0xffffffffu, c0, 1);
      c1 += __shfl_xor_sync(0xffffffffu, c1, 1);
      c0 += __shfl_xor_sync(0xffffffffu, c0, 2);
      c1 += __shfl_xor_sync(0xffffffffu, c1, 2);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] += c0;
        o[i][1] += c0;
        o[i][2] += c1;
        o[i][3] += c1;
      }
    }
  }
  // First d of accumulator pair i of this lane (o[i][0], o[i][1] in columns 2t, 2t + 1)
  static __device__ __forceinline__ int d_of(int i, int e) {
    const int t = threadIdx.x & 3;
    if (FMT == kKvBf16) return i * 8 + 2 * t + e;
    return 8 * (2 * t + e + 8 * (i >> 3)) + (i & 7);
  }
};

// ---------------------------------------------------------------- split form
// Key tiles of one sequence (all of its rows at once): the tiles that hold
// sinks, then those from the window's first key on.
struct SeqTiles {
  int first, n, len, pos0, lo, sink_tiles, lo_tile, tiles;
};
template <int TILE>
__device__ __forceinline__ SeqTiles seq_tiles(const AttnParams& p, int b) {
  SeqTiles s;
  const KvSeq q = kv_seq(p.kv, b);
  s.first = q.first;
  s.n = q.n;
  s.len = q.len;
  s.pos0 = q.len - q.n;
  s.lo = p.window > 0 ? max(0, s.pos0 - p.window + 1) : 0;
  s.lo_tile = s.lo / TILE;
  s.sink_tiles = min((min(p.sinks, s.len) + TILE - 1) / TILE, s.lo_tile);
  // a sequence with new tokens has at least one tile, which writes its rows
  s.tiles = q.n > 0 ? max(1, s.sink_tiles + (s.len + TILE - 1) / TILE - s.lo_tile) : 0;
  return s;
}

template <int D, int FMT>
struct SplitCfg {
  static constexpr int NT = 4;                                 // 8-key products of a step
  static constexpr int KEYS = NT * 8;                          // keys of a warp's step
  static constexpr int WARPS = FMT == kKvBf16 ? 4 : 8;
  static constexpr int STAGES = 3;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int TILE = KEYS * WARPS;                    // keys of a unit
  typedef Tile<D, FMT, KEYS> Layout;
  static constexpr int RING = WARPS * STAGES * Layout::kBytes;
  static constexpr int MERGE = WARPS * kRowsMax * (D + 2) * 4; // the merge buffer reuses the ring
  static constexpr int SMEM = (RING > MERGE ? RING : MERGE);
  static constexpr int BLOCKS = 2 * (SMEM + 1024) <= 227 * 1024 ? 2 : 1;   // resident blocks of an SM
};

// Copies of one warp step: lane l resolves key l's page, the lanes then copy the
// rows chunk by chunk. Keys that no row sees become zeros.
template <int D, int FMT, int KEYS>
__device__ __forceinline__ void load_step(const AttnParams& p, int b, int head, int key, const Sight& sight, uint32_t dst) {
  typedef Tile<D, FMT, KEYS> T;
  static_assert(KEYS == 32, "one lane per key");
  const int lane = threadIdx.x & 31;
  int page = -1, row = 0;
  if (sight.any(key + lane)) {
    page = kv_page(p.kv, b, key + lane);
    row = kv_row_in_page(p.kv, head, key + lane);
  }
  const long long off = page >= 0 ? page * p.kv.page_stride + static_cast<long long>(row) * (T::kChunks * 16) : -1;
  constexpr int PER = 32 / T::kChunks;   // rows of one copy instruction
#pragma unroll
  for (int i = 0; i < KEYS / PER; ++i) {
    const int r = i * PER + lane / T::kChunks, c = lane % T::kChunks;
    const long long o = __shfl_sync(0xffffffffu, off, r);
    const int n = o >= 0 ? 16 : 0;
    const long long a = o >= 0 ? o + c * 16 : 0;
    cp16(dst + T::k_chunk(r, c), p.kv.k + a, n);
    cp16(dst + T::v_chunk(r, c), p.kv.v + a, n);
  }
  if (FMT == kKvInt4) {
    const long long a = page >= 0 ? page * p.kv.scale_stride + row : 0;
    const int n = page >= 0 ? 4 : 0;
    cp4(dst + T::kKs + lane * 4, p.kv.k_scale + a, n);
    cp4(dst + T::kVs + lane * 4, p.kv.v_scale + a, n);
  }
}

// Where row r of a piece lives in q and out; r < rows.
__device__ __forceinline__ long long q_row(const AttnParams& p, int first, int head, int r) {
  const int token = first + r / p.group, hq = head * p.group + r % p.group;
  return static_cast<long long>(hq) * p.kv.M + token;
}

// N consecutive values of row r from d0 on, divided by the row's sum; the lane
// that holds d = 0 writes the log-sum-exp.
template <int D, int N>
__device__ __forceinline__ void store_row_part(const AttnParams& p, int first, int head, int r, int d0, const float (&v)[N],
                                               float top, float sum) {
  const int token = first + r / p.group, hq = head * p.group + r % p.group;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  bf16* dst = p.out + (static_cast<long long>(token) * p.Hq + hq) * D + d0;
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<uint2*>(dst + i) =
        make_uint2(pack_bf16x2(v[i] * inv, v[i + 1] * inv), pack_bf16x2(v[i + 2] * inv, v[i + 3] * inv));
  if (d0 == 0 && p.lse)
    p.lse[static_cast<long long>(hq) * p.kv.M + token] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

template <int D, int FMT>
__global__ void __launch_bounds__(SplitCfg<D, FMT>::THREADS, SplitCfg<D, FMT>::BLOCKS)
    k8_attend_split(const __grid_constant__ AttnParams p) {
  typedef SplitCfg<D, FMT> C;
  typedef typename C::Layout L;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int scan[C::WARPS];
  __shared__ int found[4];   // sequence, units before it, ...
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();

  // ---- deal the units: prefix sums over the sequences' tiles
  const int Hkv = p.kv.Hkv;
  auto block_scan = [&](int v, int& total) {   // inclusive scan over the block's threads
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      if (w < warp) before += scan[w];
      all += scan[w];
    }
    total = all;
    return x + before;
  };
  long long U = 0;
  for (int i = 0; i < p.kv.B; i += C::THREADS) {
    const int b = i + threadIdx.x;
    int total;
    block_scan(b < p.kv.B ? seq_tiles<C::TILE>(p, b).tiles : 0, total);
    U += total;
  }
  U *= Hkv;
  const int G = static_cast<int>(min(static_cast<long long>(gridDim.x), U));
  if (static_cast<int>(blockIdx.x) >= G) return;
  const long long u0 = blockIdx.x * U / G, u1 = (blockIdx.x + 1) * U / G;
  // the sequence that holds unit u0, and the units before it
  long long before = 0;
  int b = 0;
  for (int i = 0; i < p.kv.B; i += C::THREADS) {
    const int j = i + threadIdx.x;
    const int v = j < p.kv.B ? seq_tiles<C::TILE>(p, j).tiles : 0;
    int total;
    const int x = block_scan(v, total);
    if (before + static_cast<long long>(total) * Hkv > u0) {
      const long long end = before + static_cast<long long>(x) * Hkv;
      if (end > u0 && end - static_cast<long long>(v) * Hkv <= u0) {
        found[0] = j;
        found[1] = x - v;
      }
      __syncthreads();
      b = found[0];
      before += static_cast<long long>(found[1]) * Hkv;
      break;
    }
    before += static_cast<long long>(total) * Hkv;
  }

  const uint32_t ring = smem_u32(smem) + warp * (C::STAGES * L::kBytes);
  Rows16<D, FMT, C::NT> r16;
  SeqTiles st = seq_tiles<C::TILE>(p, b);
  for (long long u = u0; u < u1;) {
    while (u >= before + static_cast<long long>(st.tiles) * Hkv) {
      before += static_cast<long long>(st.tiles) * Hkv;
      st = seq_tiles<C::TILE>(p, ++b);   // u < u1 <= U: such a sequence exists
    }
    const int head = static_cast<int>((u - before) / st.tiles);
    const long long s0 = before + static_cast<long long>(head) * st.tiles, s1 = s0 + st.tiles;
    const int t0 = static_cast<int>(u - s0), t1 = static_cast<int>(min(u1, s1) - s0);
    Sight sight;
    sight.pos0 = st.pos0;
    sight.rows = st.n * p.group;
    sight.group = p.group;
    sight.len = st.len;
    sight.window = p.window;
    sight.sinks = p.sinks;
    sight.lo = st.lo;
    sight.last = st.pos0 + st.n - 1;
    // this warp's keys of tile i
    auto key_of = [&](int i) {
      return (i < st.sink_tiles ? i : st.lo_tile + i - st.sink_tiles) * C::TILE + warp * C::KEYS;
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) {
      if (t0 + i < t1) load_step<D, FMT, C::KEYS>(p, b, head, key_of(t0 + i), sight, ring + i * L::kBytes);
      cp_commit();
    }
    {
      const int g = lane >> 2, a0 = min(g, sight.rows - 1), a1 = min(g + 8, sight.rows - 1);
      r16.load_q(g < sight.rows ? p.q + q_row(p, st.first, head, a0) * D : nullptr,
                 g + 8 < sight.rows ? p.q + q_row(p, st.first, head, a1) * D : nullptr);
      r16.p0 = st.pos0 + a0 / p.group;
      r16.p1 = st.pos0 + a1 / p.group;
      r16.reset();
    }
    int slot = 0;
    for (int i = t0; i < t1; ++i) {
      const int nx = i + C::STAGES - 1;
      const int ns = slot == 0 ? C::STAGES - 1 : slot - 1;
      if (nx < t1) load_step<D, FMT, C::KEYS>(p, b, head, key_of(nx), sight, ring + ns * L::kBytes);
      cp_commit();
      cp_wait<C::STAGES - 1>();
      __syncwarp();
      const int key = key_of(i);
      // a step none of whose keys is seen is skipped (behind the end, between sinks and window)
      if (key < st.len && (key + C::KEYS > st.lo || key < p.sinks))
        r16.template step<C::KEYS>(ring + slot * L::kBytes, 0, key, sight, p.scale_log2);
      __syncwarp();
      slot = slot == C::STAGES - 1 ? 0 : slot + 1;
    }
    cp_wait<0>();
    // ---- the warps' rows together
    r16.finish();
    __syncthreads();
    float* mo = reinterpret_cast<float*>(smem);                      // [warp][16][D]
    float* mm = mo + C::WARPS * kRowsMax * D;                        // [warp][16] maximum, then sum
    float* ml = mm + C::WARPS * kRowsMax;
    {
      const int g = lane >> 2;
      float* w0 = mo + (warp * kRowsMax + g) * D;
      float* w1 = w0 + 8 * D;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = r16.d_of(i, e);
          w0[d] = r16.o[i][e];
          w1[d] = r16.o[i][2 + e];
        }
      }
      if ((lane & 3) == 0) {
        mm[warp * kRowsMax + g] = r16.m0;
        mm[warp * kRowsMax + g + 8] = r16.m1;
        ml[warp * kRowsMax + g] = r16.l0;
        ml[warp * kRowsMax + g + 8] = r16.l1;
      }
    }
    __syncthreads();
    constexpr int PER = kRowsMax * D / C::THREADS;   // values of a thread, in one row
    const int row = threadIdx.x * PER / D, d0 = threadIdx.x * PER % D;
    float acc[PER], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) top = fmaxf(top, mm[w * kRowsMax + row]);
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      const float f = top == -INFINITY ? 0.f : ex2(mm[w * kRowsMax + row] - top);
      sum += f * ml[w * kRowsMax + row];
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = fmaf(f, mo[(w * kRowsMax + row) * D + d0 + e], acc[e]);
    }
    const bool whole = t0 == 0 && t1 == st.tiles;
    if (whole) {
      if (row < sight.rows) store_row_part<D, PER>(p, st.first, head, row, d0, acc, top, sum);
    } else {
      // partial sums: slot 2i + 1 for a head that begins in this block, 2i for one begun before
      const int c0 = unit_owner(s0, G, U), c1 = unit_owner(s1 - 1, G, U);
      float* mine = p.part + static_cast<long long>(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * kPartFloats;
#pragma unroll
      for (int e = 0; e < PER; e += 4)
        __stcg(reinterpret_cast<float4*>(mine + row * D + d0 + e), make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]));
      if (d0 == 0) {
        __stcg(mine + kRowsMax * D + row, top);
        __stcg(mine + kRowsMax * D + kRowsMax + row, sum);
      }
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) found[2] = atom_add_acq_rel_gpu(p.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
      __syncthreads();
      if (found[2]) {
        __threadfence();
        top = -INFINITY;
        for (int c = c0; c <= c1; ++c)
          top = fmaxf(top, __ldcg(p.part + static_cast<long long>(2 * c + (c == c0)) * kPartFloats + kRowsMax * D + row));
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = 0.f;
        for (int c = c0; c <= c1; ++c) {
          const float* s = p.part + static_cast<long long>(2 * c + (c == c0)) * kPartFloats;
          const float f = top == -INFINITY ? 0.f : ex2(__ldcg(s + kRowsMax * D + row) - top);
          sum += f * __ldcg(s + kRowsMax * D + kRowsMax + row);
#pragma unroll
          for (int e = 0; e < PER; e += 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(s + row * D + d0 + e));
            acc[e] = fmaf(f, x.x, acc[e]);
            acc[e + 1] = fmaf(f, x.y, acc[e + 1]);
            acc[e + 2] = fmaf(f, x.z, acc[e + 2]);
            acc[e + 3] = fmaf(f, x.w, acc[e + 3]);
          }
        }
        if (row < sight.rows) store_row_part<D, PER>(p, st.first, head, row, d0, acc, top, sum);
        if (threadIdx.x == 0) p.counters[c0] = 0;
      }
    }
    __syncthreads();   // the merge buffer is the ring again
    u = before + static_cast<long long>(head) * st.tiles + t1;
  }
}

// ---------------------------------------------------------------- rows form
template <int D, int FMT>
struct RowsCfg {
  static constexpr int WARPS = 8;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ROWS = WARPS * 16;
  static constexpr int NT = 4;
  static constexpr int TILE = 64;          // keys of a block tile
  static constexpr int STAGES = 2;
  typedef Tile<D, FMT, TILE> Layout;
  static constexpr int SMEM = STAGES * Layout::kBytes;
};

template <int D, int FMT>
__global__ void __launch_bounds__(RowsCfg<D, FMT>::THREADS, 1) k8_attend_rows(const __grid_constant__ AttnParams p) {
  typedef RowsCfg<D, FMT> C;
  typedef typename C::Layout L;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const int b = blockIdx.z, head = blockIdx.y;
  const KvSeq q = kv_seq(p.kv, b);
  const int rows = q.n * p.group;
  // the longest (last) row tiles first
  const int tile = static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x);
  const int r0 = tile * C::ROWS;
  if (r0 >= rows) return;
  const int r1 = min(r0 + C::ROWS, rows);
  Sight sight;
  sight.pos0 = q.len - q.n + r0 / p.group;
  sight.last = q.len - q.n + (r1 - 1) / p.group;
  sight.rows = rows;
  sight.group = p.group;
  sight.len = min(q.len, sight.last + 1);
  sight.window = p.window;
  sight.sinks = p.sinks;
  sight.lo = p.window > 0 ? max(0, sight.pos0 - p.window + 1) : 0;
  const int lo_tile = sight.lo / C::TILE;
  const int sink_tiles = min((min(p.sinks, max(sight.len, 0)) + C::TILE - 1) / C::TILE, lo_tile);
  const int tiles = sight.len > 0 ? sink_tiles + (sight.len + C::TILE - 1) / C::TILE - lo_tile : 0;
  auto key_of = [&](int i) { return (i < sink_tiles ? i : lo_tile + i - sink_tiles) * C::TILE; };

  Rows16<D, FMT, C::NT> r16;
  const int g = lane >> 2;
  const int a0 = r0 + warp * 16 + g, a1 = a0 + 8;
  r16.load_q(a0 < rows ? p.q + q_row(p, q.first, head, a0) * D : nullptr,
             a1 < rows ? p.q + q_row(p, q.first, head, a1) * D : nullptr);
  r16.p0 = q.len - q.n + min(a0, rows - 1) / p.group;
  r16.p1 = q.len - q.n + min(a1, rows - 1) / p.group;
  r16.reset();
  // a warp's own range of positions, for its masks
  Sight mine = sight;
  mine.pos0 = q.len - q.n + min(r0 + warp * 16, rows - 1) / p.group;
  mine.last = q.len - q.n + min(r0 + warp * 16 + 15, rows - 1) / p.group;
  const bool live = r0 + warp * 16 < rows;

  // copies of one block tile: 8 warps take 8 keys each
  auto load = [&](int i, int stage) {
    const uint32_t dst = smem_u32(smem) + stage * L::kBytes;
    const int key0 = key_of(i);
    constexpr int PER = C::TILE / C::WARPS;   // keys of a warp
    int page = -1, row = 0;
    if (lane < PER && sight.any(key0 + warp * PER + lane)) {
      page = kv_page(p.kv, b, key0 + warp * PER + lane);
      row = kv_row_in_page(p.kv, head, key0 + warp * PER + lane);
    }
    const long long off = page >= 0 ? page * p.kv.page_stride + static_cast<long long>(row) * (L::kChunks * 16) : -1;
    constexpr int INSTR = (PER * L::kChunks + 31) / 32;
#pragma unroll
    for (int k = 0; k < INSTR; ++k) {
      const int at = k * 32 + lane, r = at / L::kChunks, c = at % L::kChunks;
      const long long o = __shfl_sync(0xffffffffu, off, r < PER ? r : 0);
      if (r < PER) {
        const int n = o >= 0 ? 16 : 0;
        const long long a = o >= 0 ? o + c * 16 : 0;
        cp16(dst + L::k_chunk(warp * PER + r, c), p.kv.k + a, n);
        cp16(dst + L::v_chunk(warp * PER + r, c), p.kv.v + a, n);
      }
    }
    if (FMT == kKvInt4 && lane < PER) {
      const long long a = page >= 0 ? page * p.kv.scale_stride + row : 0;
      const int n = page >= 0 ? 4 : 0;
      cp4(dst + L::kKs + (warp * PER + lane) * 4, p.kv.k_scale + a, n);
      cp4(dst + L::kVs + (warp * PER + lane) * 4, p.kv.v_scale + a, n);
    }
  };

  if (tiles > 0) load(0, 0);
  cp_commit();
  for (int i = 0; i < tiles; ++i) {
    if (i + 1 < tiles) load(i + 1, (i + 1) & 1);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    if (live) {
      const int key0 = key_of(i);
#pragma unroll 1
      for (int k = 0; k < C::TILE; k += C::NT * 8) {
        const int key = key0 + k;
        // skip what none of this warp's rows sees
        if (key > mine.last || (mine.window > 0 && key + C::NT * 8 <= mine.pos0 - mine.window + 1 && key >= mine.sinks))
          continue;
        r16.template step<C::TILE>(smem_u32(smem) + (i & 1) * L::kBytes, k, key, mine, p.scale_log2);
      }
    }
    __syncthreads();
  }
  cp_wait<0>();
  r16.finish();
  // ---- rows out
  auto put = [&](int r, int h, float top, float sum) {
    if (r >= rows) return;
    const int token = q.first + r / p.group, hq = head * p.group + r % p.group;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    bf16* dst = p.out + (static_cast<long long>(token) * p.Hq + hq) * D;
    if (FMT == kKvBf16) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<uint32_t*>(dst + r16.d_of(i, 0)) = pack_bf16x2(r16.o[i][2 * h] * inv, r16.o[i][2 * h + 1] * inv);
    } else {   // a lane holds whole runs of 8 d
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = r16.o[w * 8 + i][2 * h + e] * inv;
          *reinterpret_cast<uint4*>(dst + r16.d_of(w * 8, e)) = pack8(f);
        }
      }
    }
    if ((lane & 3) == 0 && p.lse)
      p.lse[static_cast<long long>(hq) * p.kv.M + token] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
  };
  put(a0, 0, r16.m0, r16.l0);
  put(a1, 1, r16.m1, r16.l1);
}

}  // namespace k8
}  // namespace fnl
