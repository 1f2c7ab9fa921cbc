// K8: attention of a few new tokens over the paged cache, softmax(scale q k^T) v
// with a causal mask, a sliding window and first tokens that stay visible.
//
// One pass over the keys with the running maximum and sum of the softmax
// (base 2: the scores carry scale * log2 e). The rows of a sequence and key head
// are its new tokens times the `group` query heads that share that head, token
// by token: row r is token r / group, head r % group. Every key and value row is
// read once for all of them.
//
// HBM bound: the keys and values are read once, with 2 * rows products per
// element, far below what the tensor pipe can do. So the register-level mma form
// is used, keys as the 16-row operand and the rows as its 8 columns: S^T = K Q^T
// and O^T = V^T P^T. Scores and probabilities stay in registers (P^T is S^T's
// fragment transposed lane by lane), a decode step of up to 8 heads per key head
// wastes no half tile, and a key or value fragment is unpacked once for all rows.
//
// Each warp streams its own keys through its own ring of asynchronous copies (bf16
// pages: 16 bytes a lane, swizzled for ldmatrix; 4-bit pages: bulk copies of whole
// runs of rows, whose few instructions leave the issue slots to the unpacking) and
// keeps its own softmax state, so the main loop has no block barrier. The
// (sequence, key head, key tile) units of the whole batch are dealt evenly over
// the blocks, so ragged lengths cost nothing; a block's first and last pieces may
// share their rows with other blocks, which leave fp32 partial sums that the last
// one to arrive adds in block order (results do not depend on the order of
// arrival).
//
// 4-bit pages: a key's code enters the product as the exact bf16 value 128 + code
// (two bit operations for two codes); the row's scale and minimum are applied to
// the score, s (q . c) + (m - 128 s) sum(q), in fp32. For the values, code - 8
// is formed exactly in bf16 (centred, so that the sum over many keys keeps its
// low bits), p * s is the rounded operand, and sum(p (m + 8 s)) is added at the
// end. Neither keys nor values are ever rounded.
//
// Rounding: the probabilities enter the second product as bf16 (relative error
// 2^-8 at most each, the same size as the output's own rounding); their sum is
// taken in fp32 before that rounding.
//
// Keys that no row may see (behind the sequence's end, before the window) cannot
// reach a result, whatever their slots hold, NaN included. Of bf16 pages they are
// never read: their copies write zeros. Of 4-bit pages whole runs of up to 64 rows
// of a page are copied; their scores are replaced and their scales taken as zeros. A row that sees nothing gives 0 (log-sum-exp -inf); NaN in a
// row's q or scores stays in that row and its log-sum-exp.
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
  unsigned long long wait_ns;   // limit of the waits for copies
  float* part;        // partial sums: two slots a block, each of the form's own kPartFloats
  unsigned* counters; // arrivals at a shared piece: one a block, zero between launches
  int stall;          // fault injection for the status-path tests: block 0 withholds its first copies
};

namespace k8 {

constexpr float kGrowth = 8.f;   // accumulators are rescaled when a row's maximum (base 2) has grown by more: the
                                 // probabilities stay below 256, which bf16 and fp32 hold as exactly as below 1
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
  asm(   // not volatile: independent products may be interleaved
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of 16-bit values, a row over four lanes: transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Bulk copy of neighbouring bytes, 16-byte aligned at both ends.
__device__ __forceinline__ void bulk_load_at(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// The wait that an aborting role ends with: bounded, records nothing.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > FNL_WAIT_NS) return;
}
// two codes at bits 0-3 and 16-19 -> bf16 pair 128 + code
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t r;   // (w & mask) | 128.0 in one instruction
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(0x000F000Fu), "r"(0x43004300u));
  return r;
}
// the same, centred: code - 8 (exact)
__device__ __forceinline__ uint32_t code_pair8(uint32_t w) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(code_pair(w)), "r"(0x43084308u));   // 136
  return r;
}

// Layout of one warp step of KEYS keys in shared memory: key rows, value rows,
// then (4-bit) the scale pairs of both.
template <int D, int FMT, int KEYS>
struct Tile {
  static constexpr int kRow = FMT == kKvBf16 ? D * 2 : D / 2;
  static constexpr int kV = KEYS * kRow;
  static constexpr int kKs = 2 * kV;
  static constexpr int kVs = kKs + KEYS * 4;
  static constexpr int kBytes = FMT == kKvBf16 ? kKs : kVs + KEYS * 4;
  static constexpr int kChunks = kRow / 16;   // 16-byte chunks of a row
  // bf16 chunks are XORed with the row number: ldmatrix reads one chunk of 8 rows
  static __device__ __forceinline__ uint32_t chunk(int row, int c) {
    return row * kRow + ((FMT == kKvBf16 ? c ^ (row & 7) : c) << 4);
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

// Softmax state and accumulators of NR * 8 rows held by one warp, and the step
// over KEYS keys in shared memory. Lane (g, t) = (lane / 4, lane % 4) holds, of each
// 8 rows, rows 2t and 2t + 1: scores of the keys g, g + 8, .. and accumulators of
// the d that its mma rows g and g + 8 stand for.
template <int D, int FMT, int NR, int KEYS>
struct RowState {
  static constexpr int KQ = D / 16, KT = KEYS / 16;
  uint32_t q[KQ][NR][2];
  float o[KQ][NR][4];
  float m[NR][2], l[NR][2];
  float qs[NR][2];     // 4-bit: sum of the row's q
  float cm[NR][2];     // 4-bit: sum of p (minimum + 8 scale)
  int pos[NR][2];      // positions of the rows' tokens

  // Key of mma row r (0..15) of a 16-key tile. 4-bit: a permutation that puts the
  // value rows that a lane quad reads together on both halves of the banks.
  static __device__ __forceinline__ int key_of_row(int r) {
    return FMT == kKvBf16 ? r : (r & 8) + ((r & 7) >> 1) + 4 * (r & 1);
  }
  // d of accumulator rows g (h = 0) and g + 8 (h = 1) of tile i
  static __device__ __forceinline__ int d_of(int i, int h) {
    const int g = (threadIdx.x & 31) >> 2;
    if (FMT == kKvBf16) return i * 16 + h * 8 + g;
    return D == 128 ? 16 * g + 8 * h + i : 8 * g + 4 * h + i;
  }

  // q rows g of each 8 (null: an empty row of zeros) as the column operand
  __device__ __forceinline__ void load(const bf16* (&r)[NR]) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int s = 0; s < KQ; ++s) {
        if (FMT == kKvBf16) {
          const int a = s * 16 + 2 * t;
          q[s][n][0] = r[n] ? __ldg(reinterpret_cast<const uint32_t*>(r[n] + a)) : 0u;
          q[s][n][1] = r[n] ? __ldg(reinterpret_cast<const uint32_t*>(r[n] + a + 8)) : 0u;
        } else {
          // word j of a lane's codes holds d = (D / 4) t + 8 j + 0..7; product step
          // (j, half) pairs codes (0, 4) and (1, 5), or (2, 6) and (3, 7), as they
          // come out of the word by shifts, and q follows that order of d
          const int d = (D / 4) * t + 8 * (s >> 1) + 2 * (s & 1);
          const uint16_t* x = reinterpret_cast<const uint16_t*>(r[n]);
          q[s][n][0] = x ? __ldg(x + d) | (static_cast<uint32_t>(__ldg(x + d + 4)) << 16) : 0u;
          q[s][n][1] = x ? __ldg(x + d + 1) | (static_cast<uint32_t>(__ldg(x + d + 5)) << 16) : 0u;
        }
      }
      if (FMT == kKvInt4) {
        float a = 0.f;
#pragma unroll
        for (int s = 0; s < KQ; ++s) a += bf_lo(q[s][n][0]) + bf_hi(q[s][n][0]) + bf_lo(q[s][n][1]) + bf_hi(q[s][n][1]);
        a += __shfl_xor_sync(0xffffffffu, a, 1);
        a += __shfl_xor_sync(0xffffffffu, a, 2);
        qs[n][0] = __shfl_sync(0xffffffffu, a, 8 * t);       // rows 2t and 2t + 1
        qs[n][1] = __shfl_sync(0xffffffffu, a, 8 * t + 4);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -INFINITY;
        l[n][e] = cm[n][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < KQ; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }
  }

  // Keys [key, key + KEYS) at shared address `base`.
  __device__ __forceinline__ void step(uint32_t base, int key, const Sight& sight, float scale_log2) {
    typedef Tile<D, FMT, KEYS> T;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[KT][NR][4];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int n = 0; n < NR; ++n) s[i][n][0] = s[i][n][1] = s[i][n][2] = s[i][n][3] = 0.f;
    // ---- scores
    if (FMT == kKvBf16) {
#pragma unroll
      for (int kk = 0; kk < KQ; ++kk) {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          uint32_t a[4];
          ldsm4(a, base + T::chunk(i * 16 + (lane & 15), kk * 2 + (lane >> 4)));
#pragma unroll
          for (int n = 0; n < NR; ++n) mma(s[i][n], a, q[kk][n][0], q[kk][n][1]);
        }
      }
    } else {
      uint32_t w[KT][2][D / 32];   // this lane's codes of the keys of rows g and g + 8
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const uint32_t at = base + (i * 16 + key_of_row(g)) * T::kRow + t * (D / 8);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (D == 128) {
            const uint4 x = ld_shared_v4(at + h * 8 * T::kRow);
            w[i][h][0] = x.x; w[i][h][1] = x.y; w[i][h][D / 32 - 2] = x.z; w[i][h][D / 32 - 1] = x.w;
          } else {
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[i][h][0]), "=r"(w[i][h][1]) : "r"(at + h * 8 * T::kRow));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
#pragma unroll
          for (int i = 0; i < KT; ++i) {
            const uint32_t a[4] = {code_pair(w[i][0][j] >> (8 * f)), code_pair(w[i][1][j] >> (8 * f)),
                                   code_pair(w[i][0][j] >> (8 * f + 4)), code_pair(w[i][1][j] >> (8 * f + 4))};
#pragma unroll
            for (int n = 0; n < NR; ++n) mma(s[i][n], a, q[2 * j + f][n][0], q[2 * j + f][n][1]);
          }
        }
      }
    }
    float vs[KT][2], vm[KT][2];   // 4-bit: scale of this lane's value rows, minimum + 8 scale
    const bool edge = !sight.all(key, KEYS);
    if (FMT == kKvInt4) {
#pragma unroll
      for (int i = 0; i < KT; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = i * 16 + h * 8 + key_of_row(g);
          uint32_t x, y;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(base + T::kKs + j * 4));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(y) : "r"(base + T::kVs + j * 4));
          const float sx = kv_scale_of(x), mx = fmaf(-128.f, sx, kv_min_of(x));
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            s[i][n][2 * h] = fmaf(sx, s[i][n][2 * h], mx * qs[n][0]);
            s[i][n][2 * h + 1] = fmaf(sx, s[i][n][2 * h + 1], mx * qs[n][1]);
          }
          vs[i][h] = kv_scale_of(y);
          vm[i][h] = fmaf(8.f, vs[i][h], kv_min_of(y));
        }
      }
    }
    // ---- masks, only where some row does not see some key
    if (edge) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = key + i * 16 + h * 8 + key_of_row(g);
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!sight.sees(pos[n][e], j)) s[i][n][2 * h + e] = -INFINITY;
          if (FMT == kKvInt4 && !sight.any(j)) vs[i][h] = vm[i][h] = 0.f;   // such slots may hold anything
        }
    }
    // ---- running maximum
    float x[NR][2];
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
        for (int i = 1; i < KT; ++i) y = fmaxf(y, fmaxf(s[i][n][e], s[i][n][2 + e]));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16)) * scale_log2;
        x[n][e] = y;
        grow |= y > m[n][e] + kGrowth;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool up = x[n][e] > m[n][e] + kGrowth;
          const float f = up ? ex2(m[n][e] - x[n][e]) : 1.f;
          if (up) m[n][e] = x[n][e];
          l[n][e] *= f;
          cm[n][e] *= f;
#pragma unroll
          for (int i = 0; i < KQ; ++i) {
            o[i][n][e] *= f;
            o[i][n][2 + e] *= f;
          }
        }
    }
    // ---- probabilities, transposed into the second product's column operand
    uint32_t pb[KT][NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const float b0 = m[n][0] == -INFINITY ? 0.f : m[n][0], b1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float e0 = ex2(fmaf(s[i][n][2 * h], scale_log2, -b0)), e1 = ex2(fmaf(s[i][n][2 * h + 1], scale_log2, -b1));
          l[n][0] += e0;
          l[n][1] += e1;
          if (FMT == kKvInt4) {
            cm[n][0] = fmaf(e0, vm[i][h], cm[n][0]);
            cm[n][1] = fmaf(e1, vm[i][h], cm[n][1]);
            e0 *= vs[i][h];
            e1 *= vs[i][h];
          }
          pb[i][n][h] = transpose8(pack_bf16x2(e0, e1));
        }
    }
    // ---- the second product
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      if (FMT == kKvBf16) {
#pragma unroll
        for (int d = 0; d < KQ; ++d) {
          uint32_t a[4];
          ldsm4t(a, base + T::kV + T::chunk(i * 16 + ((lane >> 4) << 3) + (lane & 7), d * 2 + ((lane >> 3) & 1)));
#pragma unroll
          for (int n = 0; n < NR; ++n) mma(o[d][n], a, pb[i][n][0], pb[i][n][1]);
        }
      } else {
        // rows 2t, 2t + 1, 2t + 8, 2t + 9 of the 16: keys t, t + 4, t + 8, t + 12
        constexpr int W = D / 64;   // words of a lane in a row: 2g, 2g + 1 (D = 128), or g
        const uint32_t at = base + T::kV + (i * 16 + t) * T::kRow + g * (4 * W);
        uint32_t x[4][W];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (W == 2)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x[r][0]), "=r"(x[r][W - 1]) : "r"(at + r * 4 * T::kRow));
          else
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[r][0]) : "r"(at + r * 4 * T::kRow));
        }
        // the same code of two rows side by side: codes 0..3 of a word, then 4..7
        uint32_t lo[2][W], hi[2][W];
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            lo[k][w] = __byte_perm(x[2 * k][w], x[2 * k + 1][w], 0x5410);
            hi[k][w] = __byte_perm(x[2 * k][w], x[2 * k + 1][w], 0x7632);
          }
#pragma unroll
        for (int d = 0; d < KQ; ++d) {
          const int c = 4 * (d & 3);
          // D = 128: code d of word 2g and of word 2g + 1; D = 64: codes d and d + 4 of word g
          const uint32_t y0 = D == 128 && d >= 4 ? hi[0][0] : lo[0][0], y2 = D == 128 && d >= 4 ? hi[1][0] : lo[1][0];
          const uint32_t y1 = D == 128 && d < 4 ? lo[0][W - 1] : hi[0][W - 1], y3 = D == 128 && d < 4 ? lo[1][W - 1] : hi[1][W - 1];
          const uint32_t a[4] = {code_pair8(y0 >> c), code_pair8(y1 >> c), code_pair8(y2 >> c), code_pair8(y3 >> c)};
#pragma unroll
          for (int n = 0; n < NR; ++n) mma(o[d][n], a, pb[i][n][0], pb[i][n][1]);
        }
      }
    }
  }

  // Sums over the lanes that hold other keys; the 4-bit minimum term joins the accumulators.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
          if (FMT == kKvInt4) cm[n][e] += __shfl_xor_sync(0xffffffffu, cm[n][e], x);
        }
        if (FMT == kKvInt4) {
#pragma unroll
          for (int i = 0; i < KQ; ++i) {
            o[i][n][e] += cm[n][e];
            o[i][n][2 + e] += cm[n][e];
          }
        }
      }
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

template <int D, int FMT, int NR>
struct SplitCfg {
  static constexpr bool BULK = FMT == kKvInt4;                 // bulk copies (else 16-byte asynchronous ones)
  static constexpr int ROWS = NR * 8;                          // rows of a piece
  // keys of a warp's step, warps, steps in the ring, resident blocks of an SM: chosen
  // by measurement. bf16 pages are bound by memory: 192 KB of ring, two thirds of it
  // in flight. 4-bit pages take longer to unpack than to read (64 sequences of 2000 to
  // 12000: issue slots 50 % used, DRAM 42 %): 64-key steps (fewer loop and copy
  // instructions) with as many warps as their registers leave, two blocks of 6 for 8
  // rows (those 64 sequences: 136 us; 32-key steps with 16 warps 150, with
  // 8 warps 181), one of 8 for 16 rows, whose state is twice as large (130003 keys:
  // 67 us; two blocks of 6 98, 32-key steps with 12 warps 83).
  static constexpr int KEYS = FMT == kKvBf16 ? 32 : 64;
  static constexpr int WARPS = FMT == kKvBf16 ? 4 : (NR == 1 ? 6 : 8);
  static constexpr int STAGES = FMT == kKvBf16 ? 3 : 2;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int TILE = KEYS * WARPS;                    // keys of a unit
  typedef Tile<D, FMT, KEYS> Layout;
  static constexpr int RING = WARPS * STAGES * Layout::kBytes;
  static constexpr int MERGE = WARPS * ROWS * (D + 2) * 4;     // the merge buffer reuses the ring
  static constexpr int SMEM = (RING > MERGE ? RING : MERGE);
  static constexpr int BLOCKS = FMT == kKvBf16 ? (D == 128 ? 1 : 2) : (NR == 1 ? 2 : 1);
  static_assert(BLOCKS * (SMEM + 1536) <= 227 * 1024, "shared memory of an SM");
};

// Bulk copies of warp steps of 4-bit pages. A step is up to KEYS / 16 runs of
// neighbouring rows (a run: the part of one page inside it), each four copies:
// keys, values and their scale pairs. Lane 4 r + w issues copy w of run r; the page
// of the next step is looked up while the present one's copies are issued.
template <int D, int KEYS>
struct BulkLanes {
  typedef Tile<D, kKvInt4, KEYS> T;
  const uint8_t* base;
  long long page_stride;
  int row_bytes, dst, run, offset;   // offset: first key of this lane's run in the step
  bool active;

  __device__ __forceinline__ void init(const KvParams& kv) {
    const int lane = threadIdx.x & 31, which = lane & 3;
    run = min(1 << kv.page_shift, KEYS);
    offset = (lane >> 2) * run;
    active = offset < KEYS;
    const bool scales = which >= 2;
    base = which == 0 ? kv.k : which == 1 ? kv.v
                             : reinterpret_cast<const uint8_t*>(which == 2 ? kv.k_scale : kv.v_scale);
    page_stride = scales ? kv.scale_stride * 4 : kv.page_stride;
    row_bytes = scales ? 4 : T::kRow;
    dst = (which == 0 ? 0 : which == 1 ? T::kV : which == 2 ? T::kKs : T::kVs) + offset * row_bytes;
  }
  // page of this lane's run of the step at `key`, -1 when nobody sees it
  __device__ __forceinline__ int page(const KvParams& kv, int b, int key, const Sight& sight) const {
    const int k = key + offset;
    return active && k < sight.len && (k + run > sight.lo || k < sight.sinks) ? kv_page(kv, b, k) : -1;
  }
  __device__ __forceinline__ void issue(const KvParams& kv, int head, int key, int page, uint32_t stage, uint64_t* bar) const {
    const int lane = threadIdx.x & 31;
    const uint32_t runs = __popc(__ballot_sync(0xffffffffu, page >= 0)) >> 2;
    if (lane == 0) {
      if (runs) mbar_arrive_expect_tx(bar, runs * run * (2 * T::kRow + 8));
      else mbar_arrive(bar);
    }
    __syncwarp();
    if (page >= 0)
      bulk_load_at(stage + dst, base + page * page_stride + static_cast<long long>(kv_row_in_page(kv, head, key + offset)) * row_bytes,
                   run * row_bytes, bar);
  }
};

// Copies of one warp step of bf16 pages: lane l resolves key l's page, the lanes then copy the
// rows chunk by chunk. Keys that no row sees become zeros.
template <int D, int KEYS>
__device__ __forceinline__ void load_step(const AttnParams& p, int b, int head, int key, const Sight& sight, uint32_t dst) {
  typedef Tile<D, kKvBf16, KEYS> T;
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
    cp16(dst + T::chunk(r, c), p.kv.k + a, n);
    cp16(dst + T::kV + T::chunk(r, c), p.kv.v + a, n);
  }
}

// Where row r of a piece lives in q and out; r < rows.
__device__ __forceinline__ long long q_row(const AttnParams& p, int first, int head, int r) {
  const int token = first + r / p.group, hq = head * p.group + r % p.group;
  return static_cast<long long>(hq) * p.kv.M + token;
}

__device__ __forceinline__ long long lse_bytes(const AttnParams& p) { return static_cast<long long>(p.Hq) * p.kv.M * 4; }
__device__ __forceinline__ long long out_bytes(const AttnParams& p, int D) {
  return static_cast<long long>(p.Hq) * p.kv.M * (2 * D);
}

// N consecutive values of row r from d0 on, divided by the row's sum; the lane
// that holds d = 0 writes the log-sum-exp.
template <int D, int N>
__device__ __forceinline__ void store_row_part(const AttnParams& p, int first, int head, int r, int d0, const float (&v)[N],
                                               float top, float sum) {
  const int token = first + r / p.group, hq = head * p.group + r % p.group;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;   // (a sum that is NaN stays one)
  bf16* dst = p.out + (static_cast<long long>(token) * p.Hq + hq) * D + d0;
#pragma unroll
  for (int i = 0; i < N; i += 4)
    kv_store(p.kv, dst + i, make_uint2(pack_bf16x2(v[i] * inv, v[i + 1] * inv), pack_bf16x2(v[i + 2] * inv, v[i + 3] * inv)),
             p.out, out_bytes(p, D));
  if (d0 == 0 && p.lse)
    kv_store(p.kv, p.lse + static_cast<long long>(hq) * p.kv.M + token, sum != 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY,
             p.lse, lse_bytes(p));
}

template <int D, int FMT, int NR>
__global__ void __launch_bounds__(SplitCfg<D, FMT, NR>::THREADS, SplitCfg<D, FMT, NR>::BLOCKS)
    k8_attend_split(const __grid_constant__ AttnParams p) {
  typedef SplitCfg<D, FMT, NR> C;
  typedef typename C::Layout L;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int scan[C::WARPS];
  __shared__ int found[3];   // sequence of the first unit, tiles before it; whether this block arrived last
  __shared__ uint64_t full[C::WARPS][C::STAGES];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (C::BULK) {
    if (lane < C::STAGES) mbar_init(&full[warp][lane], 1);
    if (threadIdx.x == 0) abort_flag = 0;
    fence_mbar_init();
    __syncwarp();   // (the block's barriers below order the flag)
  }
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
  RowState<D, FMT, NR, C::KEYS> state;
  BulkLanes<D, C::KEYS> bulk;
  if (C::BULK) bulk.init(p.kv);
  uint32_t issued = 0, used = 0;   // steps of this warp so far (bulk form): slot and parity of each
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
    int page = -1;   // bulk form: this lane's page of the next step to copy
    auto withheld = [&](uint32_t n) { return p.stall != 0 && n == 0 && warp == 0 && blockIdx.x == 0; };   // of step n
    auto issue = [&](int i) {
      const uint32_t slot = issued % C::STAGES;
      if (!withheld(issued)) bulk.issue(p.kv, head, key_of(i), page, ring + slot * L::kBytes, &full[warp][slot]);
      ++issued;
      page = i + 1 < t1 ? bulk.page(p.kv, b, key_of(i + 1), sight) : -1;
    };
    if constexpr (C::BULK) {
      page = bulk.page(p.kv, b, key_of(t0), sight);
      for (int i = t0; i < min(t0 + C::STAGES, t1); ++i) issue(i);
    } else {
#pragma unroll
      for (int i = 0; i < C::STAGES - 1; ++i) {
        if (t0 + i < t1) load_step<D, C::KEYS>(p, b, head, key_of(t0 + i), sight, ring + i * L::kBytes);
        cp_commit();
      }
    }
    {
      const bf16* r[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const int row = n * 8 + (lane >> 2);
        r[n] = row < sight.rows ? p.q + q_row(p, st.first, head, row) * D : nullptr;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          state.pos[n][e] = st.pos0 + min(n * 8 + 2 * (lane & 3) + e, sight.rows - 1) / p.group;
      }
      state.load(r);
    }
    int slot = 0;
    bool ok = true;
    for (int i = t0; i < t1; ++i) {
      const int key = key_of(i);
      // a step none of whose keys is seen is skipped (behind the end, between sinks and window)
      const bool any = key < st.len && (key + C::KEYS > st.lo || key < p.sinks);
      if constexpr (C::BULK) {
        const uint32_t at = used % C::STAGES;
        ok = warp_wait(&full[warp][at], (used / C::STAGES) & 1, &abort_flag, p.kv.status, kStatusWaitFull, p.wait_ns);
        if (!ok) break;
        ++used;
        if (any) state.step(ring + at * L::kBytes, key, sight, p.scale_log2);
        __syncwarp();   // every lane has read the slot
        if (i + C::STAGES < t1) issue(i + C::STAGES);
      } else {
        const int nx = i + C::STAGES - 1;
        const int ns = slot == 0 ? C::STAGES - 1 : slot - 1;
        if (nx < t1) load_step<D, C::KEYS>(p, b, head, key_of(nx), sight, ring + ns * L::kBytes);
        cp_commit();
        cp_wait<C::STAGES - 1>();
        __syncwarp();
        if (any) state.step(ring + slot * L::kBytes, key, sight, p.scale_log2);
        __syncwarp();
        slot = slot == C::STAGES - 1 ? 0 : slot + 1;
      }
    }
    if (C::BULK) {
      if (!ok)   // this warp's copies in flight land before the ring is used for anything else
        for (; used != issued; ++used)
          if (!withheld(used)) drain_wait(&full[warp][used % C::STAGES], (used / C::STAGES) & 1);
    } else {
      cp_wait<0>();
    }
    // ---- the warps' rows together
    state.finish();
    __syncthreads();
    if (C::BULK && abort_flag) return;   // every copy has landed; check() reports the status
    float* mo = reinterpret_cast<float*>(smem);                      // [warp][row][D]
    float* mm = mo + C::WARPS * C::ROWS * D;                        // [warp][row] maximum, then sum
    float* ml = mm + C::WARPS * C::ROWS;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = n * 8 + 2 * (lane & 3) + e;
        float* w = mo + (warp * C::ROWS + row) * D;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          w[state.d_of(i, 0)] = state.o[i][n][e];
          w[state.d_of(i, 1)] = state.o[i][n][2 + e];
        }
        if (lane < 4) {
          mm[warp * C::ROWS + row] = state.m[n][e];
          ml[warp * C::ROWS + row] = state.l[n][e];
        }
      }
    __syncthreads();
    constexpr int PER = C::THREADS * 4 >= C::ROWS * D ? 4 : C::THREADS * 8 >= C::ROWS * D ? 8 : 16;
    static_assert(PER * C::THREADS >= C::ROWS * D && D % PER == 0, "values of a thread: 4, 8 or 16 of one row");
    const bool works = static_cast<int>(threadIdx.x) * PER < C::ROWS * D;
    const int row = works ? threadIdx.x * PER / D : 0, d0 = threadIdx.x * PER % D;
    float acc[PER], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) top = fmaxf(top, mm[w * C::ROWS + row]);
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      const float f = top == -INFINITY ? 0.f : ex2(mm[w * C::ROWS + row] - top);
      sum += f * ml[w * C::ROWS + row];
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = fmaf(f, mo[(w * C::ROWS + row) * D + d0 + e], acc[e]);
    }
    const bool whole = t0 == 0 && t1 == st.tiles;
    if (whole) {
      if (works && row < sight.rows) store_row_part<D, PER>(p, st.first, head, row, d0, acc, top, sum);
    } else {
      // partial sums: slot 2i + 1 for a head that begins in this block, 2i for one begun before
      const int c0 = unit_owner(s0, G, U), c1 = unit_owner(s1 - 1, G, U);
      float* mine = p.part + static_cast<long long>(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * kPartFloats;
      if (works) {
#pragma unroll
        for (int e = 0; e < PER; e += 4)
          kv_store_cg(p.kv, mine + row * D + d0 + e, make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]), mine,
                      kPartFloats * 4);
      }
      if (works && d0 == 0) {
        kv_store_cg(p.kv, mine + C::ROWS * D + row, top, mine, kPartFloats * 4);
        kv_store_cg(p.kv, mine + C::ROWS * D + C::ROWS + row, sum, mine, kPartFloats * 4);
      }
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) found[2] = atom_add_acq_rel_gpu(p.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
      __syncthreads();
      if (found[2]) {
        __threadfence();
        // four parts' loads at a time (a head over every block has dozens of parts)
        constexpr int AT_ONCE = 4;
        auto slot_of = [&](int c) { return p.part + static_cast<long long>(2 * c + (c == c0)) * kPartFloats; };
        top = -INFINITY;
        for (int c = c0; c <= c1; c += AT_ONCE) {
          float x[AT_ONCE];
#pragma unroll
          for (int k = 0; k < AT_ONCE; ++k) x[k] = __ldcg(slot_of(min(c + k, c1)) + C::ROWS * D + row);
#pragma unroll
          for (int k = 0; k < AT_ONCE; ++k) top = fmaxf(top, x[k]);
        }
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = 0.f;
        for (int c = c0; c <= c1; c += AT_ONCE) {
          float f[AT_ONCE], l[AT_ONCE];
          float4 x[AT_ONCE][PER / 4];
#pragma unroll
          for (int k = 0; k < AT_ONCE; ++k) {
            const float* s = slot_of(min(c + k, c1));
            f[k] = __ldcg(s + C::ROWS * D + row);
            l[k] = __ldcg(s + C::ROWS * D + C::ROWS + row);
#pragma unroll
            for (int e = 0; e < PER / 4; ++e) x[k][e] = __ldcg(reinterpret_cast<const float4*>(s + row * D + d0) + e);
          }
#pragma unroll
          for (int k = 0; k < AT_ONCE; ++k) {
            const float g = top == -INFINITY || c + k > c1 ? 0.f : ex2(f[k] - top);
            sum = fmaf(g, l[k], sum);
#pragma unroll
            for (int e = 0; e < PER / 4; ++e) {
              acc[4 * e] = fmaf(g, x[k][e].x, acc[4 * e]);
              acc[4 * e + 1] = fmaf(g, x[k][e].y, acc[4 * e + 1]);
              acc[4 * e + 2] = fmaf(g, x[k][e].z, acc[4 * e + 2]);
              acc[4 * e + 3] = fmaf(g, x[k][e].w, acc[4 * e + 3]);
            }
          }
        }
        if (works && row < sight.rows) store_row_part<D, PER>(p, st.first, head, row, d0, acc, top, sum);
        if (threadIdx.x == 0) p.counters[c0] = 0;
      }
    }
    if (C::BULK) fence_proxy_async_smem();   // the merge buffer's stores come before the next bulk copies
    __syncthreads();   // the merge buffer is the ring again
    u = before + static_cast<long long>(head) * st.tiles + t1;
  }
}

}  // namespace k8
}  // namespace fnl
