// K7: a batch's new keys and values into their pages, with the rotation of q
// and k by position on the way, and the read-back of a batch's rows.
//
// Rotation of the first `rot` values of a head by the token's angles (cos and
// sin from the caller's fp32 tables): (a, b) -> (a cos - b sin, b cos + a sin)
// for the pairs (i, i + rot / 2), or (2i, 2i + 1) in the interleaved order.
// Each product and each sum is rounded to fp32 by itself (no contraction), so
// the rounding to bf16 that follows, and the 4-bit codes taken from it, are the
// same wherever the formula is evaluated in fp32 this way.
//
// 4-bit pages: the row's minimum is exact in bf16 (its values are bf16), the
// scale is (max - min) / 15 rounded up to bf16, so 15 steps reach the maximum
// and every value is within half a scale of its code.
//
// HBM bound: every byte of q, k and v is read once and written once. A thread
// owns one 16-value piece (two 16-byte loads) of a token's heads and walks over
// the heads, so the 16 cos/sin values are loaded once per token and stay in
// registers; loads of kRows rows are issued before the first is used.
#pragma once

#include "kv_common.cuh"

namespace fnl {

constexpr int kKvThreads = 256;

struct AppendParams {
  KvParams kv;
  const bf16* q;
  const bf16* k;
  const bf16* v;
  bf16* q_out;
  const float* cos;   // [max_pos][rot / 2], null when rot == 0
  const float* sin;
  int Hq, rot, max_pos, tokens;   // tokens: tokens per block (a power of two)
};

// First elements of the two 8-value parts of piece c: for the half-split
// rotation the parts pair element by element, elsewhere they are neighbours.
template <bool INTERLEAVED>
__device__ __forceinline__ void piece_at(int c, int rot, int& e0, int& e1) {
  e0 = c * 16;
  e1 = e0 + 8;
  if (!INTERLEAVED && e0 < rot) {
    e0 = c * 8;
    e1 = e0 + (rot >> 1);
  }
}

// min and max of a row held by LANES neighbouring lanes
template <int LANES>
__device__ __forceinline__ void row_min_max(const float (&a)[8], const float (&b)[8], float& lo, float& hi) {
  lo = fminf(a[0], b[0]);
  hi = fmaxf(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, fminf(a[i], b[i]));
    hi = fmaxf(hi, fmaxf(a[i], b[i]));
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
}

// Codes round((x - lo) / s) of eight values, the first in the low nibble. The
// quotient's nearest integer comes from the product with 1 / s and is right wherever
// the remainder stays clear of half a step, which the remainder, exact in one fma,
// shows; else (ties and their neighbours) the quotient itself is rounded. Integers
// are taken from floats by adding 1.5 * 2^23, four codes at a time.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float lo, float s, float inv) {
  constexpr float kMagic = 12582912.f;
  if (!(s > 0.f)) return 0u;
  const float clear = s * 0.4999995f;
  float c[8];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __fsub_rn(x[i], lo);
    c[i] = __fsub_rn(fmaf(t, inv, kMagic), kMagic);
    near |= !(fabsf(fmaf(-c[i], s, t)) < clear);   // (also where a value or 1 / s is not finite)
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], lo), s)), 0.f), 15.f);
  }
  const float w0 = fmaf(fmaf(fmaf(c[3], 16.f, c[2]), 16.f, c[1]), 16.f, c[0]) + kMagic;
  const float w1 = fmaf(fmaf(fmaf(c[7], 16.f, c[6]), 16.f, c[5]), 16.f, c[4]) + kMagic;
  return __byte_perm(__float_as_uint(w0), __float_as_uint(w1), 0x5410);
}

// 4-bit pages: four resident blocks an SM, which hide more of the wait for loads (the first stall; issue slots 63 %
// used, DRAM 51 %) although the bound of 64 registers spills 28 bytes a thread (13 prompts appended and read back:
// 120 us with three, 115 with four; 88 + 24 us apart, their bytes 60 + 14). bf16 pages: the compiler's own choice of registers (0: no bound); held to three
// blocks, 12 sequences of 330 to 1000 tokens took 33 instead of 30 us.
template <int D, int FMT, bool INTERLEAVED>
__global__ void __launch_bounds__(kKvThreads, FMT == kKvInt4 ? 4 : 0) k7_append(const __grid_constant__ AppendParams p) {
  constexpr int LANES = D / 16;               // threads of one row
  constexpr int UNITS = kKvThreads / LANES;   // rows in flight per block
  // rows loaded before the first is used; coding makes the unrolled code of four too long for the
  // instruction cache (13 prompts appended to 4-bit pages and read back, three blocks an SM: 122 us with four, 120
  // with two). The q rows, which are not coded, go in the same loop.
  constexpr int kRows = FMT == kKvInt4 ? 2 : 4;
  pdl_wait();
  const int T = p.tokens;
  const int c = threadIdx.x % LANES, unit = threadIdx.x / LANES;
  const int m0 = blockIdx.x * T;
  const int m = m0 + unit % T;
  const int lane_head = unit / T, heads = UNITS / T;
  const int M = p.kv.M, Hkv = p.kv.Hkv;
  int b = kv_find_seq(p.kv, m0);
  while (b < p.kv.B && p.kv.cu_q[b + 1] <= m) ++b;
  bool live = b < p.kv.B && m < M;
  int pos = 0, page = -1;
  if (live) {
    const KvSeq s = kv_seq(p.kv, b);
    pos = s.len - s.n + (m - s.first);
    live = m >= s.first && m < s.first + s.n;
    if (live && (pos < 0 || (p.rot > 0 && pos >= p.max_pos))) {
      kv_flag(p.kv);
      live = false;
    }
    if (live) page = kv_page(p.kv, b, pos);
  }
  int e0, e1;
  piece_at<INTERLEAVED>(c, p.rot, e0, e1);
  const bool turn = c * 16 < p.rot;
  float cs[8], sn[8];
  if (turn && live) {
    const long long at = static_cast<long long>(pos) * (p.rot >> 1) + c * 8;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p.cos + at + i));
      const float4 y = __ldg(reinterpret_cast<const float4*>(p.sin + at + i));
      cs[i] = x.x; cs[i + 1] = x.y; cs[i + 2] = x.z; cs[i + 3] = x.w;
      sn[i] = y.x; sn[i + 1] = y.y; sn[i + 2] = y.z; sn[i + 3] = y.w;
    }
  }
  const int row_in_page = kv_row_in_page(p.kv, 0, pos);
  const int first = p.rot > 0 ? 0 : p.Hq;   // without a rotation q is not touched
  const int rows = p.Hq + 2 * Hkv;
  // the same number of turns for every lane of a warp (the 4-bit form shuffles)
  for (int r0 = first; r0 < rows; r0 += heads * kRows) {
    uint4 x0[kRows], x1[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + i * heads + lane_head;
      if (live && r < rows) {
        const bf16* src = r < p.Hq ? p.q + (static_cast<long long>(r) * M + m) * D
                          : r < p.Hq + Hkv ? p.k + (static_cast<long long>(r - p.Hq) * M + m) * D
                                           : p.v + (static_cast<long long>(r - p.Hq - Hkv) * M + m) * D;
        x0[i] = *reinterpret_cast<const uint4*>(src + e0);
        x1[i] = *reinterpret_cast<const uint4*>(src + e1);
      } else {
        x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + i * heads + lane_head;
      const bool is_v = r >= p.Hq + Hkv;
      if (turn && !is_v) {
        float a[8], d[8], ya[8], yd[8];
        unpack8(x0[i], a);
        unpack8(x1[i], d);
        if (INTERLEAVED) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ya[2 * j] = __fsub_rn(__fmul_rn(a[2 * j], cs[j]), __fmul_rn(a[2 * j + 1], sn[j]));
            ya[2 * j + 1] = __fadd_rn(__fmul_rn(a[2 * j + 1], cs[j]), __fmul_rn(a[2 * j], sn[j]));
            yd[2 * j] = __fsub_rn(__fmul_rn(d[2 * j], cs[4 + j]), __fmul_rn(d[2 * j + 1], sn[4 + j]));
            yd[2 * j + 1] = __fadd_rn(__fmul_rn(d[2 * j + 1], cs[4 + j]), __fmul_rn(d[2 * j], sn[4 + j]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ya[j] = __fsub_rn(__fmul_rn(a[j], cs[j]), __fmul_rn(d[j], sn[j]));
            yd[j] = __fadd_rn(__fmul_rn(d[j], cs[j]), __fmul_rn(a[j], sn[j]));
          }
        }
        x0[i] = pack8(ya);
        x1[i] = pack8(yd);
      }
      if (FMT == kKvInt4 && __any_sync(0xffffffffu, r >= p.Hq && r < rows)) {   // (q rows are not coded)
        float a[8], d[8], lo, hi;
        unpack8(x0[i], a);
        unpack8(x1[i], d);
        row_min_max<LANES>(a, d, lo, hi);
        // (max - min) / 15, rounded up to bf16: any bit below the upper half carries into it
        const float s = __uint_as_float((__float_as_uint(__fdiv_rn(__fsub_rn(hi, lo), 15.f)) + 0xFFFFu) & 0xFFFF0000u);
        const float inv = __fdiv_rn(1.f, s);
        if (live && page >= 0 && r >= p.Hq && r < rows) {
          const int h = is_v ? r - p.Hq - Hkv : r - p.Hq;
          const int row = (h << p.kv.page_shift) + row_in_page;
          const long long page_rows = static_cast<long long>(Hkv) << p.kv.page_shift;
          uint8_t* base = (is_v ? p.kv.v : p.kv.k) + page * p.kv.page_stride;
          uint8_t* dst = base + static_cast<long long>(row) * (D / 2);
          kv_store(p.kv, dst + (e0 >> 1), codes8(a, lo, s, inv), base, page_rows * (D / 2));
          kv_store(p.kv, dst + (e1 >> 1), codes8(d, lo, s, inv), base, page_rows * (D / 2));
          if (c == 0) {
            uint32_t* pairs = (is_v ? p.kv.v_scale : p.kv.k_scale) + page * p.kv.scale_stride;
            kv_store(p.kv, pairs + row, (__float_as_uint(s) >> 16) | (__float_as_uint(lo) & 0xFFFF0000u), pairs, page_rows * 4);
          }
        }
      }
      if (live && r < rows && (FMT == kKvBf16 || r < p.Hq)) {
        bf16* dst = nullptr;
        const void* base = p.q_out;
        long long size = static_cast<long long>(p.Hq) * M * (D * 2);
        if (r < p.Hq) {
          dst = p.q_out + (static_cast<long long>(r) * M + m) * D;
        } else if (page >= 0) {
          const int h = is_v ? r - p.Hq - Hkv : r - p.Hq;
          const int row = (h << p.kv.page_shift) + row_in_page;
          uint8_t* to = (is_v ? p.kv.v : p.kv.k) + page * p.kv.page_stride;
          dst = reinterpret_cast<bf16*>(to + static_cast<long long>(row) * (D * 2));
          base = to;
          size = (static_cast<long long>(Hkv) << p.kv.page_shift) * (D * 2);
        }
        if (dst) {
          kv_store(p.kv, dst + e0, x0[i], base, size);
          kv_store(p.kv, dst + e1, x1[i], base, size);
        }
      }
    }
  }
}

// Read-back: k_out and v_out [Hkv][M][D] bf16 of the batch's new tokens.
struct GatherParams {
  KvParams kv;
  bf16* k_out;
  bf16* v_out;
  int tokens;
};

template <int D, int FMT>
__global__ void __launch_bounds__(kKvThreads) k7_gather(const __grid_constant__ GatherParams p) {
  constexpr int LANES = D / 16;
  constexpr int UNITS = kKvThreads / LANES;
  pdl_wait();
  const int T = p.tokens;
  const int c = threadIdx.x % LANES, unit = threadIdx.x / LANES;
  const int m0 = blockIdx.x * T;
  const int m = m0 + unit % T;
  const int lane_head = unit / T, heads = UNITS / T;
  const int M = p.kv.M, Hkv = p.kv.Hkv;
  int b = kv_find_seq(p.kv, m0);
  while (b < p.kv.B && p.kv.cu_q[b + 1] <= m) ++b;
  if (b >= p.kv.B || m >= M) return;
  const KvSeq s = kv_seq(p.kv, b);
  const int pos = s.len - s.n + (m - s.first);
  if (m < s.first || m >= s.first + s.n || pos < 0) return;   // kv_seq has flagged it
  const int page = kv_page(p.kv, b, pos);
  if (page < 0) return;
  const int row_in_page = kv_row_in_page(p.kv, 0, pos);
#pragma unroll 4
  for (int r = lane_head; r < 2 * Hkv; r += heads) {
    const bool is_v = r >= Hkv;
    const int h = is_v ? r - Hkv : r;
    const int row = (h << p.kv.page_shift) + row_in_page;
    const uint8_t* src = (is_v ? p.kv.v : p.kv.k) + page * p.kv.page_stride;
    uint4 y0, y1;
    if (FMT == kKvBf16) {
      const uint4* x = reinterpret_cast<const uint4*>(src + static_cast<long long>(row) * (D * 2) + c * 32);
      y0 = x[0];
      y1 = x[1];
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(src + static_cast<long long>(row) * (D / 2) + c * 8);
      const uint32_t pair = (is_v ? p.kv.v_scale : p.kv.k_scale)[page * p.kv.scale_stride + row];
      const float sc = kv_scale_of(pair), lo = kv_min_of(pair);
      float f0[8], f1[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {   // code * scale is exact in fp32 (4 + 8 bits): one rounding
        f0[i] = fmaf(static_cast<float>((w.x >> (4 * i)) & 15u), sc, lo);
        f1[i] = fmaf(static_cast<float>((w.y >> (4 * i)) & 15u), sc, lo);
      }
      y0 = pack8(f0);
      y1 = pack8(f1);
    }
    bf16* out = is_v ? p.v_out : p.k_out;
    bf16* dst = out + (static_cast<long long>(h) * M + m) * D + c * 16;
    const long long size = static_cast<long long>(Hkv) * M * (D * 2);
    kv_store(p.kv, dst, y0, out, size);
    kv_store(p.kv, dst + 8, y1, out, size);
  }
}

}  // namespace fnl
