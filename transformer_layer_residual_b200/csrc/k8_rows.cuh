#pragma once
#include "k8_attend.cuh"
namespace fnl {
namespace k8 {
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Layout of one warp step (split form) or one block tile (rows form) of KEYS
// keys in shared memory.
template <int D, int FMT, int KEYS>
struct RowsTile {
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
    typedef RowsTile<D, FMT, KEYS> T;
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

// ---------------------------------------------------------------- rows form
template <int D, int FMT>
struct RowsCfg {
  static constexpr int WARPS = 8;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ROWS = WARPS * 16;
  static constexpr int NT = 4;
  static constexpr int TILE = 64;          // keys of a block tile
  static constexpr int STAGES = 2;
  typedef RowsTile<D, FMT, TILE> Layout;
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
