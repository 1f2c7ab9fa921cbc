// K9: attention of many new tokens over the paged cache on the tcgen05 tensor
// cores. The mathematics, the row order (token by token, the heads of a group
// side by side) and the masks are K8's.
//
// A block owns 256 rows of one sequence and key head as two tiles of 128 that
// take turns: while the tensor pipe works on one tile's products, the other
// tile's softmax runs. Per 128 keys and tile: S = Q K^T into TMEM (both operands
// from shared memory, fp32), one thread per row reads its 128 scores, writes the
// probabilities back over them as packed bf16, and O += P V with P read from
// TMEM as the A operand and V from shared memory as it was loaded (rows = keys,
// the transposed-B form), so neither S nor P touches shared memory. TMEM: two S
// tiles of 128 columns and two O tiles of D.
//
// Roles (12 warps): 0 copies K and V tiles by TMA, page by page, into a ring;
// 1 issues the products; 4-7 and 8-11 are the two tiles' softmax, which also
// fetch Q and write the result. A row's accumulators are rescaled only when its
// maximum has grown by more than 8 (a factor of 256) since the last time: the
// probabilities stay below 256, exact enough in bf16's and fp32's floating
// formats, and most key tiles need no pass over O.
//
// Tensor bound by design: a key tile costs 4 * 128 * 128 * D multiply-adds on the
// tensor pipe (2048 cycles at D = 128) against 2 * 128 * 128 exponentials on the
// special-function units (2048 cycles).
//
// Slots that no row of the block sees are not copied (whole pages) or are zeroed
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
// D[tmem] (+)= A[tmem] * B[smem desc]: A is bf16, two consecutive k packed in a
// 32-bit column, row = lane.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
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

namespace k9 {

constexpr int WARPS = 12;
constexpr int THREADS = WARPS * 32;
constexpr int TILE = 128;              // keys of a tile, rows of a sub-tile
constexpr int ROWS = 2 * TILE;
constexpr int REG_SOFTMAX = 208, REG_OTHER = 72;   // 256 * 208 + 128 * 72 <= 384 * 168, the launch's registers
constexpr uint32_t TMEM_COLS = 512;
constexpr float GROWTH = 8.f;          // rescale when the maximum (base 2) has grown by more

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = TILE * D * 2;   // Q sub-tile, K tile, V tile: HALVES blocks of 128 x 64
  static constexpr int HALF_BYTES = TILE * 128;
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr int SMEM = 2 * TILE_BYTES + STAGES * TILE_BYTES + 1024 + 256;
  static constexpr uint32_t S0 = 0, O0 = 256;       // TMEM columns: S at 0 and 128 (P over it), O at 256 and 256 + D
};

struct Ctrl {
  uint64_t full[8], empty[8], s_full[2], p_full[2], o_full[2], q_full, drain;
  uint32_t tmem_base;
  uint32_t armed, armed_parity;   // ring slots with a copy issued, and the parity of each one's last
  int abort_flag;
};

struct Params {
  AttnParams a;
  int stall;   // fault injection for the status-path tests: block 0 withholds its first key tile
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    k9_prompt(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ Params prm) {
  typedef Cfg<D> C;
  const AttnParams& p = prm.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * C::TILE_BYTES;
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(ring + C::STAGES * C::TILE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctrl->s_full[s], 1);
      mbar_init(&ctrl->p_full[s], 4);
      mbar_init(&ctrl->o_full[s], 1);
    }
    mbar_init(&ctrl->q_full, 8);
    mbar_init(&ctrl->drain, 1);
    ctrl->abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  const int b = blockIdx.z, head = blockIdx.y;
  const KvSeq seq = kv_seq(p.kv, b);
  const int rows = seq.n * p.group;
  const int r0 = (static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x)) * ROWS;   // the longest first
  if (r0 >= rows) return;
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  volatile int* abortf = &ctrl->abort_flag;
  int* status = p.kv.status;

  // ---- what the block's rows see
  const int pos_first = seq.len - seq.n;                     // position of the sequence's first new token
  k8::Sight sight;
  sight.pos0 = pos_first + r0 / p.group;
  sight.last = pos_first + (min(r0 + ROWS, rows) - 1) / p.group;
  sight.rows = rows;
  sight.group = p.group;
  sight.len = min(seq.len, sight.last + 1);
  sight.window = p.window;
  sight.sinks = p.sinks;
  sight.lo = p.window > 0 ? max(0, sight.pos0 - p.window + 1) : 0;
  const int lo_tile = sight.lo / TILE;
  const int sink_tiles = min((min(p.sinks, max(sight.len, 0)) + TILE - 1) / TILE, lo_tile);
  auto key_of = [&](int i) { return (i < sink_tiles ? i : lo_tile + i - sink_tiles) * TILE; };
  // key tiles of each sub-tile: the second one's rows reach further
  auto tiles_of = [&](int s) {
    const int first = r0 + s * TILE;
    if (first >= rows) return 0;
    const int end = min(seq.len, pos_first + (min(first + TILE, rows) - 1) / p.group + 1);
    return end > 0 ? sink_tiles + (end + TILE - 1) / TILE - lo_tile : 0;
  };
  const int n0 = tiles_of(0), n1 = tiles_of(1), n = max(n0, n1);

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_OTHER));
    const int page = 1 << p.kv.page_shift;
    const int bp = min(page, TILE);                          // keys of one copy
    const int copies = (TILE / bp) * C::HALVES;              // at most 16 lanes
    const int part = lane / C::HALVES, half = lane % C::HALVES;
    int slot = 0;
    uint32_t ph = 0, armed = 0, parity = 0;
    bool withhold = prm.stall != 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int key = key_of(i) + part * bp;
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
    uint32_t ph = 0;
    auto advance = [&]() {
      if (++slot == C::STAGES) {
        slot = 0;
        ph ^= 1u;
      }
    };
    auto qk = [&](int s, int at) {
      if (lane == 0) {
        const uint32_t q = smem_u32(smem) + s * C::TILE_BYTES, k = smem_u32(ring) + at * C::TILE_BYTES;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = (kk >> 2) * C::HALF_BYTES + (kk & 3) * 32;
          umma_bf16(tmem + C::S0 + s * TILE, sw128_desc(q + o), sw128_desc(k + o), idesc_qk, kk > 0);
        }
        umma_commit(&ctrl->s_full[s]);
      }
      __syncwarp();
    };
    auto pv = [&](int s, int at, bool first) {
      if (lane == 0) {
        const uint32_t v = smem_u32(ring) + at * C::TILE_BYTES;
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
          umma_bf16_ts(tmem + C::O0 + s * D, tmem + C::S0 + s * TILE + kk * 8, sw128_mn_desc(v + kk * 2048, C::HALF_BYTES),
                       idesc_pv, !first || kk > 0);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (lane == 0) umma_commit(bar);
      __syncwarp();
    };
    bool ok = n == 0 || (warp_wait(&ctrl->q_full, 0, abortf, status, kStatusWaitConv, p.wait_ns) &&
                         warp_wait(&ctrl->full[slot], ph, abortf, status, kStatusWaitFull, p.wait_ns));
    if (ok && n > 0) {
      tc_fence_after();
      if (n0 > 0) qk(0, slot);
      if (n1 > 0) qk(1, slot);
      commit(&ctrl->empty[slot]);
      advance();
    }
    for (int i = 0; i < n && ok; ++i) {
      // V of tile i at `slot`, K of tile i + 1 behind it
      const int vs = slot;
      ok = warp_wait(&ctrl->full[slot], ph, abortf, status, kStatusWaitFull, p.wait_ns);
      if (!ok) break;
      const int key = key_of(i);
      if (key + TILE > sight.len || (key < sight.lo && key + TILE > sight.sinks)) {
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
      const int ks = slot;
      bool have_k = false;
      for (int s = 0; s < 2 && ok; ++s) {
        const int ns = s ? n1 : n0;
        if (i < ns) {
          ok = warp_wait(&ctrl->p_full[s], i & 1, abortf, status, kStatusWaitConv, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          pv(s, vs, i == 0);
          if (i + 1 == ns) commit(&ctrl->o_full[s]);
        }
        if (s == 1) commit(&ctrl->empty[vs]);
        if (i + 1 < ns) {
          if (!have_k) {
            ok = warp_wait(&ctrl->full[ks], ph, abortf, status, kStatusWaitFull, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            have_k = true;
          }
          qk(s, ks);
        }
      }
      if (ok && i + 1 < n) {
        commit(&ctrl->empty[ks]);
        advance();
      }
    }
    if (!ok || *abortf) {   // every product issued is done before TMEM is freed
      commit(&ctrl->drain);
      if (lane == 0) k8::drain_wait(&ctrl->drain, 0);
      __syncwarp();
    }
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_OTHER));
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFTMAX));
    const int s = (warp - 4) >> 2, quarter = warp & 3;
    const int r = r0 + s * TILE + quarter * 32 + lane;       // this thread's row
    {   // Q: the 8 warps fetch 256 rows, 16 bytes a lane, into the swizzled tiles
      constexpr int CH = D / 8;
      const int t = threadIdx.x - 128;
#pragma unroll 4
      for (int idx = t; idx < ROWS * CH; idx += 256) {
        const int row = idx / CH, c = idx % CH;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r0 + row < rows) x = ldg16(p.q + k8::q_row(p, seq.first, head, r0 + row) * D + c * 8);
        st_shared_v4(smem_u32(smem) + (row / TILE) * C::TILE_BYTES + (c >> 3) * C::HALF_BYTES + (row % TILE) * 128 +
                         (((c & 7) ^ (row & 7)) << 4),
                     x);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->q_full);
    }
    const int ns = s ? n1 : n0;
    const int pos = pos_first + min(r, rows - 1) / p.group;
    // the warp's own span of positions, for its masks
    k8::Sight mine = sight;
    mine.pos0 = pos_first + min(r0 + s * TILE + quarter * 32, rows - 1) / p.group;
    mine.last = pos_first + min(r0 + s * TILE + quarter * 32 + 31, rows - 1) / p.group;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + C::S0 + s * TILE, to = tmem + lanes + C::O0 + s * D;
    const float scale = p.scale_log2;
    float top = -INFINITY;   // the maximum that the sum and the accumulators are relative to
    f32x2 sum2 = pk2(0.f, 0.f);
    bool ok = true;
    for (int i = 0; i < ns; ++i) {
      ok = warp_wait(&ctrl->s_full[s], i & 1, abortf, status, kStatusWaitTmemFull, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      uint32_t x[TILE];
#pragma unroll
      for (int c = 0; c < TILE; c += 32) tmem_ld32(ts + c, x + c);
      tmem_ld_wait();
      const int key = key_of(i);
      if (!mine.all(key, TILE)) {
        const int hi = pos - key, wlo = p.window > 0 ? hi - p.window + 1 : -(1 << 30), sk = p.sinks - key;
#pragma unroll
        for (int c = 0; c < TILE; ++c)
          if (!(c <= hi && (c >= wlo || c < sk))) x[c] = 0xff800000u;   // -inf
      }
      float m = -INFINITY;
#pragma unroll
      for (int c = 0; c < TILE; c += 2) m = fmaxf(m, fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
      m *= scale;
      if (__any_sync(0xffffffffu, m > top + GROWTH || (top == -INFINITY && m > top))) {
        const bool grow = m > top + GROWTH || top == -INFINITY;
        const float f = grow && top != -INFINITY ? k8::ex2(top - m) : 1.f;
        if (grow) top = m;
        float a, c;
        unpk2(sum2, a, c);
        sum2 = pk2(a * f, c * f);
        if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {   // (before the first product O holds nothing)
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
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const f32x2 t = fma2(pk2(__uint_as_float(x[h * 32 + 2 * c]), __uint_as_float(x[h * 32 + 2 * c + 1])), scale2, base2);
          float a, d;
          unpk2(t, a, d);
          a = k8::ex2(a);
          d = k8::ex2(d);
          sum2 = add2(sum2, pk2(a, d));
          w[c] = pack_bf16x2(a, d);
        }
        tmem_st16(ts + h * 16, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->p_full[s]);
    }
    // ---- the result
    float a, c;
    unpk2(sum2, a, c);
    const float sum = a + c;
    if (ok && ns > 0) {
      ok = warp_wait(&ctrl->o_full[s], 0, abortf, status, kStatusWaitTmemFull, p.wait_ns);
      tc_fence_after();
    }
    if (ok) {
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const int rr = min(r, rows - 1);
      const int token = seq.first + rr / p.group, hq = head * p.group + rr % p.group;
      bf16* dst = p.out + (static_cast<long long>(token) * p.Hq + hq) * D;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        if (ns > 0) {
          tmem_ld32(to + c0, o);
          tmem_ld_wait();
        }
        if (r < rows) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = sum > 0.f ? __uint_as_float(o[e + j]) * inv : 0.f;
            *reinterpret_cast<uint4*>(dst + c0 + e) = pack8(f);
          }
        }
      }
      if (r < rows && p.lse)
        p.lse[static_cast<long long>(hq) * p.kv.M + token] = sum > 0.f ? (top + log2f(sum)) * k8::kLn2 : -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
  if (warp == 0 && *abortf)   // after an abort nobody has waited for the copies in flight
    for (int s = 0; s < C::STAGES; ++s)
      if (ctrl->armed & (1u << s)) k8::drain_wait(&ctrl->full[s], (ctrl->armed_parity >> s) & 1);
}

}  // namespace k9
}  // namespace fnl
