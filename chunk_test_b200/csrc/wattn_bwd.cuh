// wattn_bwd.cuh -- the gradients of the window attention with sinks on the
// tensor cores (bf16).  Mask and formulas: wattn_common.cuh.
//
// With P = exp(scale q k - lse), D = rowsum(dout out), dS = P (dout V^T - D):
//   dQ = scale dS K        a CTA holds 128 queries and walks their key tiles
//   dK = scale dS^T Q      a CTA holds 128 keys and walks the queries that see
//   dV = P^T dout          them, over the group's heads
// One kernel, four modes: dQ, dK and dV in one (d <= 128), dK, dV (above).  Each
// gradient is accumulated by one CTA in TMEM, so there are no atomics and the
// order of every sum is fixed.  S and dout V^T are formed again for each mode: 7
// products up to d = 128 and 8 above, where 5 would do with all accumulators in
// TMEM beside S and dP; it has 512 columns.
//
// Resident operands A1 (Q or K) and A2 (dout or V), 128 rows; streamed tiles
// of 128 rows B1 (K or Q) and B2 (V or dout).  128, because a product of N = 64
// takes as long as one of N = 128: both read the same 4 KB of A per 16 channels
// (tiles of 64 rows measured 1589 us where 128 took 1035 at B 2, H 6, T 8192,
// d 256, window 2048).  Roles:
//   warp 0      TMA producer of A and B1.
//   warp 10     TMA producer of B2.
//   warp 1      issues S = A1 B1^T, dP = A2 B2^T and dX += dS B1 (dV: P B2),
//               dS in TMEM in bf16 over S.  One thread; the tensor pipe forms
//               dP(n+1), and S(n+1) where TMEM holds two (d <= 128, dV), while
//               dS(n) is computed.
//   warps 2-9   dS (dV: P): two threads per row, 64 columns each.
// Bound by latency: up to d = 128 by the elementwise work of a tile (16384
// exponentials, 1024 clocks, and as many differences and products), which the
// passes of 9 tiles repeat; at d = 256 by the chain S, dS, dX of one tile (about
// 5400 clocks for 3 x 1024 of products), for TMEM holds one S beside 256 columns of
// dX, and shared memory one B1.  Measured: B 2, H 6, T 8192, d 256, window 2048,
// 4 sinks: dQ 325 us, dK and dV 580 in a row of calls; B 2, 12 heads on 4, T 4001,
// d 128, window 1000, 8 sinks: 102 and 175.
#pragma once

#include "wattn_fwd.cuh"

namespace lact {

__device__ __forceinline__ float4 ld_shared_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

enum WattnMode { WATTN_DQ, WATTN_DK, WATTN_DV, WATTN_DKV };   // DKV: d <= 128

struct WattnBwdParams {
  CUtensorMap tmA1, tmA2;   // q, dout (dQ) or k, v (dK, dV), box {64, 128}
  CUtensorMap tmB1, tmB2;   // k, v (dQ) or q, dout (dK, dV), box {64, 128}
  CUtensorMap tmX64;        // B1 (dV: B2), box {64, 64}
  WattnParams a;
  int nitems, per_head;     // items in all, and per (batch, head of A)
  int sink_tiles, parts;    // dK, dV: the split of the sink tiles (KeyPart)
};

// An item: 128 rows of A and the tiles of 128 rows of B that it walks.
template <int MODE>
struct BwdItem {
  int b, ha, a0;            // batch, head and first row of A
  int pos;                  // position of A's first row
  int len, count;           // the sequence's length, tiles of B
  int hb0, per, lo, hi;     // dK, dV: first head of B, tiles per head, query positions [lo, hi)
  int sink_tiles, first;    // dQ: tiles of 128 keys of the sinks, first of the window's
  int kt, part;
  __device__ __forceinline__ BwdItem(const WattnBwdParams& q, int item) {
    const WattnParams& p = q.a;
    if (MODE == WATTN_DQ) {
      const TileAt at = query_tile_at(p, q.per_head, item);
      b = at.b;
      ha = at.h;
      hb0 = ha / p.group;
      a0 = at.m * 128;
      pos = a0 + p.T - p.Tq;
      len = seq_len(p, b);
      const int last = min(min(pos + 128, p.T), len) - 1;
      first = max(0, pos - p.window + 1) >> 7;
      sink_tiles = min((p.sinks + 127) >> 7, first);
      count = pos < len ? sink_tiles + (last >> 7) - first + 1 : 0;
    } else {
      // all key heads at one tile together, the last tiles, which fewer queries see, last
      const int heads = p.B * p.Hkv, x = item / heads;
      b = item % heads / p.Hkv;
      ha = item % p.Hkv;
      hb0 = ha * p.group;
      const int split = q.sink_tiles * q.parts;
      kt = x < split ? x / q.parts : x - split + q.sink_tiles;
      part = x < split ? x % q.parts : 0;
      a0 = pos = kt * 128;
      len = seq_len(p, b);
      const KeyPart kp = key_part(kt, part, 128, p.window, p.T, p.far_rows);
      lo = max(kp.lo, p.T - p.Tq);
      hi = min(kp.hi, len);
      per = hi > lo ? (hi - lo + 127) >> 7 : 0;
      count = per * p.group;
    }
  }
  __device__ __forceinline__ int head(int n) const { return MODE == WATTN_DQ ? hb0 : hb0 + n / per; }
  // the position of B's first row
  __device__ __forceinline__ int at(int n) const {
    if (MODE == WATTN_DQ) return (n < sink_tiles ? n : first + n - sink_tiles) << 7;
    return lo + (n % per) * 128;
  }
};

template <int D, int MODE>
struct BwdCfg {
  static constexpr int kKb = D / 64;
  static constexpr bool kDv = MODE == WATTN_DV;
  static constexpr bool kBoth = MODE == WATTN_DKV;
  static_assert(!kBoth || D <= 128, "both accumulators beside S and dP");
  static constexpr int kSB = kDv || (D <= 128 && !kBoth) ? 2 : 1;      // buffers of S (and of dS or P, which go over it)
  static constexpr int kCol = kDv ? 128 : MODE != WATTN_DQ ? 256 : 0;   // lse and delta of a tile's columns
  static constexpr int kABytes = kKb * 16384;
  static constexpr int kAll = kDv ? kABytes : 2 * kABytes;
  // two sets of resident operands where they fit: the next item's first tile is
  // begun under this item's last
  static constexpr int kRA = D == 64 ? 2 : 1;
  static constexpr int kTile = kKb * 16384;                // a B tile of 128 rows
  // The operand of the last product (B1; dV: B2) stays until that product is
  // done: whole tiles.  The other one is K-major only and goes by blocks of 64
  // channels (DKV: it is an operand of dV too, and its blocks stay as well).
  static constexpr int kBlocks = (230400 - kSB * kCol * 4 - kRA * kAll) / 16384;  // 16 KB blocks there is room for
  static constexpr int kRx = kBlocks >= 3 * kKb + 2 ? 3 : kBlocks >= 2 * kKb + 2 ? 2 : 1;
  // a single X slot is refilled by halves of 64 rows: the product that reads it
  // is done with the first half before the second
  static constexpr int kHx = kRx == 1 ? 2 : 1;
  static constexpr int kRy0 = kBlocks - kRx * kKb, kRy = kRy0 > 2 * kKb ? 2 * kKb : kRy0;
  static_assert(kRy >= 2 && (!kBoth || kRy == 2 * kKb), "room for two blocks (DKV: tiles)");
  static constexpr int kOffX = kRA * kAll, kOffY = kOffX + kRx * kTile, kOffCol = kOffY + kRy * 16384;
  static constexpr int kOffBar = kOffCol + kSB * kCol * 4;
  // afull[RA] aempty[RA] | xfull[] xempty[] | yfull[] yempty[] | sfull[SB] pfull[SB] dfull dread cfull | gfull gempty
  static constexpr int kBars = 2 * kRA + kRx + kRx * kHx + 2 * kRy + 2 * kSB + 3 + 2;
  static constexpr int kSmem = kOffBar + kBars * 8 + 16 + 1024;
  static constexpr int kThreads = 352;
  // columns: the accumulator (DKV: dK), DKV's dV, S, dP (dV has none)
  static constexpr uint32_t kColX = 0, kColV = 128, kColS = 256, kColD = kSB == 2 ? 128 : 384;
};

template <int D, int MODE>
__global__ void __launch_bounds__(352, 1) k_wattn_bwd(const __grid_constant__ WattnBwdParams p) {
  using C = BwdCfg<D, MODE>;
  constexpr int RX = C::kRx, RY = C::kRy, KB = C::kKb, SB = C::kSB, RA = C::kRA, HX = C::kHx;
  constexpr bool DV = C::kDv, BOTH = C::kBoth;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t *afull = bar, *aempty = afull + RA, *xfull = aempty + RA, *xempty = xfull + RX, *yfull = xempty + RX * HX,
           *yempty = yfull + RY, *sfull = yempty + RY, *pfull = sfull + SB, *dfull = pfull + SB,
           *dread = dfull + 1, *cfull = dread + 1, *gfull = cfull + 1, *gempty = gfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + C::kBars);

  griddep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (__syncthreads_or(*reinterpret_cast<volatile int*>(&g_status))) return;   // an earlier wait gave up
  if (threadIdx.x == 0) {
    for (int i = 0; i < RA; ++i) {
      mbar_init(&afull[i], 1);
      mbar_init(&aempty[i], 1);
    }
    for (int i = 0; i < RX; ++i) {
      mbar_init(&xfull[i], 1);
      for (int k = 0; k < HX; ++k) mbar_init(&xempty[i * HX + k], 1);
    }
    for (int i = 0; i < RY; ++i) {
      mbar_init(&yfull[i], 1);
      mbar_init(&yempty[i], 1);
    }
    for (int i = 0; i < SB; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 8);
    }
    mbar_init(dfull, 1);
    mbar_init(dread, 8);
    mbar_init(cfull, 8);
    mbar_init(gfull, 1);
    mbar_init(gempty, 8);
    fence_barrier_init();
    tma_prefetch_map(&p.tmA1);
    tma_prefetch_map(&p.tmA2);
    tma_prefetch_map(&p.tmB1);
    tma_prefetch_map(&p.tmB2);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync_converged();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  const int off = p.a.T - p.a.Tq;                     // position of query row 0

  if (warp == 0 || warp == 10) {
    // ---------------------------------------------------------- producers
    // X: the operand of the last product, whole tiles; Y: the other one, by blocks
    if (lane == 0) {
      const bool x = warp == 0;
      // X by boxes of 128 / HX rows, Y of 128
      const CUtensorMap* map = x ? (HX == 2 ? &p.tmX64 : DV ? &p.tmB2 : &p.tmB1) : DV ? &p.tmB1 : &p.tmB2;
      int ib = 0, ic = 0;
      bool ok = true;
      for (int item = blockIdx.x; ok && item < p.nitems; item += gridDim.x) {
        const BwdItem<MODE> t(p, item);
        if (t.count == 0) continue;
        if (x) {
          const int s = ic % RA;
          if (ic >= RA && !mbar_wait(&aempty[s], ((ic / RA) - 1) & 1)) break;
          ++ic;
          mbar_arrive_expect_tx(&afull[s], C::kAll);
          for (int kb = 0; kb < KB; ++kb) {
            uint8_t* dst = smem + s * C::kAll + kb * 16384;
            tma_load_4d(dst, &p.tmA1, &afull[s], kb * 64, t.a0, t.ha, t.b);
            if (!DV) tma_load_4d(dst + C::kABytes, &p.tmA2, &afull[s], kb * 64, t.a0, t.ha, t.b);
          }
        }
        for (int n = 0; ok && n < t.count; ++n) {
          const int row = t.at(n) - (MODE == WATTN_DQ ? 0 : off), hb = t.head(n);
          if (x) {
            const int s = ib % RX;
            for (int k = 0; ok && k < HX; ++k) {
              if (ib >= RX && !mbar_wait(&xempty[s * HX + k], ((ib / RX) - 1) & 1)) { ok = false; break; }
              if (k == 0) mbar_arrive_expect_tx(&xfull[s], C::kTile);
              for (int kb = 0; kb < KB; ++kb)
                tma_load_4d(smem + C::kOffX + s * C::kTile + kb * 16384 + k * 8192, map, &xfull[s], kb * 64,
                            row + k * 64, hb, t.b);
            }
            ++ib;
          } else {
            for (int kb = 0; kb < KB; ++kb, ++ib) {
              const int s = ib % RY;
              if (ib >= RY && !mbar_wait(&yempty[s], ((ib / RY) - 1) & 1)) { ok = false; break; }
              mbar_arrive_expect_tx(&yfull[s], 16384);
              tma_load_4d(smem + C::kOffY + s * 16384, map, &yfull[s], kb * 64, row, hb, t.b);
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- products
    if (lane == 0) {
      constexpr uint32_t ids = idesc_bf16(128, 128, false, false), idx = idesc_bf16(128, D, false, true);
      const uint32_t sbase = smem_u32(smem);
      const uint64_t a1 = smem_desc_sw128(sbase, 16u, 1024u), a2 = smem_desc_sw128(sbase + C::kABytes, 16u, 1024u),
                     xk = smem_desc_sw128(sbase + C::kOffX, 16u, 1024u),
                     xm = smem_desc_sw128(sbase + C::kOffX, 16384u, 1024u),
                     yk = smem_desc_sw128(sbase + C::kOffY, 16u, 1024u),
                     ym = smem_desc_sw128(sbase + C::kOffY, 16384u, 1024u);
      int iy = 0;
      // S of tile h in all, with the tile X(h) (dV: with Y)
      auto with_x = [&](int h, int abuf) -> bool {
        const int x = h % RX;
        if (!mbar_wait(&xfull[x], (h / RX) & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(tmem + C::kColS + (h % SB) * 128, desc_at(a1, abuf * C::kAll + kb * 16384 + k * 32),
                      desc_at(xk, x * C::kTile + kb * 16384 + k * 32), ids, (kb | k) ? 1u : 0u);
        umma_commit(&sfull[h % SB]);
        return true;
      };
      // a resident operand with the next tile of Y, by blocks
      auto with_y = [&](uint32_t d, uint64_t a, int abuf, int from, int to) -> bool {
        for (int kb = from; kb < to; ++kb, ++iy) {
          const int s = iy % RY;
          if (!mbar_wait(&yfull[s], (iy / RY) & 1)) return false;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(d, desc_at(a, abuf * C::kAll + kb * 16384 + k * 32), desc_at(yk, s * 16384 + k * 32), ids,
                      (kb | k) ? 1u : 0u);
          if (!BOTH) umma_commit(&yempty[s]);
        }
        return true;
      };
      // The tile whose S (and dP) is next: `ahead` of the one whose dX is, by one
      // tile, over the items' ends too where there are two sets of A.
      int nt = blockIdx.x, nn = 0, ncount = 0, ia = 0, h = 0;
      auto settle = [&]() {
        while (nt < p.nitems && (ncount = BwdItem<MODE>(p, nt).count) == 0) nt += gridDim.x;
      };
      // dP (and S, where TMEM holds two) of the next tile, dP as far as Y's ring goes
      constexpr int KD = DV || SB == 2 || RY >= KB ? KB : RY;
      auto next_d = [&]() -> bool {
        if (nn == 0 && !mbar_wait(&afull[ia % RA], (ia / RA) & 1)) return false;
        if constexpr (DV) {
          if (!with_y(tmem + C::kColS + (h % SB) * 128, a1, ia % RA, 0, KB)) return false;
          umma_commit(&sfull[h % SB]);
        } else {
          if (SB == 2 && !with_x(h, ia % RA)) return false;
          if (h > 0 && !mbar_wait(dread, (h - 1) & 1)) return false;   // the last dP has been read
          if (!with_y(tmem + C::kColD, a2, ia % RA, 0, KD)) return false;
          if (KD == KB) umma_commit(dfull);
        }
        return true;
      };
      // The blocks of dP that the ring did not hold: they come while dX of the last
      // tile is formed and X is refilled, instead of holding that dX up (dQ at d 256:
      // 327 us, 306 with them so).
      auto rest_of_d = [&]() -> bool {
        if (KD < KB) {
          if (!with_y(tmem + C::kColD, a2, ia % RA, KD, KB)) return false;
          umma_commit(dfull);
        }
        return true;
      };
      auto next_done = [&]() {
        if (nn + 1 == ncount) {
          umma_commit(&aempty[ia % RA]);
          ++ia;
          nn = 0;
          nt += gridDim.x;
          settle();
        } else {
          ++nn;
        }
        ++h;
      };
      settle();
      int g = 0, items = 0;                           // tiles, items with an accumulator
      bool ok = true, begun = false;
      for (int item = blockIdx.x; ok && item < p.nitems; item += gridDim.x) {
        const BwdItem<MODE> t(p, item);
        if (t.count == 0) continue;
        for (int n = 0; ok && n < t.count; ++n, ++g) {
          // tile g itself, as far as it could not be begun under the last one
          if (!begun && !next_d()) { ok = false; break; }
          if (SB == 1 && (!rest_of_d() || !with_x(g, ia % RA))) { ok = false; break; }
          if (SB == 1 || !begun) next_done();
          // the next one, where its resident operands can be there
          begun = nt < p.nitems && (RA == 2 || nn > 0);
          if (begun) {
            if (!next_d()) { ok = false; break; }
            if (SB == 2) next_done();
          }
          const int s = g % RX;
          if (n == 0 && items > 0 && !mbar_wait(gempty, (items - 1) & 1)) { ok = false; break; }
          if (DV && !mbar_wait(&xfull[s], (g / RX) & 1)) { ok = false; break; }
          if (!mbar_wait(&pfull[g % SB], (g / SB) & 1)) { ok = false; break; }
          const uint32_t pa = tmem + C::kColS + (g % SB) * 128;
          tc_fence_after();
#pragma unroll
          for (int k = 0; BOTH && k < 8; ++k)   // P: columns 0..15 of each 32, dS: 16..31
            umma_bf16_ta(tmem + C::kColV, pa + (k >> 1) * 32 + (k & 1) * 8,
                         desc_at(ym, (g % (RY / KB)) * C::kTile + k * 2048), idx, (n == 0 && k == 0) ? 0u : 1u);
          if (BOTH)
            for (int kb = 0; kb < KB; ++kb) umma_commit(&yempty[(g % (RY / KB)) * KB + kb]);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            umma_bf16_ta(tmem + C::kColX, pa + (BOTH ? (k >> 1) * 32 + 16 + (k & 1) * 8 : (k >> 2) * 64 + (k & 3) * 8),
                         desc_at(xm, s * C::kTile + k * 2048), idx, (n == 0 && k == 0) ? 0u : 1u);
            if (k % (8 / HX) == 8 / HX - 1) umma_commit(&xempty[s * HX + k / (8 / HX)]);
          }
          if (n + 1 == t.count) umma_commit(gfull);
        }
        ++items;
      }
    }
  } else {
    // ---------------------------------------------------------- elementwise
    const int half = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t td = tq + C::kColD + half * 64;
    const float c2 = p.a.scale * 1.4426950408889634f;
    const int window = p.a.window, sinks = p.a.sinks;
    // -lse (log2) [128] and -delta [128] of a tile's columns, as many as there are S buffers
    float* cols = reinterpret_cast<float*>(smem + C::kOffCol);
    const int mycol = threadIdx.x - 64;                          // 0..255
    int g = 0, ic = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < p.nitems; item += gridDim.x) {
      const BwdItem<MODE> t(p, item);
      const int mine = t.pos + r;                     // this row's position
      float rl = 0.f, rd = 0.f;                       // -lse (log2), -delta
      if (MODE == WATTN_DQ && mine < t.len && t.a0 + r < p.a.Tq) {
        const int64_t at = (static_cast<int64_t>(t.b) * p.a.H + t.ha) * p.a.Tq + t.a0 + r;
        rl = p.a.lse[at] * -1.4426950408889634f;
        rd = -p.a.delta[at];
      }
      for (int n = 0; n < t.count; ++n, ++g) {
        const int t0 = t.at(n), b0 = t0 + half * 64;  // positions of the tile's and of this half's first column
        const uint32_t ts = tq + C::kColS + (g % SB) * 128 + half * 64;
        const uint32_t col_s = smem_u32(cols) + (g % SB) * C::kCol * 4 + half * 256;
        float x = 0.f;
        if (MODE != WATTN_DQ) {
          // the columns' statistics: one value per thread
          const int i = t0 + (mycol & 127);
          if (i < t.hi && (!DV || mycol < 128)) {
            const int64_t at = (static_cast<int64_t>(t.b) * p.a.H + t.head(n)) * p.a.Tq + i - off;
            x = mycol < 128 ? p.a.lse[at] * -1.4426950408889634f : -p.a.delta[at];
          }
        }
        float dp[64];
        if (!DV) {
          // dP first, so that its buffer is free while dS is computed
          if (!mbar_wait_warp(dfull, g & 1)) { ok = false; break; }
          tc_fence_after();
          tmem_ld32(td, dp);
          tmem_ld32(td + 32, dp + 32);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dread);
        }
        if (!mbar_wait_warp(&sfull[g % SB], (g / SB) & 1)) { ok = false; break; }
        if (MODE != WATTN_DQ) {
          // S came after the last dS from this buffer, so its statistics have been read
          if (mycol < C::kCol) cols[(g % SB) * C::kCol + mycol] = x;
          __syncwarp();
          if (lane == 0) mbar_arrive(cfull);
        }
        // the last product's rows behind the sequence: a dS of 0 times whatever is there must stay 0
        if (t.len < t0 + 128) {
          const int s = g % RX, keep = max(t.len - t0, 0);
          if (!mbar_wait_warp(&xfull[s], (g / RX) & 1)) { ok = false; break; }
          const uint32_t xb = smem_u32(smem) + C::kOffX + s * C::kTile;
          for (int e = keep * 8 + mycol; e < 1024; e += 256)
            for (int kb = 0; kb < KB; ++kb) {
              st_shared_v4(xb + kb * 16384 + e * 16, 0, 0, 0, 0);
              if (BOTH)   // Y's blocks are there: dP has been formed from them
                st_shared_v4(smem_u32(smem) + C::kOffY + (g % (RY / KB)) * C::kTile + kb * 16384 + e * 16, 0, 0, 0, 0);
            }
          fence_async_smem();
        }
        if (MODE != WATTN_DQ && !mbar_wait_warp(cfull, g & 1)) { ok = false; break; }
        tc_fence_after();
        bool whole;
        int clo, chi, csk;                            // columns c with clo < c <= chi, or c <= chi below csk
        if (MODE == WATTN_DQ) {
          whole = b0 + 63 <= t.pos && (b0 > t.pos + 127 - window || b0 + 63 < sinks) && t.pos + 127 < t.len;
          chi = mine < t.len ? mine - b0 : -1;
          clo = mine - window - b0;
          csk = sinks - b0;                           // columns below it are sinks
        } else {
          whole = b0 >= t.pos + 127 && (b0 + 63 - window < t.pos || t.pos + 127 < sinks) && b0 + 63 < t.hi;
          // query column c sees this key when it is at or past it and in its window, or anywhere for a sink
          const int top = mine < sinks ? t.hi - 1 : min(t.hi - 1, mine + window - 1);
          chi = top - b0;
          clo = mine - 1 - b0;
          csk = 0;
        }
        // a warp none of whose rows sees a column: a sink tile's other keys, or beside the diagonal
        const bool none = !whole && __all_sync(0xffffffffu, chi < 0 || ((clo >= 63 || chi <= clo) && csk <= 0));
        uint32_t hw[32];
        if (none) {
#pragma unroll
          for (int c = 0; c < 32; ++c) hw[c] = 0;
          if (BOTH) {
            tmem_st16u(ts, hw);
            tmem_st16u(ts + 16, hw);
            tmem_st16u(ts + 32, hw);
            tmem_st16u(ts + 48, hw);
          }
        } else {
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 32) {
            float s[32];
            tmem_ld32(ts + c0, s);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              float4 l4 = make_float4(rl, rl, rl, rl), d4 = make_float4(rd, rd, rd, rd);
              if (MODE != WATTN_DQ) {
                l4 = ld_shared_v4(col_s + (c0 + c) * 4);
                if (!DV)
                  d4 = ld_shared_v4(col_s + 512 + (c0 + c) * 4);
              }
              const float2 ll[2] = {make_float2(l4.x, l4.y), make_float2(l4.z, l4.w)};
              const float2 dd[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                float2 e = fma_f32x2(make_float2(s[c + k], s[c + k + 1]), make_float2(c2, c2), ll[k / 2]);
                e.x = ex2_approx(e.x);
                e.y = ex2_approx(e.y);
                const int d = c0 + c + k;
                if (BOTH) {
                  s[c + k] = e.x;
                  s[c + k + 1] = e.y;
                }
                if (!DV) e = mul_f32x2(e, add_f32x2(make_float2(dp[d], dp[d + 1]), dd[k / 2]));
                (BOTH ? dp[d] : s[c + k]) = e.x;
                (BOTH ? dp[d + 1] : s[c + k + 1]) = e.y;
              }
            }
            if (!whole) {
              const uint32_t see = visible_bits(clo, chi, csk, c0);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(see >> c & 1)) {
                  s[c] = 0.f;
                  if (BOTH) dp[c0 + c] = 0.f;
                }
            }
            // the last product's operand: half a step, 2^-8 of each
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              hw[(BOTH ? 0 : c0 / 2) + c] = pack_bf16x2(s[2 * c], s[2 * c + 1]);
              if (BOTH) hw[16 + c] = pack_bf16x2(dp[c0 + 2 * c], dp[c0 + 2 * c + 1]);
            }
            if (BOTH) {   // P and dS over the 32 columns that this thread has read
              tmem_st16u(ts + c0, hw);
              tmem_st16u(ts + c0 + 16, hw + 16);
            }
          }
        }
        // over the first half of the 64 columns that this thread has read
        if (!BOTH) {
          tmem_st16u(ts, hw);
          tmem_st16u(ts + 16, hw + 16);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[g % SB]);
      }
      if (!ok) break;
      // the gradient's rows: this half of the channels (DKV: the first half dK, the second dV)
      if (t.count > 0) {
        if (!mbar_wait_warp(gfull, ic & 1)) break;
        ++ic;
        tc_fence_after();
      }
      const bool is_v = DV || (BOTH && half == 1);
      const float mul = is_v ? 1.0f : p.a.scale;
      const int row = t.a0 + r;
      const bool in = row < (MODE == WATTN_DQ ? p.a.Tq : p.a.T);
      const bool zero = t.count == 0 || (MODE == WATTN_DQ && mine >= t.len);
      const View4& o = MODE == WATTN_DQ ? p.a.dq : is_v ? p.a.dv : p.a.dk;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(o.p) + t.b * o.sb + t.ha * o.sh + static_cast<int64_t>(row) * o.st;
      const bool partial = MODE != WATTN_DQ && t.kt < p.sink_tiles;
      float* pd = nullptr;
      if (partial)
        pd = p.a.part + ((((static_cast<int64_t>(t.b) * p.a.Hkv + t.ha) * p.sink_tiles + t.kt) * p.parts + t.part) * 2 +
                         (is_v ? 1 : 0)) * (128 * D) + r * D;
#pragma unroll 1
      for (int c0 = BOTH ? 0 : half * (D / 2); c0 < (BOTH ? D : (half + 1) * (D / 2)); c0 += 32) {
        float x[32];
        if (t.count > 0) {
          __syncwarp();
          tmem_ld32(tq + (BOTH && is_v ? C::kColV : C::kColX) + c0, x);
          tmem_ld_wait();
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = zero ? 0.f : x[c] * mul;
        if (partial) {
#pragma unroll
          for (int c = 0; c < 32; c += 4) *reinterpret_cast<float4*>(pd + c0 + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
        } else if (in) {
#pragma unroll
          for (int c = 0; c < 32; c += 8)
            if (c0 + c < p.a.d)
              st_global_v4(dst + c0 + c, pack_bf16x2(x[c], x[c + 1]), pack_bf16x2(x[c + 2], x[c + 3]),
                           pack_bf16x2(x[c + 4], x[c + 5]), pack_bf16x2(x[c + 6], x[c + 7]));
        }
      }
      if (t.count > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(gempty);
      }
    }
  }
  tc_fence_before();
  cta_sync_converged();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace lact
