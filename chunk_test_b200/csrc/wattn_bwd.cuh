// wattn_bwd.cuh -- the gradients of the window attention with sinks on the
// tensor cores (bf16).  Mask and formulas: wattn_common.cuh.
//
// With P = exp(scale q k - lse), D = rowsum(dout out), dS = P (dout V^T - D):
//   dQ = scale dS K        a CTA holds 128 queries and walks their key tiles
//   dK = scale dS^T Q      a CTA holds 128 keys and walks the queries that see
//   dV = P^T dout          them, over the group's heads
// One kernel, three modes; each gradient is accumulated by one CTA in TMEM, so
// there are no atomics and the order of every sum is fixed.  S (and dout V^T)
// are formed again for each of the three: 8 products where 5 would do with
// 512 + 256 columns of accumulators at d = 256, and TMEM has 512.
//
// Resident operands A1 (Q or K) and A2 (dout or V), 128 rows; streamed tiles
// of 64 rows B1 (K or Q) and B2 (V or dout).  64 rows, because with A1 and A2
// (128 KB at d = 256) only 96 KB are left for the stream.  Roles:
//   warp 0     TMA producer.
//   warp 1     issues S = A1 B1^T, dP = A2 B2^T into one of two TMEM buffers,
//              and dX += dS B1 (dV: P B2) with dS in TMEM in bf16.
//   warps 2-9  two groups of four, one per buffer; a thread owns one row.
// Bound by the tensor pipe: an M 128, N 64 product reads 6 KB of shared memory
// for 32 clocks of products and takes 48.
#pragma once

#include "wattn_fwd.cuh"

namespace lact {

enum WattnMode { WATTN_DQ, WATTN_DK, WATTN_DV };

struct WattnBwdParams {
  CUtensorMap tmA1, tmA2;   // box {64, 128}: q, dout (dQ) or k, v (dK, dV)
  CUtensorMap tmB1, tmB2;   // box {64, 64}: k, v (dQ) or q, dout (dK, dV)
  WattnParams a;
  int nitems, per_head;     // items in all, and per (batch, head of A)
  int sink_tiles, parts;    // dK, dV: the split of the sink tiles (KeyPart)
};

// An item: 128 rows of A and the tiles of 64 rows of B that it walks.
template <int MODE>
struct BwdItem {
  int b, ha, a0;            // batch, head and first row of A
  int pos;                  // position of A's first row
  int len, count;           // the sequence's length, tiles of B
  int hb0, per, lo, hi;     // dK, dV: first head of B, tiles per head, query positions [lo, hi)
  int sink_tiles, first;    // dQ: tiles of 64 keys of the sinks, first of the window's
  int kt, part;
  __device__ __forceinline__ BwdItem(const WattnBwdParams& q, int item) {
    const WattnParams& p = q.a;
    const int x = item % q.per_head, ba = item / q.per_head;
    if (MODE == WATTN_DQ) {
      b = ba / p.H;
      ha = ba % p.H;
      hb0 = ha / p.group;
      a0 = x * 128;
      pos = a0 + p.T - p.Tq;
      len = seq_len(p, b);
      const int last = min(min(pos + 128, p.T), len) - 1;
      first = max(0, pos - p.window + 1) >> 6;
      sink_tiles = min((p.sinks + 63) >> 6, first);
      count = pos < len ? sink_tiles + (last >> 6) - first + 1 : 0;
    } else {
      b = ba / p.Hkv;
      ha = ba % p.Hkv;
      hb0 = ha * p.group;
      const int split = q.sink_tiles * q.parts;
      kt = x < split ? x / q.parts : x - split + q.sink_tiles;
      part = x < split ? x % q.parts : 0;
      a0 = pos = kt * 128;
      len = seq_len(p, b);
      const KeyPart kp = key_part(kt, part, 128, p.window, p.T, p.far_rows);
      lo = max(kp.lo, p.T - p.Tq);
      hi = min(kp.hi, len);
      per = hi > lo ? (hi - lo + 63) >> 6 : 0;
      count = per * p.group;
    }
  }
  __device__ __forceinline__ int head(int n) const { return MODE == WATTN_DQ ? hb0 : hb0 + n / per; }
  // the position of B's first row
  __device__ __forceinline__ int at(int n) const {
    if (MODE == WATTN_DQ) return (n < sink_tiles ? n : first + n - sink_tiles) << 6;
    return lo + (n % per) * 64;
  }
};

template <int D, int MODE>
struct BwdCfg {
  static constexpr int kKb = D / 64;
  static constexpr int kABytes = kKb * 16384;
  static constexpr int kAll = MODE == WATTN_DV ? kABytes : 2 * kABytes;
  static constexpr int kBBytes = kKb * 8192;              // a tile of 64 rows
  static constexpr int kTiles = (229376 - kAll) / kBBytes > 6 ? 6 : (229376 - kAll) / kBBytes;   // of both rings
  // dV holds B2 until its product is done, the others B1
  static constexpr int kR1 = MODE == WATTN_DV ? kTiles / 2 : (kTiles + 1) / 2;
  static constexpr int kR2 = kTiles - kR1;
  // B2 is a K-major operand in dQ and dK: its 64-channel blocks come and go singly
  static constexpr int kS2 = MODE == WATTN_DV ? kR2 : kR2 * kKb;
  static constexpr int kB2Slot = MODE == WATTN_DV ? kBBytes : 8192;
  static constexpr int kOffB1 = kAll, kOffB2 = kOffB1 + kR1 * kBBytes, kOffCol = kOffB2 + kR2 * kBBytes;
  static constexpr int kOffBar = kOffCol + 2 * 2 * 64 * 4;   // lse and delta of two tiles' columns
  // afull aempty | b1full[] b1empty[] | b2full[] b2empty[] | sfull[2] pfull[2] cfull[2] | xfull xempty
  static constexpr int kBars = 2 + 2 * kR1 + 2 * kS2 + 6 + 2;
  static constexpr int kSmem = kOffBar + kBars * 8 + 16 + 1024;
  static constexpr int kThreads = 320;
  static constexpr uint32_t kColX = 0, kColS = 256;          // buffers of 64 + 64 columns
};

template <int D, int MODE>
__global__ void __launch_bounds__(320, 1) k_wattn_bwd(const __grid_constant__ WattnBwdParams p) {
  using C = BwdCfg<D, MODE>;
  constexpr int R1 = C::kR1, S2 = C::kS2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t *afull = bar, *aempty = bar + 1, *b1full = bar + 2, *b1empty = b1full + R1, *b2full = b1empty + R1,
           *b2empty = b2full + S2, *sfull = b2empty + S2, *pfull = sfull + 2, *cfull = pfull + 2, *xfull = cfull + 2,
           *xempty = xfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + C::kBars);

  griddep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (__syncthreads_or(*reinterpret_cast<volatile int*>(&g_status))) return;   // an earlier wait gave up
  if (threadIdx.x == 0) {
    mbar_init(afull, 1);
    mbar_init(aempty, 1);
    for (int i = 0; i < R1; ++i) {
      mbar_init(&b1full[i], 1);
      mbar_init(&b1empty[i], 1);
    }
    for (int i = 0; i < S2; ++i) {
      mbar_init(&b2full[i], 1);
      mbar_init(&b2empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
      mbar_init(&cfull[i], 4);
    }
    mbar_init(xfull, 1);
    mbar_init(xempty, 8);
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

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      int i1 = 0, i2 = 0, ic = 0;
      bool ok = true;
      for (int item = blockIdx.x; ok && item < p.nitems; item += gridDim.x) {
        const BwdItem<MODE> t(p, item);
        if (t.count == 0) continue;
        if (ic > 0 && !mbar_wait(aempty, (ic - 1) & 1)) break;
        ++ic;
        mbar_arrive_expect_tx(afull, C::kAll);
        for (int kb = 0; kb < C::kKb; ++kb) {
          tma_load_4d(smem + kb * 16384, &p.tmA1, afull, kb * 64, t.a0, t.ha, t.b);
          if (MODE != WATTN_DV)
            tma_load_4d(smem + C::kABytes + kb * 16384, &p.tmA2, afull, kb * 64, t.a0, t.ha, t.b);
        }
        for (int n = 0; ok && n < t.count; ++n) {
          const int row = t.at(n) - (MODE == WATTN_DQ ? 0 : off), hb = t.head(n);
          {
            const int s = i1 % R1;
            if (i1 >= R1 && !mbar_wait(&b1empty[s], ((i1 / R1) - 1) & 1)) { ok = false; break; }
            mbar_arrive_expect_tx(&b1full[s], C::kBBytes);
            for (int kb = 0; kb < C::kKb; ++kb)
              tma_load_4d(smem + C::kOffB1 + s * C::kBBytes + kb * 8192, &p.tmB1, &b1full[s], kb * 64, row, hb, t.b);
            ++i1;
          }
          if (MODE == WATTN_DV) {
            const int s = i2 % S2;
            if (i2 >= S2 && !mbar_wait(&b2empty[s], ((i2 / S2) - 1) & 1)) { ok = false; break; }
            mbar_arrive_expect_tx(&b2full[s], C::kBBytes);
            for (int kb = 0; kb < C::kKb; ++kb)
              tma_load_4d(smem + C::kOffB2 + s * C::kBBytes + kb * 8192, &p.tmB2, &b2full[s], kb * 64, row, hb, t.b);
            ++i2;
          } else {
            for (int kb = 0; kb < C::kKb; ++kb, ++i2) {
              const int s = i2 % S2;
              if (i2 >= S2 && !mbar_wait(&b2empty[s], ((i2 / S2) - 1) & 1)) { ok = false; break; }
              mbar_arrive_expect_tx(&b2full[s], 8192);
              tma_load_4d(smem + C::kOffB2 + s * 8192, &p.tmB2, &b2full[s], kb * 64, row, hb, t.b);
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- products
    constexpr uint32_t ids = idesc_bf16(128, 64, false, false), idx = idesc_bf16(128, D, false, true);
    const uint32_t sbase = smem_u32(smem);
    int i1 = 0, i2 = 0, sc = 0, pc = 0, ica = 0, icx = 0;
    int nt = blockIdx.x, nn = 0, ncount = 0;          // the next tile whose scores are due
    auto settle = [&]() {
      while (nt < p.nitems && (ncount = BwdItem<MODE>(p, nt).count) == 0) nt += gridDim.x;
    };
    // rows of a 64-row tile at or past `keep` become zeros (64 channels x 128 B blocks)
    auto clear = [&](uint32_t base, int keep) {
      if (keep >= 64) return;
      for (int e = max(keep, 0) * 8 + lane; e < 512; e += 32)
        for (int kb = 0; kb < C::kKb; ++kb) st_shared_v4(base + kb * 8192 + e * 16, 0, 0, 0, 0);
      fence_async_smem();
      __syncwarp();
    };
    auto scores = [&]() -> bool {
      const BwdItem<MODE> t(p, nt);
      if (nn == 0 && !mbar_wait_warp(afull, ica & 1)) return false;
      const uint32_t sd = tmem + C::kColS + (sc & 1) * 128;
      const int s1 = i1 % R1;
      if (!mbar_wait_warp(&b1full[s1], (i1 / R1) & 1)) return false;
      tc_fence_after();
      const uint32_t b1 = sbase + C::kOffB1 + s1 * C::kBBytes;
      // rows behind the sequence: a dS of 0 times whatever is there must stay 0
      if (MODE != WATTN_DV) clear(b1, t.len - t.at(nn));
      if (lane == 0) {
        for (int kb = 0; kb < C::kKb; ++kb)
          mma_kblock<false, false>(sd, sbase + kb * 16384, 0, b1 + kb * 8192, 0, ids, kb == 0);
        if (MODE == WATTN_DV) umma_commit(&b1empty[s1]);
      }
      __syncwarp();
      ++i1;
      if (MODE != WATTN_DV) {
        for (int kb = 0; kb < C::kKb; ++kb, ++i2) {
          const int s = i2 % S2;
          if (!mbar_wait_warp(&b2full[s], (i2 / S2) & 1)) return false;
          tc_fence_after();
          if (lane == 0) {
            mma_kblock<false, false>(sd + 64, sbase + C::kABytes + kb * 16384, 0, sbase + C::kOffB2 + s * 8192, 0, ids,
                                     kb == 0);
            umma_commit(&b2empty[s]);
          }
          __syncwarp();
        }
      }
      const bool end = nn + 1 == ncount;
      if (lane == 0) {
        umma_commit(&sfull[sc & 1]);
        if (end) umma_commit(aempty);
      }
      __syncwarp();
      ++sc;
      if (end) {
        ++ica;
        nn = 0;
        nt += gridDim.x;
        settle();
      } else {
        ++nn;
      }
      return true;
    };
    settle();
    bool ok = nt >= p.nitems || scores();
    for (int item = blockIdx.x; ok && item < p.nitems; item += gridDim.x) {
      const BwdItem<MODE> t(p, item);
      if (t.count == 0) continue;
      for (int n = 0; ok && n < t.count; ++n, ++pc) {
        if (nt < p.nitems && !scores()) { ok = false; break; }
        if (n == 0 && icx > 0 && !mbar_wait_warp(xempty, (icx - 1) & 1)) { ok = false; break; }
        if (!mbar_wait_warp(&pfull[pc & 1], (pc >> 1) & 1)) { ok = false; break; }
        const uint32_t pa = tmem + C::kColS + (pc & 1) * 128;
        const int s = MODE == WATTN_DV ? pc % S2 : pc % R1;
        const uint32_t xb = sbase + (MODE == WATTN_DV ? C::kOffB2 : C::kOffB1) + s * C::kBBytes;
        if (MODE == WATTN_DV) {
          if (!mbar_wait_warp(&b2full[s], (pc / S2) & 1)) { ok = false; break; }
          clear(xb, t.len - t.at(n));
        }
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16_ta(tmem + C::kColX, pa + k * 8, smem_desc_sw128(xb + k * 2048u, 8192u, 1024u), idx,
                         (n == 0 && k == 0) ? 0u : 1u);
          umma_commit(MODE == WATTN_DV ? &b2empty[s] : &b1empty[s]);
          if (n + 1 == t.count) umma_commit(xfull);
        }
        __syncwarp();
      }
      ++icx;
    }
  } else {
    // ---------------------------------------------------------- elementwise
    const int group = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t ts = tq + C::kColS + group * 128;
    const float c2 = p.a.scale * 1.4426950408889634f;
    const int window = p.a.window, sinks = p.a.sinks;
    float* cols = reinterpret_cast<float*>(smem + C::kOffCol) + group * 128;   // lse (log2), delta
    const uint32_t col_s = smem_u32(cols);
    int sc = 0, ic = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < p.nitems; item += gridDim.x) {
      const BwdItem<MODE> t(p, item);
      const int mine = t.pos + r;                     // this row's position
      float rl = 0.f, rd = 0.f;
      if (MODE == WATTN_DQ && mine < t.len && t.a0 + r < p.a.Tq) {
        const int64_t at = (static_cast<int64_t>(t.b) * p.a.H + t.ha) * p.a.Tq + t.a0 + r;
        rl = p.a.lse[at] * 1.4426950408889634f;
        rd = p.a.delta[at];
      }
      for (int n = 0; n < t.count; ++n, ++sc) {
        if ((sc & 1) != group) continue;
        const int b0 = t.at(n);                       // position of the tile's first column
        float x = 0.f;
        if (MODE != WATTN_DQ) {
          // the columns' statistics: one value per thread
          const int i = b0 + (r & 63);
          if (i < t.hi) {
            const int64_t at = (static_cast<int64_t>(t.b) * p.a.H + t.head(n)) * p.a.Tq + i - off;
            x = r < 64 ? p.a.lse[at] * 1.4426950408889634f : (MODE == WATTN_DK ? p.a.delta[at] : 0.f);
          }
        }
        if (!mbar_wait_warp(&sfull[group], (sc >> 1) & 1)) { ok = false; break; }
        if (MODE != WATTN_DQ) {
          // S came after the group's last dS, so the last tile's statistics have been read
          cols[r] = x;
          __syncwarp();
          if (lane == 0) mbar_arrive(&cfull[group]);
          if (!mbar_wait_warp(&cfull[group], (sc >> 1) & 1)) { ok = false; break; }
        }
        tc_fence_after();
        bool whole;
        int clo, chi, csk;                            // columns c with clo < c <= chi, or csk's side
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
          csk = -1;
        }
        uint32_t hw[32];
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          float s[32], dp[32];
          tmem_ld16(ts + c0, s);
          tmem_ld16(ts + c0 + 16, s + 16);
          if (MODE != WATTN_DV) {
            tmem_ld16(ts + 64 + c0, dp);
            tmem_ld16(ts + 64 + c0 + 16, dp + 16);
          }
          tmem_ld_wait();
#pragma unroll
          for (int c4 = 0; c4 < 32; c4 += 4) {
            float4 l4, d4;
            if (MODE != WATTN_DQ) {
              asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(l4.x), "=f"(l4.y), "=f"(l4.z), "=f"(l4.w) : "r"(col_s + (c0 + c4) * 4));
              if (MODE == WATTN_DK)
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(d4.x), "=f"(d4.y), "=f"(d4.z), "=f"(d4.w) : "r"(col_s + 256 + (c0 + c4) * 4));
            }
            const float ll[4] = {l4.x, l4.y, l4.z, l4.w}, dd[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int c = c4 + k;
              const float pr = ex2_approx(fmaf(s[c], c2, -(MODE == WATTN_DQ ? rl : ll[k])));
              s[c] = MODE == WATTN_DV ? pr : pr * (dp[c] - (MODE == WATTN_DQ ? rd : dd[k]));
            }
          }
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c0 + c > chi || (c0 + c <= clo && c0 + c >= csk)) s[c] = 0.f;
          }
          // the last product's operand: half a step, 2^-8 of each
#pragma unroll
          for (int c = 0; c < 16; ++c) hw[c0 / 2 + c] = pack_bf16x2(s[2 * c], s[2 * c + 1]);
        }
        tmem_st16u(ts, hw);
        tmem_st16u(ts + 16, hw + 16);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[group]);
      }
      if (!ok) break;
      // the gradient's rows: this group's half of the channels
      if (t.count > 0) {
        if (!mbar_wait_warp(xfull, ic & 1)) break;
        ++ic;
        tc_fence_after();
      }
      const float mul = MODE == WATTN_DV ? 1.0f : p.a.scale;
      const int row = t.a0 + r;
      const bool in = row < (MODE == WATTN_DQ ? p.a.Tq : p.a.T);
      const bool zero = t.count == 0 || (MODE == WATTN_DQ && mine >= t.len);
      const View4& o = MODE == WATTN_DQ ? p.a.dq : MODE == WATTN_DK ? p.a.dk : p.a.dv;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(o.p) + t.b * o.sb + t.ha * o.sh + static_cast<int64_t>(row) * o.st;
      const bool partial = MODE != WATTN_DQ && t.kt < p.sink_tiles;
      float* pd = nullptr;
      if (partial)
        pd = p.a.part + ((((static_cast<int64_t>(t.b) * p.a.Hkv + t.ha) * p.sink_tiles + t.kt) * p.parts + t.part) * 2 +
                         (MODE == WATTN_DV ? 1 : 0)) * (128 * D) + r * D;
#pragma unroll 1
      for (int c0 = group * (D / 2); c0 < (group + 1) * (D / 2); c0 += 16) {
        float x[16];
        if (t.count > 0) {
          __syncwarp();
          tmem_ld16(tq + C::kColX + c0, x);
          tmem_ld_wait();
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = zero ? 0.f : x[c] * mul;
        if (partial) {
#pragma unroll
          for (int c = 0; c < 16; c += 4) *reinterpret_cast<float4*>(pd + c0 + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
        } else if (in) {
#pragma unroll
          for (int c = 0; c < 16; c += 8)
            if (c0 + c < p.a.d)
              st_global_v4(dst + c0 + c, pack_bf16x2(x[c], x[c + 1]), pack_bf16x2(x[c + 2], x[c + 3]),
                           pack_bf16x2(x[c + 4], x[c + 5]), pack_bf16x2(x[c + 6], x[c + 7]));
        }
      }
      if (t.count > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(xempty);
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
