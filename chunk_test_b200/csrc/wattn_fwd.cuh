// wattn_fwd.cuh -- the window attention with sinks on the tensor cores (bf16).
// Mask and formulas: wattn_common.cuh.
//
// A tile is 128 queries of one head; it walks the key tiles (128 keys) of the
// sinks and of its window with an online softmax.  Roles of a CTA:
//   warp 0     TMA producer of the queries and keys: a key slot is 128 keys x
//              64 channels (16 KB), freed as soon as its part of S is done.
//              (NS = 1: of the values too.)
//   warp 1     issues S_j = Q K_j^T and O += P_j V_j (tcgen05, M = 128).
//   warps 2-5  softmax, one query row per thread; P_j goes back to TMEM in
//              bf16, over S_j, and is the second product's A operand from
//              there, so shared memory carries K, V and Q only.
//   warp 6     (NS = 2) TMA producer of the values, in slots of 64 keys x all
//              channels (128 keys at d = 64).
// Head dims up to 128: two CTAs per SM with one score buffer each (NS = 1); one
// CTA's products run under the other's exponentials.  Above: one CTA per SM
// and two score buffers (NS = 2), S_{j+1} issued before P_j is ready.
//
// Bound by the exponentials (16 per clock and SM: 1024 clocks a tile of 128 x
// 128, as many as both products at d = 128) up to d = 128, by the tensor pipe
// (2048 clocks a tile at d = 256) above.
#pragma once

#include "swa_flash.cuh"
#include "wattn_common.cuh"

namespace lact {

// 4-D tiled load (channel, token, head, batch)
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// A wait made by a whole warp, with one outcome for all of its lanes.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// D[tmem] (+)= A[tmem] * B[smem], bf16: A's row r is lane r, two elements of K per column.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]));
}

struct WattnFwdParams {
  CUtensorMap tmQ;    // [d, Tq, H, B], box {64, 128}
  CUtensorMap tmK;    // [d, T, Hkv, B], box {64, 128}
  CUtensorMap tmV;    // [d, T, Hkv, B], box {64, kVKeys}
  WattnParams a;
  int nb, ntiles;     // 128-query tiles per head, in all
};

// One query tile and the key tiles it walks: the sinks' before its window,
// then its window's.
struct QueryTile {
  int b, h, hk, q0, i0, len, sink_tiles, first, count;
  __device__ __forceinline__ QueryTile(const WattnParams& p, int nb, int tile) {
    const int bh = tile / nb;
    b = bh / p.H;
    h = bh % p.H;
    hk = h / p.group;
    q0 = (tile % nb) * 128;
    i0 = q0 + p.T - p.Tq;
    len = seq_len(p, b);
    const int last = min(min(i0 + 128, p.T), len) - 1;    // last position of the tile that is a token
    first = max(0, i0 - p.window + 1) >> 7;
    sink_tiles = min((p.sinks + 127) >> 7, first);
    count = i0 < len ? sink_tiles + (last >> 7) - first + 1 : 0;
  }
  __device__ __forceinline__ int key0(int n) const { return (n < sink_tiles ? n : first + n - sink_tiles) << 7; }
};

template <int D>
struct WattnCfg {
  static_assert(D % 64 == 0 && D >= 64 && D <= 256, "padded head dim");
  static constexpr int kNS = D <= 128 ? 1 : 2;            // score buffers
  static constexpr int kCtas = D <= 128 ? 2 : 1;          // CTAs per SM
  static constexpr int kWarps = kNS == 1 ? 6 : 7;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kKb = D / 64;                      // key slots of a tile
  static constexpr int kVKeys = D == 64 ? 128 : 64;
  static constexpr int kVSlots = 128 / kVKeys;            // value slots of a tile
  static constexpr int kVBox = kVKeys * 128;              // bytes of one box {64, kVKeys}
  static constexpr int kKSlot = 16384, kVSlot = kKb * kVBox;
  static constexpr int kQBytes = kKb * 16384;
  // slots of the two rings: 96 to 98 KB for one of two CTAs, 224 KB for a single one
  static constexpr int kKR = D == 64 ? 3 : D == 128 ? 2 : D == 192 ? 5 : 4;
  static constexpr int kVR = D <= 128 ? 2 : D == 192 ? 4 : 3;
  static constexpr int kOffK = kQBytes, kOffV = kOffK + kKR * kKSlot, kOffBar = kOffV + kVR * kVSlot;
  // qfull qempty | kfull[] kempty[] | vfull[] vempty[] | sfull[NS] pfull[NS] | pvdone ofull oempty
  static constexpr int kBars = 2 + 2 * kKR + 2 * kVR + 2 * kNS + 3;
  static constexpr int kSmem = kOffBar + kBars * 8 + 16 + 1024;
  static constexpr uint32_t kColO = 0, kColS = kNS == 1 ? 128 : 256, kCols = kNS == 1 ? 256 : 512;
};

template <int D>
__global__ void __launch_bounds__(WattnCfg<D>::kThreads, WattnCfg<D>::kCtas)
    k_wattn_fwd(const __grid_constant__ WattnFwdParams p) {
  using C = WattnCfg<D>;
  constexpr int NS = C::kNS, KR = C::kKR, VR = C::kVR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t *qfull = bar, *qempty = bar + 1, *kfull = bar + 2, *kempty = kfull + KR, *vfull = kempty + KR,
           *vempty = vfull + VR, *sfull = vempty + VR, *pfull = sfull + NS, *pvdone = pfull + NS, *ofull = pvdone + 1, *oempty = ofull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + C::kBars);

  griddep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (__syncthreads_or(*reinterpret_cast<volatile int*>(&g_status))) return;   // an earlier wait gave up
  if (threadIdx.x == 0) {
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    for (int i = 0; i < KR; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < VR; ++i) {
      mbar_init(&vfull[i], 1);
      mbar_init(&vempty[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
    }
    mbar_init(pvdone, 1);
    mbar_init(ofull, 1);
    mbar_init(oempty, 4);
    fence_barrier_init();
    tma_prefetch_map(&p.tmQ);
    tma_prefetch_map(&p.tmK);
    tma_prefetch_map(&p.tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync_converged();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  if (warp == 0 || (NS == 2 && warp == 6)) {
    // ---------------------------------------------------------- producers
    if (lane == 0) {
      const bool keys = warp == 0, values = NS == 1 || warp == 6;
      int ik = 0, iv = 0, tc = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < p.ntiles; tile += gridDim.x) {
        const QueryTile t(p.a, p.nb, tile);
        if (t.count == 0) continue;
        if (keys) {
          if (tc > 0 && !mbar_wait(qempty, (tc - 1) & 1)) break;
          ++tc;
          mbar_arrive_expect_tx(qfull, C::kQBytes);
          for (int kb = 0; kb < C::kKb; ++kb)
            tma_load_4d(smem + kb * 16384, &p.tmQ, qfull, kb * 64, t.q0, t.h, t.b);
        }
        for (int n = 0; ok && n < t.count; ++n) {
          const int j0 = t.key0(n);
          for (int kb = 0; keys && ok && kb < C::kKb; ++kb, ++ik) {
            const int s = ik % KR;
            if (ik >= KR && !mbar_wait(&kempty[s], ((ik / KR) - 1) & 1)) { ok = false; break; }
            mbar_arrive_expect_tx(&kfull[s], C::kKSlot);
            tma_load_4d(smem + C::kOffK + s * C::kKSlot, &p.tmK, &kfull[s], kb * 64, j0, t.hk, t.b);
          }
          for (int vs = 0; values && ok && vs < C::kVSlots; ++vs, ++iv) {
            const int s = iv % VR;
            if (iv >= VR && !mbar_wait(&vempty[s], ((iv / VR) - 1) & 1)) { ok = false; break; }
            mbar_arrive_expect_tx(&vfull[s], C::kVSlot);
            for (int nb = 0; nb < C::kKb; ++nb)
              tma_load_4d(smem + C::kOffV + s * C::kVSlot + nb * C::kVBox, &p.tmV, &vfull[s], nb * 64,
                          j0 + vs * C::kVKeys, t.hk, t.b);
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- products
    constexpr uint32_t ids = idesc_bf16(128, 128, false, false), ido = idesc_bf16(128, D, false, true);
    const uint32_t sbase = smem_u32(smem);
    int ik = 0, iv = 0, sc = 0, pc = 0, tcq = 0, tco = 0;
    // the next key tile whose scores are due
    int qt = blockIdx.x, qn = 0, qcount = 0;
    auto settle = [&]() {
      while (qt < p.ntiles && (qcount = QueryTile(p.a, p.nb, qt).count) == 0) qt += gridDim.x;
    };
    auto scores = [&]() -> bool {
      if (qn == 0 && !mbar_wait_warp(qfull, tcq & 1)) return false;
      const uint32_t sd = tmem + C::kColS + (sc % NS) * 128;
      for (int kb = 0; kb < C::kKb; ++kb, ++ik) {
        const int s = ik % KR;
        if (!mbar_wait_warp(&kfull[s], (ik / KR) & 1)) return false;
        tc_fence_after();
        if (lane == 0) {
          mma_kblock<false, false>(sd, sbase + kb * 16384, 0, sbase + C::kOffK + s * C::kKSlot, 0, ids, kb == 0);
          umma_commit(&kempty[s]);
        }
        __syncwarp();
      }
      const bool end = qn + 1 == qcount;
      if (lane == 0) {
        umma_commit(&sfull[sc % NS]);
        if (end) umma_commit(qempty);
      }
      __syncwarp();
      ++sc;
      if (end) {
        ++tcq;
        qn = 0;
        qt += gridDim.x;
        settle();
      } else {
        ++qn;
      }
      return true;
    };
    settle();
    bool ok = qt >= p.ntiles || scores();
    for (int tile = blockIdx.x; ok && tile < p.ntiles; tile += gridDim.x) {
      const QueryTile t(p.a, p.nb, tile);
      if (t.count == 0) continue;
      for (int n = 0; ok && n < t.count; ++n, ++pc) {
        if (NS == 2 && qt < p.ntiles && !scores()) { ok = false; break; }
        if (n == 0 && tco > 0 && !mbar_wait_warp(oempty, (tco - 1) & 1)) { ok = false; break; }
        if (!mbar_wait_warp(&pfull[pc % NS], (pc / NS) & 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t pa = tmem + C::kColS + (pc % NS) * 128;
        const int j0 = t.key0(n);
        for (int vs = 0; vs < C::kVSlots; ++vs, ++iv) {
          const int s = iv % VR;
          if (!mbar_wait_warp(&vfull[s], (iv / VR) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t vb = sbase + C::kOffV + s * C::kVSlot;
          // rows behind the sequence: a probability of 0 times whatever is there must stay 0
          const int keep = t.len - (j0 + vs * C::kVKeys);
          if (keep < C::kVKeys) {
            for (int e = max(keep, 0) * 8 + lane; e < C::kVKeys * 8; e += 32)
              for (int nb = 0; nb < C::kKb; ++nb) st_shared_v4(vb + nb * C::kVBox + e * 16, 0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
          }
          if (lane == 0) {
#pragma unroll
            for (int k = 0; k < C::kVKeys / 16; ++k)
              umma_bf16_ta(tmem + C::kColO, pa + (vs * C::kVKeys + k * 16) / 2,
                           smem_desc_sw128(vb + k * 2048u, C::kVBox, 1024u), ido, (n == 0 && vs == 0 && k == 0) ? 0u : 1u);
            umma_commit(&vempty[s]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) {
          umma_commit(pvdone);
          if (n + 1 == t.count) umma_commit(ofull);
        }
        __syncwarp();
        if (NS == 1 && qt < p.ntiles && !scores()) ok = false;
      }
      ++tco;
    }
  } else if (warp < 6) {
    // ---------------------------------------------------------- softmax
    // The reference maximum of a row is raised only when a tile's maximum is
    // above it by more than 8 in log2 units; the output row in TMEM is
    // rescaled then (the whole warp: TMEM accesses are collective).  The
    // probabilities stay below 2^8, their sum in 32 bits.
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float c2 = p.a.scale * 1.4426950408889634f;
    const int window = p.a.window, sinks = p.a.sinks;
    int sc = 0, tc = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < p.ntiles; tile += gridDim.x) {
      const QueryTile t(p.a, p.nb, tile);
      const int i = t.i0 + r, last = t.i0 + 127;
      float mx = -INFINITY, sum = 0.f;
      for (int n = 0; n < t.count; ++n, ++sc) {
        const int sb = sc % NS, j0 = t.key0(n);
        if (!mbar_wait_warp(&sfull[sb], (sc / NS) & 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t ts = tq + C::kColS + sb * 128;
        float sv[128];
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 16) tmem_ld16(ts + c0, sv + c0);
        tmem_ld_wait();
        const bool whole = j0 + 127 <= t.i0 && (j0 > last - window || j0 + 127 < sinks) && last < t.len;
        if (!whole) {
          const int hi = i < t.len ? i - j0 : -1, lo = i - window - j0, sk = sinks - j0;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > hi || (c <= lo && c >= sk)) sv[c] = -INFINITY;
        }
        float b8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) b8[c] = sv[c];
#pragma unroll
        for (int c = 8; c < 128; ++c) b8[c & 7] = fmaxf(b8[c & 7], sv[c]);
        const float bm = fmaxf(fmaxf(fmaxf(b8[0], b8[1]), fmaxf(b8[2], b8[3])),
                               fmaxf(fmaxf(b8[4], b8[5]), fmaxf(b8[6], b8[7])));
        float fix = 1.0f;
        bool grow = false;
        if (mx == -INFINITY) {
          mx = bm;   // no earlier key of this row: its output row and sum are zero
        } else if ((bm - mx) * c2 > 8.0f) {
          grow = true;
          fix = ex2_approx((mx - bm) * c2);
          mx = bm;
        }
        if (__any_sync(0xffffffffu, grow)) {
          // S_n was issued after P V of tile n - 2 (NS = 2) or n - 1 (NS = 1)
          if (NS == 2 && !mbar_wait_warp(pvdone, (sc - 1) & 1)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            float o[16];
            __syncwarp();
            tmem_ld16(tq + C::kColO + c0, o);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] *= fix;
            tmem_st16(tq + C::kColO + c0, o);
          }
          sum *= fix;
        }
        const float off = mx == -INFINITY ? 0.f : -mx * c2;
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t hw[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float e0 = ex2_approx(fmaf(sv[c0 + 2 * c], c2, off));
            const float e1 = ex2_approx(fmaf(sv[c0 + 2 * c + 1], c2, off));
            ps[c & 3] += e0 + e1;
            hw[c] = pack_bf16x2(e0, e1);   // the second product's operand: half a step, 2^-8 of each
          }
          tmem_st16u(ts + c0 / 2, hw);
        }
        sum += (ps[0] + ps[1]) + (ps[2] + ps[3]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[sb]);
      }
      if (!ok) break;
      // out = O / sum, lse = the reference maximum + log sum
      const bool in = t.q0 + r < p.a.Tq;
      const bool some = i < t.len;       // a token sees at least itself
      const float inv = some ? 1.0f / sum : 0.f;
      if (in)
        p.a.lse[(static_cast<int64_t>(t.b) * p.a.H + t.h) * p.a.Tq + t.q0 + r] =
            some ? fmaf(mx, p.a.scale, logf(sum)) : -INFINITY;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.a.out.p) + t.b * p.a.out.sb + t.h * p.a.out.sh +
                           static_cast<int64_t>(t.q0 + r) * p.a.out.st;
      if (t.count == 0) {
        if (in)
          for (int c = 0; c < p.a.d; c += 8) st_global_v4(dst + c, 0, 0, 0, 0);
        continue;
      }
      if (!mbar_wait_warp(ofull, tc & 1)) break;
      ++tc;
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        __syncwarp();
        tmem_ld16(tq + C::kColO + c0, o);
        tmem_ld16(tq + C::kColO + c0 + 16, o + 16);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (in && c0 + 8 * g < p.a.d) {
#pragma unroll
            for (int c = 0; c < 8; ++c) o[8 * g + c] = some ? o[8 * g + c] * inv : 0.f;
            st_global_v4(dst + c0 + 8 * g, pack_bf16x2(o[8 * g], o[8 * g + 1]), pack_bf16x2(o[8 * g + 2], o[8 * g + 3]),
                         pack_bf16x2(o[8 * g + 4], o[8 * g + 5]), pack_bf16x2(o[8 * g + 6], o[8 * g + 7]));
          }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(oempty);
    }
  }
  tc_fence_before();
  cta_sync_converged();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

}  // namespace lact
