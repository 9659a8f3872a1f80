// wattn_fwd.cuh -- the window attention with sinks on the tensor cores (bf16).
// Mask and formulas: wattn_common.cuh.
//
// A tile is 128 queries of one head; it walks the key tiles (128 keys) of the
// sinks and of its window with an online softmax.  Where the sinks end with at
// most 32 keys of a tile, that tile is 32 keys wide in every step.  Roles:
//   warp 0     TMA producer of the queries and keys (NS = 1: of the values too).
//   warp 1     issues S_j = Q K_j^T and O += P_j V_j (tcgen05, M = 128), in the
//              order S_(j+1), P_j V_j (NS = 2): S_(j+1) first, because the softmax
//              that waits for it is as long as both products.  One thread; it
//              waits and commits as little as the rings allow, each of which
//              costs 50 to 100 clocks in which it feeds nothing.
//   warps 2-5  softmax, one query row per thread; P_j goes back to TMEM in
//              bf16, over S_j, and is the second product's A operand from
//              there, so shared memory carries K, V and Q only.  The output
//              leaves through a staging tile and bulk tensor stores (16-byte
//              stores of a row per thread took 6600 clocks a query tile at d 256).
//   warp 6     (NS = 2) TMA producer of the values, in slots of 64 keys.
// Head dims up to 128: two CTAs per SM with one score buffer each (NS = 1); one
// CTA's products run under the other's exponentials.  Above: one CTA per SM
// and two score buffers (NS = 2).
//
// Bound, above d = 128, by the tensor pipe and what the issuing thread waits:
// about 3000 clocks a tile for 2048 of products at d = 256 (B 2, H 6, T 32768,
// window 2048, 4 sinks: 862 us in a row of calls, 929 TFLOP/s, where the 1000 W
// cap holds the clock down; 766 us after a pause).  Up to d = 128 by the latency of
// S, softmax and P V in turn: 2900 clocks a tile and SM for 1024 of products and
// as many of exponentials at 16 per clock (B 3 of up to 5000 tokens, 12 heads on
// 4, d 128, window 1000: 107 us).
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

// 4-D tiled store from shared memory (bulk-group completion); clips at the tensor's ends
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
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

// 32 lanes x 32 columns; thread t of the warp gets lane 32 (warp % 4) + t.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Two 32-bit operations in one instruction.
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Bits 0..31: the columns base + bit below `n`.
__device__ __forceinline__ uint32_t bits_below(int n, int base) {
  const int k = n - base;
  return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u;
}
// The visible ones of columns base .. base + 31: lo < c <= hi, or c < sk.
__device__ __forceinline__ uint32_t visible_bits(int lo, int hi, int sk, int base) {
  return bits_below(hi + 1, base) & (~bits_below(lo + 1, base) | bits_below(sk, base));
}

// Shared-memory descriptors of one operand differ by their start address only.
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }
// Keeps the compiler from forming a loop's descriptors ahead of the loop, where
// they spill.
__device__ __forceinline__ uint64_t here(uint64_t desc) {
  asm volatile("" : "+l"(desc));
  return desc;
}

struct WattnFwdParams {
  CUtensorMap tmQ;          // [d, Tq, H, B], box {64, 128}
  CUtensorMap tmK, tmV;     // [d, T, Hkv, B], boxes {64, 128}, {64, kVKeys}
  CUtensorMap tmK32, tmV32; // the same, box {64, 32}: a narrow sink tile
  CUtensorMap tmO;          // out, box {32, 32}, 64-byte swizzle
  WattnParams a;
  int nb, ntiles;           // 128-query tiles per head, in all
};

// One query tile and the key tiles it walks: the sinks' before its window,
// then its window's.
struct QueryTile {
  int b, h, hk, q0, i0, len, sink_tiles, first, count;
  int narrow;   // the sink tile of which at most 32 keys are sinks, or -1
  __device__ __forceinline__ QueryTile(const WattnParams& p, int nb, int tile) {
    const TileAt at = query_tile_at(p, nb, tile);
    b = at.b;
    h = at.h;
    hk = h / p.group;
    q0 = at.m * 128;
    i0 = q0 + p.T - p.Tq;
    len = seq_len(p, b);
    const int last = min(min(i0 + 128, p.T), len) - 1;    // last position of the tile that is a token
    first = max(0, i0 - p.window + 1) >> 7;
    sink_tiles = min((p.sinks + 127) >> 7, first);
    count = i0 < len ? sink_tiles + (last >> 7) - first + 1 : 0;
    narrow = sink_tiles > 0 && p.sinks - ((sink_tiles - 1) << 7) <= 32 ? sink_tiles - 1 : -1;
  }
  __device__ __forceinline__ int key0(int n) const { return (n < sink_tiles ? n : first + n - sink_tiles) << 7; }
};

template <int D>
struct WattnCfg {
  static_assert(D % 64 == 0 && D >= 64 && D <= 256, "padded head dim");
  static constexpr int kNS = D <= 128 ? 1 : 2;            // score buffers
  static constexpr int kCtas = D <= 128 ? 2 : 1;          // CTAs per SM
  static constexpr int kThreads = kNS == 1 ? 192 : 224;
  static constexpr int kKb = D / 64;
  static constexpr int kQBytes = kKb * 16384;
  // key slots of 128 keys x kKBlk 64-channel blocks, value slots of kVKeys keys
  static constexpr int kKBlk = D == 256 ? 2 : kKb, kKPer = kKb / kKBlk;
  static constexpr int kVKeys = kNS == 1 ? 128 : 64, kVPer = 128 / kVKeys;
  static constexpr int kVBox = kVKeys * 128;              // bytes of one box {64, kVKeys}
  static constexpr int kKSlot = kKBlk * 16384, kVSlot = kKb * kVBox;
  static constexpr int kKR = D == 128 ? 1 : 2, kVR = D == 128 ? 1 : 2;
  static constexpr int kOffK = kQBytes, kOffV = kOffK + kKR * kKSlot, kOffStage = kOffV + kVR * kVSlot;
  static constexpr int kStages = kNS == 1 ? 2 : 4;        // staging tiles of a softmax warp: 32 rows x 32 channels
  static constexpr int kOffBar = kOffStage + 4 * kStages * 2048;
  // qfull qempty | kfull[] kempty[] | vfull[] vempty[] | sfull[NS] pfull[NS] | pvdone ofull oempty
  static constexpr int kBars = 2 + 2 * kKR + 2 * kVR + 2 * kNS + 3;
  static constexpr int kSmem = kOffBar + kBars * 8 + 16;
  static constexpr uint32_t kColO = 0, kColS = kNS == 1 ? 128 : 256, kCols = kNS == 1 ? 256 : 512;
};

template <int D>
__global__ void __launch_bounds__(WattnCfg<D>::kThreads, WattnCfg<D>::kCtas)
    k_wattn_fwd(const __grid_constant__ WattnFwdParams p) {
  using C = WattnCfg<D>;
  constexpr int NS = C::kNS, KR = C::kKR, VR = C::kVR;
  // The swizzled tiles want 1024-byte alignment.  Without static shared memory the
  // dynamic part starts on it; it is checked below, since two CTAs leave no room
  // to round up.
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t *qfull = bar, *qempty = bar + 1, *kfull = bar + 2, *kempty = kfull + KR, *vfull = kempty + KR,
           *vempty = vfull + VR, *sfull = vempty + VR, *pfull = sfull + NS, *pvdone = pfull + NS,
           *ofull = pvdone + 1, *oempty = ofull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + C::kBars);

  griddep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (__syncthreads_or(*reinterpret_cast<volatile int*>(&g_status))) return;   // an earlier wait gave up
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) atomicExch(&g_status, kStatusTimeout);
    return;
  }
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
          const bool narrow = n == t.narrow;
          for (int ks = 0; keys && ok && ks < C::kKPer; ++ks, ++ik) {
            const int s = ik % KR;
            if (ik >= KR && !mbar_wait(&kempty[s], ((ik / KR) - 1) & 1)) { ok = false; break; }
            mbar_arrive_expect_tx(&kfull[s], narrow ? C::kKSlot / 4 : C::kKSlot);
            for (int kb = 0; kb < C::kKBlk; ++kb)
              tma_load_4d(smem + C::kOffK + s * C::kKSlot + kb * 16384, narrow ? &p.tmK32 : &p.tmK, &kfull[s],
                          (ks * C::kKBlk + kb) * 64, j0, t.hk, t.b);
          }
          for (int vs = 0; values && ok && vs < (narrow ? 1 : C::kVPer); ++vs, ++iv) {
            const int s = iv % VR;
            if (iv >= VR && !mbar_wait(&vempty[s], ((iv / VR) - 1) & 1)) { ok = false; break; }
            mbar_arrive_expect_tx(&vfull[s], narrow ? C::kKb * 4096 : C::kVSlot);
            for (int nb = 0; nb < C::kKb; ++nb)
              tma_load_4d(smem + C::kOffV + s * C::kVSlot + nb * C::kVBox, narrow ? &p.tmV32 : &p.tmV, &vfull[s],
                          nb * 64, j0 + vs * C::kVKeys, t.hk, t.b);
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t sbase = smem_u32(smem);
      const uint64_t qd = smem_desc_sw128(sbase, 16u, 1024u), kd = smem_desc_sw128(sbase + C::kOffK, 16u, 1024u),
                     vd = smem_desc_sw128(sbase + C::kOffV, C::kVBox, 1024u);
      constexpr uint32_t ids = idesc_bf16(128, 128, false, false), ids32 = idesc_bf16(128, 32, false, false),
                         ido = idesc_bf16(128, D, false, true);
      int ik = 0, iv = 0;
      // S of the sc-th key tile in all; `n` counts from 0 in each query tile
      auto scores = [&](int sc, bool narrow) -> bool {
        const uint32_t sd = tmem + C::kColS + (sc % NS) * 128;
        const uint32_t id = narrow ? ids32 : ids;
        for (int ks = 0; ks < C::kKPer; ++ks, ++ik) {
          const int s = ik % KR;
          if (!mbar_wait(&kfull[s], (ik / KR) & 1)) return false;
          tc_fence_after();
          const uint64_t qk = here(desc_at(qd, ks * C::kKBlk * 16384)), kk = here(desc_at(kd, s * C::kKSlot));
#pragma unroll
          for (int kb = 0; kb < C::kKBlk; ++kb)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16(sd, desc_at(qk, kb * 16384 + k * 32), desc_at(kk, kb * 16384 + k * 32), id, (ks | kb | k) ? 1u : 0u);
          umma_commit(&kempty[s]);
        }
        umma_commit(&sfull[sc % NS]);
        return true;
      };
      auto output = [&](int pc, bool narrow, bool first, bool last) -> bool {
        if (!mbar_wait(&pfull[pc % NS], (pc / NS) & 1)) return false;
        const uint32_t pa = tmem + C::kColS + (pc % NS) * 128;
        for (int vs = 0; vs < (narrow ? 1 : C::kVPer); ++vs, ++iv) {
          const int s = iv % VR;
          if (!mbar_wait(&vfull[s], (iv / VR) & 1)) return false;
          tc_fence_after();
          const uint64_t vk = here(desc_at(vd, s * C::kVSlot));
#pragma unroll
          for (int k = 0; k < C::kVKeys / 16; ++k)
            if (k < 2 || !narrow)
              umma_bf16_ta(tmem + C::kColO, pa + vs * C::kVKeys / 2 + k * 8,
                           desc_at(vk, k * 2048),
                           ido, (first && vs == 0 && k == 0) ? 0u : 1u);
          umma_commit(&vempty[s]);
        }
        if (NS == 2) umma_commit(pvdone);
        if (last) umma_commit(ofull);
        return true;
      };
      int sc = 0, pc = 0, tc = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < p.ntiles; tile += gridDim.x) {
        const QueryTile t(p.a, p.nb, tile);
        if (t.count == 0) continue;
        if (!mbar_wait(qfull, tc & 1) || !scores(sc++, t.narrow == 0)) break;
        if (t.count == 1) umma_commit(qempty);
        for (int n = 0; ok && n < t.count; ++n, ++pc) {
          // S of the next key tile.  NS = 2: ahead of this one's product, over the P
          // of the last; NS = 1: behind it, over this P.  In order, so nothing waits.
          if (NS == 2 && n + 1 < t.count) ok = scores(sc++, n + 1 == t.narrow);
          if (ok && n == 0 && tc > 0 && !mbar_wait(oempty, (tc - 1) & 1)) ok = false;
          ok = ok && output(pc, n == t.narrow, n == 0, n + 1 == t.count);
          if (NS == 1 && ok && n + 1 < t.count) ok = scores(sc++, n + 1 == t.narrow);
          if (ok && n + 2 == t.count) umma_commit(qempty);
        }
        ++tc;
      }
    }
  } else {
    // ---------------------------------------------------------- softmax
    // The reference maximum of a row is raised only when a tile's maximum is
    // above it by more than 8 in log2 units; the output row in TMEM is
    // rescaled then (the whole warp: TMEM accesses are collective).  The
    // probabilities stay below 2^8, their sum in 32 bits.
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float c2 = p.a.scale * 1.4426950408889634f;
    const int window = p.a.window, sinks = p.a.sinks;
    int sc = 0, iv = 0, tc = 0, nst = 0;
    bool ok = true;
    float mx, sum;
    // one key tile; false where a wait gave up
    auto step = [&](const QueryTile& t, int n) -> bool {
      const bool narrow = n == t.narrow;
      const int cols = narrow ? 32 : 128;
      const int sb = sc % NS, j0 = t.key0(n), i = t.i0 + r, last = t.i0 + 127;
      if (!mbar_wait_warp(&sfull[sb], (sc / NS) & 1)) return false;
      tc_fence_after();
      const uint32_t ts = tq + C::kColS + sb * 128;
      const bool whole = !narrow && j0 + 127 <= t.i0 && (j0 > last - window || j0 + 127 < sinks) && last < t.len;
      const int hi = i < t.len ? i - j0 : -1, lo = i - window - j0, sk = sinks - j0;
      // W columns at a time, as far as the tile goes (a narrow one: the first W, masked
      // behind its 32).  The upper half is loaded twice, for the maximum and for the
      // exponentials: a row of 128 scores in registers spills where two CTAs share an
      // SM.  Two threads a row, which meet for the maximum, measured 137 us on the
      // ragged batch where this takes 107.
      constexpr int W = 64;
      // scores of columns [c0, c0 + W), at -inf where they are not visible
      auto load = [&](float* sv, int c0) {
#pragma unroll
        for (int c = 0; c < W; c += 32) tmem_ld32(ts + c0 + c, sv + c);
        tmem_ld_wait();
        if (!whole) {
#pragma unroll
          for (int w = 0; w < W; w += 32) {
            const uint32_t see = visible_bits(lo, hi, sk, c0 + w);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(see >> c & 1)) sv[w + c] = -INFINITY;
          }
        }
      };
      float sv[W], b4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c0 = 128 - W; c0 >= 0; c0 -= W) {
        if (c0 >= cols) continue;
        load(sv, c0);
#pragma unroll
        for (int c = 0; c < W; c += 8) {
          b4[0] = max3(b4[0], sv[c], sv[c + 1]);
          b4[1] = max3(b4[1], sv[c + 2], sv[c + 3]);
          b4[2] = max3(b4[2], sv[c + 4], sv[c + 5]);
          b4[3] = max3(b4[3], sv[c + 6], sv[c + 7]);
        }
      }
      const float bm = fmaxf(max3(b4[0], b4[1], b4[2]), b4[3]);
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
        // NS = 1: S_n came behind the last product; NS = 2: wait for it
        if (NS == 2 && !mbar_wait_warp(pvdone, (sc - 1) & 1)) return false;
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
      float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += W) {
        if (c0 >= cols) break;
        if (c0 > 0) load(sv, c0);
#pragma unroll
        for (int w = 0; w < W; w += 32) {
          uint32_t hw[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float2 e = fma_f32x2(make_float2(sv[w + 2 * c], sv[w + 2 * c + 1]), make_float2(c2, c2),
                                 make_float2(off, off));
            e.x = ex2_approx(e.x);
            e.y = ex2_approx(e.y);
            ps[c & 1] = add_f32x2(ps[c & 1], e);
            hw[c] = pack_bf16x2(e.x, e.y);   // the second product's operand: half a step, 2^-8 of each
          }
          tmem_st16u(ts + (c0 + w) / 2, hw);   // over columns that this thread has read
        }
      }
      sum += (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y);
      // value rows behind the sequence: a probability of 0 times whatever is there must stay 0
      const int per = narrow ? 1 : C::kVPer, rows = narrow ? 32 : C::kVKeys;
      if (t.len < j0 + cols) {
        for (int vs = 0; vs < per; ++vs) {
          const int s = (iv + vs) % VR, keep = max(t.len - (j0 + vs * rows), 0);
          if (!mbar_wait_warp(&vfull[s], ((iv + vs) / VR) & 1)) return false;
          const uint32_t vb = smem_u32(smem) + C::kOffV + s * C::kVSlot;
          for (int e = keep * 8 + r; e < rows * 8; e += 128)
            for (int nb = 0; nb < C::kKb; ++nb) st_shared_v4(vb + nb * C::kVBox + e * 16, 0, 0, 0, 0);
        }
        fence_async_smem();
      }
      iv += per;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[sb]);
      ++sc;
      return true;
    };
    for (int tile = blockIdx.x; ok && tile < p.ntiles; tile += gridDim.x) {
      const QueryTile t(p.a, p.nb, tile);
      mx = -INFINITY;
      sum = 0.f;
      for (int n = 0; ok && n < t.count; ++n)
        ok = step(t, n);
      if (!ok) break;
      // out = O / sum, lse = the reference maximum + log sum
      const bool in = t.q0 + r < p.a.Tq;
      const bool some = t.i0 + r < t.len;       // a token sees at least itself
      const float inv = some ? 1.0f / sum : 0.f;
      if (in)
        p.a.lse[(static_cast<int64_t>(t.b) * p.a.H + t.h) * p.a.Tq + t.q0 + r] =
            some ? fmaf(mx, p.a.scale, logf(sum)) : -INFINITY;
      if (t.count > 0) {
        if (!mbar_wait_warp(ofull, tc & 1)) break;
        ++tc;
        tc_fence_after();
      }
      // rows of 64 bytes in 64-byte swizzle; rows and channels outside are clipped by the store.
      // A warp without a row below Tq stages nothing: each step that writes a staging tile also
      // commits a group, which the wait below counts on.
      const int channels = t.q0 + quarter * 32 < p.a.Tq ? p.a.d : 0;
      const uint32_t stage = smem_u32(smem + C::kOffStage) + (warp - 2) * C::kStages * 2048;
#pragma unroll 1
      for (int c0 = 0; c0 < channels; c0 += 32, ++nst) {
        float o[32];
        if (t.count > 0) {
          __syncwarp();
          tmem_ld32(tq + C::kColO + c0, o);
          tmem_ld_wait();
        }
        const uint32_t to = stage + (nst % C::kStages) * 2048;
        if (lane == 0) {   // the store that last read this staging tile is done with it
          asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(C::kStages - 1) : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
          for (int c = 8 * g; c < 8 * g + 8; ++c) o[c] = some ? o[c] * inv : 0.f;
          st_shared_v4(to + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4), pack_bf16x2(o[8 * g], o[8 * g + 1]),
                       pack_bf16x2(o[8 * g + 2], o[8 * g + 3]), pack_bf16x2(o[8 * g + 4], o[8 * g + 5]),
                       pack_bf16x2(o[8 * g + 6], o[8 * g + 7]));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_4d(&p.tmO, to, c0, t.q0 + quarter * 32, t.h, t.b);
          bulk_commit_group();
        }
      }
      if (t.count == 0) continue;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(oempty);
    }
    if (lane == 0) bulk_wait_all();   // the last stores, before the shared memory goes
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
