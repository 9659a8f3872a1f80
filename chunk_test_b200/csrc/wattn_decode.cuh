// wattn_decode.cuh -- the window attention with sinks for one new token per
// sequence, over a rolling cache.
//
// The cache of a key head holds sinks + window slots: the token at position p
// is in slot p when p < sinks, else in slot sinks + (p - sinks) % window.  A
// sequence that has seen `pos` tokens writes the new one (position pos) into
// its slot and attends to all min(pos + 1, sinks + window) filled slots: these
// are exactly the visible keys.  No CTA reads the new token's slot from the
// cache; its key and value come from the call's k and v, so the CTA that
// writes the slot races with nobody.
//
// Bound by HBM (each key and value is read once for up to 8 of the group's heads,
// again for each 8 more) and, for few sequences, by latency: the slots of one (sequence, key head)
// are split over a thread-block cluster, whose CTAs join their softmax
// statistics and sums through distributed shared memory in rank order -- one
// launch, no workspace, no atomics, the same bits on every run.  Measured: 64
// sequences of 0 to 16512 tokens, 12 heads on 4, d 128, window 8192: 157 us, 5.1
// TB/s; one sequence, 6 heads, d 256, window 2048: 8.7 us in a graph of such calls,
// of which 2 are bytes.
#pragma once

#include <cooperative_groups.h>

#include "swa_flash.cuh"
#include "wattn_common.cuh"

namespace lact {

constexpr int kDecThreads = 256, kDecWarps = 8, kDecHeads = 8;

struct DecodeParams {
  View4 q, out, kn, vn;        // [B, H, 1, d], [B, Hkv, 1, d]; st unused
  void *kc, *vc;               // [B, Hkv, sinks + window, d]
  const int* seen;             // [B]
  float scale;
  int H, Hkv, group, d, window, sinks, hgroups;   // hgroups: blocks of 8 heads of a group
};

struct DecodeSlots {
  int b, hk, h0, heads;        // sequence, key head, first query head, query heads of this CTA
  int pos, fresh;              // the new token's position and slot
  int lo, hi;                  // slots of this CTA
};

__device__ __forceinline__ DecodeSlots decode_slots(const DecodeParams& p, int rank, int ranks) {
  DecodeSlots s;
  const int item = blockIdx.y;
  const int hg = item % p.hgroups, bk = item / p.hgroups;
  s.b = bk / p.Hkv;
  s.hk = bk % p.Hkv;
  s.h0 = s.hk * p.group + hg * kDecHeads;
  s.heads = min(kDecHeads, p.group - hg * kDecHeads);
  s.pos = p.seen[s.b];
  s.fresh = s.pos < p.sinks ? s.pos : p.sinks + (s.pos - p.sinks) % p.window;
  const int n = static_cast<int>(min(static_cast<int64_t>(s.pos) + 1, static_cast<int64_t>(p.sinks) + p.window));
  const int per = ((n + ranks - 1) / ranks + 15) / 16 * 16;
  s.lo = min(rank * per, n);
  s.hi = min(s.lo + per, n);
  return s;
}

__device__ __forceinline__ void mma_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A load that is used once.  Not the non-coherent path: the last step's kernel may
// still write its token while this one starts (it waits before its first load).
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// One warp's statistics and sums over its slots: m, l [8 heads], acc [8][DP]
// in shared memory; then the CTA's, then the cluster's.  Scores are in log2
// units.  `wm`, `wl` [warps][8], `wacc` [warps][8][DP].
template <typename T, int DP>
__device__ __forceinline__ void decode_join(const DecodeParams& p, const DecodeSlots& s, float* wm, float* wl,
                                            float* wacc, int rank, int ranks) {
  namespace cg = cooperative_groups;
  __shared__ float cm[kDecHeads], cl[kDecHeads], fac[kDecWarps][kDecHeads];
  __syncthreads();
  if (threadIdx.x < kDecHeads) {
    const int h = threadIdx.x;
    float m = -INFINITY;
    for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, wm[w * kDecHeads + h]);
    float l = 0.f;
    for (int w = 0; w < kDecWarps; ++w) {
      const float f = wm[w * kDecHeads + h] == -INFINITY ? 0.f : exp2f(wm[w * kDecHeads + h] - m);
      fac[w][h] = f;
      l += f * wl[w * kDecHeads + h];
    }
    cm[h] = m;
    cl[h] = l;
  }
  __syncthreads();
  // the CTA's sums, in place of warp 0's
  for (int e = threadIdx.x; e < s.heads * DP; e += kDecThreads) {
    const int h = e / DP;
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) x += fac[w][h] * wacc[w * kDecHeads * DP + e];
    wacc[e] = x;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  const int n = s.heads * DP, per = (n + ranks - 1) / ranks;
  T* out = static_cast<T*>(p.out.p) + s.b * p.out.sb + s.h0 * p.out.sh;
  for (int e = rank * per + threadIdx.x; e < min(n, (rank + 1) * per); e += kDecThreads) {
    const int h = e / DP, c = e % DP;
    float m = -INFINITY;
    for (int r = 0; r < ranks; ++r) m = fmaxf(m, *cluster.map_shared_rank(&cm[h], r));
    float x = 0.f, l = 0.f;
    for (int r = 0; r < ranks; ++r) {
      const float rm = *cluster.map_shared_rank(&cm[h], r);
      const float f = rm == -INFINITY ? 0.f : exp2f(rm - m);
      l += f * *cluster.map_shared_rank(&cl[h], r);
      x += f * *cluster.map_shared_rank(&wacc[e], r);
    }
    if (c < p.d) {
      const float y = x / l;
      if constexpr (sizeof(T) == 4) out[h * p.out.sh + c] = y;
      else out[h * p.out.sh + c] = __float2bfloat16(y);
    }
  }
  cluster.sync();   // no CTA leaves while another reads its shared memory
}

// A sequence with a negative count is inactive: out 0, its cache untouched.
template <typename T>
__device__ __forceinline__ bool decode_inactive(const DecodeParams& p, const DecodeSlots& s, int rank) {
  if (s.pos >= 0) return false;
  if (rank == 0) {
    T* out = static_cast<T*>(p.out.p) + s.b * p.out.sb + s.h0 * p.out.sh;
    for (int e = threadIdx.x; e < s.heads * p.d; e += kDecThreads) out[e / p.d * p.out.sh + e % p.d] = T(0.f);
  }
  return true;
}

// the new token into its slot, by the last CTA of the first block of heads
template <typename T>
__device__ __forceinline__ void decode_write(const DecodeParams& p, const DecodeSlots& s, const T* kn, const T* vn,
                                             T* kc, T* vc) {
  constexpr int kV = 16 / sizeof(T);
  for (int e = threadIdx.x; e < 2 * (p.d / kV); e += kDecThreads) {
    const int c = (e >> 1) * kV;
    const int64_t to = static_cast<int64_t>(s.fresh) * p.d + c;
    if (e & 1) *reinterpret_cast<uint4*>(vc + to) = *reinterpret_cast<const uint4*>(vn + c);
    else *reinterpret_cast<uint4*>(kc + to) = *reinterpret_cast<const uint4*>(kn + c);
  }
}

// bf16: a warp takes 16 slots at a time.  The scores of up to 8 heads are one
// 16 x 8 product per 8 slots and 16 channels (mma.sync: rows are heads, the
// upper eight empty), the output 16 channels x 8 heads per 16 slots, with the
// channels permuted so that every lane's operands are 16-byte loads straight
// from the cache: nothing is staged.  Tensor throughput is no limit here; the
// instruction is used because 8 heads on the CUDA cores would be.
template <int DP>
__global__ void __launch_bounds__(kDecThreads, DP <= 128 ? 2 : 1) k_wattn_decode_bf16(const DecodeParams p) {
  using B16 = __nv_bfloat16;
  extern __shared__ float dec_smem[];
  float *wm = dec_smem, *wl = wm + kDecWarps * kDecHeads, *wacc = wl + kDecWarps * kDecHeads;
  griddep_launch();
  griddep_wait();
  const int rank = blockIdx.x, ranks = gridDim.x;
  const DecodeSlots s = decode_slots(p, rank, ranks);
  if (decode_inactive<B16>(p, s, rank)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t head = (static_cast<int64_t>(s.b) * p.Hkv + s.hk) * (static_cast<int64_t>(p.sinks) + p.window) * p.d;
  B16 *kc = static_cast<B16*>(p.kc) + head, *vc = static_cast<B16*>(p.vc) + head;
  const B16* kn = static_cast<const B16*>(p.kn.p) + s.b * p.kn.sb + s.hk * p.kn.sh;
  const B16* vn = static_cast<const B16*>(p.vn.p) + s.b * p.vn.sb + s.hk * p.vn.sh;
  if (rank == ranks - 1 && s.h0 == s.hk * p.group) decode_write<B16>(p, s, kn, vn, kc, vc);

  // q of head g, channels 32 kk + 8 t .. + 7: the rows of the scores' product
  uint4 qr[DP / 32];
  const B16* qp = static_cast<const B16*>(p.q.p) + s.b * p.q.sb + (s.h0 + g) * p.q.sh;
#pragma unroll
  for (int kk = 0; kk < DP / 32; ++kk) {
    const int c = 32 * kk + 8 * t;
    qr[kk] = (g < s.heads && c < p.d) ? *reinterpret_cast<const uint4*>(qp + c) : make_uint4(0, 0, 0, 0);
  }
  const float c2 = p.scale * 1.4426950408889634f;
  float acc[DP / 64][4][4] = {};
  float m = -INFINITY, l = 0.f;   // of head g (l: this lane's slots)
  for (int s0 = s.lo + warp * 16; s0 < s.hi; s0 += kDecWarps * 16) {
    uint4 kr[2][DP / 32], vr[4][DP / 64];
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
      const int slot = s0 + nb * 8 + g;
      const B16* row = slot == s.fresh ? kn : kc + static_cast<int64_t>(slot) * p.d;
#pragma unroll
      for (int kk = 0; kk < DP / 32; ++kk) {
        const int c = 32 * kk + 8 * t;
        kr[nb][kk] = (slot < s.hi && c < p.d) ? ld_stream(row + c) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int slot = s0 + 2 * t + (i & 1) + (i >> 1) * 8;
      const B16* row = slot == s.fresh ? vn : vc + static_cast<int64_t>(slot) * p.d;
#pragma unroll
      for (int vg = 0; vg < DP / 64; ++vg) {
        const int c = 64 * vg + 8 * g;
        // slots past the end: zeros, whatever the cache holds there
        vr[i][vg] = (slot < s.hi && c < p.d) ? ld_stream(row + c) : make_uint4(0, 0, 0, 0);
      }
    }
    float sc[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < DP / 32; ++kk)
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        mma_16816(sc[nb], qr[kk].x, 0u, qr[kk].y, 0u, kr[nb][kk].x, kr[nb][kk].y);
        mma_16816(sc[nb], qr[kk].z, 0u, qr[kk].w, 0u, kr[nb][kk].z, kr[nb][kk].w);
      }
    float top = -INFINITY;
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sc[nb][i] = s0 + nb * 8 + 2 * t + i < s.hi ? sc[nb][i] * c2 : -INFINITY;
        top = fmaxf(top, sc[nb][i]);
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
    const float fix = ex2_approx(m - base);
    m = mn;
    float e[2][2];
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) e[nb][i] = ex2_approx(sc[nb][i] - base);
    l = l * fix + ((e[0][0] + e[0][1]) + (e[1][0] + e[1][1]));
    // the products' probabilities in bf16 (half a step, 2^-8 of each); the sum keeps 32 bits
    const uint32_t p0 = pack_bf16x2(e[0][0], e[0][1]), p1 = pack_bf16x2(e[1][0], e[1][1]);
    if (__any_sync(0xffffffffu, fix != 1.f)) {
      const float f0 = __shfl_sync(0xffffffffu, fix, 8 * t), f1 = __shfl_sync(0xffffffffu, fix, 8 * t + 4);
#pragma unroll
      for (int vg = 0; vg < DP / 64; ++vg)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[vg][i][0] *= f0; acc[vg][i][1] *= f1; acc[vg][i][2] *= f0; acc[vg][i][3] *= f1;
        }
    }
#pragma unroll
    for (int vg = 0; vg < DP / 64; ++vg) {
      const uint32_t* r0 = reinterpret_cast<const uint32_t*>(&vr[0][vg]);
      const uint32_t* r1 = reinterpret_cast<const uint32_t*>(&vr[1][vg]);
      const uint32_t* r2 = reinterpret_cast<const uint32_t*>(&vr[2][vg]);
      const uint32_t* r3 = reinterpret_cast<const uint32_t*>(&vr[3][vg]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // rows: channel 8 g + i and 8 g + 4 + i of the group of 64
        const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
        mma_16816(acc[vg][i], __byte_perm(r0[i / 2], r1[i / 2], sel), __byte_perm(r0[2 + i / 2], r1[2 + i / 2], sel),
                  __byte_perm(r2[i / 2], r3[i / 2], sel), __byte_perm(r2[2 + i / 2], r3[2 + i / 2], sel), p0, p1);
      }
    }
  }
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (t == 0) {
    wm[warp * kDecHeads + g] = m;
    wl[warp * kDecHeads + g] = l;
  }
  float* wa = wacc + warp * kDecHeads * DP;
#pragma unroll
  for (int vg = 0; vg < DP / 64; ++vg)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 64 * vg + 8 * g + i;
      wa[(2 * t) * DP + c] = acc[vg][i][0];
      wa[(2 * t + 1) * DP + c] = acc[vg][i][1];
      wa[(2 * t) * DP + c + 4] = acc[vg][i][2];
      wa[(2 * t + 1) * DP + c + 4] = acc[vg][i][3];
    }
  decode_join<B16, DP>(p, s, wm, wl, wacc, rank, ranks);
}

// float32: a warp takes one slot at a time, a lane DP/32 of its channels;
// products and sums in 32 bits.  GH: heads computed, at least this CTA's.
template <int DP, int GH>
__global__ void __launch_bounds__(kDecThreads, 1) k_wattn_decode_f32(const DecodeParams p) {
  extern __shared__ float dec_smem[];
  float *wm = dec_smem, *wl = wm + kDecWarps * kDecHeads, *wacc = wl + kDecWarps * kDecHeads;
  griddep_launch();
  griddep_wait();
  const int rank = blockIdx.x, ranks = gridDim.x;
  const DecodeSlots s = decode_slots(p, rank, ranks);
  if (decode_inactive<float>(p, s, rank)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t head = (static_cast<int64_t>(s.b) * p.Hkv + s.hk) * (static_cast<int64_t>(p.sinks) + p.window) * p.d;
  float *kc = static_cast<float*>(p.kc) + head, *vc = static_cast<float*>(p.vc) + head;
  const float* kn = static_cast<const float*>(p.kn.p) + s.b * p.kn.sb + s.hk * p.kn.sh;
  const float* vn = static_cast<const float*>(p.vn.p) + s.b * p.vn.sb + s.hk * p.vn.sh;
  if (rank == ranks - 1 && s.h0 == s.hk * p.group) decode_write<float>(p, s, kn, vn, kc, vc);
  constexpr int kC = DP / 64;   // pairs of channels 2 lane + 64 i
  float2 q[GH][kC], acc[GH][kC] = {};
  float m[GH], l[GH];
  const float* qp = static_cast<const float*>(p.q.p) + s.b * p.q.sb + s.h0 * p.q.sh;
#pragma unroll
  for (int h = 0; h < GH; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 2 * lane + 64 * i;
      q[h][i] = (h < s.heads && c < p.d) ? *reinterpret_cast<const float2*>(qp + h * p.q.sh + c) : make_float2(0.f, 0.f);
    }
  }
  const float c2 = p.scale * 1.4426950408889634f;
  constexpr int kU = 4;   // slots in flight
  for (int s0 = s.lo + warp * kU; s0 < s.hi; s0 += kDecWarps * kU) {
    float2 kr[kU][kC], vr[kU][kC];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int slot = s0 + j;
      const float* kp = slot == s.fresh ? kn : kc + static_cast<int64_t>(slot) * p.d;
      const float* vp = slot == s.fresh ? vn : vc + static_cast<int64_t>(slot) * p.d;
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int c = 2 * lane + 64 * i;
        const bool in = slot < s.hi && c < p.d;
        kr[j][i] = in ? *reinterpret_cast<const float2*>(kp + c) : make_float2(0.f, 0.f);
        vr[j][i] = in ? *reinterpret_cast<const float2*>(vp + c) : make_float2(0.f, 0.f);
      }
    }
#pragma unroll
    for (int h = 0; h < GH; ++h) {
      float x[kU];
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        x[j] = 0.f;
#pragma unroll
        for (int i = 0; i < kC; ++i) x[j] = fmaf(q[h][i].y, kr[j][i].y, fmaf(q[h][i].x, kr[j][i].x, x[j]));
      }
#pragma unroll
      for (int w = 16; w; w >>= 1)
#pragma unroll
        for (int j = 0; j < kU; ++j) x[j] += __shfl_xor_sync(0xffffffffu, x[j], w);
      float top = m[h];
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        x[j] = s0 + j < s.hi ? x[j] * c2 : -INFINITY;
        top = fmaxf(top, x[j]);
      }
      const float base = top == -INFINITY ? 0.f : top, fix = exp2f(m[h] - base);
      m[h] = top;
      l[h] *= fix;
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        acc[h][i].x *= fix;
        acc[h][i].y *= fix;
      }
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        const float e = exp2f(x[j] - base);
        l[h] += e;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          acc[h][i].x = fmaf(e, vr[j][i].x, acc[h][i].x);
          acc[h][i].y = fmaf(e, vr[j][i].y, acc[h][i].y);
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < GH; ++h) {
    if (lane == 0) {
      wm[warp * kDecHeads + h] = m[h];
      wl[warp * kDecHeads + h] = l[h];
    }
#pragma unroll
    for (int i = 0; i < kC; ++i)
      *reinterpret_cast<float2*>(wacc + (warp * kDecHeads + h) * DP + 2 * lane + 64 * i) = acc[h][i];
  }
  decode_join<float, DP>(p, s, wm, wl, wacc, rank, ranks);
}

// A prompt's keys and values into the cache: positions below the sinks and the
// last `window` others, each into its slot; other slots keep what they hold.
struct FillParams {
  View4 k, v;                  // [B, Hkv, T, d]
  void *kc, *vc;
  const int* lengths;          // [B] or null
  int64_t n;                   // rows that can be written: B Hkv min(T, sinks + window)
  int Hkv, T, row_vecs, window, sinks, esz;
};
__global__ void __launch_bounds__(256) k_wattn_fill(const FillParams p) {
  griddep_launch();
  griddep_wait();
  const int64_t slots = static_cast<int64_t>(p.sinks) + p.window;
  const int most = static_cast<int>(min(static_cast<int64_t>(p.T), slots));
  const int64_t n = p.n * p.row_vecs;
  for (int64_t e = blockIdx.x * 256LL + threadIdx.x; e < n; e += gridDim.x * 256LL) {
    const int c = static_cast<int>(e % p.row_vecs);
    const int r = static_cast<int>(e / p.row_vecs % most), bk = static_cast<int>(e / p.row_vecs / most);
    const int b = bk / p.Hkv, hk = bk % p.Hkv;
    const int len = p.lengths ? max(0, min(p.lengths[b], p.T)) : p.T;
    // row r: the r-th of the sequence's kept positions
    const int skip = max(0, len - static_cast<int>(min(slots, static_cast<int64_t>(p.T))));
    const int pos = r < p.sinks ? r : r + skip;
    if (pos >= len) continue;
    const int64_t slot = pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % p.window;
    const int64_t to = ((static_cast<int64_t>(bk) * slots + slot) * p.row_vecs + c) * 16;
    const int64_t kf = (b * p.k.sb + hk * p.k.sh + pos * p.k.st) * p.esz + c * 16;
    const int64_t vf = (b * p.v.sb + hk * p.v.sh + pos * p.v.st) * p.esz + c * 16;
    *reinterpret_cast<uint4*>(static_cast<char*>(p.kc) + to) = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.k.p) + kf);
    *reinterpret_cast<uint4*>(static_cast<char*>(p.vc) + to) = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.v.p) + vf);
  }
}

}  // namespace lact
