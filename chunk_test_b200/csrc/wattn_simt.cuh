// wattn_simt.cuh -- the window attention with sinks in 32 bits on the CUDA
// cores: float32 inputs, products and sums (the tensor cores would round the
// operands).  Formulas and mask: wattn_common.cuh.
//
// Tiles of 32 rows (64 above d = 128) against tiles of 32 in shared memory, 4
// threads a row; small tiles, so that a short sequence fills more SMs, as long as
// two CTAs or more share one.  A thread holds 4 x 2 scores and 4 rows x (D/16)
// columns of each product that runs over the other axis.  Bound by latency where
// there are few CTAs (B 1, H 4, T 1025, d 64, window 256: dQ 54 us, dK and dV 58),
// else by the FP32 pipe and the shared-memory reads that feed it.
#pragma once

#include "wattn_common.cuh"

namespace lact {

constexpr int kSimtN = 32;

template <int D>
struct SimtCfg {
  static constexpr int kM = D <= 128 ? 32 : 64, kThreads = 4 * kM;
  static constexpr int kLd = D + 4;                     // row pitch: a row starts 4 banks after the last
  static constexpr int kMain = kM * kLd, kOther = kSimtN * kLd, kP = kM * (kSimtN + 1);
  static constexpr int kFwdSmem = (kMain + 2 * kOther + kP) * 4;
  static constexpr int kBwdSmem = (2 * kMain + 2 * kOther + 2 * kP) * 4;
  static constexpr int kC = D / 16;                     // columns of a thread
};

// rows [r0, r0 + ROWS) of a [T, d] head into shared memory; rows at or past
// `end` (or below `begin`) and channels past d become zeros
template <int ROWS, int D>
__device__ __forceinline__ void simt_load(float* dst, const float* src, int64_t st, int r0, int begin, int end, int d) {
  constexpr int kV = D / 4;
  for (int e = threadIdx.x; e < ROWS * kV; e += SimtCfg<D>::kThreads) {
    const int r = e / kV, c = (e % kV) * 4, row = r0 + r;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row >= begin && row < end && c < d) v = *reinterpret_cast<const float4*>(src + row * st + c);
    *reinterpret_cast<float4*>(dst + r * SimtCfg<D>::kLd + c) = v;
  }
}

// acc[i][j] += A[4 ty + i] . B[tx + 16 j] over D channels
template <int D>
__device__ __forceinline__ void simt_dot(const float* a, const float* b, int ty, int tx, float acc[4][2]) {
  constexpr int ld = SimtCfg<D>::kLd;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 x[4], y[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * ld + c);
#pragma unroll
    for (int j = 0; j < 2; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * ld + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, acc[i][j]))));
  }
}

// acc[i][c] += sum_n P[4 ty + i][n] B[n][column c of this thread]; columns 4 tx + 64 k + 0..3
template <int D>
__device__ __forceinline__ void simt_mul(const float* pm, const float* b, int ty, int tx, float (*acc)[SimtCfg<D>::kC]) {
  constexpr int ld = SimtCfg<D>::kLd;
#pragma unroll 2
  for (int n = 0; n < kSimtN; ++n) {
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pm[(4 * ty + i) * (kSimtN + 1) + n];
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      const float4 y = *reinterpret_cast<const float4*>(b + n * ld + 4 * tx + 64 * k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][4 * k] = fmaf(w[i], y.x, acc[i][4 * k]);
        acc[i][4 * k + 1] = fmaf(w[i], y.y, acc[i][4 * k + 1]);
        acc[i][4 * k + 2] = fmaf(w[i], y.z, acc[i][4 * k + 2]);
        acc[i][4 * k + 3] = fmaf(w[i], y.w, acc[i][4 * k + 3]);
      }
    }
  }
}

// The key tiles of kSimtN that a query tile at positions [i0, i1) sees: those
// of the sinks before the window, then the window's.
struct SimtKeys {
  int sink_tiles, first, count;   // tiles 0 .. sink_tiles - 1, then first ..
};
__device__ __forceinline__ SimtKeys simt_keys(int i0, int i1, int window, int sinks) {
  SimtKeys r;
  r.first = max(0, i0 - window + 1) / kSimtN;
  const int last = (i1 - 1) / kSimtN;
  r.sink_tiles = min((sinks + kSimtN - 1) / kSimtN, r.first);
  r.count = r.sink_tiles + last - r.first + 1;
  return r;
}

__device__ __forceinline__ bool wattn_sees(int i, int j, int window, int sinks, int len) {
  return j <= i && (j > i - window || j < sinks) && i < len;
}

template <int D>
__global__ void __launch_bounds__(SimtCfg<D>::kThreads) k_wattn_fwd_f32(const WattnParams p) {
  using C = SimtCfg<D>;
  extern __shared__ float sm[];
  float *sq = sm, *sk = sq + C::kMain, *sv = sk + C::kOther, *sp = sv + C::kOther;
  griddep_wait();
  const int bh = blockIdx.y, b = bh / p.H, h = bh % p.H, hk = h / p.group;
  const int q0 = blockIdx.x * C::kM, off = p.T - p.Tq;
  const int i0 = q0 + off, i1 = min(q0 + C::kM, p.Tq) + off;
  const int len = seq_len(p, b), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float* q = static_cast<const float*>(p.q.p) + b * p.q.sb + h * p.q.sh;
  const float* k = static_cast<const float*>(p.k.p) + b * p.k.sb + hk * p.k.sh;
  const float* v = static_cast<const float*>(p.v.p) + b * p.v.sb + hk * p.v.sh;
  simt_load<C::kM, D>(sq, q, p.q.st, q0, 0, min(p.Tq, len - off), p.d);
  float acc[4][C::kC], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < C::kC; ++c) acc[i][c] = 0.f;
  }
  const SimtKeys keys = simt_keys(i0, min(i1, max(len, i0 + 1)), p.window, p.sinks);
  const int tiles = i0 < len ? keys.count : 0;
  for (int n = 0; n < tiles; ++n) {
    const int j0 = (n < keys.sink_tiles ? n : keys.first + n - keys.sink_tiles) * kSimtN;
    __syncthreads();
    simt_load<kSimtN, D>(sk, k, p.k.st, j0, 0, len, p.d);
    simt_load<kSimtN, D>(sv, v, p.v.st, j0, 0, len, p.d);
    __syncthreads();
    float s[4][2] = {};
    simt_dot<D>(sq, sk, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i0 + 4 * ty + i;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s[i][j] = wattn_sees(row, j0 + tx + 16 * j, p.window, p.sinks, len) ? s[i][j] * p.scale : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mn = fmaxf(m[i], top);
      const float base = mn == -INFINITY ? 0.f : mn, fix = expf(m[i] - base);
      m[i] = mn;
      float add = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float e = expf(s[i][j] - base);
        add += e;
        sp[(4 * ty + i) * (kSimtN + 1) + tx + 16 * j] = e;
      }
#pragma unroll
      for (int x = 8; x; x >>= 1) add += __shfl_xor_sync(0xffffffffu, add, x);
      l[i] = l[i] * fix + add;
#pragma unroll
      for (int c = 0; c < C::kC; ++c) acc[i][c] *= fix;
    }
    __syncwarp();   // a warp reads only the rows of P that it wrote
    simt_mul<D>(sp, sv, ty, tx, acc);
  }
  griddep_launch();   // not before: the next kernel's blocks would pile up on the SMs that this one leaves free
  float* o = static_cast<float*>(p.out.p) + b * p.out.sb + h * p.out.sh;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + 4 * ty + i;
    if (row >= p.Tq) break;
    const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
    for (int k4 = 0; k4 < D / 64; ++k4) {
      const int c = 4 * tx + 64 * k4;
      if (c < p.d)
        *reinterpret_cast<float4*>(o + row * p.out.st + c) =
            make_float4(acc[i][4 * k4] * inv, acc[i][4 * k4 + 1] * inv, acc[i][4 * k4 + 2] * inv, acc[i][4 * k4 + 3] * inv);
    }
    if (tx == 0) p.lse[static_cast<int64_t>(bh) * p.Tq + row] = l[i] > 0.f ? m[i] + logf(l[i]) : -INFINITY;
  }
}

// delta[b, h, t] = sum_c dout out in 32 bits; 0 past the length.  LANES lanes of
// a warp per row, 16 bytes each at a time.
template <typename T, int LANES>
__global__ void __launch_bounds__(256) k_wattn_delta(const WattnParams p) {
  griddep_launch();
  griddep_wait();
  const int64_t rows = static_cast<int64_t>(p.B) * p.H * p.Tq;
  constexpr int kV = 16 / sizeof(T), kRows = 256 / LANES;
  const int lane = threadIdx.x % LANES;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t row = r0 + threadIdx.x / LANES;
    float s = 0.f;
    if (row < rows) {
      const int t = static_cast<int>(row % p.Tq), bh = static_cast<int>(row / p.Tq), b = bh / p.H, h = bh % p.H;
      if (t + p.T - p.Tq < seq_len(p, b)) {
        const T* o = static_cast<const T*>(p.out.p) + b * p.out.sb + h * p.out.sh + t * p.out.st;
        const T* g = static_cast<const T*>(p.dout.p) + b * p.dout.sb + h * p.dout.sh + t * p.dout.st;
        for (int c = lane * kV; c < p.d; c += LANES * kV) {
          float x[kV], y[kV];
          load_vec<kV>(o + c, x);
          load_vec<kV>(g + c, y);
#pragma unroll
          for (int i = 0; i < kV; ++i) s = fmaf(x[i], y[i], s);
        }
      }
    }
#pragma unroll
    for (int x = LANES / 2; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (row < rows && lane == 0) p.delta[row] = s;
  }
}

// dQ of kM queries: over the key tiles, P = exp(S - lse), dS = P (dO V^T - delta) scale, dQ += dS K.
template <int D>
__global__ void __launch_bounds__(SimtCfg<D>::kThreads) k_wattn_dq_f32(const WattnParams p) {
  using C = SimtCfg<D>;
  extern __shared__ float sm[];
  float *sq = sm, *sg = sq + C::kMain, *sk = sg + C::kMain, *sv = sk + C::kOther, *sp = sv + C::kOther;
  griddep_wait();
  const int bh = blockIdx.y, b = bh / p.H, h = bh % p.H, hk = h / p.group;
  const int q0 = blockIdx.x * C::kM, off = p.T - p.Tq;
  const int i0 = q0 + off, i1 = min(q0 + C::kM, p.Tq) + off;
  const int len = seq_len(p, b), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float* q = static_cast<const float*>(p.q.p) + b * p.q.sb + h * p.q.sh;
  const float* g = static_cast<const float*>(p.dout.p) + b * p.dout.sb + h * p.dout.sh;
  const float* k = static_cast<const float*>(p.k.p) + b * p.k.sb + hk * p.k.sh;
  const float* v = static_cast<const float*>(p.v.p) + b * p.v.sb + hk * p.v.sh;
  const int qend = min(p.Tq, len - off);
  simt_load<C::kM, D>(sq, q, p.q.st, q0, 0, qend, p.d);
  simt_load<C::kM, D>(sg, g, p.dout.st, q0, 0, qend, p.d);
  float acc[4][C::kC] = {}, lse[4], del[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + 4 * ty + i;
    lse[i] = row < qend ? p.lse[static_cast<int64_t>(bh) * p.Tq + row] : 0.f;
    del[i] = row < qend ? p.delta[static_cast<int64_t>(bh) * p.Tq + row] : 0.f;
  }
  const SimtKeys keys = simt_keys(i0, min(i1, max(len, i0 + 1)), p.window, p.sinks);
  const int tiles = i0 < len ? keys.count : 0;
  for (int n = 0; n < tiles; ++n) {
    const int j0 = (n < keys.sink_tiles ? n : keys.first + n - keys.sink_tiles) * kSimtN;
    __syncthreads();
    simt_load<kSimtN, D>(sk, k, p.k.st, j0, 0, len, p.d);
    simt_load<kSimtN, D>(sv, v, p.v.st, j0, 0, len, p.d);
    __syncthreads();
    float s[4][2] = {}, dp[4][2] = {};
    simt_dot<D>(sq, sk, ty, tx, s);
    simt_dot<D>(sg, sv, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool see = wattn_sees(i0 + 4 * ty + i, j0 + tx + 16 * j, p.window, p.sinks, len);
        const float pr = see ? expf(s[i][j] * p.scale - lse[i]) : 0.f;
        sp[(4 * ty + i) * (kSimtN + 1) + tx + 16 * j] = see ? pr * (dp[i][j] - del[i]) * p.scale : 0.f;
      }
    __syncwarp();
    simt_mul<D>(sp, sk, ty, tx, acc);
  }
  griddep_launch();
  float* o = static_cast<float*>(p.dq.p) + b * p.dq.sb + h * p.dq.sh;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = q0 + 4 * ty + i;
    if (row >= p.Tq) break;
#pragma unroll
    for (int k4 = 0; k4 < D / 64; ++k4) {
      const int c = 4 * tx + 64 * k4;
      if (c < p.d)
        *reinterpret_cast<float4*>(o + row * p.dq.st + c) =
            make_float4(acc[i][4 * k4], acc[i][4 * k4 + 1], acc[i][4 * k4 + 2], acc[i][4 * k4 + 3]);
    }
  }
}

// dK, dV of kM keys over one part of the query positions (KeyPart) and the
// group's heads: dV += P^T dO, dK += dS^T Q.  A sink tile's parts go to
// `part` [B Hkv][sink tiles][parts][2][kM][D], the others to dk and dv.
template <int D>
__global__ void __launch_bounds__(SimtCfg<D>::kThreads) k_wattn_dkv_f32(const WattnParams p, int sink_tiles, int parts) {
  using C = SimtCfg<D>;
  extern __shared__ float sm[];
  float *sk = sm, *sv = sk + C::kMain, *sq = sv + C::kMain, *sg = sq + C::kOther, *sp = sg + C::kOther, *sd = sp + C::kP;
  griddep_wait();
  // blockIdx.x: the sink tiles' parts first, then the other tiles
  const int item = blockIdx.x, split = sink_tiles * parts;
  const int kt = item < split ? item / parts : item - split + sink_tiles;
  const int part = item < split ? item % parts : 0;
  const int bk = blockIdx.y, b = bk / p.Hkv, hk = bk % p.Hkv;
  const int j0 = kt * C::kM, off = p.T - p.Tq, len = seq_len(p, b);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const KeyPart kp = key_part(kt, part, C::kM, p.window, p.T, p.far_rows);
  const int lo = max(kp.lo, off), hi = min(kp.hi, len);
  const float* k = static_cast<const float*>(p.k.p) + b * p.k.sb + hk * p.k.sh;
  const float* v = static_cast<const float*>(p.v.p) + b * p.v.sb + hk * p.v.sh;
  simt_load<C::kM, D>(sk, k, p.k.st, j0, 0, len, p.d);
  simt_load<C::kM, D>(sv, v, p.v.st, j0, 0, len, p.d);
  float ak[4][C::kC] = {}, av[4][C::kC] = {};
  for (int h = hk * p.group; h < (hk + 1) * p.group; ++h) {
    const float* q = static_cast<const float*>(p.q.p) + b * p.q.sb + h * p.q.sh;
    const float* g = static_cast<const float*>(p.dout.p) + b * p.dout.sb + h * p.dout.sh;
    const int64_t row0 = (static_cast<int64_t>(b) * p.H + h) * p.Tq;
    for (int i0 = lo; i0 < hi; i0 += kSimtN) {
      __syncthreads();
      simt_load<kSimtN, D>(sq, q, p.q.st, i0 - off, 0, hi - off, p.d);
      simt_load<kSimtN, D>(sg, g, p.dout.st, i0 - off, 0, hi - off, p.d);
      __syncthreads();
      float s[4][2] = {}, dp[4][2] = {};
      simt_dot<D>(sk, sq, ty, tx, s);
      simt_dot<D>(sv, sg, ty, tx, dp);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = i0 + tx + 16 * j;
        const float lse = i < hi ? p.lse[row0 + i - off] : 0.f, del = i < hi ? p.delta[row0 + i - off] : 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool see = i < hi && wattn_sees(i, j0 + 4 * ty + r, p.window, p.sinks, len);
          const float pr = see ? expf(s[r][j] * p.scale - lse) : 0.f;
          sp[(4 * ty + r) * (kSimtN + 1) + tx + 16 * j] = pr;
          sd[(4 * ty + r) * (kSimtN + 1) + tx + 16 * j] = see ? pr * (dp[r][j] - del) * p.scale : 0.f;
        }
      }
      __syncwarp();
      simt_mul<D>(sp, sg, ty, tx, av);
      simt_mul<D>(sd, sq, ty, tx, ak);
    }
  }
  griddep_launch();
  const bool direct = kt >= sink_tiles;
  float* po = direct ? nullptr
                     : p.part + ((static_cast<int64_t>(bk) * sink_tiles + kt) * parts + part) * 2 * C::kM * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = j0 + 4 * ty + i;
#pragma unroll
    for (int k4 = 0; k4 < D / 64; ++k4) {
      const int c = 4 * tx + 64 * k4;
      const float4 x = make_float4(ak[i][4 * k4], ak[i][4 * k4 + 1], ak[i][4 * k4 + 2], ak[i][4 * k4 + 3]);
      const float4 y = make_float4(av[i][4 * k4], av[i][4 * k4 + 1], av[i][4 * k4 + 2], av[i][4 * k4 + 3]);
      if (!direct) {
        *reinterpret_cast<float4*>(po + (4 * ty + i) * D + c) = x;
        *reinterpret_cast<float4*>(po + (C::kM + 4 * ty + i) * D + c) = y;
      } else if (row < p.T && c < p.d) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.dk.p) + b * p.dk.sb + hk * p.dk.sh + row * p.dk.st + c) = x;
        *reinterpret_cast<float4*>(static_cast<float*>(p.dv.p) + b * p.dv.sb + hk * p.dv.sh + row * p.dv.st + c) = y;
      }
    }
  }
}

// The sink tiles' gradients: the sum of their parts, in order, one rounding.
// part [B Hkv][sink tiles][parts][2][bn][DP], DP the padded head dim.
template <typename T>
__global__ void __launch_bounds__(256) k_wattn_sink_sums(const WattnParams p, int sink_tiles, int parts, int bn, int DP) {
  griddep_launch();
  griddep_wait();
  const int64_t plane = static_cast<int64_t>(bn) * DP;
  const int vecs = DP / 4;
  const int64_t n = static_cast<int64_t>(p.B) * p.Hkv * sink_tiles * 2 * bn * vecs;
  for (int64_t e = blockIdx.x * 256 + threadIdx.x; e < n; e += static_cast<int64_t>(gridDim.x) * 256) {
    const int c = static_cast<int>(e % vecs) * 4, r = static_cast<int>(e / vecs % bn);
    const int which = static_cast<int>(e / vecs / bn % 2);
    const int kt = static_cast<int>(e / vecs / bn / 2 % sink_tiles), bk = static_cast<int>(e / vecs / bn / 2 / sink_tiles);
    const int row = kt * bn + r;
    if (row >= p.T || c >= p.d) continue;
    const float* src = p.part + (static_cast<int64_t>(bk) * sink_tiles + kt) * parts * 2 * plane + which * plane +
                       static_cast<int64_t>(r) * DP + c;
    float4 s = *reinterpret_cast<const float4*>(src);
    for (int k = 1; k < parts; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(src + k * 2 * plane);
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    const View4& o = which ? p.dv : p.dk;
    T* dst = static_cast<T*>(o.p) + bk / p.Hkv * o.sb + bk % p.Hkv * o.sh + row * o.st + c;
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(dst) = s;
    else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

}  // namespace lact
