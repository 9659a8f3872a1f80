// rotary_kernels.cuh -- rotary positions of the block's queries and keys, with
// the per head and channel scales and offsets of its attention half
// ("LaCT架构核心思想解析" §1.1) in the same pass, and the backward of both.
//
// Forward, per head h and token at position p, x' = x * scale[h] + offset[h],
// then for each rotated pair i (channels (2i, 2i+1), or (i, i + rot/2) in the
// half layout) with the angle t = p * freqs[i]:
//   y_a = amp (x'_a cos t - x'_b sin t),  y_b = amp (x'_b cos t + x'_a sin t);
// channels from rot on are x'.  Backward: g = the rotation by -t of dy (times
// amp), dx = g * scale, dscale = sum_{b,t} g x, doffset = sum_{b,t} g.
//
// Bound by HBM: each element is read and written once (the backward of the
// scales also reads x).  A thread owns a few channels of one head and walks the
// block's tokens, so scales, offsets and their gradients' sums stay in its
// registers; the angles of a tile of tokens are formed once per block, in
// shared memory, for all of its heads: p * freqs[i] in 64 bits, because a
// position of 10^6 leaves a 32-bit product only 4 bits below the turn, then
// the fraction of the turn goes to sincospif in 32.
#pragma once

#include "sm100.cuh"

namespace lact {

// One [B, heads, T, d] tensor: channels contiguous, strides in elements.
struct View4 {
  void* p;
  int64_t sb, sh, st;
};

constexpr int kRotaryThreads = 384;    // of a block, 512 where a thread owns single channels
constexpr int kRotaryTile = 16;        // tokens whose angles are held at a time
// upper half of the turn that marks the pairs which pad a row's last vector: a NaN
// of its own, so that a frequency that is not a number is still one
constexpr int kPadTurn = 0x7ff85ad0;

struct RotaryParams {
  View4 xq, xk;            // forward: inputs; backward: inputs, for the scales' gradients (else null)
  View4 yq, yk;            // forward: outputs; backward: the outputs' gradients
  View4 dq, dk;            // backward: the inputs' gradients
  const double* freqs;     // [rot / 2], radians per position
  const int* positions;    // [B, T] or null: start + t
  const float *q_scale, *q_offset, *k_scale, *k_offset;   // [H, d], [Hkv, d] or null
  float* partial;          // backward of the scales: [blocks][2][H + Hkv][d]
  int64_t start;
  int64_t T;
  int B, H, Hkv, d, rot;
  int units, rot_units;    // threads of a head; those that rotate
  int rows;                // heads of a block
  int per_block, ranges;   // tokens of a block, blocks of a sequence
  float amp;
};

template <int V>
__device__ __forceinline__ void load_vec(const float* p, float* x) {
  static_assert(V == 4, "16 bytes");
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float* x) {
  if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else *p = x[0];
}
template <int V>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float* x) {
  static_assert(V == 8, "16 bytes");
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// the one rounding of a bf16 result: to nearest, ties to even
template <int V>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float* x) {
  if constexpr (V == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  else if constexpr (V == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  else *p = __float2bfloat16(x[0]);
}
template <int V>
__device__ __forceinline__ void load_params(const float* p, float* x) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) load_vec<4>(p + i, x + i);
  } else {
    x[0] = *p;
  }
}

// 16 or 8 bytes (V = 8 or 4) or one element (V = 1) as loaded
template <typename T, int V>
struct Raw {
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    if constexpr (sizeof(T) == 4) {
      x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
      x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    } else {
      const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(h[i] << 16);
        x[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
      }
    }
  }
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xffff0000u);
  }
};
template <typename T>
struct Raw<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T* p) { w = *p; }
  __device__ __forceinline__ void get(float* x) const { x[0] = static_cast<float>(w); }
};

// A thread owns `V` channels at c0 and, for rotated units of the half layout,
// the V partners at c0 + rot/2: both elements of every pair it touches, so the
// output may be the input itself.  V is 4 when rot/2 is a multiple of it, 16
// bytes for interleaved pairs, else 1: eight bf16 channels a thread, whose
// scales, offsets and sums leave room for two blocks of 12 warps an SM (16-byte
// halves, 16 channels a thread, left 12 warps: 181 us where this takes 154, 5.2
// TB/s, at B 2, 12 heads, T 32768, d 256; the rest goes to the angles, a
// quarter of the instructions, between two barriers).  The backward of the
// scales keeps 16 sums more and loads one token at a time (75 us where batches
// of two spill and take 82, at T 8192).
// Block (x, y): tokens [x % ranges * per_block, ..) of sequence x / ranges, heads
// [y * rows, (y + 1) * rows); thread u + units * r: unit u of head y * rows + r.
template <typename T, int V, bool INTER, bool BWD, bool AFF>
__global__ void __launch_bounds__(V == 1 ? 512 : kRotaryThreads, V == 1 ? 1 : 2) k_rotary(const RotaryParams p) {
  // [kRotaryTile][pairs of a unit][rot_units]: (amp cos, amp sin), then the pairs' turns per position in that order
  extern __shared__ float2 trig[];
  griddep_launch();
  griddep_wait();
  constexpr int kHalf = INTER ? 1 : 2;           // vectors of a rotated unit
  constexpr int kPairs = INTER ? V / 2 : V;      // pairs of a rotated unit
  constexpr int kUnroll = AFF && BWD ? 1 : 4;    // tokens in flight
  const int b = blockIdx.x / p.ranges;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x % p.ranges) * p.per_block;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(p.per_block), p.T - t0));
  const int u = threadIdx.x % p.units, r = threadIdx.x / p.units;
  const int hh = blockIdx.y * p.rows + r;
  const bool active = r < p.rows && hh < p.H + p.Hkv, isq = hh < p.H;
  const int h = isq ? hh : hh - p.H;
  const bool rotated = u < p.rot_units;
  const int nvec = active ? (rotated ? kHalf : 1) : 0;
  const int c0 = (INTER || rotated) ? u * V : p.rot + (u - p.rot_units) * V;
  const int c1 = c0 + p.rot / 2;
  const View4& xv = isq ? p.xq : p.xk;
  const View4& yv = isq ? p.yq : p.yk;
  const View4& dv = isq ? p.dq : p.dk;
  // what is rotated and what is written
  const View4& src = BWD ? yv : xv;
  const View4& dst = BWD ? dv : yv;
  const int64_t ss = src.st, ds = dst.st, xs = xv.st;
  const T* s0 = static_cast<const T*>(src.p) + b * src.sb + h * src.sh + t0 * ss;
  T* o0 = static_cast<T*>(dst.p) + b * dst.sb + h * dst.sh + t0 * ds;
  const T* x0 = (BWD && AFF) ? static_cast<const T*>(xv.p) + b * xv.sb + h * xv.sh + t0 * xs : nullptr;
  float sc[kHalf][V], of[kHalf][V], as[kHalf][V], ao[kHalf][V];
  if constexpr (AFF) {
#pragma unroll
    for (int k = 0; k < kHalf; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i) as[k][i] = ao[k][i] = 0.f;
      if (k < nvec) {
        load_params<V>((isq ? p.q_scale : p.k_scale) + h * p.d + (k ? c1 : c0), sc[k]);
        if constexpr (!BWD) load_params<V>((isq ? p.q_offset : p.k_offset) + h * p.d + (k ? c1 : c0), of[k]);
      }
    }
  }
  const int row_pairs = kPairs * p.rot_units;    // pairs past rot / 2 pad the last vector: angle 0
  double* turns = reinterpret_cast<double*>(trig + kRotaryTile * row_pairs);
  for (int x = threadIdx.x; x < row_pairs; x += blockDim.x) {
    const int i = (x % p.rot_units) * kPairs + x / p.rot_units;
    turns[x] = 2 * i < p.rot ? p.freqs[i] * 0.15915494309189533577 : __hiloint2double(kPadTurn, 0);   // 1 / (2 pi)
  }
  const int step_t = blockDim.x / row_pairs, step_x = blockDim.x % row_pairs;
  const int first_t = threadIdx.x / row_pairs, first_x = threadIdx.x % row_pairs;
  for (int base = 0; base < ntok; base += kRotaryTile) {
    const int nt = min(kRotaryTile, ntok - base);
    __syncthreads();
    for (int t = first_t, x = first_x; t < nt;) {
      const int64_t tok = t0 + base + t;
      const int64_t pos = p.positions ? p.positions[b * p.T + tok] : p.start + tok;
      const double turn = turns[x], n = static_cast<double>(pos) * turn;
      float s, c;
      sincospif(static_cast<float>(2.0 * (n - rint(n))), &s, &c);
      const bool pad = INTER && __double2hiint(turn) == kPadTurn;   // passes through
      trig[t * row_pairs + x] = make_float2(pad ? 1.f : p.amp * c, pad ? 0.f : p.amp * (BWD ? -s : s));
      t += step_t;
      x += step_x;
      if (x >= row_pairs) {
        x -= row_pairs;
        ++t;
      }
    }
    __syncthreads();
    if (nvec == 0) continue;
    for (int tb = 0; tb < nt; tb += kUnroll) {
      Raw<T, V> raw[kUnroll][kHalf], rx[kUnroll][kHalf];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (tb + j < nt) {
          const int64_t t = base + tb + j;
#pragma unroll
          for (int k = 0; k < kHalf; ++k)
            if (k < nvec) {
              raw[j][k].load(s0 + t * ss + (k ? c1 : c0));
              if constexpr (AFF && BWD) rx[j][k].load(x0 + t * xs + (k ? c1 : c0));
            }
        }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        if (tb + j >= nt) break;
        const int64_t t = base + tb + j;
        float a[kHalf][V];
#pragma unroll
        for (int k = 0; k < kHalf; ++k) {
          if (k < nvec) raw[j][k].get(a[k]);
          if constexpr (AFF && !BWD) {
#pragma unroll
            for (int i = 0; i < V; ++i) a[k][i] = fmaf(a[k][i], sc[k][i], of[k][i]);
          }
        }
        if (rotated) {
          const float2* cs = trig + (tb + j) * row_pairs + u;
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            const float2 w = cs[i * p.rot_units];
            float& xa = INTER ? a[0][2 * i] : a[0][i];
            float& xb = INTER ? a[0][2 * i + 1] : a[kHalf - 1][i];
            const float ya = xa * w.x - xb * w.y, yb = xb * w.x + xa * w.y;
            xa = ya;
            xb = yb;
          }
        }
        if constexpr (AFF && BWD) {
#pragma unroll
          for (int k = 0; k < kHalf; ++k)
            if (k < nvec) {
              float x[V];
              rx[j][k].get(x);
#pragma unroll
              for (int i = 0; i < V; ++i) {
                as[k][i] = fmaf(a[k][i], x[i], as[k][i]);
                ao[k][i] += a[k][i];
                a[k][i] *= sc[k][i];
              }
            }
        }
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
          if (k < nvec) store_vec<V>(o0 + t * ds + (k ? c1 : c0), a[k]);
      }
    }
  }
  if constexpr (AFF && BWD) {
    // this block's sums, in 32 bits and in the tokens' order
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float* out = p.partial + ((static_cast<int64_t>(blockIdx.x) * 2 + which) * (p.H + p.Hkv) + hh) * p.d;
#pragma unroll
      for (int k = 0; k < kHalf; ++k)
        if (k < nvec) {
          if constexpr (V >= 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) store_vec<4>(out + (k ? c1 : c0) + i, (which ? ao[k] : as[k]) + i);
          } else {
            out[k ? c1 : c0] = which ? ao[k][0] : as[k][0];
          }
        }
    }
  }
}

// The scales' and offsets' gradients: the sum of the blocks' partial sums
// [blocks][2][H + Hkv][d], 32 columns a block, 16 interleaved chains per column
// joined in a fixed order.
__global__ void __launch_bounds__(512) k_rotary_sums(const float* partial, int tiles, int H, int Hkv, int d,
                                                     float* dq_scale, float* dq_offset, float* dk_scale,
                                                     float* dk_offset) {
  __shared__ float part[16][33];
  griddep_launch();
  griddep_wait();
  const int n = 2 * (H + Hkv) * d;
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < n)
    for (int t = g; t < tiles; t += 16) s += partial[static_cast<int64_t>(t) * n + col];
  part[g][lane] = s;
  __syncthreads();
  if (g == 0 && col < n) {
    s = part[0][lane];
#pragma unroll
    for (int k = 1; k < 16; ++k) s += part[k][lane];
    const int which = col / ((H + Hkv) * d), at = col % ((H + Hkv) * d);
    if (at < H * d) (which ? dq_offset : dq_scale)[at] = s;
    else if (Hkv > 0) (which ? dk_offset : dk_scale)[at - H * d] = s;
  }
}

}  // namespace lact
