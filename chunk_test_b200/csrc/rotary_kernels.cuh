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
// scales also reads x).  A block takes a tile of tokens and walks the heads,
// so an angle is formed once and used by every head: p * freqs[i] in 64 bits,
// because a position of 10^6 leaves a 32-bit product only 4 bits below the
// turn, then the fraction of the turn goes to sincospif in 32.
#pragma once

#include "sm100.cuh"

namespace lact {

// One [B, heads, T, d] tensor: channels contiguous, strides in elements.
struct View4 {
  void* p;
  int64_t sb, sh, st;
};

// 512 threads where a thread owns single channels (up to 511 units of a row)
template <int V>
constexpr int kRotaryThreads = V == 1 ? 512 : 256;

struct RotaryParams {
  View4 xq, xk;            // forward: inputs; backward: inputs, for the scales' gradients (else null)
  View4 yq, yk;            // forward: outputs; backward: the outputs' gradients
  View4 dq, dk;            // backward: the inputs' gradients
  const double* freqs;     // [rot / 2], radians per position
  const int* positions;    // [B, T] or null: start + t
  const float *q_scale, *q_offset, *k_scale, *k_offset;   // [H, d], [Hkv, d] or null
  float* partial;          // backward of the scales: [token tiles][2][H + Hkv][d]
  int64_t start;
  int64_t T;
  int B, H, Hkv, d, rot, pairs;   // pairs: rot / 2 rounded up to a whole vector
  int tile, heads_per_block;      // tokens of a block, heads of a block
  float amp;
};

template <int V>
__device__ __forceinline__ void load_vec(const float* p, float* x) {
  if constexpr (V == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    x[0] = *p;
  }
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float* x) {
  if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else *p = x[0];
}
template <int V>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float* x) {
  if constexpr (V == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    x[0] = __bfloat162float(*p);
  }
}
// the one rounding of a bf16 result: to nearest, ties to even
template <int V>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float* x) {
  if constexpr (V == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
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

// A thread owns `V` channels at c0 and, for rotated units of the half layout,
// the V partners at c0 + rot/2: both elements of every pair it touches, so the
// output may be the input itself.  V is the 16-byte vector when rot/2 is a
// multiple of it (interleaved pairs: always), else 1.
template <typename T, int V, bool INTER, bool BWD, bool AFF>
__global__ void __launch_bounds__(kRotaryThreads<V>) k_rotary(const RotaryParams p) {
  extern __shared__ float2 trig[];   // [tile][pairs] (amp cos, amp sin), then the sums' staging
  griddep_launch();
  griddep_wait();
  constexpr int kHalf = INTER ? 1 : 2;           // vectors of a rotated unit
  constexpr int kThreads = kRotaryThreads<V>;
  constexpr int kUnroll = V == 1 ? 2 : 4;
  const int tiles = static_cast<int>((p.T + p.tile - 1) / p.tile);
  const int b = blockIdx.x / tiles;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x % tiles) * p.tile;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.tile), p.T - t0));
  for (int e = threadIdx.x; e < nt * p.pairs; e += kThreads) {
    const int t = e / p.pairs, i = e % p.pairs;
    float2 cs = make_float2(1.f, 0.f);           // pairs that pad the last vector pass through
    if (2 * i < p.rot) {
      const int64_t pos = p.positions ? p.positions[b * p.T + t0 + t] : p.start + t0 + t;
      const double turns = static_cast<double>(pos) * p.freqs[i] * 0.15915494309189533577;   // 1 / (2 pi)
      float s, c;
      sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
      cs = make_float2(p.amp * c, p.amp * (BWD ? -s : s));
    }
    trig[e] = cs;
  }
  __syncthreads();

  const int rot_units = INTER ? (p.rot + V - 1) / V : p.rot / (2 * V);
  const int units = INTER ? p.d / V : rot_units + (p.d - p.rot) / V;
  const int rows = kThreads / units;
  const int u = threadIdx.x % units, r = threadIdx.x / units;
  const bool rotated = u < rot_units;
  const int nvec = rotated ? kHalf : 1;
  const int c0 = (INTER || rotated) ? u * V : p.rot + (u - rot_units) * V;
  const int c1 = c0 + p.rot / 2;
  const int pair0 = INTER ? c0 / 2 : c0;
  const int h1 = min(static_cast<int>(blockIdx.y + 1) * p.heads_per_block, p.H + p.Hkv);
  for (int hh = blockIdx.y * p.heads_per_block; hh < h1; ++hh) {
    const bool isq = hh < p.H;
    const int h = isq ? hh : hh - p.H;
    const View4& xv = isq ? p.xq : p.xk;
    const View4& yv = isq ? p.yq : p.yk;
    const View4& dv = isq ? p.dq : p.dk;
    // what is rotated and what is written
    const View4& src = BWD ? yv : xv;
    const View4& dst = BWD ? dv : yv;
    const T* s0 = static_cast<const T*>(src.p) + b * src.sb + h * src.sh + t0 * src.st;
    T* o0 = static_cast<T*>(dst.p) + b * dst.sb + h * dst.sh + t0 * dst.st;
    const T* x0 = (BWD && AFF) ? static_cast<const T*>(xv.p) + b * xv.sb + h * xv.sh + t0 * xv.st : nullptr;
    float sc[kHalf][V], of[kHalf][V], as[kHalf][V], ao[kHalf][V];
    if constexpr (AFF) {
      const float* sp = (isq ? p.q_scale : p.k_scale) + h * p.d;
      const float* op = BWD ? nullptr : (isq ? p.q_offset : p.k_offset) + h * p.d;
#pragma unroll
      for (int k = 0; k < kHalf; ++k) {
#pragma unroll
        for (int i = 0; i < V; ++i) as[k][i] = ao[k][i] = 0.f;
        if (k < nvec) {
          load_params<V>(sp + (k ? c1 : c0), sc[k]);
          if constexpr (!BWD) load_params<V>(op + (k ? c1 : c0), of[k]);
        }
      }
    }
    if (r < rows) {
      for (int tb = r; tb < nt; tb += kUnroll * rows) {
        float a[kUnroll][kHalf][V];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          const int t = tb + j * rows;
          if (t < nt) {
#pragma unroll
            for (int k = 0; k < kHalf; ++k)
              if (k < nvec) load_vec<V>(s0 + t * src.st + (k ? c1 : c0), a[j][k]);
          }
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          const int t = tb + j * rows;
          if (t >= nt) break;
          if constexpr (AFF && !BWD) {
#pragma unroll
            for (int k = 0; k < kHalf; ++k)
#pragma unroll
              for (int i = 0; i < V; ++i) a[j][k][i] = fmaf(a[j][k][i], sc[k][i], of[k][i]);
          }
          if (rotated) {
            const float2* cs = trig + t * p.pairs + pair0;
            if constexpr (INTER) {
#pragma unroll
              for (int i = 0; i < V; i += 2) {
                const float2 w = cs[i / 2];
                const float xa = a[j][0][i], xb = a[j][0][i + 1];
                a[j][0][i] = xa * w.x - xb * w.y;
                a[j][0][i + 1] = xb * w.x + xa * w.y;
              }
            } else {
#pragma unroll
              for (int i = 0; i < V; ++i) {
                const float2 w = cs[i];
                const float xa = a[j][0][i], xb = a[j][1][i];
                a[j][0][i] = xa * w.x - xb * w.y;
                a[j][1][i] = xb * w.x + xa * w.y;
              }
            }
          }
          if constexpr (AFF && BWD) {
#pragma unroll
            for (int k = 0; k < kHalf; ++k)
              if (k < nvec) {
                float x[V];
                load_vec<V>(x0 + t * xv.st + (k ? c1 : c0), x);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                  as[k][i] = fmaf(a[j][k][i], x[i], as[k][i]);
                  ao[k][i] += a[j][k][i];
                  a[j][k][i] *= sc[k][i];
                }
              }
          }
#pragma unroll
          for (int k = 0; k < kHalf; ++k)
            if (k < nvec) store_vec<V>(o0 + t * dst.st + (k ? c1 : c0), a[j][k]);
        }
      }
    }
    if constexpr (AFF && BWD) {
      // the block's sums over its tokens, in 32 bits and a fixed order: each
      // thread's tokens, then the rows of threads
      float* stage = reinterpret_cast<float*>(trig + p.tile * p.pairs);   // [rows][d]
      for (int which = 0; which < 2; ++which) {
        if (r < rows) {
#pragma unroll
          for (int k = 0; k < kHalf; ++k)
            if (k < nvec)
#pragma unroll
              for (int i = 0; i < V; ++i)
                stage[r * p.d + (k ? c1 : c0) + i] = which ? ao[k][i] : as[k][i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.d; c += kThreads) {
          float s = 0.f;
          for (int k = 0; k < rows; ++k) s += stage[k * p.d + c];
          p.partial[((static_cast<int64_t>(blockIdx.x) * 2 + which) * (p.H + p.Hkv) + hh) * p.d + c] = s;
        }
        __syncthreads();
      }
    }
  }
}

// The scales' and offsets' gradients: the sum of the token tiles' partial sums
// [tiles][2][H + Hkv][d], 32 columns a block, 16 interleaved chains per column
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
