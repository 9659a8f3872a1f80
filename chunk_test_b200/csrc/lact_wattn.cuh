// lact_wattn.cuh -- host side of the attention half's operators: rotary
// positions, the window attention with sinks (forward, backward) and its
// single-token form over a rolling cache.  Included by lact_api.cu after the
// launch helpers.
#pragma once

#include "wattn_decode.cuh"
#include "wattn_bwd.cuh"
#include "wattn_fwd.cuh"
#include "wattn_simt.cuh"

namespace lact {

// ------------------------------------------------------------------ arguments
struct Extent4 {
  int64_t B, H, T, d;
};

// int32 and float32 arrays that are read singly (null: absent)
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// a * b <= 65535, for numbers of any size
static bool product_ok(int64_t a, int64_t b) { return a <= 65535 && b <= 65535 && a * b <= 65535; }

static bool view_ok(const lact_tensor4* t, const Extent4& e, int esz) {
  if (!t || !t->data || !aligned16(t->data)) return false;
  const int64_t s[3] = {t->stride_b, t->stride_h, t->stride_t}, n[3] = {e.B, e.H, e.T};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] <= 0 || s[i] * esz % 16 != 0 || s[i] > (int64_t(1) << 36))) return false;
  return true;
}

// Strides of dimensions of length 1 mean nothing to the caller; they are set
// to the ones a dense tensor would have.
static View4 view4(const lact_tensor4* t, const Extent4& e) {
  View4 v{t->data, t->stride_b, t->stride_h, t->stride_t};
  if (e.T == 1) v.st = e.d;
  if (e.H == 1) v.sh = e.T > 1 ? v.st * e.T : e.d;
  if (e.B == 1) v.sb = std::max(v.sh * e.H, v.st * e.T);
  return v;
}

static int64_t span(const View4& v, const Extent4& e) {   // elements from the first to behind the last
  return (e.B - 1) * v.sb + (e.H - 1) * v.sh + (e.T - 1) * v.st + e.d;
}

// No two elements of the view share an address: by ascending stride, each
// dimension steps over all of the ones below it.
static bool injective(const View4& v, const Extent4& e) {
  std::pair<int64_t, int64_t> s[3] = {{v.sb, e.B}, {v.sh, e.H}, {v.st, e.T}};
  std::sort(s, s + 3);
  int64_t reach = e.d;
  for (auto& x : s) {
    if (x.second == 1) continue;
    if (x.first < reach) return false;
    reach = x.first * (x.second - 1) + reach;
  }
  return true;
}

// The bytes that a view covers within one period of `pitch` bytes: dimensions
// that step by whole periods add nothing; -1 where one steps over part of one.
static int64_t bytes_in_pitch(const View4& v, const Extent4& e, int64_t pitch, int esz) {
  const int64_t s[3] = {v.sb, v.sh, v.st}, n[3] = {e.B, e.H, e.T};
  int64_t w = e.d * esz;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && s[i] * esz % pitch != 0) {
      if (s[i] * esz > pitch) return -1;
      w += (n[i] - 1) * s[i] * esz;
    }
  return w;
}

// Whether two views share no memory: their spans are apart, or both are slices
// of one packed buffer, in different places of each of its rows, heads or
// sequences: modulo the stride of one of the dimensions they do not meet.
static bool apart(const View4& a, const Extent4& ea, const View4& b, const Extent4& eb, int esz) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  if (!overlaps(a.p, static_cast<size_t>(span(a, ea)) * esz, b.p, static_cast<size_t>(span(b, eb)) * esz)) return true;
  const int64_t strides[6] = {a.st, a.sh, a.sb, b.st, b.sh, b.sb}, n[6] = {ea.T, ea.H, ea.B, eb.T, eb.H, eb.B};
  for (int i = 0; i < 6; ++i) {
    if (n[i] < 2) continue;
    const int64_t pitch = strides[i] * esz;
    const int64_t wa = bytes_in_pitch(a, ea, pitch, esz), wb = bytes_in_pitch(b, eb, pitch, esz);
    if (wa < 0 || wb < 0) continue;
    const int64_t at = ((static_cast<int64_t>(pb - pa)) % pitch + pitch) % pitch;
    if (at >= wa && at + wb <= pitch) return true;
  }
  return false;
}
static bool same(const View4& a, const View4& b, const Extent4& e) {
  return a.p == b.p && (e.B == 1 || a.sb == b.sb) && (e.H == 1 || a.sh == b.sh) && (e.T == 1 || a.st == b.st);
}
static bool apart_from(const View4& a, const Extent4& e, int esz, const void* p, int64_t bytes) {
  return !p || !overlaps(a.p, static_cast<size_t>(span(a, e)) * esz, p, static_cast<size_t>(bytes));
}

// A failed call's error is reported by its status alone, not left behind for the
// caller's next check.
static cudaError_t cleared(cudaError_t e) {
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

// Raises a kernel's dynamic shared memory limit, once per device.
template <class F>
static cudaError_t set_smem(F* kernel, int bytes, bool (&done)[64], bool big_cluster = false) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && big_cluster) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

// ------------------------------------------------------------------ rotary
struct RotaryDims {
  int vec, units, rot_units, rows, head_blocks, per_block, ranges, smem;
};

static int rotary_validate(const lact_rotary_problem* p) {
  if (!p || p->B < 1 || p->H < 1 || p->Hkv < 0 || p->T < 1 || p->d < 1) return LACT_EINVAL;
  if (p->dtype != LACT_F32 && p->dtype != LACT_BF16) return LACT_EINVAL;
  if (p->d % 8 != 0 || p->d > 512 || p->rot < 2 || p->rot > p->d || p->rot % 2 != 0) return LACT_EINVAL;
  if (!product_ok(p->B, p->H) || !product_ok(p->B, p->Hkv) || p->B * (p->H + p->Hkv) > 65535) return LACT_EINVAL;
  if (p->T > (int64_t(1) << 30)) return LACT_EINVAL;
  if (p->start < 0 || p->start > (int64_t(1) << 40) || (p->interleaved & ~1)) return LACT_EINVAL;
  if (!(std::isfinite(p->amplitude))) return LACT_EINVAL;
  return LACT_OK;
}

// Vectors of 4 channels where both halves of a pair start on one (interleaved
// pairs: of 16 bytes), else single channels.  A block takes as many heads as 384
// threads (512 where a head alone has more units) hold, so angles are formed once
// for all of them.
static RotaryDims rotary_dims(const lact_rotary_problem* p, bool sums) {
  RotaryDims r;
  const int d = static_cast<int>(p->d), rot = static_cast<int>(p->rot);
  r.vec = p->interleaved ? (p->dtype == LACT_BF16 ? 8 : 4) : (rot / 2) % 4 == 0 ? 4 : 1;
  r.rot_units = p->interleaved ? static_cast<int>(cdiv(rot, r.vec)) : rot / (2 * r.vec);
  r.units = p->interleaved ? d / r.vec : r.rot_units + (d - rot) / r.vec;
  const int64_t heads = p->H + p->Hkv;
  const int64_t most = std::max<int64_t>(1, kRotaryThreads / r.units);
  r.head_blocks = static_cast<int>(cdiv(heads, std::min(heads, most)));
  // two blocks per SM: with sums one round of them, since each block writes its
  // own; without, at most 32 tokens each, so that the last round is short
  r.per_block = static_cast<int>(cdiv(p->B * p->T * r.head_blocks, 2 * kPlanSMs));
  if (!sums) r.per_block = std::min(r.per_block, 2 * kRotaryTile);
  r.per_block = static_cast<int>(std::min<int64_t>(std::max(r.per_block, 1), p->T));
  r.ranges = static_cast<int>(cdiv(p->T, r.per_block));
  r.rows = static_cast<int>(cdiv(heads, r.head_blocks));
  r.smem = (kRotaryTile + 1) * r.rot_units * (p->interleaved ? r.vec / 2 : r.vec) * 8;
  return r;
}

static size_t rotary_bwd_workspace(const lact_rotary_problem* p) {
  const RotaryDims r = rotary_dims(p, true);
  return static_cast<size_t>(rup(p->B * r.ranges * 2 * (p->H + p->Hkv) * p->d * 4, 256));
}

template <typename T, int V, bool INTER, bool BWD, bool AFF>
static cudaError_t launch_rotary(const RotaryDims& r, const RotaryParams& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.B * r.ranges), static_cast<unsigned>(r.head_blocks));
  return launch_pdl(k_rotary<T, V, INTER, BWD, AFF>, grid, dim3(static_cast<unsigned>(rup(r.units * r.rows, 32))),
                    r.smem, st, a);
}

template <bool BWD, bool AFF>
static cudaError_t launch_rotary_any(const lact_rotary_problem* p, const RotaryDims& r, const RotaryParams& a,
                                     cudaStream_t st) {
  using B16 = __nv_bfloat16;
  if (p->dtype == LACT_BF16) {
    if (p->interleaved) return launch_rotary<B16, 8, true, BWD, AFF>(r, a, st);
    return r.vec == 4 ? launch_rotary<B16, 4, false, BWD, AFF>(r, a, st)
                      : launch_rotary<B16, 1, false, BWD, AFF>(r, a, st);
  }
  if (p->interleaved) return launch_rotary<float, 4, true, BWD, AFF>(r, a, st);
  return r.vec == 4 ? launch_rotary<float, 4, false, BWD, AFF>(r, a, st)
                    : launch_rotary<float, 1, false, BWD, AFF>(r, a, st);
}

static RotaryParams rotary_params(const lact_rotary_problem* p, const RotaryDims& r, const double* freqs,
                                  const int32_t* positions) {
  RotaryParams a;
  std::memset(&a, 0, sizeof(a));
  a.freqs = freqs; a.positions = positions; a.start = p->start; a.T = p->T;
  a.B = static_cast<int>(p->B); a.H = static_cast<int>(p->H); a.Hkv = static_cast<int>(p->Hkv);
  a.d = static_cast<int>(p->d); a.rot = static_cast<int>(p->rot); a.units = r.units; a.rot_units = r.rot_units;
  a.rows = r.rows; a.per_block = r.per_block; a.ranges = r.ranges; a.amp = p->amplitude;
  return a;
}

// ------------------------------------------------------------------ window attention
// Query rows of a sink tile's far part: about the work of a near part; the
// CUDA cores take as long for a quarter of the rows.
constexpr int kWattnFarRows = 1024, kWattnFarRowsF32 = 256;
constexpr int kFewRounds = 8;         // rounds of persistent CTAs below which the short tiles go last
constexpr int kWalkedSequences = 8;   // sequences whose lengths are walked to find a tile's place

struct WattnDims {
  int64_t B, H, Hkv, T, Tq, d, DP;
  int window, sinks, dtype;
  int bn, sink_tiles, parts, key_tiles, far_rows;   // of the keys' gradients
};

static int wattn_validate(const lact_swa_sink_problem* p, WattnDims& D) {
  if (!p || p->B < 1 || p->H < 1 || p->Hkv < 1 || p->T < 1 || p->Tq < 1 || p->d < 1) return LACT_EINVAL;
  if (p->dtype != LACT_F32 && p->dtype != LACT_BF16) return LACT_EINVAL;
  if (p->H % p->Hkv != 0 || p->Tq > p->T || p->d % 8 != 0 || p->d > 256) return LACT_EINVAL;
  if (p->window < 1 || p->sinks < 0 || !std::isfinite(p->scale) || !(p->scale > 0.f))
    return LACT_EINVAL;
  if (!product_ok(p->B, p->H) || p->T > (int64_t(1) << 24)) return LACT_EINVAL;
  D.B = p->B; D.H = p->H; D.Hkv = p->Hkv; D.T = p->T; D.Tq = p->Tq; D.d = p->d;
  D.DP = rup(p->d, 64);
  D.window = static_cast<int>(std::min(p->window, p->T));
  D.sinks = static_cast<int>(std::min(p->sinks, p->T));
  if (static_cast<int64_t>(D.window) + D.sinks >= p->T) {   // no key is hidden: plain causal attention
    D.window = static_cast<int>(p->T);
    D.sinks = 0;
  }
  D.dtype = p->dtype;
  D.bn = D.dtype == LACT_BF16 ? 128 : D.DP <= 128 ? SimtCfg<128>::kM : SimtCfg<256>::kM;
  D.key_tiles = static_cast<int>(cdiv(D.T, D.bn));
  D.sink_tiles = static_cast<int>(cdiv(D.sinks, D.bn));
  // far parts of kWattnFarRows query rows, fewer and longer where the sink tiles
  // alone make four rounds of CTAs: each part's sums take workspace
  D.far_rows = D.dtype == LACT_BF16 ? kWattnFarRows : kWattnFarRowsF32;
  if (D.sink_tiles > 0) {
    const int64_t most = std::max<int64_t>(1, 4 * kPlanSMs / (D.B * D.Hkv * D.sink_tiles));
    D.far_rows = static_cast<int>(std::max<int64_t>(D.far_rows, rup(cdiv(D.T, most), 128)));
  }
  const int far = far_parts(D.bn, D.window, static_cast<int>(D.T), D.far_rows);
  if (far == 0) D.sink_tiles = 0;   // the window reaches every query: no far part
  D.parts = 1 + far;
  return LACT_OK;
}

struct WattnBufs {
  float *delta, *part;
};
static void wattn_bwd_plan(const WattnDims& D, Bump& bp, WattnBufs& b) {
  b.delta = bp.take<float>(D.B * D.H * D.Tq);
  b.part = bp.take<float>(D.B * D.Hkv * D.sink_tiles * D.parts * 2 * D.bn * D.DP);
}
static size_t wattn_bwd_workspace(const WattnDims& D) {
  Bump bp{0, 0};
  WattnBufs b;
  wattn_bwd_plan(D, bp, b);
  return static_cast<size_t>(rup(static_cast<int64_t>(bp.off), 256));
}

static WattnParams wattn_params(const WattnDims& D, float scale, const int32_t* lengths, const float* lse) {
  WattnParams a;
  std::memset(&a, 0, sizeof(a));
  a.lse = const_cast<float*>(lse); a.lengths = lengths; a.scale = scale;
  a.B = static_cast<int>(D.B); a.H = static_cast<int>(D.H); a.Hkv = static_cast<int>(D.Hkv);
  a.group = static_cast<int>(D.H / D.Hkv); a.T = static_cast<int>(D.T); a.Tq = static_cast<int>(D.Tq);
  a.d = static_cast<int>(D.d); a.window = D.window; a.sinks = D.sinks; a.far_rows = D.far_rows;
  return a;
}

// 4-D bf16 map (channel, token, head, batch) of a view, boxes of 64 channels
// (128-byte swizzle) or 32 (64-byte swizzle) x `rows` tokens; elements outside
// read as zero and are not written.
static bool map_view(CUtensorMap* m, const View4& v, const Extent4& e, uint32_t rows, uint32_t channels = 64) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(e.d), static_cast<cuuint64_t>(e.T), static_cast<cuuint64_t>(e.H),
                        static_cast<cuuint64_t>(e.B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(v.st) * 2, static_cast<cuuint64_t>(v.sh) * 2,
                           static_cast<cuuint64_t>(v.sb) * 2};
  cuuint32_t box[4] = {channels, rows, 1, 1}, es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            channels == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP>
static cudaError_t wattn_fwd_bf16(const WattnDims& D, const WattnParams& a, cudaStream_t st) {
  using C = WattnCfg<DP>;
  // 228 KB an SM, 1 KB of it reserved for each CTA
  static_assert((C::kSmem + 1024) * C::kCtas <= 228 * 1024, "dynamic shared memory above the SM's limit");
  static bool done[64] = {};
  const cudaError_t e = set_smem(k_wattn_fwd<DP>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  WattnFwdParams f;
  std::memset(&f, 0, sizeof(f));
  const Extent4 eq{D.B, D.H, D.Tq, D.d}, ek{D.B, D.Hkv, D.T, D.d};
  if (!map_view(&f.tmQ, a.q, eq, 128) || !map_view(&f.tmK, a.k, ek, 128) || !map_view(&f.tmV, a.v, ek, C::kVKeys) ||
      !map_view(&f.tmK32, a.k, ek, 32) || !map_view(&f.tmV32, a.v, ek, 32) ||
      !map_view(&f.tmO, a.out, eq, 32, 32))
    return cudaErrorInvalidValue;
  f.a = a;
  f.nb = static_cast<int>(cdiv(D.Tq, 128));
  const int64_t tiles = D.B * D.H * f.nb;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  f.ntiles = static_cast<int>(tiles);
  const int64_t places = sm_count() * C::kCtas;
  f.a.heads_first = tiles < kFewRounds * places;
  // Tiles by length, for more than one round and few: 5% less time over 193 ragged
  // batches of up to 8 sequences and 1 to 8 rounds.  Each role of a CTA walks the
  // lengths for each of its tiles, so more sequences lose by it: 32 of up to 2088
  // tokens, 12 heads on 4, d 128 take 321 us with and 235 without.
  f.a.by_length = a.lengths && D.B <= kWalkedSequences && f.a.heads_first && tiles > places;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(tiles, places)));
  return launch_pdl(k_wattn_fwd<DP>, grid, dim3(C::kThreads), C::kSmem, st, f);
}

template <int DP>
static cudaError_t wattn_fwd_f32(const WattnDims& D, const WattnParams& a, cudaStream_t st) {
  static bool done[64] = {};
  const cudaError_t e = set_smem(k_wattn_fwd_f32<DP>, SimtCfg<DP>::kFwdSmem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(cdiv(D.Tq, SimtCfg<DP>::kM)), static_cast<unsigned>(D.B * D.H));
  return launch_pdl(k_wattn_fwd_f32<DP>, grid, dim3(SimtCfg<DP>::kThreads), SimtCfg<DP>::kFwdSmem, st, a);
}
template <int DP>
static cudaError_t wattn_dq_f32(const WattnDims& D, const WattnParams& a, cudaStream_t st) {
  static bool done[64] = {};
  static_assert(SimtCfg<DP>::kBwdSmem <= kMaxSmemPerBlock, "dynamic shared memory above the per-CTA limit");
  const cudaError_t e = set_smem(k_wattn_dq_f32<DP>, SimtCfg<DP>::kBwdSmem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(cdiv(D.Tq, SimtCfg<DP>::kM)), static_cast<unsigned>(D.B * D.H));
  return launch_pdl(k_wattn_dq_f32<DP>, grid, dim3(SimtCfg<DP>::kThreads), SimtCfg<DP>::kBwdSmem, st, a);
}
template <int DP>
static cudaError_t wattn_dkv_f32(const WattnDims& D, const WattnParams& a, cudaStream_t st) {
  static bool done[64] = {};
  const cudaError_t e = set_smem(k_wattn_dkv_f32<DP>, SimtCfg<DP>::kBwdSmem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(D.sink_tiles * D.parts + D.key_tiles - D.sink_tiles),
                  static_cast<unsigned>(D.B * D.Hkv));
  return launch_pdl(k_wattn_dkv_f32<DP>, grid, dim3(SimtCfg<DP>::kThreads), SimtCfg<DP>::kBwdSmem, st, a, D.sink_tiles, D.parts);
}

template <int DP, int MODE>
static cudaError_t wattn_bwd_bf16(const WattnDims& D, const WattnParams& a, cudaStream_t st) {
  using C = BwdCfg<DP, MODE>;
  static_assert(C::kSmem <= kMaxSmemPerBlock, "dynamic shared memory above the per-CTA limit");
  static bool done[64] = {};
  const cudaError_t e = set_smem(k_wattn_bwd<DP, MODE>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  WattnBwdParams f;
  std::memset(&f, 0, sizeof(f));
  const Extent4 eq{D.B, D.H, D.Tq, D.d}, ek{D.B, D.Hkv, D.T, D.d};
  CUtensorMap *q = MODE == WATTN_DQ ? &f.tmA1 : &f.tmB1, *g = MODE == WATTN_DQ ? &f.tmA2 : &f.tmB2;
  CUtensorMap *k = MODE == WATTN_DQ ? &f.tmB1 : &f.tmA1, *v = MODE == WATTN_DQ ? &f.tmB2 : &f.tmA2;
  if (!map_view(q, a.q, eq, 128) || !map_view(g, a.dout, eq, 128) || !map_view(k, a.k, ek, 128) ||
      !map_view(v, a.v, ek, 128) ||
      !(MODE == WATTN_DQ ? map_view(&f.tmX64, a.k, ek, 64) : map_view(&f.tmX64, MODE == WATTN_DV ? a.dout : a.q, eq, 64)))
    return cudaErrorInvalidValue;
  f.a = a;
  f.sink_tiles = D.sink_tiles;
  f.parts = D.parts;
  f.per_head = MODE == WATTN_DQ ? static_cast<int>(cdiv(D.Tq, 128)) : D.sink_tiles * (D.parts - 1) + D.key_tiles;
  const int64_t items = D.B * (MODE == WATTN_DQ ? D.H : D.Hkv) * f.per_head;
  if (items > INT32_MAX) return cudaErrorInvalidValue;
  f.nitems = static_cast<int>(items);
  f.a.heads_first = items < kFewRounds * sm_count();
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(items, sm_count())));
  return launch_pdl(k_wattn_bwd<DP, MODE>, grid, dim3(C::kThreads), C::kSmem, st, f);
}

#define LACT_BY_DP(DPV, ...)                  \
  switch (DPV) {                               \
    case 64: { constexpr int DP = 64; return cleared(__VA_ARGS__); }   \
    case 128: { constexpr int DP = 128; return cleared(__VA_ARGS__); } \
    case 192: { constexpr int DP = 192; return cleared(__VA_ARGS__); } \
    default: { constexpr int DP = 256; return cleared(__VA_ARGS__); }  \
  }

template <typename T, int LANES>
static cudaError_t launch_wattn_delta_as(const WattnDims& D, const WattnParams& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(cdiv(D.B * D.H * D.Tq, 256 / LANES), kPlanSMs * 32)));
  return launch_pdl(k_wattn_delta<T, LANES>, grid, dim3(256), 0, st, a);
}
static cudaError_t launch_wattn_delta(const WattnDims& D, const WattnParams& a, cudaStream_t st) {
  using B16 = __nv_bfloat16;
  if (D.dtype == LACT_F32) return launch_wattn_delta_as<float, 32>(D, a, st);
  if (D.d <= 64) return launch_wattn_delta_as<B16, 8>(D, a, st);
  return D.d <= 128 ? launch_wattn_delta_as<B16, 16>(D, a, st) : launch_wattn_delta_as<B16, 32>(D, a, st);
}
static cudaError_t launch_wattn_sums(const WattnDims& D, const WattnParams& a, cudaStream_t st) {
  const int64_t n = D.B * D.Hkv * D.sink_tiles * 2 * D.bn * (D.DP / 4);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(cdiv(n, 256), kPlanSMs * 16)));
  const int DP = static_cast<int>(D.DP);
  return D.dtype == LACT_F32
             ? launch_pdl(k_wattn_sink_sums<float>, grid, dim3(256), 0, st, a, D.sink_tiles, D.parts, D.bn, DP)
             : launch_pdl(k_wattn_sink_sums<__nv_bfloat16>, grid, dim3(256), 0, st, a, D.sink_tiles, D.parts, D.bn, DP);
}

static void wattn_fwd_run(const WattnDims& D, const WattnParams& a, cudaStream_t st, Launcher& L) {
  L.st = st;
  L(K_WATTN_FWD, [&]() -> cudaError_t {
    LACT_BY_DP(D.DP, D.dtype == LACT_F32 ? wattn_fwd_f32<DP>(D, a, st) : wattn_fwd_bf16<DP>(D, a, st))
  });
}

static void wattn_bwd_run(const WattnDims& D, const WattnParams& a, cudaStream_t st, Launcher& L) {
  L.st = st;
  L(K_WATTN_ELEM, [&] { return cleared(launch_wattn_delta(D, a, st)); });
  L(K_WATTN_DQ, [&]() -> cudaError_t {
    LACT_BY_DP(D.DP, D.dtype == LACT_F32 ? wattn_dq_f32<DP>(D, a, st) : (wattn_bwd_bf16<DP, WATTN_DQ>(D, a, st)))
  });
  if (D.dtype == LACT_F32) {
    L(K_WATTN_DKV, [&]() -> cudaError_t { LACT_BY_DP(D.DP, wattn_dkv_f32<DP>(D, a, st)) });
  } else {
    // both in one pass where TMEM holds both accumulators beside S and dP
    if (D.DP <= 128) {
      L(K_WATTN_DKV, [&] { return cleared(D.DP == 64 ? wattn_bwd_bf16<64, WATTN_DKV>(D, a, st) : wattn_bwd_bf16<128, WATTN_DKV>(D, a, st)); });
    } else {
      L(K_WATTN_DKV, [&] { return cleared(D.DP == 192 ? wattn_bwd_bf16<192, WATTN_DK>(D, a, st) : wattn_bwd_bf16<256, WATTN_DK>(D, a, st)); });
      L(K_WATTN_DKV, [&] { return cleared(D.DP == 192 ? wattn_bwd_bf16<192, WATTN_DV>(D, a, st) : wattn_bwd_bf16<256, WATTN_DV>(D, a, st)); });
    }
  }
  if (D.sink_tiles > 0) L(K_WATTN_ELEM, [&] { return cleared(launch_wattn_sums(D, a, st)); });
}

// ------------------------------------------------------------------ single-token form
static int decode_validate(const lact_swa_sink_problem* p) {
  if (!p || p->B < 1 || p->H < 1 || p->Hkv < 1 || p->d < 1) return LACT_EINVAL;
  if (p->dtype != LACT_F32 && p->dtype != LACT_BF16) return LACT_EINVAL;
  if (p->H % p->Hkv != 0 || p->d % 8 != 0 || p->d > 256) return LACT_EINVAL;
  if (p->window < 1 || p->sinks < 0 || !std::isfinite(p->scale) || !(p->scale > 0.f))
    return LACT_EINVAL;
  if (p->window > (int64_t(1) << 30) || p->sinks > (int64_t(1) << 30)) return LACT_EINVAL;
  // the kernels count slots in 32 bits, rounded up to whole steps of the cluster's CTAs
  if (p->sinks + p->window > (int64_t(1) << 31) - 1024) return LACT_EINVAL;
  if (!product_ok(p->B, p->H)) return LACT_EINVAL;
  return LACT_OK;
}

// CTAs of one (sequence, key head): doubled while the whole grid would leave
// SMs idle and each CTA keeps 16 slots for each of its warps.  More CTAs than
// that cost more in joining full windows than they balance (4 key heads, d 128,
// windows of 8192: 64 full sequences 184 us with one, 190 with two, 201 with four;
// at lengths from none to the whole window 162, 157 and 154; 32 full ones 101 with
// two, 105 with four; 8 full ones 37 with eight, 55 with sixteen).  16 is the
// largest cluster.
static int decode_ranks(int64_t items, int64_t slots) {
  int r = 1;
  while (r < 16 && items * r < kPlanSMs && slots >= static_cast<int64_t>(r) * 2 * kDecWarps * 16) r *= 2;
  return r;
}

template <class F>
static cudaError_t launch_decode_as(F* kernel, int smem, bool (&done)[64], const DecodeParams& a, int64_t items,
                                    cudaStream_t st) {
  cudaError_t e = set_smem(kernel, smem, done, true);
  if (e != cudaSuccess) return e;
  const int ranks = decode_ranks(items, static_cast<int64_t>(a.sinks) + a.window);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks, static_cast<unsigned>(items));
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int DP>
static cudaError_t launch_decode(int dtype, const DecodeParams& a, int64_t items, cudaStream_t st) {
  constexpr int smem = (2 * kDecWarps * kDecHeads + kDecWarps * kDecHeads * DP) * 4;
  if (dtype == LACT_BF16) {
    static bool done[64] = {};
    return launch_decode_as(k_wattn_decode_bf16<DP>, smem, done, a, items, st);
  }
  const int heads = std::min(a.group, kDecHeads);
  static bool done1[64] = {}, done4[64] = {}, done8[64] = {};
  if (heads == 1) return launch_decode_as(k_wattn_decode_f32<DP, 1>, smem, done1, a, items, st);
  if (heads <= 4) return launch_decode_as(k_wattn_decode_f32<DP, 4>, smem, done4, a, items, st);
  return launch_decode_as(k_wattn_decode_f32<DP, 8>, smem, done8, a, items, st);
}

static cudaError_t launch_decode_any(int64_t DPV, int dtype, const DecodeParams& a, int64_t items, cudaStream_t st) {
  LACT_BY_DP(DPV, launch_decode<DP>(dtype, a, items, st))
}

}  // namespace lact

// ------------------------------------------------------------------ entry points
extern "C" {

size_t lact_rotary_bwd_workspace_bytes(const lact_rotary_problem* p) {
  return lact::rotary_validate(p) == LACT_OK ? lact::rotary_bwd_workspace(p) : 0;
}

int lact_rotary_fwd(const lact_rotary_problem* p, const lact_tensor4* q, const lact_tensor4* k, const double* freqs,
                    const int32_t* positions, const float* q_scale, const float* q_offset, const float* k_scale,
                    const float* k_offset, const lact_tensor4* q_out, const lact_tensor4* k_out, void* stream) {
  using namespace lact;
  const int rc = rotary_validate(p);
  if (rc != LACT_OK) return rc;
  const int esz = p->dtype == LACT_BF16 ? 2 : 4;
  const Extent4 eq{p->B, p->H, p->T, p->d}, ek{p->B, p->Hkv, p->T, p->d};
  const bool has_k = p->Hkv > 0, affine = q_scale != nullptr;
  if (!freqs || !aligned16(freqs) || !aligned4(positions) || !view_ok(q, eq, esz) || !view_ok(q_out, eq, esz)) return LACT_EINVAL;
  if (has_k && (!view_ok(k, ek, esz) || !view_ok(k_out, ek, esz))) return LACT_EINVAL;
  const float* params[] = {q_scale, q_offset, k_scale, k_offset};
  for (int i = 0; i < (has_k ? 4 : 2); ++i)
    if ((params[i] != nullptr) != affine || !aligned16(params[i])) return LACT_EINVAL;
  const RotaryDims r = rotary_dims(p, false);
  RotaryParams a = rotary_params(p, r, freqs, positions);
  a.xq = view4(q, eq); a.yq = view4(q_out, eq);
  if (!injective(a.yq, eq)) return LACT_EINVAL;
  if (!same(a.xq, a.yq, eq) && !apart(a.xq, eq, a.yq, eq, esz)) return LACT_EINVAL;
  if (has_k) {
    a.xk = view4(k, ek); a.yk = view4(k_out, ek);
    if (!injective(a.yk, ek) || !apart(a.yq, eq, a.yk, ek, esz) || !apart(a.yq, eq, a.xk, ek, esz) ||
        !apart(a.xq, eq, a.yk, ek, esz) || (!same(a.xk, a.yk, ek) && !apart(a.xk, ek, a.yk, ek, esz)))
      return LACT_EINVAL;
  }
  a.q_scale = q_scale; a.q_offset = q_offset; a.k_scale = k_scale; a.k_offset = k_offset;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  Launcher L{false, st};
  L(K_ROTARY, [&] { return cleared(affine ? launch_rotary_any<false, true>(p, r, a, st) : launch_rotary_any<false, false>(p, r, a, st)); });
  return L.err;
}

int lact_rotary_bwd(const lact_rotary_problem* p, const lact_tensor4* dq_out, const lact_tensor4* dk_out,
                    const double* freqs, const int32_t* positions, const lact_tensor4* q, const lact_tensor4* k,
                    const float* q_scale, const float* k_scale, const lact_tensor4* dq, const lact_tensor4* dk,
                    float* dq_scale, float* dq_offset, float* dk_scale, float* dk_offset, void* workspace,
                    size_t workspace_bytes, void* stream) {
  using namespace lact;
  const int rc = rotary_validate(p);
  if (rc != LACT_OK) return rc;
  const int esz = p->dtype == LACT_BF16 ? 2 : 4;
  const Extent4 eq{p->B, p->H, p->T, p->d}, ek{p->B, p->Hkv, p->T, p->d};
  const bool has_k = p->Hkv > 0, affine = q_scale != nullptr;
  if (!freqs || !aligned16(freqs) || !aligned4(positions) || !view_ok(dq_out, eq, esz) || !view_ok(dq, eq, esz)) return LACT_EINVAL;
  if (has_k && (!view_ok(dk_out, ek, esz) || !view_ok(dk, ek, esz))) return LACT_EINVAL;
  if (has_k && (k_scale != nullptr) != affine) return LACT_EINVAL;
  if (!aligned16(q_scale) || !aligned16(k_scale)) return LACT_EINVAL;
  const RotaryDims r = rotary_dims(p, affine);
  RotaryParams a = rotary_params(p, r, freqs, positions);
  a.yq = view4(dq_out, eq); a.dq = view4(dq, eq);
  if (!injective(a.dq, eq) || (!same(a.yq, a.dq, eq) && !apart(a.yq, eq, a.dq, eq, esz))) return LACT_EINVAL;
  if (has_k) {
    a.yk = view4(dk_out, ek); a.dk = view4(dk, ek);
    if (!injective(a.dk, ek) || !apart(a.dq, eq, a.dk, ek, esz) || !apart(a.dq, eq, a.yk, ek, esz) ||
        !apart(a.yq, eq, a.dk, ek, esz) || (!same(a.yk, a.dk, ek) && !apart(a.yk, ek, a.dk, ek, esz)))
      return LACT_EINVAL;
  }
  if (affine) {
    if (!view_ok(q, eq, esz) || (has_k && !view_ok(k, ek, esz))) return LACT_EINVAL;
    a.xq = view4(q, eq);
    if (!apart(a.xq, eq, a.dq, eq, esz)) return LACT_EINVAL;
    if (has_k) {
      a.xk = view4(k, ek);
      if (!apart(a.xk, ek, a.dq, eq, esz) || !apart(a.xq, eq, a.dk, ek, esz) || !apart(a.xk, ek, a.dk, ek, esz))
        return LACT_EINVAL;
    }
    float* g[] = {dq_scale, dq_offset, dk_scale, dk_offset};
    for (int i = 0; i < (has_k ? 4 : 2); ++i) {
      const int64_t n = (i < 2 ? p->H : p->Hkv) * p->d * 4;
      if (!g[i] || !aligned16(g[i])) return LACT_EINVAL;
      if (!apart_from(a.dq, eq, esz, g[i], n) || (has_k && !apart_from(a.dk, ek, esz, g[i], n))) return LACT_EINVAL;
      for (int j = 0; j < i; ++j)
        if (overlaps(g[i], n, g[j], (j < 2 ? p->H : p->Hkv) * p->d * 4)) return LACT_EINVAL;
    }
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LACT_EINVAL;
    if (workspace_bytes < rotary_bwd_workspace(p)) return LACT_ENOSPC;
    a.partial = static_cast<float*>(workspace);
  }
  a.q_scale = q_scale; a.k_scale = k_scale;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  Launcher L{false, st};
  L(K_ROTARY, [&] { return cleared(affine ? launch_rotary_any<true, true>(p, r, a, st) : launch_rotary_any<true, false>(p, r, a, st)); });
  if (affine)
    L(K_ROTARY_SUMS, [&] {
      const int64_t n = 2 * (p->H + p->Hkv) * p->d;
      return cleared(launch_pdl(k_rotary_sums, dim3(static_cast<unsigned>(cdiv(n, 32))), dim3(512), 0, st,
                                static_cast<const float*>(a.partial), static_cast<int>(p->B * r.ranges), a.H, a.Hkv,
                                a.d, dq_scale, dq_offset, dk_scale, dk_offset));
    });
  return L.err;
}

int lact_swa_sink_fwd(const lact_swa_sink_problem* p, const lact_tensor4* q, const lact_tensor4* k,
                      const lact_tensor4* v, const int32_t* lengths, const lact_tensor4* out, float* lse,
                      void* stream) {
  using namespace lact;
  WattnDims D;
  const int rc = wattn_validate(p, D);
  if (rc != LACT_OK) return rc;
  const int esz = D.dtype == LACT_BF16 ? 2 : 4;
  const Extent4 eq{D.B, D.H, D.Tq, D.d}, ek{D.B, D.Hkv, D.T, D.d};
  if (!view_ok(q, eq, esz) || !view_ok(k, ek, esz) || !view_ok(v, ek, esz) || !view_ok(out, eq, esz)) return LACT_EINVAL;
  if (!lse || !aligned4(lse) || !aligned4(lengths)) return LACT_EINVAL;
  WattnParams a = wattn_params(D, p->scale, lengths, lse);
  a.q = view4(q, eq); a.k = view4(k, ek); a.v = view4(v, ek); a.out = view4(out, eq);
  if (!injective(a.out, eq) || !apart(a.q, eq, a.out, eq, esz) || !apart(a.k, ek, a.out, eq, esz) ||
      !apart(a.v, ek, a.out, eq, esz))
    return LACT_EINVAL;
  const int64_t n = D.B * D.H * D.Tq * 4;
  if (!apart_from(a.q, eq, esz, lse, n) || !apart_from(a.k, ek, esz, lse, n) || !apart_from(a.v, ek, esz, lse, n) ||
      !apart_from(a.out, eq, esz, lse, n))
    return LACT_EINVAL;
  Launcher L{false, static_cast<cudaStream_t>(stream)};
  wattn_fwd_run(D, a, static_cast<cudaStream_t>(stream), L);
  return L.err;
}

size_t lact_swa_sink_bwd_workspace_bytes(const lact_swa_sink_problem* p) {
  lact::WattnDims D;
  return lact::wattn_validate(p, D) == LACT_OK ? lact::wattn_bwd_workspace(D) : 0;
}

int lact_swa_sink_bwd(const lact_swa_sink_problem* p, const lact_tensor4* q, const lact_tensor4* k,
                      const lact_tensor4* v, const lact_tensor4* out, const float* lse, const lact_tensor4* dout,
                      const int32_t* lengths, const lact_tensor4* dq, const lact_tensor4* dk, const lact_tensor4* dv,
                      void* workspace, size_t workspace_bytes, void* stream) {
  using namespace lact;
  WattnDims D;
  const int rc = wattn_validate(p, D);
  if (rc != LACT_OK) return rc;
  const int esz = D.dtype == LACT_BF16 ? 2 : 4;
  const Extent4 eq{D.B, D.H, D.Tq, D.d}, ek{D.B, D.Hkv, D.T, D.d};
  const lact_tensor4* qs[] = {q, out, dout, dq};
  const lact_tensor4* ks[] = {k, v, dk, dv};
  for (const lact_tensor4* x : qs)
    if (!view_ok(x, eq, esz)) return LACT_EINVAL;
  for (const lact_tensor4* x : ks)
    if (!view_ok(x, ek, esz)) return LACT_EINVAL;
  if (!lse || !aligned4(lse) || !aligned4(lengths)) return LACT_EINVAL;
  WattnParams a = wattn_params(D, p->scale, lengths, lse);
  a.q = view4(q, eq); a.k = view4(k, ek); a.v = view4(v, ek); a.out = view4(out, eq); a.dout = view4(dout, eq);
  a.dq = view4(dq, eq); a.dk = view4(dk, ek); a.dv = view4(dv, ek);
  const View4 in[] = {a.q, a.out, a.dout, a.k, a.v}, res[] = {a.dq, a.dk, a.dv};
  for (int i = 0; i < 3; ++i) {
    const Extent4& e = i ? ek : eq;
    if (!injective(res[i], e) || !apart_from(res[i], e, esz, lse, D.B * D.H * D.Tq * 4)) return LACT_EINVAL;
    for (int j = 0; j < 5; ++j)
      if (!apart(res[i], e, in[j], j < 3 ? eq : ek, esz)) return LACT_EINVAL;
    for (int j = 0; j < i; ++j)
      if (!apart(res[i], e, res[j], j ? ek : eq, esz)) return LACT_EINVAL;
  }
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LACT_EINVAL;
  if (workspace_bytes < wattn_bwd_workspace(D)) return LACT_ENOSPC;
  Bump bp{reinterpret_cast<uintptr_t>(workspace), 0};
  WattnBufs b;
  wattn_bwd_plan(D, bp, b);
  a.delta = b.delta; a.part = b.part;
  Launcher L{false, static_cast<cudaStream_t>(stream)};
  wattn_bwd_run(D, a, static_cast<cudaStream_t>(stream), L);
  return L.err;
}

int lact_swa_sink_decode(const lact_swa_sink_problem* p, const lact_tensor4* q, const lact_tensor4* k,
                         const lact_tensor4* v, void* k_cache, void* v_cache, const int32_t* seen,
                         const lact_tensor4* out, void* stream) {
  using namespace lact;
  const int rc = decode_validate(p);
  if (rc != LACT_OK) return rc;
  if (p->T != 1 || p->Tq != 1) return LACT_EINVAL;
  const int esz = p->dtype == LACT_BF16 ? 2 : 4;
  const Extent4 eq{p->B, p->H, 1, p->d}, ek{p->B, p->Hkv, 1, p->d};
  if (!view_ok(q, eq, esz) || !view_ok(out, eq, esz) || !view_ok(k, ek, esz) || !view_ok(v, ek, esz)) return LACT_EINVAL;
  if (!seen || !aligned4(seen) || !k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)) return LACT_EINVAL;
  DecodeParams a;
  std::memset(&a, 0, sizeof(a));
  a.q = view4(q, eq); a.out = view4(out, eq); a.kn = view4(k, ek); a.vn = view4(v, ek);
  const int64_t bytes = p->B * p->Hkv * (p->sinks + p->window) * p->d * esz;
  if (overlaps(k_cache, bytes, v_cache, bytes) || !injective(a.out, eq)) return LACT_EINVAL;
  if (!apart(a.out, eq, a.q, eq, esz) || !apart(a.out, eq, a.kn, ek, esz) || !apart(a.out, eq, a.vn, ek, esz))
    return LACT_EINVAL;
  for (void* c : {k_cache, v_cache})
    if (!apart_from(a.q, eq, esz, c, bytes) || !apart_from(a.out, eq, esz, c, bytes) ||
        !apart_from(a.kn, ek, esz, c, bytes) || !apart_from(a.vn, ek, esz, c, bytes))
      return LACT_EINVAL;
  a.kc = k_cache; a.vc = v_cache; a.seen = seen; a.scale = p->scale;
  a.H = static_cast<int>(p->H); a.Hkv = static_cast<int>(p->Hkv); a.group = static_cast<int>(p->H / p->Hkv);
  a.d = static_cast<int>(p->d); a.window = static_cast<int>(p->window); a.sinks = static_cast<int>(p->sinks);
  a.hgroups = static_cast<int>(cdiv(a.group, kDecHeads));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  Launcher L{false, st};
  L(K_WATTN_DECODE, [&] { return cleared(launch_decode_any(rup(p->d, 64), p->dtype, a, p->B * p->Hkv * a.hgroups, st)); });
  return L.err;
}

int lact_swa_cache_fill(const lact_swa_sink_problem* p, const lact_tensor4* k, const lact_tensor4* v,
                        const int32_t* lengths, void* k_cache, void* v_cache, void* stream) {
  using namespace lact;
  if (!p) return LACT_EINVAL;
  lact_swa_sink_problem keys = *p;   // there are no queries
  keys.H = p->Hkv;
  const int rc = decode_validate(&keys);
  if (rc != LACT_OK) return rc;
  if (p->T < 1 || p->T > (int64_t(1) << 24)) return LACT_EINVAL;
  const int esz = p->dtype == LACT_BF16 ? 2 : 4;
  const Extent4 ek{p->B, p->Hkv, p->T, p->d};
  if (!view_ok(k, ek, esz) || !view_ok(v, ek, esz) || !aligned4(lengths)) return LACT_EINVAL;
  if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)) return LACT_EINVAL;
  FillParams a;
  std::memset(&a, 0, sizeof(a));
  a.k = view4(k, ek); a.v = view4(v, ek);
  const int64_t slots = p->sinks + p->window, bytes = p->B * p->Hkv * slots * p->d * esz;
  if (overlaps(k_cache, bytes, v_cache, bytes)) return LACT_EINVAL;
  for (void* c : {k_cache, v_cache})
    if (!apart_from(a.k, ek, esz, c, bytes) || !apart_from(a.v, ek, esz, c, bytes)) return LACT_EINVAL;
  a.kc = k_cache; a.vc = v_cache; a.lengths = lengths;
  a.n = p->B * p->Hkv * std::min(p->T, slots);
  a.Hkv = static_cast<int>(p->Hkv); a.T = static_cast<int>(p->T); a.row_vecs = static_cast<int>(p->d * esz / 16);
  a.window = static_cast<int>(p->window); a.sinks = static_cast<int>(p->sinks); a.esz = esz;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  Launcher L{false, st};
  L(K_WATTN_ELEM, [&] {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(cdiv(a.n * a.row_vecs, 256), kPlanSMs * 16)));
    return cleared(launch_pdl(k_wattn_fill, grid, dim3(256), 0, st, a));
  });
  return L.err;
}

}  // extern "C"
