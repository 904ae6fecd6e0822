// delta_tiles.h -- fp32 matrix-instruction tiles shared by the gated delta
// rule's kernels (v_mfma_f32_16x16x4_f32: 16 of k in four steps).
#pragma once

#include "delta.h"
#include "mfma_common.h"

namespace ssd {

// c += A B over 16 of k: lane l holds row (A) or column (B) l % 16, and of k
// 4 (l / 16) + r in element r; c holds column l % 16, rows 4 (l / 16) + r, so
// a result tile is the B operand of the next product over its rows.
__device__ __forceinline__ f32x4 mfma16(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
  return c;
}

// A triangular matrix on the bf16 path: operand tiles (16 rows x 32 of k, in lane
// order, 8 of k a lane), of which the diagonal leaves four whole and two half
// empty. Those two share the fifth tile's 16 bytes a lane.
//   lower, rows i, k columns: (0,0)h (1,0) (2,0) (3,0) (2,1)h (3,1)
//   upper:                    (0,0) (0,1) (1,0)h (1,1) (2,1) (3,1)h
constexpr int kTriTiles = 5, kTileElems = 512;
__host__ __device__ constexpr int lower_tile(int i, int ks) {
  return i == 0 || (i == 2 && ks == 1) ? 4 : ks == 0 ? i - 1 : 3;
}
__host__ __device__ constexpr int upper_tile(int i, int ks) {
  return i == 3 || (i == 1 && ks == 0) ? 4 : i + ks;
}
// Of the 8 of k that a lane holds of a shared tile, which 4: the second operand's
// are the last. In the operand they are the first 4 (lower) or last 4 (upper).
__device__ __forceinline__ bf16x8 lower_operand(bf16x8 t, int i, int ks) {
  const bf16 z = (bf16)0.f;
  if (i == 0) return bf16x8{t[0], t[1], t[2], t[3], z, z, z, z};
  if (i == 2 && ks == 1) return bf16x8{t[4], t[5], t[6], t[7], z, z, z, z};
  return t;
}
__device__ __forceinline__ bf16x8 upper_operand(bf16x8 t, int i, int ks) {
  const bf16 z = (bf16)0.f;
  if (i == 1 && ks == 0) return bf16x8{z, z, z, z, t[0], t[1], t[2], t[3]};
  if (i == 3) return bf16x8{z, z, z, z, t[4], t[5], t[6], t[7]};
  return t;
}

constexpr f32x4 kZero4 = {0.f, 0.f, 0.f, 0.f};

__device__ __forceinline__ f32x4 ldf4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
__device__ __forceinline__ void stf4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }

// Four consecutive elements widened to fp32.
__device__ __forceinline__ f32x4 widen4(const float *p) { return ldf4(p); }
__device__ __forceinline__ f32x4 widen4(const bf16 *p) {
  const bf16x4 v = *reinterpret_cast<const bf16x4 *>(p);
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

// Eight values of an operand in two bf16 each.
struct Split {
  bf16x8 hi, lo;
};
__device__ __forceinline__ bf16x8 pack8(f32x4 a, f32x4 b) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 v = {pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(b[0], b[1]), pack2(b[2], b[3])};
  return __builtin_bit_cast(bf16x8, v);
}
// a, b as two bf16 each: rounded, and the rest rounded.
__device__ __forceinline__ Split split8(f32x4 a, f32x4 b) {
  Split s;
  s.hi = pack8(a, b);
  f32x4 ra, rb;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    ra[r] = a[r] - (float)s.hi[r];
    rb[r] = b[r] - (float)s.hi[4 + r];
  }
  s.lo = pack8(ra, rb);
  return s;
}

// Stage `len` of 64 token rows (ld apart, N columns) as fp32 rows of W floats
// in LDS; the rest is zero.
template <int W, typename T>
__device__ __forceinline__ void stage_rows_f32(float *to, const T *from, size_t ld, int N, int len) {
  for (int e = threadIdx.x; e < kDeltaChunk * (W / 4); e += blockDim.x) {
    const int t = e / (W / 4), c = 4 * (e % (W / 4));
    f32x4 v = kZero4;
    if (t < len && c < N) v = widen4(from + t * ld + c);
    stf4(to + t * W + c, v);
  }
}

// Decay prefix (base 2) and write strengths of a chunk, by the first wave.
template <typename T>
__device__ __forceinline__ void stage_gates(float *sG, float *sB, const DeltaArgs &a, int64_t start,
                                            int h, int len) {
  if (threadIdx.x < kDeltaChunk) {
    const int t = threadIdx.x;
    const size_t at = (size_t)(start + min(t, len - 1)) * a.H + h;
    const float gl = t < len ? delta_log2_decay(ld<T>(a.g, at)) : 0.f;
    sG[t] = wave_inclusive_sum(gl);
    sB[t] = t < len ? ld<T>(a.beta, at) : 0.f;
  }
}

}  // namespace ssd
