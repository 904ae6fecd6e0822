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

constexpr f32x4 kZero4 = {0.f, 0.f, 0.f, 0.f};

__device__ __forceinline__ f32x4 ldf4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
__device__ __forceinline__ void stf4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }

// Four consecutive elements widened to fp32.
__device__ __forceinline__ f32x4 widen4(const float *p) { return ldf4(p); }
__device__ __forceinline__ f32x4 widen4(const bf16 *p) {
  const bf16x4 v = *reinterpret_cast<const bf16x4 *>(p);
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
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
