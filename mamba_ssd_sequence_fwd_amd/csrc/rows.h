// rows.h -- eight consecutive channels of one token row, as a lane holds them:
// loads, exact widening to fp32 and rounded stores for bf16 and fp32 rows, the
// 8-bit checkpoint form of a row, and SiLU. Shared by the kernels that stream
// token rows (convolution front, group norm, checkpoints).
#pragma once

#include "ssd_internal.h"

namespace ssd {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Two values rounded to nearest even, in one instruction as a pair.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Eight consecutive elements of one row, widened exactly to fp32, and back.
// load_once reads with the nontemporal hint, for rows no other lane reads.
// Rows are stored with nontemporal stores: nothing in the call reads them
// again, and keeping them out of the caches was measured 20-25% faster on the
// 2.7B-shaped front (nontemporal loads as well were slower).
template <typename T> struct Row8;
template <> struct Row8<bf16> {
  uint4 q;
  __device__ __forceinline__ void load(const void *p, size_t i) {
    q = *reinterpret_cast<const uint4 *>(static_cast<const bf16 *>(p) + i);
  }
  __device__ __forceinline__ void load_once(const void *p, size_t i) {
    const u32x4_t v = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4_t *>(static_cast<const bf16 *>(p) + i));
    q = make_uint4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void *p, size_t i, const float (&v)[8]) {
    u32x4_t q;
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
    __builtin_nontemporal_store(q, reinterpret_cast<u32x4_t *>(static_cast<bf16 *>(p) + i));
  }
};
template <> struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void *p, size_t i) {
    const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    a = s[0];
    b = s[1];
  }
  __device__ __forceinline__ void load_once(const void *p, size_t i) {
    const f32x4_t *s = reinterpret_cast<const f32x4_t *>(static_cast<const float *>(p) + i);
    const f32x4_t u = __builtin_nontemporal_load(s), v = __builtin_nontemporal_load(s + 1);
    a = make_float4(u[0], u[1], u[2], u[3]);
    b = make_float4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ __forceinline__ void store(void *p, size_t i, const float (&v)[8]) {
    f32x4_t *d = reinterpret_cast<f32x4_t *>(static_cast<float *>(p) + i);
    const f32x4_t lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
    __builtin_nontemporal_store(lo, d);
    __builtin_nontemporal_store(hi, d + 1);
  }
};

// Four consecutive elements of one row, for kernels that hold much per channel.
template <typename T> struct Row4;
template <> struct Row4<bf16> {
  uint2 q;
  __device__ __forceinline__ void load(const void *p, size_t i) {
    q = *reinterpret_cast<const uint2 *>(static_cast<const bf16 *>(p) + i);
  }
  __device__ __forceinline__ void widen(float (&v)[4]) const {
    v[0] = __uint_as_float(q.x << 16);
    v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16);
    v[3] = __uint_as_float(q.y & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(void *p, size_t i, const float (&v)[4]) {
    u32x2_t q;
#pragma unroll
    for (int k = 0; k < 2; ++k) q[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
    __builtin_nontemporal_store(q, reinterpret_cast<u32x2_t *>(static_cast<bf16 *>(p) + i));
  }
};
template <> struct Row4<float> {
  float4 a;
  __device__ __forceinline__ void load(const void *p, size_t i) {
    a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
  }
  __device__ __forceinline__ void widen(float (&v)[4]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
  static __device__ __forceinline__ void store(void *p, size_t i, const float (&v)[4]) {
    const f32x4_t q = {v[0], v[1], v[2], v[3]};
    __builtin_nontemporal_store(q, reinterpret_cast<f32x4_t *>(static_cast<float *>(p) + i));
  }
};

// v * sigmoid(v) on the hardware exp and reciprocal units: for very negative
// v the exponential overflows to +inf and the result is -0, for very
// positive v it is v.
__device__ __forceinline__ float silu(float v) {
  constexpr float kLog2e = 1.4426950408889634f;
  return v * __builtin_amdgcn_rcpf(1.f + exp2_fast(-v * kLog2e));
}

// sigmoid(v), the same way. silu(v) = v s and silu'(v) = s (1 + v (1 - s)):
// for very negative v both are 0 (s is exactly 0 there, v finite).
__device__ __forceinline__ float sigmoid(float v) {
  constexpr float kLog2e = 1.4426950408889634f;
  return __builtin_amdgcn_rcpf(1.f + exp2_fast(-v * kLog2e));
}

// ---- 8-bit checkpoint rows ---------------------------------------------------
// Blocks of kCkptBlock consecutive channels of a row share a step 2^s, the
// least power of two (s >= -125) for which the block's largest magnitude
// rounds to at most 127 steps; each element is kept as the nearest whole
// number of steps (int8, ties to even), so it is off by at most half a step.
// The block's byte is s + 127, the exponent field of the step itself:
// decoding is a shift and a product that is exact, in bf16 too (7 bits; only
// the last 0.4% of fp32's range rounds past it, to infinity). A
// block that holds an infinity or NaN has byte 255 and zeros: the step reads
// as infinity and 0 * infinity decodes to NaN with no test.
constexpr int kCkptBlock = 32;
constexpr int kCkptLanes = kCkptBlock / 8;  // lanes that share a block

__host__ __device__ inline int ckpt_blocks(int channels) {
  return (channels + kCkptBlock - 1) / kCkptBlock;
}

// A checkpoint of (rows, channels): contiguous.
struct Ckpt {
  int8_t *q;    // (rows, channels)
  uint8_t *e;   // (rows, ckpt_blocks(channels))
};

// Eight channels of a checkpoint row.
struct RowQ8 {
  uint2 q;
  uint32_t e;
  __device__ __forceinline__ void load(const Ckpt &k, size_t row, int channels, int c0) {
    q = *reinterpret_cast<const uint2 *>(k.q + row * channels + c0);
    e = k.e[row * ckpt_blocks(channels) + c0 / kCkptBlock];
  }
  __device__ __forceinline__ void load_once(const Ckpt &k, size_t row, int channels, int c0) {
    const u32x2_t v = __builtin_nontemporal_load(
        reinterpret_cast<const u32x2_t *>(k.q + row * channels + c0));
    q = make_uint2(v[0], v[1]);
    e = k.e[row * ckpt_blocks(channels) + c0 / kCkptBlock];
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    const float step = __uint_as_float(e << 23);
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = step * (float)(((int32_t)(w[k / 4] << (24 - 8 * (k & 3)))) >> 24);
  }
};

// Four channels of a checkpoint row.
struct RowQ4 {
  uint32_t q, e;
  __device__ __forceinline__ void load(const Ckpt &k, size_t row, int channels, int c0) {
    q = *reinterpret_cast<const uint32_t *>(k.q + row * channels + c0);
    e = k.e[row * ckpt_blocks(channels) + c0 / kCkptBlock];
  }
  __device__ __forceinline__ void widen(float (&v)[4]) const {
    const float step = __uint_as_float(e << 23);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = step * (float)(((int32_t)(q << (24 - 8 * k))) >> 24);
  }
};

// Maximum over the four lanes of a quad (all four must be active).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  constexpr int kXor1 = 0xb1, kXor2 = 0x4e;  // quad_perm [1,0,3,2] and [2,3,0,1]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kXor1, 0xf, 0xf, true));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kXor2, 0xf, 0xf, true));
}

// Quantise a lane's N = 8 or 4 channels; the lanes of a quad or of two
// neighbouring quads hold one block (lanes past the last channel hold zeros).
// Rounding to nearest even comes from one fused multiply-add onto 1.5 * 2^23,
// whose low byte is then the int8: the product by a power of two is exact.
template <int N>
__device__ __forceinline__ void quantise(const float (&v)[N], uint32_t (&q)[N / 4], uint32_t &e) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
  m = quad_max(m);
  if (N == 4) {
    constexpr int kHalfMirror = 0x141;  // the other quad of eight lanes
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kHalfMirror, 0xf, 0xf, true));
  }
  // the exponent field of the step: 127 steps hold the block unless its
  // largest mantissa is at least 127.5 / 64, which rounds up to 128
  const bool bad = m >= 0x7f800000u;
  const int b = max((int)((m + 0x10000u) >> 23) - 6, 2);
  const float inv = __uint_as_float((uint32_t)(254 - min(b, 249)) << 23);
  uint32_t w[N];
#pragma unroll
  for (int k = 0; k < N; ++k) w[k] = __float_as_uint(__builtin_fmaf(v[k], inv, 12582912.f));
  // low bytes of four words into one
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    const uint32_t lo = __builtin_amdgcn_perm(w[4 * k + 1], w[4 * k], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(w[4 * k + 3], w[4 * k + 2], 0x04000c0cu);
    q[k] = bad ? 0u : lo | hi;
  }
  e = bad ? 255u : (uint32_t)b;
}

// Store a lane's part of a checkpoint row (the first lane of each block
// stores its byte); `live` is false on lanes past the last channel.
template <int N>
__device__ __forceinline__ void store_ckpt(const Ckpt &k, size_t row, int channels, int c0,
                                           const float (&v)[N], bool live) {
  uint32_t q[N / 4], e;
  quantise<N>(v, q, e);
  if (live) {
    int8_t *to = k.q + row * channels + c0;
    if constexpr (N == 8) {
      const u32x2_t s = {q[0], q[1]};
      __builtin_nontemporal_store(s, reinterpret_cast<u32x2_t *>(to));
    } else {
      __builtin_nontemporal_store(q[0], reinterpret_cast<uint32_t *>(to));
    }
    if (c0 % kCkptBlock == 0)
      k.e[row * ckpt_blocks(channels) + c0 / kCkptBlock] = (uint8_t)e;
  }
}

}  // namespace ssd
