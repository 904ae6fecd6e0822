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
// A chunk's matrices in a row, each in kTriLevels bf16 or fewer, level by level: the
// values rounded, and what the roundings before left, rounded.
constexpr int kTriTiles = 5, kTileElems = 512, kTriLevels = 3;
constexpr int kLevelElems = kTriTiles * kTileElems, kMatrixElems = kTriLevels * kLevelElems;
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

// Place (in elements) of (row, col) in a staged tile with rows of W bf16: the
// 16-byte pieces of a row are permuted so that the 256 bytes which LDS gives at
// once hold 16 rows of one piece (a row operand), and two neighbouring pieces of
// 8 rows, 0 to 7 or 0 to 3 and 8 to 11 (a transposed read).
template <int W>
__device__ __forceinline__ int tile_swizzle(int row) {
  if (W >= 128) {
    const int h = (row & 3) | ((((row >> 2) ^ (row >> 3)) & 1) << 2);
    return 2 * h + ((row >> 3) & 1);
  }
  if (W == 64) return 2 * (((row >> 1) & 1) | ((((row >> 2) ^ (row >> 3)) & 1) << 1)) + ((row >> 3) & 1);
  if (W == 32) return 2 * (((row >> 2) ^ (row >> 3)) & 1) + ((row >> 3) & 1);
  return (row >> 3) & 1;
}
template <int W>
__device__ __forceinline__ int place(int row, int col) {
  return row * W + (((col >> 3) ^ tile_swizzle<W>(row)) << 3) + (col & 7);
}

// ROWS rows of W columns (row stride ld; zeros from column n and row len on) into
// such a tile, asynchronously, by WV waves; and `n` KiB in a row.
template <int W, int ROWS, int WV, bool kAnew = false>
__device__ void stage_tile(bf16 *tile, const bf16 *src, size_t ld, int n, int len);
// The same of K such tiles of one shape.
template <int W, int ROWS, int WV, bool kAnew, int K>
__device__ void stage_tiles(bf16 *const (&tile)[K], const bf16 *const (&src)[K], size_t ld, int n,
                            int len);
template <int WV>
__device__ void stage_block(bf16 *to, const void *src, int n);

#ifdef __HIP_DEVICE_COMPILE__  // (the host pass has no type for buffer descriptors)
// Buffer descriptor of `bytes` from p: loads past them give zeros.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void *p, uint32_t bytes) {
  constexpr int kRaw = 0x00027000;  // untyped dwords
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, bytes, kRaw);
}

// Only the descriptor changes from call to call: a lane's offset stays in one
// register (kAnew: in none, it is worked out again).
template <int W, int ROWS, int WV, bool kAnew, int K>
__device__ __forceinline__ void stage_tiles(bf16 *const (&tile)[K], const bf16 *const (&src)[K],
                                            size_t ld, int n, int len) {
  constexpr int R = 512 / W, NI = ROWS / R;  // rows of an instruction, instructions
  constexpr int kSame = WV * R % 16 == 0 ? 1 : 16 / (WV * R);  // until the swizzle repeats
  int lane = threadIdx.x & 63;
  if (kAnew) asm volatile("" : "+v"(lane));
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rl = lane / (W / 8), pc = lane % (W / 8);
  uint32_t off[kSame];
#pragma unroll
  for (int k = 0; k < kSame; ++k) {
    const int s = (wave + WV * k) * R + rl, c = pc ^ tile_swizzle<W>(s);
    off[k] = 8 * c < n ? (uint32_t)s * (uint32_t)(ld * 2) + 16u * (uint32_t)c : 0x80000000u;
  }
#pragma unroll
  for (int t = 0; t < K; ++t) {
    const Buffer rows =
        buffer_of(src[t], (uint32_t)(len - 1) * (uint32_t)(ld * 2) + 2u * (uint32_t)n);
#pragma unroll
    for (int k = 0; k < (NI + WV - 1) / WV; ++k) {
      if (NI % WV != 0 && wave + WV * k >= NI) break;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rows, (lds_void *)(tile[t] + (wave + WV * k) * 512), 16,
          off[k % kSame] + (uint32_t)(k / kSame * kSame * WV * R) * (uint32_t)(ld * 2), 0, 0, 0);
    }
  }
}
template <int W, int ROWS, int WV, bool kAnew>
__device__ __forceinline__ void stage_tile(bf16 *tile, const bf16 *src, size_t ld, int n, int len) {
  bf16 *const t[1] = {tile};
  const bf16 *const s[1] = {src};
  stage_tiles<W, ROWS, WV, kAnew>(t, s, ld, n, len);
}
template <int WV>
__device__ __forceinline__ void stage_block(bf16 *to, const void *src, int n) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Buffer block = buffer_of(src, (uint32_t)n * 1024u);
  for (int m = wave; m < n; m += WV)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(block, (lds_void *)(to + m * 512), 16,
                                             lane * 16 + m * 1024, 0, 0, 0);
}
#endif

// Eight values of an operand in two bf16 each (2^-17 off), or three (2^-26).
struct Split {
  bf16x8 hi, lo;
};
struct Split3 {
  bf16x8 hi, mid, lo;
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
__device__ __forceinline__ Split3 split8x3(f32x4 a, f32x4 b) {
  Split3 s;
  s.hi = pack8(a, b);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    a[r] -= (float)s.hi[r];
    b[r] -= (float)s.hi[4 + r];
  }
  const Split rest = split8(a, b);
  s.mid = rest.hi;
  s.lo = rest.lo;
  return s;
}

}  // namespace ssd
