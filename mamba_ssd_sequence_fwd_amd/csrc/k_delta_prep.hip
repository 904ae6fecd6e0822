// k_delta_prep.hip -- the triangular matrices of each chunk of the gated delta
// rule: T = (I + L)^-1 and M (delta.h), or T, T^T and M^T for the backward pass.
//
// One wave takes one chunk and a few heads of one group. K K^T and Q K^T are
// products of the group's rows, kept in registers for its heads as 16 x 16
// tiles on and below the diagonal, transposed: a lane holds 4 consecutive
// columns j of one row i. In that layout a tile of L is the left operand of
// the fp32 matrix instruction (lane l: row l % 16, columns 4 (l / 16) + r at
// step r) and a result tile its right operand, so the block inversion
//   T_ij = -T_ii sum_{j <= k < i} L_ik T_kj
// passes from product to product in registers, in fp32: T multiplies every
// value that enters the state. Only the four diagonal blocks go through LDS,
// where 64 lanes invert them at once by forward substitution, one column a
// lane. (Substitution, not powers of L: with equal keys the powers of a
// 16 x 16 block reach 6435 and cancel, the substitution's values stay within
// those of the inverse.)
#include "delta_tiles.h"

namespace ssd {

// Index of lower tile (i, j), j <= i.
__host__ __device__ constexpr int tri(int i, int j) { return i * (i + 1) / 2 + j; }

// acc[tri(i, j)] = rows j of X against rows i of Y (lane: row i % 16, 4
// columns j): 64 rows each, `ld` apart, N columns, rows past len read as the
// last one. Both products that share the rows K are taken in one walk.
template <typename T>
__device__ __forceinline__ void tri_products(const T *K, const T *Q, size_t ld, int N, int len,
                                             f32x4 (&kk)[10], f32x4 (&qk)[10], bool transposed_q) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
#pragma unroll
  for (int e = 0; e < 10; ++e) kk[e] = qk[e] = f32x4{0.f, 0.f, 0.f, 0.f};
  if constexpr (sizeof(T) == 2) {
    for (int n0 = 0; n0 < N; n0 += 32) {
      bf16x8 k[4], q[4];
      const int col = n0 + 8 * lg;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const size_t row = (size_t)min(16 * t + lr, len - 1) * ld + min(col, N - 8);
        k[t] = ldg8((const bf16 *)K + row);
        q[t] = ldg8((const bf16 *)Q + row);
        if (col >= N) k[t] = q[t] = zero8();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          kk[tri(i, j)] = mfma(k[j], k[i], kk[tri(i, j)]);
          qk[tri(i, j)] = transposed_q ? mfma(q[i], k[j], qk[tri(i, j)])
                                       : mfma(k[j], q[i], qk[tri(i, j)]);
        }
    }
  } else {
    for (int n0 = 0; n0 < N; n0 += 16) {
      f32x4 k[4], q[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const size_t row = (size_t)min(16 * t + lr, len - 1) * ld + n0 + 4 * lg;
        k[t] = *reinterpret_cast<const f32x4 *>(K + row);
        q[t] = *reinterpret_cast<const f32x4 *>(Q + row);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          kk[tri(i, j)] = mfma16(k[j], k[i], kk[tri(i, j)]);
          qk[tri(i, j)] = transposed_q ? mfma16(q[i], k[j], qk[tri(i, j)])
                                       : mfma16(k[j], q[i], qk[tri(i, j)]);
        }
    }
  }
}

// T (64, 64) fp32 rows, tiles above the diagonal not written.
__device__ __forceinline__ void store_rows_f32(float *to, int i, int j, f32x4 v) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  *reinterpret_cast<f32x4 *>(to + (16 * i + lr) * kDeltaChunk + 16 * j + 4 * lg) = v;
}

template <typename T, DeltaTri W>
__global__ __launch_bounds__(64) void k_delta_prep_f32(DeltaArgs a, int per) {
  __shared__ float sG[kDeltaChunk], sB[kDeltaChunk];
  __shared__ f32x4 sD[4][16][5];  // diagonal blocks: rows of L, then columns of T
  const int lane = threadIdx.x, lr = lane & 15, lg = lane >> 4;
  const int parts = (a.hpg + per - 1) / per;
  int unit = blockIdx.x;
  const int hp = unit % parts;
  unit /= parts;
  const int grp = unit % a.G, slot = unit / a.G;
  int64_t start;
  int len;
  if (!delta_chunk(a, slot, start, len)) return;

  f32x4 kk[10], qk[10];
  const size_t row0 = ((size_t)start * a.G + grp) * a.N;
  tri_products<T>((const T *)a.B + row0, (const T *)a.C + row0, (size_t)a.G * a.N, a.N, len, kk,
                  qk, W == kTriBackward);

  const int h1 = grp * a.hpg + min(a.hpg, (hp + 1) * per);
  for (int h = grp * a.hpg + hp * per; h < h1; ++h) {
    {
      const size_t at = (size_t)(start + min(lane, len - 1)) * a.H + h;
      const float gl = lane < len ? delta_log2_decay(ld<T>(a.g, at)) : 0.f;
      sG[lane] = wave_inclusive_sum(gl);
      sB[lane] = lane < len ? ld<T>(a.beta, at) : 0.f;
    }
    __syncthreads();
    f32x4 gr[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) gr[t] = *reinterpret_cast<const f32x4 *>(sG + 16 * t + 4 * lg);
    float *out = (float *)a.tri + ((size_t)slot * a.H + h) * ((W == kTriForward ? 2 : 3) * 4096);

    // L, and M beside it
    f32x4 Lt[10];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float gi = sG[16 * i + lr], bi = sB[16 * i + lr];
#pragma unroll
      for (int j = 0; j <= i; ++j) {
        f32x4 m;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool below = j < i || 4 * lg + r < lr;
          const float e = exp2_fast(gi - gr[j][r]);
          Lt[tri(i, j)][r] = below ? bi * kk[tri(i, j)][r] * e : 0.f;
          if (W == kTriForward) m[r] = below || 4 * lg + r == lr ? qk[tri(i, j)][r] * e : 0.f;
        }
        if (W == kTriForward) store_rows_f32(out + 4096, i, j, m);
      }
    }
    if (W == kTriBackward) {  // M^T: lane holds column j, 4 rows i
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float gj = sG[16 * j + lr];
#pragma unroll
        for (int i = j; i < 4; ++i) {
          f32x4 m;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            m[r] = j < i || lr <= 4 * lg + r ? qk[tri(i, j)][r] * exp2_fast(gr[i][r] - gj) : 0.f;
          store_rows_f32(out + 8192, j, i, m);
        }
      }
    }

    // diagonal blocks: lane (b, j) = (lg, lr) takes column j of block b
#pragma unroll
    for (int b = 0; b < 4; ++b) sD[b][lr][lg] = Lt[tri(b, b)];
    __syncthreads();
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == lr ? 1.f : 0.f;
#pragma unroll
      for (int q = 0; q < (i + 3) / 4; ++q) {
        const f32x4 l = sD[lg][i][q];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (4 * q + r < i) v -= l[r] * t[4 * q + r];
      }
      t[i] = v;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      sD[lg][lr][q] = f32x4{t[4 * q], t[4 * q + 1], t[4 * q + 2], t[4 * q + 3]};
    __syncthreads();
    f32x4 Tt[10], Ta[4];  // Tt: lane column j, 4 rows i; Ta: lane row i, 4 columns
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      Tt[tri(b, b)] = sD[b][lr][lg];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        Ta[b][r] = reinterpret_cast<const float *>(&sD[b][4 * lg + r][0])[lr];
      store_rows_f32(out, b, b, Ta[b]);
      if (W == kTriBackward) store_rows_f32(out + 4096, b, b, Tt[tri(b, b)]);
    }
#pragma unroll
    for (int d = 1; d < 4; ++d)
#pragma unroll
      for (int j = 0; j + d < 4; ++j) {
        const int i = j + d;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = j; k < i; ++k) x = mfma16(Lt[tri(i, k)], Tt[tri(k, j)], x);
        x = -x;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        Tt[tri(i, j)] = mfma16(Ta[i], x, zero);
        store_rows_f32(out, i, j, mfma16(x, Ta[i], zero));
        if (W == kTriBackward) store_rows_f32(out + 4096, j, i, Tt[tri(i, j)]);
      }
    __syncthreads();
  }
}

size_t delta_tri_bytes(bool bf16_path, DeltaTri which) {
  return (size_t)(which == kTriForward ? 2 : 3) * 4096 * sizeof(float);
}

hipError_t launch_delta_prep(const DeltaArgs &a, bool bf16_io, DeltaTri which, hipStream_t s) {
  if (a.nslots == 0) return hipSuccess;
  const int per = 1;
  const dim3 grid((unsigned)((int64_t)a.nslots * a.G * ((a.hpg + per - 1) / per))), block(64);
  if (bf16_io) {
    if (which == kTriForward)
      hipLaunchKernelGGL((k_delta_prep_f32<bf16, kTriForward>), grid, block, 0, s, a, per);
    else
      hipLaunchKernelGGL((k_delta_prep_f32<bf16, kTriBackward>), grid, block, 0, s, a, per);
  } else {
    if (which == kTriForward)
      hipLaunchKernelGGL((k_delta_prep_f32<float, kTriForward>), grid, block, 0, s, a, per);
    else
      hipLaunchKernelGGL((k_delta_prep_f32<float, kTriBackward>), grid, block, 0, s, a, per);
  }
  return hipGetLastError();
}

}  // namespace ssd
