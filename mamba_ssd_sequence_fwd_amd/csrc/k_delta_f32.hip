// k_delta_f32.hip -- the gated delta rule's chunks in fp32 arithmetic
// (delta.h has the formulas): the walk over a sequence's chunks, the same
// walk backwards, and the gradients of each chunk.
//
// The columns of the state (one per value channel) never mix, so a wave takes
// 16 of them through all chunks with the state in registers: S is a stack of
// 16 x 16 result tiles (rows: state channels n), and every product of the walk
// contracts over the rows of tiles that the wave holds already (S, R, U),
// which makes them right operands as they are. The left operands, rows of K
// and Q, are staged in LDS for the workgroup's waves; T and M (k_delta_prep's)
// come through the caches into registers. The bound is the fp32 matrix rate (1/16 of
// the bf16 rate): 68 products of 16 x 16 x 16 a chunk and wave at N = 64, 4.1 us.
// Measured (MI355X), 36 sequences and heads of 64 x 64 and 5 chunks: 44 us, 36
// workgroups on 36 compute units, a chunk every 8.8 us (its rows staged, its four
// products one after the other); 48 and up to 8: the two walks of the backward pass 73
// us together (about 135 one after the other), the gradients 43 us. Every sequence is
// walked whole: 1 x 16384 tokens of 32 heads of 128 x 128 take 3330 us.
#include "delta_tiles.h"

namespace ssd {

// `len` of 64 token rows of K and Q (or of K alone: null), N columns each, as rows
// of 16 NT + 4 floats in LDS (the last 4 are for the banks), the rest zero. All of a
// thread's loads for up to 128 columns are on their way at once (one after the other
// they took as long as the chunk's products).
template <int NT>
__device__ __forceinline__ void stage_rows(float *toK, float *toQ, const float *K, const float *Q,
                                           size_t ld, int N, int len) {
  constexpr int W = 16 * NT + 4, kRow = 4 * NT, kAll = kDeltaChunk * kRow;
  constexpr int kAtOnce = NT < 8 ? NT : 8;
  for (int e0 = threadIdx.x; e0 < kAll; e0 += kAtOnce * (int)blockDim.x) {
    f32x4 k[kAtOnce], q[kAtOnce];
#pragma unroll
    for (int b = 0; b < kAtOnce; ++b) {
      const int e = e0 + b * (int)blockDim.x, t = e / kRow, c = 4 * (e % kRow);
      const size_t at = (size_t)min(t, len - 1) * ld + min(c, N - 4);
      k[b] = ldf4(K + at);
      if (Q) q[b] = ldf4(Q + at);
    }
#pragma unroll
    for (int b = 0; b < kAtOnce; ++b) {
      const int e = e0 + b * (int)blockDim.x, t = e / kRow, c = 4 * (e % kRow);
      const bool in = t < len && c < N;
      stf4(toK + t * W + c, in ? k[b] : kZero4);
      if (Q) stf4(toQ + t * W + c, in ? q[b] : kZero4);
    }
  }
}

// decay_sums (sG and sE) and write strengths of a chunk, by the first wave.
__device__ __forceinline__ void stage_gates(float *sG, float *sE, float *sB, const DeltaArgs &a, int64_t start,
                                            int h, int len) {
  if (threadIdx.x < kDeltaChunk) {
    const int t = threadIdx.x;
    const size_t at = (size_t)(start + min(t, len - 1)) * a.H + h;
    const float gl = t < len ? delta_log2_decay(((const float *)a.g)[at]) : 0.f;
    const DecaySum gam = decay_sums(gl);
    sG[t] = gam.hi;
    sE[t] = gam.lo;
    sB[t] = t < len ? ((const float *)a.beta)[at] : 0.f;
  }
}

// Left operand from staged rows: K^T (row n0 + lr, tokens t0 + 4 lg + r).
template <int W>
__device__ __forceinline__ f32x4 column_operand(const float *rows, int t0, int n0) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const float *p = rows + (t0 + 4 * lg) * W + n0 + lr;
  return f32x4{p[0], p[W], p[2 * W], p[3 * W]};
}
template <int W>
__device__ __forceinline__ f32x4 row_operand(const float *rows, int t0, int n0) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  return ldf4(rows + (t0 + lr) * W + n0 + 4 * lg);
}

// 16 columns from p0 of 4 token rows (t0 + 4 lg + r), zeros past len.
__device__ __forceinline__ f32x4 value_tile(const float *v, size_t ld, int t0, int len) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  f32x4 o;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int t = t0 + 4 * lg + r;
    const float x = v[min(t, len - 1) * ld + lr];
    o[r] = t < len ? x : 0.f;
  }
  return o;
}

// Forward (kStates false): y and the final state. For the backward pass
// (kStates true): the state entering each chunk, as (P, N), and U.
template <int NT, bool kStates>
__device__ __forceinline__ void chain_f32(const DeltaArgs &a, int unit, float *lds) {
  constexpr int W = 16 * NT + 4;
  float *sG = lds, *sE = sG + kDeltaChunk, *sB = sE + kDeltaChunk, *sK = sB + kDeltaChunk;
  float *sQ = sK + kDeltaChunk * W;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int waves = blockDim.x >> 6, blocks = a.P / (16 * waves);
  const int p0 = ((unit % blocks) * waves + (threadIdx.x >> 6)) * 16;
  unit /= blocks;
  const int h = unit % a.H, seq = unit / a.H, grp = h / a.hpg;
  int64_t lo, hi;
  delta_seq(a, seq, lo, hi);
  const int slot0 = delta_slot0(a, seq, lo);
  const size_t srow = (((size_t)seq * a.H + h) * a.P + p0 + lr) * a.N + 4 * lg;

  f32x4 S[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    S[n] = a.h0 && 16 * n < a.N ? ldf4(a.h0 + srow + 16 * n) : kZero4;

  const size_t ldk = (size_t)a.G * a.N, ldx = (size_t)a.H * a.P;
  int c = 0;
  for (int64_t at = lo; at < hi; at += kDeltaChunk, ++c) {
    const int len = (int)min((int64_t)kDeltaChunk, hi - at);
    const size_t sh = (size_t)(slot0 + c) * a.H + h;
    __syncthreads();
    const size_t rows = (at * a.G + grp) * a.N;
    stage_rows<NT>(sK, sQ, (const float *)a.B + rows, kStates ? nullptr : (const float *)a.C + rows,
                  ldk, a.N, len);
    stage_gates(sG, sE, sB, a, at, h, len);
    // (on their way while K S is computed)
    const float *tri = (const float *)a.tri + sh * ((kStates ? 3 : 2) * 4096);
    const float *x = (const float *)a.x + ((size_t)at * a.H + h) * a.P + p0;
    f32x4 V[4], T[10], M[10];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      V[i] = value_tile(x, ldx, 16 * i, len);
#pragma unroll
      for (int j = 0; j <= i; ++j) {
        const int e = (16 * i + lr) * kDeltaChunk + 16 * j + 4 * lg;
        T[i * (i + 1) / 2 + j] = ldf4(tri + e);
        if (!kStates) M[i * (i + 1) / 2 + j] = ldf4(tri + 4096 + e);
      }
    }
    __syncthreads();

    f32x4 R[4], O[4], U[4], e[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4 ks = kZero4, qs = kZero4;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        ks = mfma16(row_operand<W>(sK, 16 * t, 16 * n), S[n], ks);
        if (!kStates) qs = mfma16(row_operand<W>(sQ, 16 * t, 16 * n), S[n], qs);
      }
      const f32x4 gm = ldf4(sG + 16 * t + 4 * lg), b = ldf4(sB + 16 * t + 4 * lg);
      const f32x4 v = V[t];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        e[t][r] = exp2_fast(gm[r]);
        R[t][r] = b[r] * (v[r] - e[t][r] * ks[r]);
        O[t][r] = e[t][r] * qs[r];
      }
    }
    const float gc = sG[kDeltaChunk - 1], rc = sE[kDeltaChunk - 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      U[i] = kZero4;
#pragma unroll
      for (int j = 0; j <= i; ++j)
        U[i] = mfma16(T[i * (i + 1) / 2 + j], R[j], U[i]);
    }
    if (!kStates) {
      float *y = (float *)a.y + ((size_t)at * a.H + h) * a.P + p0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j <= i; ++j)
          O[i] = mfma16(M[i * (i + 1) / 2 + j], U[j], O[i]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * i + 4 * lg + r;
          if (t < len) y[t * ldx + lr] = O[i][r];
        }
      }
    } else {
      float *st = (float *)a.st0 + (sh * a.P + p0 + lr) * a.N + 4 * lg;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (16 * n < a.N) stf4(st + 16 * n, S[n]);
      float *u = (float *)a.u + sh * kDeltaChunk * a.P + p0 + lr;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) u[(16 * i + 4 * lg + r) * a.P] = U[i][r];
    }
    const float ec = exp2_fast(gc);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4 d = (gc - ldf4(sG + 16 * t + 4 * lg)) + (rc - ldf4(sE + 16 * t + 4 * lg));
#pragma unroll
      for (int r = 0; r < 4; ++r) U[t][r] *= exp2_fast(d[r]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      S[n] *= ec;
#pragma unroll
      for (int t = 0; t < 4; ++t) S[n] = mfma16(column_operand<W>(sK, 16 * t, 16 * n), U[t], S[n]);
    }
  }
  if (a.hT && !kStates) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (16 * n < a.N) stf4(a.hT + srow + 16 * n, S[n]);
  }
}

// Backwards: dL/dS entering from behind each chunk, as (P, N), dL/dR, and the
// gradient of the initial state.
//   dU = M^T dY + e^{gam_c - gam} (K dS),  dR = T^T dU
//   dS <- e^{gam_c} dS + Q^T (e^gam dY) - K^T (beta e^gam dR)
template <int NT>
__device__ __forceinline__ void reverse_f32(const DeltaArgs &a, int unit, float *lds) {
  constexpr int W = 16 * NT + 4;
  float *sG = lds, *sE = sG + kDeltaChunk, *sB = sE + kDeltaChunk, *sK = sB + kDeltaChunk;
  float *sQ = sK + kDeltaChunk * W;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int waves = blockDim.x >> 6, blocks = a.P / (16 * waves);
  const int p0 = ((unit % blocks) * waves + (threadIdx.x >> 6)) * 16;
  unit /= blocks;
  const int h = unit % a.H, seq = unit / a.H, grp = h / a.hpg;
  int64_t lo, hi;
  delta_seq(a, seq, lo, hi);
  const int slot0 = delta_slot0(a, seq, lo);
  const size_t srow = (((size_t)seq * a.H + h) * a.P + p0 + lr) * a.N + 4 * lg;

  f32x4 S[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    S[n] = a.dhT && 16 * n < a.N ? ldf4(a.dhT + srow + 16 * n) : kZero4;

  const size_t ldk = (size_t)a.G * a.N, ldx = (size_t)a.H * a.P;
  const int chunks = (int)((hi - lo + kDeltaChunk - 1) / kDeltaChunk);
  for (int c = chunks - 1; c >= 0; --c) {
    const int64_t at = lo + (int64_t)c * kDeltaChunk;
    const int len = (int)min((int64_t)kDeltaChunk, hi - at);
    const size_t sh = (size_t)(slot0 + c) * a.H + h;
    __syncthreads();
    const size_t rows = (at * a.G + grp) * a.N;
    stage_rows<NT>(sK, sQ, (const float *)a.B + rows, (const float *)a.C + rows, ldk, a.N, len);
    stage_gates(sG, sE, sB, a, at, h, len);
    // (on their way while K dS is computed)
    const float *tri = (const float *)a.tri + sh * (3 * 4096);
    const float *dy = (const float *)a.dy + ((size_t)at * a.H + h) * a.P + p0;
    f32x4 Y[4], Tt[10], Mt[10];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Y[i] = value_tile(dy, ldx, 16 * i, len);
#pragma unroll
      for (int j = 0; j <= i; ++j) {
        const int e = (16 * j + lr) * kDeltaChunk + 16 * i + 4 * lg;
        Tt[i * (i + 1) / 2 + j] = ldf4(tri + 4096 + e);
        Mt[i * (i + 1) / 2 + j] = ldf4(tri + 8192 + e);
      }
    }
    __syncthreads();
    const float gc = sG[kDeltaChunk - 1], rc = sE[kDeltaChunk - 1];

    float *st = (float *)a.st1 + (sh * a.P + p0 + lr) * a.N + 4 * lg;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (16 * n < a.N) stf4(st + 16 * n, S[n]);

    f32x4 U[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4 ks = kZero4;
#pragma unroll
      for (int n = 0; n < NT; ++n) ks = mfma16(row_operand<W>(sK, 16 * t, 16 * n), S[n], ks);
      const f32x4 d = (gc - ldf4(sG + 16 * t + 4 * lg)) + (rc - ldf4(sE + 16 * t + 4 * lg));
#pragma unroll
      for (int r = 0; r < 4; ++r) U[t][r] = exp2_fast(d[r]) * ks[r];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = j; i < 4; ++i)
        U[j] = mfma16(Mt[i * (i + 1) / 2 + j], Y[i], U[j]);
    f32x4 R[4];
    float *dr = (float *)a.dr + sh * kDeltaChunk * a.P + p0 + lr;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      R[j] = kZero4;
#pragma unroll
      for (int i = j; i < 4; ++i)
        R[j] = mfma16(Tt[i * (i + 1) / 2 + j], U[i], R[j]);
#pragma unroll
      for (int r = 0; r < 4; ++r) dr[(16 * j + 4 * lg + r) * a.P] = R[j][r];
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4 gm = ldf4(sG + 16 * t + 4 * lg), b = ldf4(sB + 16 * t + 4 * lg);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = exp2_fast(gm[r]);
        Y[t][r] *= e;
        R[t][r] *= -b[r] * e;
      }
    }
    const float ec = exp2_fast(gc);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      S[n] *= ec;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        S[n] = mfma16(column_operand<W>(sQ, 16 * t, 16 * n), Y[t], S[n]);
        S[n] = mfma16(column_operand<W>(sK, 16 * t, 16 * n), R[t], S[n]);
      }
    }
  }
  if (a.dh0) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (16 * n < a.N) stf4(a.dh0 + srow + 16 * n, S[n]);
  }
}

template <int NT>
__global__ __launch_bounds__(256) void k_delta_chain_f32(DeltaArgs a) {
  extern __shared__ float lds[];
  chain_f32<NT, false>(a, (int)blockIdx.x, lds);
}

// The backward pass's two walks, which do not need each other: half of the
// workgroups each, the longer way first.
template <int NT>
__global__ __launch_bounds__(256) void k_delta_both_f32(DeltaArgs a) {
  extern __shared__ float lds[];
  const int half = (int)gridDim.x / 2, b = (int)blockIdx.x;
  if (b < half)
    reverse_f32<NT>(a, b, lds);
  else
    chain_f32<NT, true>(a, b - half, lds);
}

// Sum over the 16 lanes that share lg (columns of a result tile).
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// The gradients of one (chunk, head), a wave per 16 tokens. With D the decay
// factors e^{gam_i - gam_j}, dM = dY U^T (i >= j), dL = -dR U^T (i > j):
//   dx = beta dR
//   dQ = e^gam dY S^T + (dM D) K
//   dK = -beta e^gam dR S^T + e^{gam_c - gam} U dS^T + (dM D)^T Q + (dL beta D) K + (dL beta D)^T K
//   dbeta = dR . V - e^gam K . (dR S^T) + sum_j dL (K K^T) D
//   dg_t = sum_{i >= t} [e^gam Q . (dY S^T) - beta e^gam K . (dR S^T)]_i
//        + sum_{i < t} [e^{gam_c - gam} K . (U dS^T)]_i
//        + sum_{i >= t > j} (dM M + dL L)_ij + e^{gam_c} <S, dS>
// The pair sum is taken as suffix sums of row sums less column sums of one
// matrix, so that pairs on one side of t cancel to fp32 rounding.
__global__ __launch_bounds__(256) void k_delta_grad_f32(DeltaArgs a) {
  constexpr int W1 = kDeltaChunk + 4;
  __shared__ float sG[kDeltaChunk], sE[kDeltaChunk], sB[kDeltaChunk];
  __shared__ float sM[kDeltaChunk * W1], sL[kDeltaChunk * W1];  // dM D, dL beta D
  __shared__ float sZ[kDeltaChunk], sP[kDeltaChunk], sC[4][kDeltaChunk], sS[4];
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4, w = threadIdx.x >> 6;
  const int h = blockIdx.x % a.H, slot = blockIdx.x / a.H, grp = h / a.hpg;
  int64_t start;
  int len;
  if (!delta_chunk(a, slot, start, len)) return;
  const size_t sh = (size_t)slot * a.H + h;
  const size_t ldk = (size_t)a.G * a.N, ldx = (size_t)a.H * a.P;
  const float *K = (const float *)a.B + ((size_t)start * a.G + grp) * a.N;
  const float *Q = (const float *)a.C + ((size_t)start * a.G + grp) * a.N;
  const float *X = (const float *)a.x + ((size_t)start * a.H + h) * a.P;
  const float *dY = (const float *)a.dy + ((size_t)start * a.H + h) * a.P;
  const float *U = (const float *)a.u + sh * kDeltaChunk * a.P;
  const float *dR = (const float *)a.dr + sh * kDeltaChunk * a.P;
  const float *S0 = (const float *)a.st0 + sh * a.P * a.N;
  const float *S1 = (const float *)a.st1 + sh * a.P * a.N;
  stage_gates(sG, sE, sB, a, start, h, len);
  for (int e = threadIdx.x; e < 4 * kDeltaChunk; e += 256) (&sC[0][0])[e] = 0.f;
  __syncthreads();

  const int ti = 16 * w + lr;                    // this lane's token as a row of a left operand
  const int tr = min(ti, len - 1);
  const bool live = ti < len;
  const f32x4 gm = ldf4(sG + 16 * w + 4 * lg), bt = ldf4(sB + 16 * w + 4 * lg);
  const f32x4 toEnd = (sG[kDeltaChunk - 1] - gm) + (sE[kDeltaChunk - 1] - ldf4(sE + 16 * w + 4 * lg));
  const float gi = sG[ti], ei = sE[ti], bi = sB[ti];

  // pairs: rows i of this wave's tile, columns j of tiles up to it (lane: row
  // i, 4 columns j)
  float rowsum = 0.f, betasum = 0.f;
  for (int j = 0; j <= w; ++j) {
    f32x4 kk = kZero4, qk = kZero4, dm = kZero4, dl = kZero4;
    const int tj = min(16 * j + lr, len - 1);
    for (int n = 4 * lg; n < a.N; n += 16) {
      const f32x4 kj = ldf4(K + tj * ldk + n);
      kk = mfma16(kj, ldf4(K + tr * ldk + n), kk);
      qk = mfma16(kj, ldf4(Q + tr * ldk + n), qk);
    }
    for (int p = 4 * lg; p < a.P; p += 16) {
      const f32x4 u = ldf4(U + (16 * j + lr) * a.P + p);
      const f32x4 y = ldf4(dY + tr * ldx + p);
      dm = mfma16(u, live ? y : kZero4, dm);
      dl = mfma16(u, ldf4(dR + ti * a.P + p), dl);
    }
    const f32x4 dg = (gi - ldf4(sG + 16 * j + 4 * lg)) + (ei - ldf4(sE + 16 * j + 4 * lg));
    f32x4 m, l, both;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = ti - (16 * j + 4 * lg + r);
      const float e = d >= 0 ? exp2_fast(dg[r]) : 0.f;
      m[r] = d >= 0 ? dm[r] * e : 0.f;
      const float lk = d > 0 ? -dl[r] * e : 0.f;
      l[r] = lk * bi;
      betasum += lk * kk[r];
      both[r] = m[r] * qk[r] + l[r] * kk[r];
      rowsum += both[r];
    }
    stf4(sM + ti * W1 + 16 * j + 4 * lg, m);
    stf4(sL + ti * W1 + 16 * j + 4 * lg, l);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float cs = sum16(both[r]);
      if (lr == 0) sC[w][16 * j + 4 * lg + r] = cs;
    }
  }
  rowsum += __shfl_xor(rowsum, 16);
  rowsum += __shfl_xor(rowsum, 32);
  betasum += __shfl_xor(betasum, 16);
  betasum += __shfl_xor(betasum, 32);

  // dx, and dR . V
  float rv = 0.f;
  for (int p = 4 * lg; p < a.P; p += 16) {
    const f32x4 r = ldf4(dR + ti * a.P + p), v = ldf4(X + tr * ldx + p);
    float *dx = (float *)a.dx + ((size_t)(start + tr) * a.H + h) * a.P + p;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (live) {
        rv += r[q] * v[q];
        dx[q] = bi * r[q];
      }
    }
  }
  rv += __shfl_xor(rv, 16);
  rv += __shfl_xor(rv, 32);
  __syncthreads();

  // dQ, dK of this wave's tokens, 16 state channels at a time (result tiles:
  // lane: channel n, 4 tokens)
  f32x4 za = kZero4, zb = kZero4, zk = kZero4;
  float ss = 0.f;
  // (to dB and dC where a group has one head)
  float *dKo = (a.hparts == 1 ? (float *)a.dB : a.part) + (size_t)h * a.N;
  float *dQo = a.hparts == 1 ? (float *)a.dC + (size_t)h * a.N : dKo + (size_t)a.T * a.H * a.N;
  for (int n0 = 0; n0 < a.N; n0 += 16) {
    f32x4 ys = kZero4, rs = kZero4, us = kZero4;
    for (int p = 4 * lg; p < a.P; p += 16) {
      f32x4 s0, s1;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s0[r] = S0[(size_t)(p + r) * a.N + n0 + lr];
        s1[r] = S1[(size_t)(p + r) * a.N + n0 + lr];
        if (w == (n0 >> 4) % 4) ss += s0[r] * s1[r];
      }
      const f32x4 y = ldf4(dY + tr * ldx + p);
      ys = mfma16(live ? y : kZero4, s0, ys);
      rs = mfma16(ldf4(dR + ti * a.P + p), s0, rs);
      us = mfma16(ldf4(U + ti * a.P + p), s1, us);
    }
    f32x4 k, q, dq, dk;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = min(16 * w + 4 * lg + r, len - 1);
      k[r] = K[t * ldk + n0 + lr];
      q[r] = Q[t * ldk + n0 + lr];
      const float e = exp2_fast(gm[r]);
      dq[r] = e * ys[r];
      const float rk = -e * rs[r], uk = exp2_fast(toEnd[r]) * us[r];
      dk[r] = bt[r] * rk + uk;
      za[r] += q[r] * dq[r] + bt[r] * k[r] * rk;
      zk[r] += k[r] * rk;
      zb[r] += k[r] * uk;
    }
    for (int j = 0; j < 4; ++j) {
      // columns n of K and Q rows of tile j as right operands
      f32x4 kj, qj;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = min(16 * j + 4 * lg + r, len - 1);
        kj[r] = K[t * ldk + n0 + lr];
        qj[r] = Q[t * ldk + n0 + lr];
      }
      if (j <= w) {
        dq = mfma16(ldf4(sM + ti * W1 + 16 * j + 4 * lg), kj, dq);
        dk = mfma16(ldf4(sL + ti * W1 + 16 * j + 4 * lg), kj, dk);
      }
      if (j >= w) {
        f32x4 mt, lt;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          mt[r] = sM[(16 * j + 4 * lg + r) * W1 + ti];
          lt[r] = sL[(16 * j + 4 * lg + r) * W1 + ti];
        }
        dk = mfma16(mt, qj, dk);
        dk = mfma16(lt, kj, dk);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * lg + r;
      if (t < len) {
        const size_t to = (size_t)(start + t) * a.H * a.N + n0 + lr;
        dKo[to] = dk[r];
        dQo[to] = dq[r];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    za[r] = sum16(za[r]);
    zb[r] = sum16(zb[r]);
    zk[r] = sum16(zk[r]);
    if (lr == 0) {
      sZ[16 * w + 4 * lg + r] = za[r];
      sP[16 * w + 4 * lg + r] = zb[r];
    }
  }
  // dbeta: rv and betasum are per row i (lanes lr), zk per row 4 lg + r
  __shared__ float sK2[kDeltaChunk], sR[kDeltaChunk];
  if (lr == 0)
#pragma unroll
    for (int r = 0; r < 4; ++r) sK2[16 * w + 4 * lg + r] = zk[r];
  if (lg == 0) sR[ti] = rowsum;
  ss = sum16(ss);
  ss += __shfl_xor(ss, 16);
  ss += __shfl_xor(ss, 32);
  if (lane == 0) sS[w] = ss;
  __syncthreads();
  if (lg == 0 && live)
    ((float *)a.dbeta)[(size_t)(start + ti) * a.H + h] = rv + betasum + sK2[ti];
  if (w == 0) {
    const float zed = sZ[lane] + sR[lane] -
                      (sC[0][lane] + sC[1][lane] + sC[2][lane] + sC[3][lane]);
    const float zp = sP[lane];
    const float pre = wave_inclusive_sum(zed), all = __shfl(pre, 63);
    const float prefix = wave_inclusive_sum(zp) - zp;
    const float ends = exp2_fast(sG[kDeltaChunk - 1]) * (sS[0] + sS[1] + sS[2] + sS[3]);
    if (lane < len)
      ((float *)a.dg)[(size_t)(start + lane) * a.H + h] =
          all - (pre - zed) + prefix + ends;
  }
}

// dB, dC of a group: the sum over the parts of its heads, in order.
template <typename T>
__global__ __launch_bounds__(256) void k_delta_heads_sum(const float *part, T *dB, T *dC, int64_t n4,
                                                         int N4, int parts, int64_t all4) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * n4) return;
  const bool q = i >= n4;
  const int64_t e = q ? i - n4 : i;
  const int64_t row = e / N4;                    // token * G + group
  const f32x4 *p = reinterpret_cast<const f32x4 *>(part) + (q ? all4 : 0) + row * parts * N4 + e % N4;
  f32x4 v = kZero4;
  for (int k = 0; k < parts; ++k) v += p[(int64_t)k * N4];
  T *to = (q ? dC : dB) + 4 * e;
#pragma unroll
  for (int r = 0; r < 4; ++r) to[r] = from_f32<T>(v[r]);
}

template <int NT>
hipError_t walk_f32(const DeltaArgs &a, bool both, hipStream_t s) {
  constexpr int W = 16 * NT + 4;
  const int waves = min(4, a.P / 16);
  const unsigned units = (unsigned)((int64_t)a.nseq * a.H * (a.P / (16 * waves)));
  const size_t lds = (3 * kDeltaChunk + 2 * kDeltaChunk * W) * sizeof(float);
  const auto f = both ? k_delta_both_f32<NT> : k_delta_chain_f32<NT>;
  if (hipError_t e = hipFuncSetAttribute((const void *)f, hipFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)lds))
    return e;
  hipLaunchKernelGGL(f, dim3(both ? 2 * units : units), dim3(64 * waves), lds, s, a);
  return hipGetLastError();
}

hipError_t launch_delta_walk_f32(const DeltaArgs &a, bool both, hipStream_t s) {
  if (a.nseq == 0) return hipSuccess;
  if (a.N <= 64) return walk_f32<4>(a, both, s);
  if (a.N <= 128) return walk_f32<8>(a, both, s);
  return walk_f32<16>(a, both, s);
}

template <typename T>
hipError_t heads_sum(const DeltaArgs &a, hipStream_t s) {
  const int64_t n4 = a.T * a.G * (a.N / 4);
  hipLaunchKernelGGL(k_delta_heads_sum<T>, dim3((unsigned)((2 * n4 + 255) / 256)), dim3(256), 0, s,
                     a.part, (T *)a.dB, (T *)a.dC, n4, a.N / 4, a.hparts, n4 * a.hparts);
  return hipGetLastError();
}

hipError_t launch_delta_heads_sum(const DeltaArgs &a, bool bf16_io, hipStream_t s) {
  return bf16_io ? heads_sum<bf16>(a, s) : heads_sum<float>(a, s);
}

hipError_t launch_delta_grad_f32(const DeltaArgs &a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  hipLaunchKernelGGL(k_delta_grad_f32, dim3((unsigned)((int64_t)a.nslots * a.H)), dim3(256), 0, s, a);
  if (const hipError_t e = hipGetLastError()) return e;
  return a.hparts == 1 ? hipSuccess : heads_sum<float>(a, s);
}

}  // namespace ssd
