// k_delta_prep.hip -- the triangular matrices of each chunk of the gated delta
// rule: T = (I + L)^-1 and M (delta.h), or T, T^T and M^T for the backward pass.
//
// (Forwards in bf16 T alone: the walk makes M from the rows that it holds.) A workgroup
// takes one chunk and some heads of one group. Q K^T and K K^T, which those share, are
// computed once, as 16 x 16 tiles on and below the diagonal,
// transposed: a lane holds 4 consecutive columns j of one row i. Each wave then
// takes heads in turn. In that layout a tile of L is the left operand of
// the fp32 matrix instruction (lane l: row l % 16, columns 4 (l / 16) + r at
// step r) and a result tile its right operand, so the block inversion
//   T_ij = -T_ii sum_{j <= k < i} L_ik T_kj
// passes from product to product in registers, in fp32: T multiplies every
// value that enters the state. Only the four diagonal blocks go through LDS,
// where 64 lanes invert them at once by forward substitution, one column a
// lane. (Substitution, not powers of L: with equal keys the powers of a
// 16 x 16 block reach 6435 and cancel, the substitution's values stay within
// those of the inverse.)
//
// Measured (MI355X): 80 heads of one group, 256 chunks forwards, 67 to 70 us: 20,480
// inverses of 64 x 64, and 315 MB written (62 us at a copy's rate). Two heads a group,
// 4096 chunks and groups: 50 to 52 us forwards; 58 to 62 backwards, of 2048 (189 MB
// written). A wave reads all of its rows of K before the first product (one tile row
// after another read K up to four times). Waves a workgroup share the group's products:
// forwards 4, or 1 for groups of up to 3 heads, backwards as many as a group has heads,
// or 4. (us by 1, 2 and 4 waves, 4 x 2048 tokens: groups of 1 head 38, 41, 50, backwards
// 76, 83, 97; of 2 heads 26, 30, 34, backwards 66, 60, 71; of 3 heads 34, 39, 38, backwards
// 82, 79, 82; of 8 heads 26, 22, 22, backwards 58, 48, 38.)
#include <type_traits>

#include "delta_tiles.h"

namespace ssd {

// LDS accesses of one wave before and after stay in order (they run in order).
__device__ __forceinline__ void wave_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// Index of lower tile (i, j), j <= i.
__host__ __device__ constexpr int tri(int i, int j) { return i * (i + 1) / 2 + j; }

// Row r, columns n.. of a tile's rows as an operand: 8 of 32 columns in bf16, 4 of
// 16 in fp32; zeros from column N on.
__device__ __forceinline__ bf16x8 operand(const bf16 *row, int n, int N) {
  const int col = n + 8 * ((threadIdx.x & 63) >> 4);
  bf16x8 v = ldg8(row + min(col, N - 8));
  return col < N ? v : zero8();
}
__device__ __forceinline__ f32x4 operand(const float *row, int n, int N) {
  const f32x4 v = ldf4(row + min(n, N - 16) + 4 * ((threadIdx.x & 63) >> 4));
  return n < N ? v : kZero4;
}
__device__ __forceinline__ f32x4 product(bf16x8 a, bf16x8 b, f32x4 c) { return mfma(a, b, c); }
__device__ __forceinline__ f32x4 product(f32x4 a, f32x4 b, f32x4 c) { return mfma16(a, b, c); }

// Tile rows 3 - v of K K^T and, where kPairs, v of Q K^T (five tiles on and below the
// diagonal) for v from LO to HI: rows j of K against rows i (lane: row i % 16, 4 columns j),
// or with kSwap Q K^T the other way round (lane: row j % 16, 4 columns i). Rows past
// len are read as the last one. NB operands' columns are on their way at once; a
// wave reads the rows of K once. The tiles go to LDS in lane order, tile (i, j) at
// tri(i, j).
template <int LO, int HI, int NB, bool kPairs, bool kSwap, typename T>
__device__ __forceinline__ void tile_rows(const T *K, const T *Q, size_t ld, int N, int len,
                                          f32x4 (*kk)[64], f32x4 (*qk)[64]) {
  constexpr int kCols = sizeof(T) == 2 ? 32 : 16;
  constexpr int kRows = (3 - LO > HI - 1 || !kPairs ? 3 - LO : HI - 1) + 1;  // of K's tiles
  const int lane = threadIdx.x & 63, lr = lane & 15;
  f32x4 k[HI - LO][4], q[HI - LO][4];
#pragma unroll
  for (int v = LO; v < HI; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) k[v - LO][j] = q[v - LO][j] = kZero4;
  for (int n0 = 0; n0 < N; n0 += NB * kCols) {
    decltype(operand(K, 0, 0)) x[kRows][NB], y[HI - LO][NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        x[j][b] = operand(K + (size_t)min(16 * j + lr, len - 1) * ld, n0 + kCols * b, N);
#pragma unroll
      for (int v = LO; v < HI && kPairs; ++v)
        y[v - LO][b] = operand(Q + (size_t)min(16 * v + lr, len - 1) * ld, n0 + kCols * b, N);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v = LO; v < HI; ++v) {
#pragma unroll
        for (int j = 0; j <= 3 - v; ++j)
          k[v - LO][j] = product(x[j][b], x[3 - v][b], k[v - LO][j]);
#pragma unroll
        for (int j = 0; j <= v && kPairs; ++j)
          q[v - LO][j] = kSwap ? product(y[v - LO][b], x[j][b], q[v - LO][j])
                               : product(x[j][b], y[v - LO][b], q[v - LO][j]);
      }
  }
#pragma unroll
  for (int v = LO; v < HI; ++v) {
#pragma unroll
    for (int j = 0; j <= 3 - v; ++j) kk[tri(3 - v, j)][lane] = k[v - LO][j];
#pragma unroll
    for (int j = 0; j <= v && kPairs; ++j) qk[tri(v, j)][lane] = q[v - LO][j];
  }
}
template <int WV, int NB, bool kPairs, bool kSwap, typename T>
__device__ __forceinline__ void group_tiles(int wave, const T *K, const T *Q, size_t ld, int N,
                                            int len, f32x4 (*kk)[64], f32x4 (*qk)[64]) {
  constexpr int R = 4 / WV;
  if (wave == 0)
    tile_rows<0, R, NB, kPairs, kSwap>(K, Q, ld, N, len, kk, qk);
  else if (wave == 1)
    tile_rows<R % 4, R % 4 + R, NB, kPairs, kSwap>(K, Q, ld, N, len, kk, qk);
  else if (wave == 2)
    tile_rows<2 * R % 4, 2 * R % 4 + R, NB, kPairs, kSwap>(K, Q, ld, N, len, kk, qk);
  else
    tile_rows<3 * R % 4, 3 * R % 4 + R, NB, kPairs, kSwap>(K, Q, ld, N, len, kk, qk);
}

// Where a chunk's matrices go. v: the ten tiles (lane: row 16 i + l % 16, columns
// 16 j + 4 (l / 16) + r) of a lower matrix, tile (i, j) at tri(i, j), or of an
// upper one, tile (j, i) at tri(i, j). As fp32 rows of 64 (tiles that are zero
// not written), or as operand tiles of the bf16 matrix instruction (a row's 8 of
// k are 4 of each tile of a pair), in kLevels bf16.
struct RowsOut {
  float *p;
  template <int kMatrix, int kLevels, bool kUpper>
  __device__ __forceinline__ void put(const f32x4 (&v)[10]) const {
    const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j <= i; ++j)
        stf4(p + kMatrix * 4096 + (16 * (kUpper ? j : i) + lr) * kDeltaChunk +
                 16 * (kUpper ? i : j) + 4 * lg, v[tri(i, j)]);
  }
};
struct TilesOut {
  bf16 *p;
  template <int kMatrix, int kLevels, bool kUpper>
  __device__ __forceinline__ void put(const f32x4 (&v)[10]) const {
    bf16 *to = p + kMatrix * kMatrixElems + 8 * (threadIdx.x & 63);
    const auto tile = [&](int t, f32x4 a, f32x4 b) {
      const auto level = [&](int l, bf16x8 v) {
        *reinterpret_cast<bf16x8 *>(to + l * kLevelElems + t * kTileElems) = v;
      };
      if (kLevels == 3) {
        const Split3 s = split8x3(a, b);
        level(0, s.hi), level(1, s.mid), level(2, s.lo);
      } else if (kLevels == 2) {
        const Split s = split8(a, b);
        level(0, s.hi), level(1, s.lo);
      } else {
        level(0, pack8(a, b));
      }
    };
    if (!kUpper) {
      tile(lower_tile(1, 0), v[tri(1, 0)], v[tri(1, 1)]);
      tile(lower_tile(2, 0), v[tri(2, 0)], v[tri(2, 1)]);
      tile(lower_tile(3, 0), v[tri(3, 0)], v[tri(3, 1)]);
      tile(lower_tile(3, 1), v[tri(3, 2)], v[tri(3, 3)]);
      tile(4, v[tri(0, 0)], v[tri(2, 2)]);
    } else {
      tile(upper_tile(0, 0), v[tri(0, 0)], v[tri(1, 0)]);
      tile(upper_tile(0, 1), v[tri(2, 0)], v[tri(3, 0)]);
      tile(upper_tile(1, 1), v[tri(2, 1)], v[tri(3, 1)]);
      tile(upper_tile(2, 1), v[tri(2, 2)], v[tri(3, 2)]);
      tile(4, v[tri(1, 1)], v[tri(3, 3)]);
    }
  }
};

// Forwards in bf16 T alone is wanted: the walk makes M itself, from Q and K in its LDS.
template <typename T, DeltaTri W>
constexpr bool kFew = sizeof(T) == 2 && W == kTriForward;

template <typename T, DeltaTri W, int WV, typename Out>
__global__ __launch_bounds__(64 * WV, WV == 1 ? 2 : 3) void k_delta_prep(DeltaArgs a, int64_t bytes, int per) {
  constexpr bool kPairs = !kFew<T, W>;
  __shared__ f32x4 sKK[10][64], sQK[kPairs ? 10 : 1][64];
  __shared__ float sGate[WV][2][kDeltaChunk];    // decay_sums
  __shared__ f32x4 sDiag[WV][4][16][5];  // diagonal blocks: rows of L, then columns of T
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int parts = (a.hpg + WV * per - 1) / (WV * per);
  if (a.order && blockIdx.x == 0) {  // the walks' order of sequences, for all
    int *chunks = reinterpret_cast<int *>(&sKK[0][0]);
    static_assert(sizeof(sKK) >= kMostOrdered * sizeof(int), "the lengths must fit");
    for (int s = threadIdx.x; s < a.nseq; s += 64 * WV) {
      int64_t lo, hi;
      delta_seq(a, s, lo, hi);
      chunks[s] = (int)((hi - lo + kDeltaChunk - 1) / kDeltaChunk);
    }
    __syncthreads();
    for (int s = threadIdx.x; s < a.nseq; s += 64 * WV) {
      const int own = chunks[s];
      int rank = 0;
      for (int o = 0; o < a.nseq; ++o) rank += chunks[o] > own || (chunks[o] == own && o < s);
      a.order[rank] = s;
    }
    __syncthreads();
  }
  int unit = xcd_unit();
  const int part = unit % parts;
  unit /= parts;
  const int grp = unit % a.G, slot = unit / a.G;
  int64_t start;
  int len;
  if (!delta_chunk(a, slot, start, len)) return;
  const size_t row0 = ((size_t)start * a.G + grp) * a.N, ld = (size_t)a.G * a.N;
  const T *K = (const T *)a.B + row0, *Q = (const T *)a.C + row0;
  // the group's products
  constexpr bool kSwap = W == kTriBackward;
  constexpr int kNarrow = sizeof(T) == 2 ? 2 : 4;  // operands of 64 columns
  if (a.N <= 64)
    group_tiles<WV, kNarrow, kPairs, kSwap>(wave, K, Q, ld, a.N, len, sKK, sQK);
  else
    group_tiles<WV, 4, kPairs, kSwap>(wave, K, Q, ld, a.N, len, sKK, sQK);
  __syncthreads();
  float *sG = sGate[wave][0], *sE = sGate[wave][1];
  f32x4 (*sD)[16][5] = sDiag[wave];
  const int h1 = min((part + 1) * WV * per, a.hpg);
  for (int hh = part * WV * per + wave; hh < h1; hh += WV) {
    const int h = grp * a.hpg + hh;
    float beta;
    {
      const size_t at = (size_t)(start + min(lane, len - 1)) * a.H + h;
      const DecaySum gam = decay_sums(lane < len ? delta_log2_decay(ssd::ld<T>(a.g, at)) : 0.f);
      sG[lane] = gam.hi;
      sE[lane] = gam.lo;
      beta = lane < len ? ssd::ld<T>(a.beta, at) : 0.f;
    }
    wave_order();
    Out out;
    out.p = reinterpret_cast<decltype(out.p)>((char *)a.tri + ((int64_t)slot * a.H + h) * bytes);
    if (kPairs) {  // M, or M^T (lane holds column j, 4 rows i)
      f32x4 qk[10];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          qk[tri(i, j)] = sQK[tri(i, j)][lane];
          const int row = 16 * (W == kTriForward ? i : j) + lr;
          const int col = 16 * (W == kTriForward ? j : i) + 4 * lg;
          const f32x4 d = (sG[row] - ldf4(sG + col)) + (sE[row] - ldf4(sE + col));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool below = j < i || (W == kTriForward ? 4 * lg + r <= lr : lr <= 4 * lg + r);
            const float e = exp2_fast(W == kTriForward ? d[r] : -d[r]);
            qk[tri(i, j)][r] = below ? qk[tri(i, j)][r] * e : 0.f;
          }
        }
      if (W == kTriForward)
        out.template put<1, 1, false>(qk);
      else
        out.template put<2, 3, true>(qk);
    }
    f32x4 Lt[10];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float gi = sG[16 * i + lr], ei = sE[16 * i + lr], bi = __shfl(beta, 16 * i + lr);
#pragma unroll
      for (int j = 0; j <= i; ++j) {
        const f32x4 kk = sKK[tri(i, j)][lane];
        const f32x4 d = (gi - ldf4(sG + 16 * j + 4 * lg)) + (ei - ldf4(sE + 16 * j + 4 * lg));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool below = j < i || 4 * lg + r < lr;
          Lt[tri(i, j)][r] = below ? bi * kk[r] * exp2_fast(d[r]) : 0.f;
        }
      }
    }

    // diagonal blocks: lane (b, j) = (lg, lr) takes column j of block b
#pragma unroll
    for (int b = 0; b < 4; ++b) sD[b][lr][lg] = Lt[tri(b, b)];
    wave_order();
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
    wave_order();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      sD[lg][lr][q] = f32x4{t[4 * q], t[4 * q + 1], t[4 * q + 2], t[4 * q + 3]};
    wave_order();
    // T: lane column j, 4 rows i; and lane row i, 4 columns j
    f32x4 Tt[10], Ta[10];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      Tt[tri(b, b)] = sD[b][lr][lg];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        Ta[tri(b, b)][r] = reinterpret_cast<const float *>(&sD[b][4 * lg + r][0])[lr];
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
        Tt[tri(i, j)] = mfma16(Ta[tri(i, i)], x, kZero4);
        Ta[tri(i, j)] = mfma16(x, Ta[tri(i, i)], kZero4);
      }
    out.template put<0, 3, false>(Ta);
    if (W == kTriBackward) out.template put<1, 3, true>(Tt);
  }
}

size_t delta_tri_bytes(bool tiles, DeltaTri which) {
  if (tiles) return (size_t)(which == kTriForward ? 1 : 3) * kMatrixElems * sizeof(bf16);
  return (size_t)(which == kTriForward ? 2 : 3) * 4096 * sizeof(float);
}

template <typename T, DeltaTri W, int WV, typename Out>
hipError_t prep_wv(const DeltaArgs &a, hipStream_t s) {
  const int64_t bytes = delta_tri_bytes(std::is_same<Out, TilesOut>::value, W);
  // Heads a wave takes in turn: the fewest with which all workgroups are on the card
  // at once, three on a compute unit and forwards in bf16, where they take fewer
  // registers and no M, four, since each makes the group's products anew. (80 heads and
  // 256 chunks forwards: 5 heads in 1024 workgroups 67 to 70 us; 7 in 768 workgroups 71 to
  // 75, 1 in 5120 workgroups 86 to 90, 20 in 256 workgroups 95 to 98.)
  constexpr int64_t kOnCard = (kFew<T, W> ? 4 : 3) * 256;
  const int64_t groups = (int64_t)a.nslots * a.G;
  const int64_t most = groups < kOnCard ? kOnCard / groups : 1;
  const int per = (int)((a.hpg + WV * most - 1) / (WV * most));
  const int64_t parts = (a.hpg + WV * per - 1) / (WV * per);
  const dim3 grid((unsigned)((int64_t)a.nslots * a.G * parts)), block(64 * WV);
  hipLaunchKernelGGL((k_delta_prep<T, W, WV, Out>), grid, block, 0, s, a, bytes, per);
  return hipGetLastError();
}

template <typename T, DeltaTri W, typename Out>
hipError_t prep(const DeltaArgs &a, hipStream_t s) {
  if constexpr (kFew<T, W>) {
    if (a.hpg <= 3) return prep_wv<T, W, 1, Out>(a, s);
  } else {
    if (a.hpg == 1) return prep_wv<T, W, 1, Out>(a, s);
    if (a.hpg == 2) return prep_wv<T, W, 2, Out>(a, s);
  }
  return prep_wv<T, W, 4, Out>(a, s);
}

hipError_t launch_delta_prep(const DeltaArgs &a, bool bf16_io, DeltaTri which, hipStream_t s) {
  if (a.nslots == 0) return hipSuccess;
  if (bf16_io)
    return which == kTriForward ? prep<bf16, kTriForward, TilesOut>(a, s)
                                : prep<bf16, kTriBackward, TilesOut>(a, s);
  return which == kTriForward ? prep<float, kTriForward, RowsOut>(a, s)
                              : prep<float, kTriBackward, RowsOut>(a, s);
}

}  // namespace ssd
