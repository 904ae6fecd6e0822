// k_delta.hip -- the gated delta rule in bf16 (delta.h has the formulas): the
// walks over a sequence's chunks, forwards and backwards, on the bf16 matrix
// instructions.
//
// The state's columns (value channels) never mix, so a wave takes 16 of them
// through all chunks with the state in fp32 result tiles and no exchange with
// other waves: each product contracts over rows of tiles that the wave holds
// (S, R, U), whose registers are right operands as they are, once rounded to
// bf16. A result tile's rows stand for state channels
// n = 32 ks + 8 (row / 4) + 4 par + row % 4, so that two tiles make an operand
// with 8 channels in a row, as the rows of K and Q lie in LDS; R and U pair
// tiles of 16 tokens, in which order k_delta_prep writes its matrices.
//
// Rounding. K, Q, V and dY are bf16 as they are. What enters a state is held in three
// bf16 (the value, and twice what rounding left of it: 2^-26 off, less than fp32's own
// half step) and multiplied with what of the other operand is not below that, so that
// the states are those of fp32 arithmetic: S in K S, R and T in T R, U in K^T U, and
// the same backwards (relative error 1.9e-7; two bf16 each gave 3.6e-6). y is rounded
// to bf16 in the end: S, M and U enter it in two bf16 (2^-17 off), so that its error is
// that rounding's, 1.66e-3 (S and M in one gave 2.44e-3). U and dR, and the
// states of a chunk's start and end, go to the gradients in two bf16.
//
// Segments. A walk's length is its chunks' latencies one after the other, and
// few sequences and heads leave most of the card idle. Then each sequence is
// cut: a first walk takes every segment at once from a state of zeros, together
// with its transition (the N unit vectors walked through it, without values);
// k_delta_join passes the states through the transitions; and the walk proper
// starts every segment from its own state.
//
// Four waves (64 columns) a workgroup share the staged K, Q and T, and M, whose tiles
// they make from K and Q among themselves; each takes 192 matrix and 830 vector
// instructions a chunk (N = 128; the latter for the parts above all). Measured (MI355X),
// 80 heads of 64, 8 x 2048 tokens: 326 to 398 us, 5 workgroups for 2 compute units; the
// matrix units are busy for 117 us of it and the vector units for 127, and a chunk's
// products wait for each other: a workgroup alone on a unit takes 5 us a chunk. Places of
// a lane in LDS are worked out anew where the registers would not hold them (a spilled
// one's load waits for the rows under way: 504 us a call with 60 bytes spilled, 441 with
// none).
#include "delta_tiles.h"

namespace ssd {

// Staged values (64 tokens x W columns): 16 columns from c0 of tokens
// t0 + 4 lg + r, as a result tile has them.
template <int W>
__device__ __forceinline__ f32x4 value_tile(const bf16 *v, int t0, int c0) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const bf16x4 w = ds_tr4(v, place<W>(t0 + 4 * lg + (lr >> 2), c0 + 4 * (lr & 3)));
  return f32x4{(float)w[0], (float)w[1], (float)w[2], (float)w[3]};
}

__device__ __forceinline__ float bits_to_f32(uint16_t w) { return __uint_as_float((uint32_t)w << 16); }

// Tables of a chunk, one entry a token: beta, beta e^gam, e^{gam_c - gam},
// e^gam; zeros in the first two past the end; and gam itself in two floats. Filled
// by one wave.
struct Gates {
  float b[kDeltaChunk], be[kDeltaChunk], lf[kDeltaChunk], ef[kDeltaChunk];
  float hi[kDeltaChunk], lo[kDeltaChunk];
};
__device__ __forceinline__ void fill_gates(Gates &G, float g, float beta, bool live) {
  const int lane = threadIdx.x & 63;
  const DecaySum gam = decay_sums(live ? delta_log2_decay(g) : 0.f);
  const float e = exp2_fast(gam.hi);
  G.b[lane] = live ? beta : 0.f;
  G.be[lane] = live ? beta * e : 0.f;
  G.lf[lane] = exp2_fast((__shfl(gam.hi, 63) - gam.hi) + (__shfl(gam.lo, 63) - gam.lo));
  G.ef[lane] = e;
  G.hi[lane] = gam.hi;
  G.lo[lane] = gam.lo;
}

// Left operand K^T: rows n (as the state's tiles have them), tokens
// 32 kt + 16 (e / 4) + 4 lg + e % 4.
template <int N>
__device__ __forceinline__ bf16x8 state_operand(const bf16 *rows, int kt, int ks, int par) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int row = 32 * kt + 4 * lg + (lr >> 2), col = 32 * ks + 8 * (lr & 3) + 4 * par;
  const bf16x4 a = ds_tr4(rows, place<N>(row, col));
  const bf16x4 b = ds_tr4(rows, place<N>(row + 16, col));
  return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// The two operands (values 32 kt + 16 (e / 4) + 4 lg + e % 4) of staged values
// as they are.
template <int W>
__device__ __forceinline__ bf16x8 value_operand(const bf16 *v, int kt, int c0) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int at = place<W>(32 * kt + 4 * lg + (lr >> 2), c0 + 4 * (lr & 3));
  const bf16x4 a = ds_tr4(v, at), b = ds_tr4(v, at + 16 * W);  // (16 rows on: the same swizzle)
  return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// This lane, anew: places worked out from it are not kept over the chunks (all of them
// would fill the registers).
__device__ __forceinline__ int lane_anew() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// Tiles (I, J), (I2, J2), ... of M: Q_i . K_j with the decay between them (lane: row i, 4
// columns j), in two bf16; and their places in the operand tiles, of which each is half of
// a lane's columns.
struct MTile {
  uint2 hi, lo;
};
template <int NK, int I, int J, int... More>
__device__ __forceinline__ void m_tiles(MTile *to, const bf16 *sK, const bf16 *sQ, const Gates &G) {
  constexpr int N = 32 * NK;
  const int lane = lane_anew(), lr = lane & 15, lg = lane >> 4;
  f32x4 v = kZero4;
#pragma unroll
  for (int ks = 0; ks < NK; ++ks) {
    const int e = place<N>(lr, 32 * ks + 8 * lg);
    v = mfma(*reinterpret_cast<const bf16x8 *>(sK + e + 16 * J * N),
             *reinterpret_cast<const bf16x8 *>(sQ + e + 16 * I * N), v);
  }
  const f32x4 d = (G.hi[16 * I + lr] - ldf4(G.hi + 16 * J + 4 * lg)) +
                  (G.lo[16 * I + lr] - ldf4(G.lo + 16 * J + 4 * lg));
#pragma unroll
  for (int r = 0; r < 4; ++r)
    v[r] = J < I || 4 * lg + r <= lr ? v[r] * exp2_fast(d[r]) : 0.f;
  to->hi = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
  v[0] -= __uint_as_float(to->hi.x << 16);
  v[1] -= __uint_as_float(to->hi.x & 0xffff0000u);
  v[2] -= __uint_as_float(to->hi.y << 16);
  v[3] -= __uint_as_float(to->hi.y & 0xffff0000u);
  to->lo = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
  if constexpr (sizeof...(More) > 0) m_tiles<NK, More...>(to + 1, sK, sQ, G);
}
template <int I, int J, int... More>
__device__ __forceinline__ void put_m_tiles(const MTile *from, bf16 *to) {
  constexpr bool kSecond = I == 2 && J == 2;  // of the shared tile
  constexpr int kHalf = kSecond ? 1 : I == 0 ? 0 : J & 1;
  bf16 *at = to + lower_tile(I, J / 2) * kTileElems + 8 * lane_anew() + 4 * kHalf;
  *reinterpret_cast<uint2 *>(at) = from->hi;
  *reinterpret_cast<uint2 *>(at + kLevelElems) = from->lo;
  if constexpr (sizeof...(More) > 0) put_m_tiles<More...>(from + 1, to);
}

// A store at a lane's 32-bit byte offset from an address that the wave shares.
template <typename V>
__device__ __forceinline__ void store_at(void *base, uint32_t off, V v) {
  *reinterpret_cast<V *>(static_cast<char *>(base) + off) = v;
}

// What a walk writes.
enum WalkMode : int {
  kWalkY = 0,      // y, and the final state
  kWalkSave = 1,   // backward pass: the state entering each chunk, and U
  kWalkLocal = 2   // a segment's own final state and its transition's columns
};

// What the walks stage, one array for each: the compiler then sees which reads do
// not meet the loads under way, and does not wait for those. (T's last
// level and M take Q's place once Q S is done, y that of the values; backwards the last
// levels of M^T and T^T take the values' place.)
template <int NK>
constexpr int kRowElems = kDeltaChunk * 32 * NK;
constexpr int kTriElems = 2 * kLevelElems;  // a matrix's first two levels

// The walk forwards of unit `unit`: 16 WV columns of a sequence or segment.
template <int NK, int WV, WalkMode kMode>
__device__ __forceinline__ void walk_forwards(const DeltaArgs &a, int unit, bf16 *sK, bf16 *sQ,
                                              bf16 *sT, bf16 *sV, Gates &G) {
  constexpr int N = 32 * NK, W = 16 * WV;  // state channels, the workgroup's columns
  constexpr bool kY = kMode == kWalkY, kLocal = kMode == kWalkLocal;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = WV == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = (kLocal ? a.P + a.N : a.P) / 16, blocks = (tiles + WV - 1) / WV;
  const int tile0 = (unit % blocks) * WV, tile = min(tile0 + wave, tiles - 1);
  const bool on = tile0 + wave < tiles;     // (a wave past the last tile repeats it)
  unit /= blocks;
  const int h = unit % a.H, sg = unit / a.H, grp = h / a.hpg;
  DeltaWalk w;
  if (!delta_walk(a, sg, w)) return;
  if (kLocal && w.last && !a.dspan) return;  // forward, nothing starts from its end
  const int p0 = 16 * tile, p = p0 + lr;
  const bool valued = !kLocal || tile0 * 16 < a.P;  // (P / 16 is a multiple of WV)

  f32x4 S[NK][2];
  {
    const float *from = nullptr;
    if (!kLocal && a.seg)
      from = a.span + (((size_t)sg * a.H + h) * (a.P + a.N) + p) * a.N;
    else if (!kLocal && a.h0)
      from = a.h0 + (((size_t)w.s * a.H + h) * a.P + p) * a.N;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks)
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const int n = 32 * ks + 8 * lg + 4 * par;
        S[ks][par] = from && n < a.N ? ldf4(from + n) : kZero4;
        if (kLocal)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[ks][par][r] = n + r == p - a.P ? 1.f : 0.f;
      }
  }

  const size_t ldk = (size_t)a.G * a.N, ldx = (size_t)a.H * a.P;
  const int chunks = (int)((w.hi - w.lo + kDeltaChunk - 1) / kDeltaChunk);
  const auto length = [&](int c) {
    return (int)min((int64_t)kDeltaChunk, w.hi - w.lo - (int64_t)c * kDeltaChunk);
  };
  const auto rows_at = [&](int c) { return (w.lo + (int64_t)c * kDeltaChunk); };
  const auto tri_at = [&](int c) {
    return (const bf16 *)a.tri + ((size_t)(w.slot + c) * a.H + h) * a.tri_stride;
  };
  uint16_t g = 0, bt = 0;  // (bits: a conversion here would wait for the loads)
  const auto fetch_rows = [&](int c) __attribute__((always_inline)) {
    const int64_t at = rows_at(c);
    stage_tile<N, kDeltaChunk, WV>(sK, (const bf16 *)a.B + (at * a.G + grp) * a.N, ldk, a.N,
                                   length(c));
    if (kY)
      stage_tile<N, kDeltaChunk, WV>(sQ, (const bf16 *)a.C + (at * a.G + grp) * a.N, ldk, a.N,
                                     length(c));
  };
  const auto fetch_tri = [&](int c) __attribute__((always_inline)) {
    if (wave == 0) {
      const size_t ga = (size_t)(rows_at(c) + min(lane, length(c) - 1)) * a.H + h;
      g = ((const uint16_t *)a.g)[ga];
      bt = ((const uint16_t *)a.beta)[ga];
    }
    stage_block<WV>(sT, tri_at(c), 2 * kTriTiles);
  };
  if (chunks > 0) {
    fetch_rows(0);
    fetch_tri(0);
  }
  for (int c = 0; c < chunks; ++c) {
    const int64_t at = rows_at(c);
    const int len = length(c);
    wait_vmem_all();
    if (wave == 0) fill_gates(G, bits_to_f32(g), bits_to_f32(bt), lane < len);
    __syncthreads();
    if (valued)
      stage_tile<W, kDeltaChunk, WV, kY>(
          sV, (const bf16 *)a.x + ((size_t)at * a.H + h) * a.P + 16 * tile0, ldx, W, len);

    // K S, and Q S transposed (lane: token lr of its tile, rows p); two tiles'
    // operands at a time, the next ones under way
    f32x4 A[4], O[4];
    {
      bf16x8 kb[2][2], qb[2][2];
      const auto keys = [&](int b) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int e = place<N>(32 * (b & 1) + 16 * u + lr, 32 * (b >> 1) + 8 * lg);
          kb[b & 1][u] = *reinterpret_cast<const bf16x8 *>(sK + e);
          if (kY) qb[b & 1][u] = *reinterpret_cast<const bf16x8 *>(sQ + e);
        }
      };
      keys(0);
#pragma unroll
      for (int t = 0; t < 4; ++t) A[t] = O[t] = kZero4;
      Split3 s;
#pragma unroll
      for (int b = 0; b < 2 * NK; ++b) {
        const int ks = b >> 1, t = 2 * (b & 1);
        if (b + 1 < 2 * NK) keys(b + 1);
        __builtin_amdgcn_sched_barrier(0);
        if ((b & 1) == 0) {
          s = split8x3(S[ks][0], S[ks][1]);
          if (kMode == kWalkSave && 32 * ks + 8 * lg < a.N) {
            bf16 *to = (bf16 *)a.st0 + (((size_t)(w.slot + c) * a.H + h) * a.P + p0) * a.N + 32 * ks;
            store_at(to, (uint32_t)(lr * a.N + 8 * lg) * 2u, s.hi);
            store_at(to + a.st_rest, (uint32_t)(lr * a.N + 8 * lg) * 2u, s.mid);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) A[t + u] = mfma(kb[b & 1][u], s.hi, A[t + u]);
        if (kY)
#pragma unroll
          for (int u = 0; u < 2; ++u) O[t + u] = mfma(s.hi, qb[b & 1][u], O[t + u]);
        if (kY)
#pragma unroll
          for (int u = 0; u < 2; ++u) O[t + u] = mfma(s.mid, qb[b & 1][u], O[t + u]);
#pragma unroll
        for (int u = 0; u < 2; ++u) A[t + u] = mfma(kb[b & 1][u], s.mid, A[t + u]);
#pragma unroll
        for (int u = 0; u < 2; ++u) A[t + u] = mfma(kb[b & 1][u], s.lo, A[t + u]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    const auto tri_tiles = [&](const bf16 *level,
                               bf16x8 (&to)[kTriTiles]) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < kTriTiles; ++k)
        to[k] = *reinterpret_cast<const bf16x8 *>(level + k * kTileElems + 8 * lane);
    };
    // M: the ten tiles Q_i K_j^T on and below the diagonal (lane: token lr of tile i, 4 tokens
    // of tile j) with their decays, shared out over the waves by the rows they read
    MTile m[kY ? 4 / WV : 1][3];
    if (kY)
#pragma unroll
      for (int k = 0; k < 4 / WV; ++k) {
        const int role = wave + WV * k;
        if (role == 0)
          m_tiles<NK, 0, 0, 1, 0, 1, 1>(m[k], sK, sQ, G);
        else if (role == 1)
          m_tiles<NK, 2, 0, 2, 1, 2, 2>(m[k], sK, sQ, G);
        else if (role == 2)
          m_tiles<NK, 3, 0, 3, 1>(m[k], sK, sQ, G);
        else
          m_tiles<NK, 3, 2, 3, 3>(m[k], sK, sQ, G);
      }
    bf16x8 T[kTriTiles];
    tri_tiles(sT, T);
    wait_vmem_all();
    __syncthreads();
    stage_block<WV>(sQ, tri_at(c) + 2 * kLevelElems, kTriTiles);
    // (behind T's last level, as operand tiles)
    if (kY)
#pragma unroll
      for (int k = 0; k < 4 / WV; ++k) {
        const int role = wave + WV * k;
        if (role == 0)
          put_m_tiles<0, 0, 1, 0, 1, 1>(m[k], sQ + kLevelElems);
        else if (role == 1)
          put_m_tiles<2, 0, 2, 1, 2, 2>(m[k], sQ + kLevelElems);
        else if (role == 2)
          put_m_tiles<3, 0, 3, 1>(m[k], sQ + kLevelElems);
        else
          put_m_tiles<3, 2, 3, 3>(m[k], sQ + kLevelElems);
      }
    __builtin_amdgcn_sched_barrier(0);
    // R, as operands
    Split3 R[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      f32x4 v[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = 2 * kt + u;
        const f32x4 b = ldf4(G.b + 16 * t + 4 * lg), be = ldf4(G.be + 16 * t + 4 * lg);
        v[u] = -be * A[t];
        if (valued) v[u] += b * value_tile<W>(sV, 16 * t, p0 - 16 * tile0);
      }
      R[kt] = split8x3(v[0], v[1]);
    }
    // U = T R, level by level of T with what of R is not below fp32's last bit
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) A[i] = kZero4;
    const auto times = [&](bf16x8 Split3::*part) __attribute__((always_inline)) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int i = 2 * kt; i < 4; ++i)
          A[i] = mfma(lower_operand(T[lower_tile(i, kt)], i, kt), R[kt].*part, A[i]);
    };
    times(&Split3::hi), times(&Split3::mid), times(&Split3::lo);
    tri_tiles(sT + kLevelElems, T);
    times(&Split3::hi), times(&Split3::mid);
    wait_vmem_all();
    __syncthreads();
    tri_tiles(sQ, T);
    if (c + 1 < chunks) fetch_tri(c + 1);
    times(&Split3::hi);
    const float ec = G.ef[kDeltaChunk - 1];
    bf16x8 kT[2][2];  // of a block of 16 channels, the next one's under way
    const auto columns = [&](int b) __attribute__((always_inline)) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) kT[b & 1][kt] = state_operand<N>(sK, kt, b >> 1, b & 1);
    };
    Split U[2];
    if (kY) {
      bf16x8 M[kTriTiles];
      tri_tiles(sQ + kLevelElems, M);
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) U[kt] = split8(A[2 * kt], A[2 * kt + 1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) O[t] *= G.ef[16 * t + lr];
      const auto times_m = [&](bf16x8 Split::*part) __attribute__((always_inline)) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int t = 2 * kt; t < 4; ++t)
            O[t] = mfma(U[kt].*part, lower_operand(M[lower_tile(t, kt)], t, kt), O[t]);
      };
      times_m(&Split::hi), times_m(&Split::lo);
      tri_tiles(sQ + 2 * kLevelElems, M);
      times_m(&Split::hi);
    } else if (!kLocal) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) U[kt] = split8(A[2 * kt], A[2 * kt + 1]);
    }
    // the state: rows of U fall by e^{gam_c - gam}
    __builtin_amdgcn_sched_barrier(0);
    columns(0);
    Split3 D[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
      D[kt] = split8x3(A[2 * kt] * ldf4(G.lf + 32 * kt + 4 * lg),
                       A[2 * kt + 1] * ldf4(G.lf + 32 * kt + 16 + 4 * lg));
#pragma unroll
    for (int b = 0; b < 2 * NK; ++b) {
      if (b + 1 < 2 * NK) columns(b + 1);
      __builtin_amdgcn_sched_barrier(0);
      f32x4 s = S[b >> 1][b & 1] * ec;
      s = mfma(kT[b & 1][0], D[0].hi, s);
      s = mfma(kT[b & 1][0], D[0].mid, s);
      s = mfma(kT[b & 1][0], D[0].lo, s);
      s = mfma(kT[b & 1][1], D[1].hi, s);
      s = mfma(kT[b & 1][1], D[1].mid, s);
      S[b >> 1][b & 1] = mfma(kT[b & 1][1], D[1].lo, s);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (kY) {
      // y by whole rows of the workgroup's columns: 16 bytes a lane
      const int own = lane_anew(), row = own & 15, col = p0 - 16 * tile0 + 4 * (own >> 4);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        *reinterpret_cast<uint2 *>(sV + place<W>(16 * t + row, col)) =
            make_uint2(pack2(O[t][0], O[t][1]), pack2(O[t][2], O[t][3]));
    } else if (!kLocal) {
      // (tokens in the order of the operands: 16 bytes a lane)
      bf16 *u = (bf16 *)a.u + (((size_t)(w.slot + c) * a.H + h) * a.P + p0) * kDeltaChunk;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        store_at(u + 32 * kt, (uint32_t)(lr * kDeltaChunk + 8 * lg) * 2u, U[kt].hi);
        store_at(u + a.u_rest + 32 * kt, (uint32_t)(lr * kDeltaChunk + 8 * lg) * 2u, U[kt].lo);
      }
    }
    __syncthreads();
    if (c + 1 < chunks) fetch_rows(c + 1);
    if (kY) {
      constexpr int kPer = 64 * 8 / W;  // rows of an instruction
      bf16 *y = (bf16 *)a.y + ((size_t)at * a.H + h) * a.P + 16 * tile0;
      const int own = lane_anew(), row = own / (W / 8), col = 8 * (own % (W / 8));
#pragma unroll
      for (int k = 0; k < kDeltaChunk / (kPer * WV); ++k) {
        const int t = (k * WV + wave) * kPer;
        const bf16x8 v = *reinterpret_cast<const bf16x8 *>(sV + place<W>(t + row, col));
        if (t + row < len) store_at(y + t * ldx, (uint32_t)(row * (int)ldx + col) * 2u, v);
      }
    }
  }
  float *to = nullptr;
  if (kLocal && on)
    to = a.span + (((size_t)sg * a.H + h) * (a.P + a.N) + p) * a.N;
  else if (kY && a.hT && w.last)
    to = a.hT + (((size_t)w.s * a.H + h) * a.P + p) * a.N;
  if (to)
#pragma unroll
    for (int ks = 0; ks < NK; ++ks)
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const int n = 32 * ks + 8 * lg + 4 * par;
        if (n < a.N) stf4(to + n, S[ks][par]);
      }
}

// Backwards, from the last chunk to the first:
//   dU = M^T dY + e^{gam_c - gam} (K dS),  dR = T^T dU
//   dS <- e^{gam_c} dS + Q^T (e^gam dY) - K^T (beta e^gam dR)
// Writes dS behind each chunk, dR, and the initial state's gradient; or
// (kLocal) a segment's dS at its start from zeros at its end.
template <int NK, int WV, bool kLocal>
__device__ __forceinline__ void walk_backwards(const DeltaArgs &a, int unit, bf16 *sK, bf16 *sQ,
                                               bf16 *sT, bf16 *sV, Gates &G) {
  constexpr int N = 32 * NK, W = 16 * WV;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = a.P / W;
  const int pw = (unit % blocks) * W, p0 = pw + 16 * wave, p = p0 + lr;
  unit /= blocks;
  const int h = unit % a.H, sg = unit / a.H, grp = h / a.hpg;
  DeltaWalk w;
  if (!delta_walk(a, sg, w)) return;
  if (kLocal && w.first) return;            // nothing ends at its start

  f32x4 S[NK][2];
  {
    const float *from = nullptr;
    if (!kLocal && a.seg)
      from = a.dspan + (((size_t)sg * a.H + h) * a.P + p) * a.N;
    else if (!kLocal && a.dhT)
      from = a.dhT + (((size_t)w.s * a.H + h) * a.P + p) * a.N;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks)
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const int n = 32 * ks + 8 * lg + 4 * par;
        S[ks][par] = from && n < a.N ? ldf4(from + n) : kZero4;
      }
  }

  const size_t ldk = (size_t)a.G * a.N, ldx = (size_t)a.H * a.P;
  const int chunks = (int)((w.hi - w.lo + kDeltaChunk - 1) / kDeltaChunk);
  const auto length = [&](int c) {
    return (int)min((int64_t)kDeltaChunk, w.hi - w.lo - (int64_t)c * kDeltaChunk);
  };
  const auto rows_at = [&](int c) { return (w.lo + (int64_t)c * kDeltaChunk); };
  const auto tri_at = [&](int c) {
    return (const bf16 *)a.tri + ((size_t)(w.slot + c) * a.H + h) * a.tri_stride;
  };
  uint16_t g = 0, bt = 0;
  // K and M^T, and what is free earlier in a chunk: Q and dY (T^T takes M^T's
  // place once dU is done)
  const auto fetch_keys = [&](int c) __attribute__((always_inline)) {
    const int64_t at = rows_at(c);
    if (wave == 0) {
      const size_t ga = (size_t)(at + min(lane, length(c) - 1)) * a.H + h;
      g = ((const uint16_t *)a.g)[ga];
      bt = ((const uint16_t *)a.beta)[ga];
    }
    stage_tile<N, kDeltaChunk, WV>(sK, (const bf16 *)a.B + (at * a.G + grp) * a.N, ldk, a.N,
                                   length(c));
    stage_block<WV>(sT, tri_at(c) + 2 * kMatrixElems, 2 * kTriTiles);
  };
  const auto fetch_rows = [&](int c) __attribute__((always_inline)) {
    const int64_t at = rows_at(c);
    stage_tile<N, kDeltaChunk, WV>(sQ, (const bf16 *)a.C + (at * a.G + grp) * a.N, ldk, a.N,
                                   length(c));
    stage_tile<W, kDeltaChunk, WV>(sV, (const bf16 *)a.dy + ((size_t)at * a.H + h) * a.P + pw, ldx,
                                   W, length(c));
  };
  const auto tri_tiles = [&](const bf16 *level,
                             bf16x8 (&to)[kTriTiles]) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kTriTiles; ++k)
      to[k] = *reinterpret_cast<const bf16x8 *>(level + k * kTileElems + 8 * lane);
  };
  if (chunks > 0) {
    fetch_keys(chunks - 1);
    fetch_rows(chunks - 1);
  }
  for (int c = chunks - 1; c >= 0; --c) {
    const int len = length(c);
    wait_vmem_all();
    if (wave == 0) fill_gates(G, bits_to_f32(g), bits_to_f32(bt), lane < len);
    __syncthreads();
    // dY as it is (rows past the end are zeros)
    bf16x8 Y[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) Y[kt] = value_operand<W>(sV, kt, p0 - pw);
    __syncthreads();
    stage_block<WV>(sV, tri_at(c) + 2 * kMatrixElems + 2 * kLevelElems, kTriTiles);
    f32x4 A[4];
    {
      bf16x8 kb[2][2];
      const auto keys = [&](int b) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          kb[b & 1][u] = *reinterpret_cast<const bf16x8 *>(
              sK + place<N>(32 * (b & 1) + 16 * u + lr, 32 * (b >> 1) + 8 * lg));
      };
      keys(0);
#pragma unroll
      for (int t = 0; t < 4; ++t) A[t] = kZero4;
      Split3 s;
#pragma unroll
      for (int b = 0; b < 2 * NK; ++b) {
        const int ks = b >> 1, t = 2 * (b & 1);
        if (b + 1 < 2 * NK) keys(b + 1);
        __builtin_amdgcn_sched_barrier(0);
        if ((b & 1) == 0) {
          s = split8x3(S[ks][0], S[ks][1]);
          if (!kLocal && 32 * ks + 8 * lg < a.N) {
            bf16 *to = (bf16 *)a.st1 + (((size_t)(w.slot + c) * a.H + h) * a.P + p0) * a.N + 32 * ks;
            store_at(to, (uint32_t)(lr * a.N + 8 * lg) * 2u, s.hi);
            store_at(to + a.st_rest, (uint32_t)(lr * a.N + 8 * lg) * 2u, s.mid);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) A[t + u] = mfma(kb[b & 1][u], s.hi, A[t + u]);
#pragma unroll
        for (int u = 0; u < 2; ++u) A[t + u] = mfma(kb[b & 1][u], s.mid, A[t + u]);
#pragma unroll
        for (int u = 0; u < 2; ++u) A[t + u] = mfma(kb[b & 1][u], s.lo, A[t + u]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // dU: M^T by levels, the last one in the values' place
    Split3 U[2];
    bf16x8 T[kTriTiles];
    const auto times_y = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int t = 0; t < 2 * kt + 2; ++t)
          A[t] = mfma(upper_operand(T[upper_tile(t, kt)], t, kt), Y[kt], A[t]);
    };
    tri_tiles(sT, T);
#pragma unroll
    for (int t = 0; t < 4; ++t) A[t] *= ldf4(G.lf + 16 * t + 4 * lg);
    times_y();
    tri_tiles(sT + kLevelElems, T);
    times_y();
    wait_vmem_all();
    __syncthreads();
    tri_tiles(sV, T);
    stage_block<WV>(sT, tri_at(c) + kMatrixElems, 2 * kTriTiles);
    times_y();
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) U[kt] = split8x3(A[2 * kt], A[2 * kt + 1]);
    __syncthreads();
    stage_block<WV>(sV, tri_at(c) + kMatrixElems + 2 * kLevelElems, kTriTiles);
    // dS <- e^{gam_c} dS + Q^T (e^gam dY), while T^T comes
    const float ec = G.ef[kDeltaChunk - 1];
    bf16x8 kT[2][2];  // of a block of 16 channels, the next one's under way
    const auto columns = [&](const bf16 *rows, int b) __attribute__((always_inline)) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) kT[b & 1][kt] = state_operand<N>(rows, kt, b >> 1, b & 1);
    };
    columns(sQ, 0);
    {
      Split3 E[2];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        f32x4 e[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4 ef = ldf4(G.ef + 32 * kt + 16 * u + 4 * lg);
#pragma unroll
          for (int r = 0; r < 4; ++r) e[u][r] = ef[r] * (float)Y[kt][4 * u + r];
        }
        E[kt] = split8x3(e[0], e[1]);
      }
#pragma unroll
      for (int b = 0; b < 2 * NK; ++b) {
        if (b + 1 < 2 * NK) columns(sQ, b + 1);
        __builtin_amdgcn_sched_barrier(0);
        f32x4 s = S[b >> 1][b & 1] * ec;
        s = mfma(kT[b & 1][0], E[0].hi, s);
        s = mfma(kT[b & 1][0], E[0].mid, s);
        s = mfma(kT[b & 1][0], E[0].lo, s);
        s = mfma(kT[b & 1][1], E[1].hi, s);
        s = mfma(kT[b & 1][1], E[1].mid, s);
        S[b >> 1][b & 1] = mfma(kT[b & 1][1], E[1].lo, s);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_vmem_all();
    __syncthreads();
    // dR = T^T dU, level by level as U = T R
#pragma unroll
    for (int t = 0; t < 4; ++t) A[t] = kZero4;
    const auto times = [&](bf16x8 Split3::*part) __attribute__((always_inline)) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int t = 0; t < 2 * kt + 2; ++t)
          A[t] = mfma(upper_operand(T[upper_tile(t, kt)], t, kt), U[kt].*part, A[t]);
    };
    tri_tiles(sV, T);
    times(&Split3::hi);
    __syncthreads();
    if (c > 0) fetch_rows(c - 1);
    tri_tiles(sT, T);
    times(&Split3::hi), times(&Split3::mid), times(&Split3::lo);
    tri_tiles(sT + kLevelElems, T);
    times(&Split3::hi), times(&Split3::mid);
    if (!kLocal) {
      bf16 *dr = (bf16 *)a.dr + (((size_t)(w.slot + c) * a.H + h) * a.P + p0) * kDeltaChunk;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const Split r = split8(A[2 * kt], A[2 * kt + 1]);
        store_at(dr + 32 * kt, (uint32_t)(lr * kDeltaChunk + 8 * lg) * 2u, r.hi);
        store_at(dr + a.u_rest + 32 * kt, (uint32_t)(lr * kDeltaChunk + 8 * lg) * 2u, r.lo);
      }
    }
    // dS <- dS - K^T (beta e^gam dR)
    columns(sK, 0);
    Split3 D[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
      D[kt] = split8x3(-ldf4(G.be + 32 * kt + 4 * lg) * A[2 * kt],
                       -ldf4(G.be + 32 * kt + 16 + 4 * lg) * A[2 * kt + 1]);
#pragma unroll
    for (int b = 0; b < 2 * NK; ++b) {
      if (b + 1 < 2 * NK) columns(sK, b + 1);
      __builtin_amdgcn_sched_barrier(0);
      f32x4 s = mfma(kT[b & 1][0], D[0].hi, S[b >> 1][b & 1]);
      s = mfma(kT[b & 1][0], D[0].mid, s);
      s = mfma(kT[b & 1][0], D[0].lo, s);
      s = mfma(kT[b & 1][1], D[1].hi, s);
      s = mfma(kT[b & 1][1], D[1].mid, s);
      S[b >> 1][b & 1] = mfma(kT[b & 1][1], D[1].lo, s);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (c > 0) {
      __syncthreads();
      fetch_keys(c - 1);
    }
  }
  float *to = nullptr;
  if (kLocal)
    to = a.dspan + (((size_t)sg * a.H + h) * a.P + p) * a.N;
  else if (a.dh0 && w.first)
    to = a.dh0 + (((size_t)w.s * a.H + h) * a.P + p) * a.N;
  if (to)
#pragma unroll
    for (int ks = 0; ks < NK; ++ks)
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const int n = 32 * ks + 8 * lg + 4 * par;
        if (n < a.N) stf4(to + n, S[ks][par]);
      }
}

// Three workgroups of four waves to a compute unit: 168 registers and 53 KB of
// LDS each.
template <int NK, int WV, WalkMode kMode>
__global__ __launch_bounds__(64 * WV, (NK <= 4 ? 3 : 1)) void k_delta_walk(DeltaArgs a) {
  constexpr bool kY = kMode == kWalkY;
  constexpr int kFree = (kY ? 3 : 1) * kLevelElems;  // what takes Q's place
  __shared__ bf16 sK[kRowElems<NK>], sT[kTriElems], sV[kDeltaChunk * 16 * WV];
  __shared__ bf16 sQ[kY && kRowElems<NK> > kFree ? kRowElems<NK> : kFree];
  __shared__ Gates G;
  const int unit = kMode == kWalkLocal
                       ? xcd_unit()
                       : delta_unit(a, (int)blockIdx.x, (int)gridDim.x, a.H * (a.P / (16 * WV)));
  if (unit >= 0) walk_forwards<NK, WV, kMode>(a, unit, sK, sQ, sT, sV, G);
}

// The backward pass's two walks at once: neither needs the other (dS goes without
// S and U), and one alone leaves most of a compute unit idle while it waits for its
// chunk's products. The first `back` workgroups walk backwards, the longer way.
template <int NK, int WV, bool kLocal>
__global__ __launch_bounds__(64 * WV, (NK <= 4 ? 3 : 1)) void k_delta_both(DeltaArgs a, int back) {
  constexpr int kValues = kDeltaChunk * 16 * WV;
  __shared__ bf16 sK[kRowElems<NK>], sQ[kRowElems<NK>], sT[kTriElems];
  __shared__ bf16 sV[kValues > kLevelElems ? kValues : kLevelElems];  // (a level takes its place)
  __shared__ Gates G;
  static_assert(kRowElems<NK> >= kLevelElems, "a level must fit where Q is");
  const int per = a.H * (a.P / (16 * WV)), b = (int)blockIdx.x;
  const int unit = b < back ? delta_unit(a, b, back, per)
                            : delta_unit(a, b - back, (int)gridDim.x - back, per);
  if (unit < 0) return;
  if (b < back)
    walk_backwards<NK, WV, kLocal>(a, unit, sK, sQ, sT, sV, G);
  else
    walk_forwards<NK, WV, kLocal ? kWalkLocal : kWalkSave>(a, unit, sK, sQ, sT, sV, G);
}

// The states at the segments' starts, in place of their own final states: with
// F a segment's transition, S <- F S + (its own). kBack: dL/dS at the segments'
// ends, dS <- F^T dS + (its own), from the last to the first. Per (sequence,
// head) and 16 columns a workgroup of WV waves, in fp32 throughout; wave w holds
// the state channels of tiles w, w + WV, ...; the state goes round through LDS.
// A transition does not depend on the state: the next one is on its way into
// registers while one is used (without that, 16 segments of 32 heads of 128 x 128
// took 130 us, not 56). `span` has a transition's
// columns as rows: span[P + j][n] = F[n][j].
template <int NT, int WV, bool kBack>
__global__ __launch_bounds__(64 * WV) void k_delta_join(DeltaArgs a) {
  constexpr int kOwn = NT / WV;  // tiles of a wave
  __shared__ float sS[2][16 * NT][17];
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4, wave = threadIdx.x >> 6;
  const int blocks = a.P / 16;
  int unit = blockIdx.x;
  const int p = (unit % blocks) * 16 + lr;
  unit /= blocks;
  const int h = unit % a.H, seq = unit / a.H;
  int64_t lo, hi;
  delta_seq(a, seq, lo, hi);
  const int64_t len = (int64_t)kDeltaChunk * a.seg;
  const int first = a.cu ? (int)(lo / len) + seq : seq * a.nseg_per;
  const int n = max(1, (int)((hi - lo + len - 1) / len));
  const float *init = kBack ? a.dhT : a.h0;
  const auto place_of = [&](int c) { return (size_t)(first + (kBack ? n - 1 - c : c)) * a.H + h; };
  f32x4 S[kOwn], F[kOwn][NT], own[kOwn];
  const auto fetch = [&](int c) __attribute__((always_inline)) {
    const size_t at = place_of(c);
    const float *from = kBack ? a.dspan + (at * a.P + p) * a.N : a.span + (at * (a.P + a.N) + p) * a.N;
    const float *f = a.span + (at * (a.P + a.N) + a.P) * a.N;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const int t = 16 * (wave + WV * k);
      if (t >= a.N) continue;
      own[k] = ldf4(from + t + 4 * lg);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (16 * j >= a.N) continue;
        if (kBack) {
          F[k][j] = ldf4(f + (size_t)(t + lr) * a.N + 16 * j + 4 * lg);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) F[k][j][r] = f[(size_t)(16 * j + 4 * lg + r) * a.N + t + lr];
        }
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    const int t = 16 * (wave + WV * k);
    S[k] = init && t < a.N ? ldf4(init + (((size_t)seq * a.H + h) * a.P + p) * a.N + t + 4 * lg)
                           : kZero4;
#pragma unroll
    for (int j = 0; j < NT; ++j) F[k][j] = kZero4;
    own[k] = kZero4;
  }
  if (n > 1) fetch(0);
  for (int c = 0; c < n; ++c) {
    const size_t at = place_of(c);
    float *to = kBack ? a.dspan + (at * a.P + p) * a.N : a.span + (at * (a.P + a.N) + p) * a.N;
    float (*s)[17] = sS[c & 1];
    f32x4 next[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const int t = 16 * (wave + WV * k);
      next[k] = own[k];
      if (t < a.N) stf4(to + t + 4 * lg, S[k]);
#pragma unroll
      for (int r = 0; r < 4; ++r) s[t + 4 * lg + r][lr] = S[k][r];
    }
    if (c + 1 == n) break;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      f32x4 b;
#pragma unroll
      for (int r = 0; r < 4; ++r) b[r] = s[16 * j + 4 * lg + r][lr];
#pragma unroll
      for (int k = 0; k < kOwn; ++k) next[k] = mfma16(F[k][j], b, next[k]);
    }
    if (c + 2 < n) fetch(c + 1);
#pragma unroll
    for (int k = 0; k < kOwn; ++k) S[k] = next[k];
  }
}

enum Walk : int { kForward, kForwardLocal, kBoth, kBothLocal };

template <int NK, int WV>
hipError_t walk_launch(const DeltaArgs &a, Walk what, hipStream_t s) {
  // (a segment's local walk forwards takes its transition's columns too)
  const int tiles = a.P / 16, more = what == kForwardLocal || what == kBothLocal ? a.N / 16 : 0;
  const int64_t seqs = a.seg ? a.nsegs : a.order ? (a.nseq + 7) / 8 * 8 : a.nseq;
  const int64_t units = seqs * a.H;
  const unsigned ahead = (unsigned)(units * ((tiles + more + WV - 1) / WV));
  const unsigned back = (unsigned)(units * (tiles / WV));
  const dim3 block(64 * WV);
  switch (what) {
    case kForward:
      hipLaunchKernelGGL((k_delta_walk<NK, WV, kWalkY>), dim3(ahead), block, 0, s, a);
      break;
    case kForwardLocal:
      hipLaunchKernelGGL((k_delta_walk<NK, WV, kWalkLocal>), dim3(ahead), block, 0, s, a);
      break;
    case kBoth:
      hipLaunchKernelGGL((k_delta_both<NK, WV, false>), dim3(back + ahead), block, 0, s, a, (int)back);
      break;
    case kBothLocal:
      hipLaunchKernelGGL((k_delta_both<NK, WV, true>), dim3(back + ahead), block, 0, s, a, (int)back);
      break;
  }
  return hipGetLastError();
}

template <int NK>
hipError_t walk_n(const DeltaArgs &a, Walk what, hipStream_t s) {
  if (a.P == 16) return walk_launch<NK, 1>(a, what, s);
  if (a.P == 32) return walk_launch<NK, 2>(a, what, s);
  return walk_launch<NK, 4>(a, what, s);
}

hipError_t walk(const DeltaArgs &a, Walk what, hipStream_t s) {
  if (a.nseq == 0) return hipSuccess;
  if (a.N <= 64) return walk_n<2>(a, what, s);
  if (a.N <= 128) return walk_n<4>(a, what, s);
  return walk_n<8>(a, what, s);
}

template <int NT, int WV>
hipError_t join_n(const DeltaArgs &a, bool back, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.nseq * a.H * (a.P / 16))), block(64 * WV);
  if (back)
    hipLaunchKernelGGL((k_delta_join<NT, WV, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_delta_join<NT, WV, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t join(const DeltaArgs &a, bool back, hipStream_t s) {
  if (a.N <= 64) return join_n<4, 4>(a, back, s);
  if (a.N <= 128) return join_n<8, 4>(a, back, s);
  return join_n<16, 8>(a, back, s);
}

// Whether and where sequences are cut. Whole, a call takes its sequences' chunks one
// after the other, while a workgroup (64 columns) on each compute unit is close to
// half of what the units give. Cut, every segment is walked twice, the N columns of
// its transition come along, and each of its joins takes a time that goes with N.
// In units of a walk's chunk (5 us at N = 128), with w walks (1, backward 2):
//   whole: chunks
//   cut:   the longer of two segments and the work, (2 w + N / P) of it, at 0.6 of
//          a chunk a workgroup (three share a unit; 1 past N = 128, where one fills
//          it), w N / 128 a segment for the joins, and w + 1 launches more
// sqrt(chunks) of them make a segment, or as many as leave two workgroups for each
// unit. Packed sequences are cut by their mean length: what they hold is not known here,
// and one long sequence among short ones is walked whole. Measured in us, whole and cut:
//   32 heads of 128, 1 x 16384 tokens   1448, 619    backward 2401, 1845
//   32 heads of 128, 1 x 2048 tokens     176, 116    backward  318,  327 (not cut)
//   24 heads of 64, 1 x 4096 tokens      334, 125    backward  451,  317
//   24 heads of 64, 2 x 4096 tokens      334, 177    backward  573,  531
//   24 heads of 64, 1 x 2048 tokens      173,  91    backward  241,  202
//   24 heads of 64, 1 x 1024 tokens       92,  67    backward  137,  129 (not cut)
//   80 heads of 64, 1 x 4096 tokens      341, 279
//   32 heads of 64, 2 x 4096, N = 64     277, 129
//   16 heads of 128, N = 256, 1 x 4096   478, 293    backward  760,  823 (not cut)
//   32 heads of 64, 2 x 2048, N = 256    254, 385 (not cut)
void delta_segments(DeltaArgs &a, bool packed, bool backward) {
  constexpr int kComputeUnits = 256;
  a.seg = a.nseg_per = a.nsegs = 0;
  if (a.nseq == 0 || a.T == 0) return;
  // (packed: on average, and at least one where there are fewer tokens than sequences)
  const int64_t all = (int64_t)kDeltaChunk * a.nseq, chunks = (a.T + all - 1) / all;
  const int64_t groups = (int64_t)a.nseq * a.H * ((a.P + 63) / 64);
  const int64_t w = backward ? 2 : 1;
  int64_t m = chunks * groups * w / (2 * kComputeUnits);
  while (m * m < chunks) ++m;
  const float fill = (float)groups * (float)chunks / kComputeUnits * (a.N <= 128 ? 0.6f : 1.f);
  const float work = fill * (2.f * (float)w + (float)a.N / (float)a.P);
  const float joins = (float)((chunks + m - 1) / m * w) * (float)a.N / 128.f;
  if (fmaxf(2.f * (float)m, work) + joins + (float)(w + 1) >= (float)chunks) return;
  a.seg = (int)m;
  a.nseg_per = (int)((a.nc_per + m - 1) / m);
  a.nsegs = packed ? (int)(a.T / (kDeltaChunk * m)) + a.nseq : a.nseq * a.nseg_per;
}

hipError_t launch_delta_forward(const DeltaArgs &a, hipStream_t s) {
  if (a.seg) {
    hipError_t e = walk(a, kForwardLocal, s);
    if (e == hipSuccess) e = join(a, false, s);
    if (e != hipSuccess) return e;
  }
  return walk(a, kForward, s);
}

hipError_t launch_delta_both_ways(const DeltaArgs &a, hipStream_t s) {
  if (a.seg) {
    hipError_t e = walk(a, kBothLocal, s);
    if (e == hipSuccess) e = join(a, false, s);
    if (e == hipSuccess) e = join(a, true, s);
    if (e != hipSuccess) return e;
  }
  return walk(a, kBoth, s);
}

}  // namespace ssd
