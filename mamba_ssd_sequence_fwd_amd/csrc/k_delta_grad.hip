// k_delta_grad.hip -- the gradients of the gated delta rule's chunks in bf16.
//
// One workgroup takes a chunk and a part of the heads of one group, head by
// head; wave w owns tokens 16 w .. 16 w + 15 and keeps their dQ and dK (fp32,
// all state channels) in registers over the heads. With D the decay factors
// e^{gam_i - gam_j}, dM = dY U^T (i >= j), dL = -dR U^T (i > j):
//   dx = beta dR
//   dQ = e^gam dY S^T + (dM D) K
//   dK = -beta e^gam dR S^T + e^{gam_c - gam} U dS^T + (dM D)^T Q + (dL beta D) K + (dL beta D)^T K
//   dbeta = dR . V - e^gam K . (dR S^T) + sum_j dL (K K^T) D
//   dg_t = sum_{i >= t} [e^gam Q . (dY S^T) - beta e^gam K . (dR S^T)]_i
//        + sum_{i < t} [e^{gam_c - gam} K . (U dS^T)]_i
//        + sum_{i >= t > j} (dM M + dL L)_ij + e^{gam_c} <S, dS>
// Results are taken transposed (lane: token, 4 state channels), so that the
// pair matrices' result tiles are right operands as they are: once as rows j of
// a column i for dQ and (dL beta D) K, once as rows i of a column j for the
// transposed products. The pair sum of dg is taken as suffix sums of row sums
// less column sums of the same fp32 products, so that pairs on one side of t
// cancel. K, Q and dY are bf16 as they are; S, dS, U, dR and the pair matrices are in
// two bf16 each (2^-17 off; a product leaves out that of the two rests), so that the
// gradients' error is the rounding of the results (1.66e-3; with one bf16 each they were
// 2.3e-3 to 3.0e-3 off). Every sum is fp32. The states pass through LDS 32 channels at
// a time, the next block under way while one is used.
//
// Measured (MI355X), 32 heads of 128 x 128, 4 x 2048 tokens: 346 to 389 us. 1456 MB
// counted (S and dS are 537 of them) take 285 us at a copy's rate; matrix instructions
// are busy for 60 us and vector instructions for 137, two workgroups a compute unit. (The
// pair matrices of each pass of value channels by themselves took 433 to 485 us.)
#include "delta_tiles.h"

namespace ssd {
namespace {

// Eight consecutive elements, and four rows of one column (transposed read).
__device__ __forceinline__ bf16x8 read8(const bf16 *t, int at) {
  return *reinterpret_cast<const bf16x8 *>(t + at);
}
__device__ __forceinline__ bf16x8 read4x2(const bf16 *t, int at, int at2) {
  const bf16x4 a = ds_tr4(t, at), b = ds_tr4(t, at2);
  return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// A lane's places in the staged tiles, of which all others follow by an XOR of
// the column and an added row: W is a power of two, the swizzle an XOR and the
// same for rows 16 apart. (Made anew for each use of the tiles: kept over the
// heads, the places themselves would fill the registers.)
template <int N, int P>
struct Places {
  int row, own4, yrow;   // row lr: columns 8 lg of K and Q, 4 lg, and 8 lg of dY
  int tile;              // transposed, result-tile order: rows 4 lg + lr / 4 of K, Q
  int tok0, tok1;        // transposed: rows 8 lg + lr / 4 (+ 4) of U, dR, tokens 8 (lr % 4)
  int st0, st1;          // the same of a block of S, columns 4 (lr % 4)
  __device__ __forceinline__ Places() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int lr = lane & 15, lg = lane >> 4, r8 = 8 * lg + (lr >> 2);
    row = place<N>(lr, 8 * lg);
    own4 = place<N>(lr, 4 * lg);
    yrow = place<P>(lr, 8 * lg);
    tile = place<N>(4 * lg + (lr >> 2), 4 * (lr & 3));
    tok0 = place<kDeltaChunk>(r8, 8 * (lr & 3));
    tok1 = place<kDeltaChunk>(r8 + 4, 8 * (lr & 3));
    st0 = place<32>(r8, 4 * (lr & 3));
    st1 = place<32>(r8 + 4, 4 * (lr & 3));
  }
  // K or Q: eight of row 16 t + lr from column 32 ks + 8 lg
  __device__ __forceinline__ bf16x8 keys(const bf16 *s, int t, int ks) const {
    return read8(s, (row ^ (32 * ks)) + 16 * t * N);
  }
  // dY: the same
  __device__ __forceinline__ bf16x8 values(const bf16 *s, int t, int ps) const {
    return read8(s, (yrow ^ (32 * ps)) + 16 * t * P);
  }
  // K or Q transposed: tokens 32 kt + 16 (e / 4) + 4 lg + e % 4 of column n0 + lr
  __device__ __forceinline__ bf16x8 columns(const bf16 *s, int kt, int n0) const {
    const int at = (tile ^ n0) + 32 * kt * N;
    return read4x2(s, at, at + 16 * N);
  }
  // U or dR (rows of value channels, a pair of tiles' tokens in the order of the
  // operands: 32 kt + 8 lg + e for token 32 kt + 16 (e / 4) + 4 lg + e % 4):
  // channels 32 ps + 8 lg + e of token 16 t + lr
  __device__ __forceinline__ Split tokens(const bf16 (*s)[P * kDeltaChunk], int ps, int t) const {
    const int x = 32 * (t >> 1), d = 4 * (t & 1) + 32 * ps * kDeltaChunk;
    return Split{read4x2(s[0], (tok0 ^ x) + d, (tok1 ^ x) + d),
                 read4x2(s[1], (tok0 ^ x) + d, (tok1 ^ x) + d)};
  }
  // a block of S: channels 32 ps + 8 lg + e of column 16 par + lr
  __device__ __forceinline__ Split state(const bf16 (*s)[P * 32], int ps, int par) const {
    const int a = (st0 ^ (16 * par)) + 32 * ps * 32, b = (st1 ^ (16 * par)) + 32 * ps * 32;
    return Split{read4x2(s[0], a, b), read4x2(s[1], a, b)};
  }
};

__device__ __forceinline__ float dot8(const Split &a, bf16x8 b) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s += ((float)a.hi[e] + (float)a.lo[e]) * (float)b[e];
  return s;
}
__device__ __forceinline__ float dot8(const Split &a, const Split &b) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    s += ((float)a.hi[e] + (float)a.lo[e]) * ((float)b.hi[e] + (float)b.lo[e]);
  return s;
}
// c += A B for operands in two bf16, of which one may be exact.
using ssd::mfma;
__device__ __forceinline__ f32x4 mfma(const Split &a, bf16x8 b, f32x4 c) {
  return ssd::mfma(a.lo, b, ssd::mfma(a.hi, b, c));
}
__device__ __forceinline__ f32x4 mfma(bf16x8 a, const Split &b, f32x4 c) {
  return ssd::mfma(a, b.lo, ssd::mfma(a, b.hi, c));
}
__device__ __forceinline__ f32x4 mfma(const Split &a, const Split &b, f32x4 c) {
  return ssd::mfma(a.lo, b.hi, ssd::mfma(a.hi, b.lo, ssd::mfma(a.hi, b.hi, c)));
}
// Sum over the four lanes that share lr.
__device__ __forceinline__ float sum_lg(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
// A sum that is added up where it is written: left to the end, with all that it is
// the sum of, it fills the registers.
__device__ __forceinline__ void keep_here(float &v) { asm volatile("" : "+v"(v)); }

// Result tiles 2 kt and 2 kt + 1 of an operand, one at a time.
__device__ __forceinline__ void set_half(bf16x8 &to, int half, f32x4 &v) {
  const uint32_t a = pack2(v[0], v[1]), b = pack2(v[2], v[3]);
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 w = __builtin_bit_cast(u32x4, to);
  w[2 * half] = a;
  w[2 * half + 1] = b;
  to = __builtin_bit_cast(bf16x8, w);
  v -= f32x4{__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u),
             __uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)};
}
__device__ __forceinline__ void set_half(Split &to, int half, f32x4 v) {
  set_half(to.hi, half, v);  // (leaves the rest in v)
  set_half(to.lo, half, v);
}

// A head's value channels are taken 32 at a time (64 past 128 state channels), twice:
// first for the pair matrices, which are sums over all of them, then with the states, 32
// state channels at a time. (32 let two workgroups share a compute unit: 71 KB of LDS and
// 256 registers up to 128 state channels; 64 leave one. Past 128 there is one anyway.)
template <int NK>
__global__ __launch_bounds__(256, (NK <= 4 ? 2 : 1)) void k_delta_grad(DeltaArgs a) {
  constexpr int PK = NK <= 4 ? 1 : 2;
  constexpr int N = 32 * NK, P = 32 * PK, C = kDeltaChunk;
  __shared__ bf16 sK[C * N], sQ[C * N], sY[C * P], sU[2][P * C], sR[2][P * C];
  __shared__ bf16 sA0[2][P * 32], sB0[2][P * 32], sA1[2][P * 32], sB1[2][P * 32];  // S, dS
  __shared__ float sG[C], sE[C], sBt[C], sZ[C], sP[C], sS[4];
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int unit = xcd_unit();
  const int part = unit % a.hparts;
  unit /= a.hparts;
  const int grp = unit % a.G, slot = unit / a.G;
  int64_t start;
  int len;
  if (!delta_chunk(a, slot, start, len)) return;
  const int per = (a.hpg + a.hparts - 1) / a.hparts;
  const int h0 = grp * a.hpg + part * per, h1 = min(h0 + per, (grp + 1) * a.hpg);
  const size_t ldk = (size_t)a.G * a.N, ldx = (size_t)a.H * a.P;
  const int own = 16 * w + lr;              // this lane's token
  const bool live = own < len;
  const size_t tok = (size_t)(start + min(own, len - 1));

  f32x4 dQ[NK][2], dK[NK][2];
#pragma unroll
  for (int nb = 0; nb < NK; ++nb)
#pragma unroll
    for (int par = 0; par < 2; ++par) dQ[nb][par] = dK[nb][par] = kZero4;
  stage_tile<N, C, 4>(sK, (const bf16 *)a.B + ((size_t)start * a.G + grp) * a.N, ldk, a.N, len);
  stage_tile<N, C, 4>(sQ, (const bf16 *)a.C + ((size_t)start * a.G + grp) * a.N, ldk, a.N, len);

  for (int h = h0; h < h1; ++h) {
    const size_t sh = (size_t)slot * a.H + h;
    // dY, U and dR of value channels pb to pb + P - 1
    const auto fetch_rows = [&](int pb) __attribute__((always_inline)) {
      const int pn = min(P, a.P - pb);
      stage_tile<P, C, 4, true>(sY, (const bf16 *)a.dy + ((size_t)start * a.H + h) * a.P + pb, ldx, pn, len);
      const bf16 *u = (const bf16 *)a.u + (sh * a.P + pb) * C;
      const bf16 *dr = (const bf16 *)a.dr + (sh * a.P + pb) * C;
      bf16 *const to[4] = {sU[0], sU[1], sR[0], sR[1]};
      const bf16 *const from[4] = {u, u + a.u_rest, dr, dr + a.u_rest};
      stage_tiles<C, P, 4, true>(to, from, C, C, pn);
    };
    // and their state channels 32 nb to 32 nb + 31
    const auto fetch_states = [&](int pb, int nb, bf16 (*A)[P * 32],
                                  bf16 (*B)[P * 32]) __attribute__((always_inline)) {
      const int n = max(min(32, a.N - 32 * nb), 0), pn = min(P, a.P - pb);
      const bf16 *s0 = (const bf16 *)a.st0 + (sh * a.P + pb) * a.N + 32 * nb;
      const bf16 *s1 = (const bf16 *)a.st1 + (sh * a.P + pb) * a.N + 32 * nb;
      bf16 *const to[4] = {A[0], A[1], B[0], B[1]};
      const bf16 *const from[4] = {s0, s0 + a.st_rest, s1, s1 + a.st_rest};
      stage_tiles<32, P, 4, true>(to, from, a.N, n, pn);
    };
    float rv = 0.f, pairs = 0.f, betas = 0.f;  // for dbeta; row sums less column sums; for dbeta
    float zq = 0.f, zk = 0.f, zu = 0.f, ss = 0.f;
    float bi, gi, ei, gc, ef, lf, be;
    const int last = (a.P - 1) / P * P;
    // dM and -dL (without masks and decays): column i = own with rows j of tiles up to this
    // wave's, and column j = own with rows i of later ones; and of this wave's (dmw, dlw)
    f32x4 dm[4], dl[4], dmw = kZero4, dlw = kZero4;
#pragma unroll
    for (int t = 0; t < 4; ++t) dm[t] = dl[t] = kZero4;
    for (int pb = 0; pb < a.P; pb += P) {
      if (h > h0 || pb > 0) __syncthreads();
      fetch_rows(pb);
      if (pb == last) fetch_states(pb, 0, sA0, sB0);
      if (w == 0 && pb == 0) {
        const size_t ga = (size_t)(start + min(lane, len - 1)) * a.H + h;
        const DecaySum gam = decay_sums(
            lane < len ? delta_log2_decay((float)((const bf16 *)a.g)[ga]) : 0.f);
        sG[lane] = gam.hi;
        sE[lane] = gam.lo;
        sBt[lane] = lane < len ? (float)((const bf16 *)a.beta)[ga] : 0.f;
      }
      wait_vmem_all();
      __syncthreads();
      const Places<N, P> at;
      bi = sBt[own];
      // this token's rows of dY, dR, U (what is staged past the end and past P is zeros)
      bf16x8 yo[PK];
      Split ro[PK], uo[PK];
#pragma unroll
      for (int ps = 0; ps < PK; ++ps) {
        yo[ps] = at.values(sY, w, ps);
        ro[ps] = at.tokens(sR, ps, w);
        uo[ps] = at.tokens(sU, ps, w);
        if (32 * ps + 8 * lg >= a.P - pb || !live) continue;
        const size_t xa = (tok * a.H + h) * a.P + pb + 32 * ps + 8 * lg;
        rv += dot8(ro[ps], ldg8((const bf16 *)a.x + xa));
        f32x4 p, q;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = bi * ((float)ro[ps].hi[e] + (float)ro[ps].lo[e]);
          q[e] = bi * ((float)ro[ps].hi[4 + e] + (float)ro[ps].lo[4 + e]);
        }
        *reinterpret_cast<bf16x8 *>((bf16 *)a.dx + xa) = pack8(p, q);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ps = 0; ps < PK; ++ps) {
          if (t <= w) {
            const Split u = at.tokens(sU, ps, t);
            dm[t] = mfma(u, yo[ps], dm[t]);
            dl[t] = mfma(u, ro[ps], dl[t]);
          } else {
            dm[t] = mfma(at.values(sY, t, ps), uo[ps], dm[t]);
            dl[t] = mfma(at.tokens(sR, ps, t), uo[ps], dl[t]);
          }
        }
      }
#pragma unroll
      for (int ps = 0; ps < PK; ++ps) {
        dmw = mfma(yo[ps], uo[ps], dmw);
        dlw = mfma(ro[ps], uo[ps], dlw);
      }
    }
    gi = sG[own], ei = sE[own], gc = sG[C - 1];
    ef = exp2_fast(gi), lf = exp2_fast((gc - gi) + (sE[C - 1] - ei)), be = bi * ef;
    // the pair matrices, and what they add to dQ and dK
    {
      // (as operands of two tiles: rows j of pairs up to this wave's, rows i of a pair
      // behind it, and rows i of this wave's in mw, lw)
      const Split none = {zero8(), zero8()};
      Split mo[2] = {none, none}, lo[2] = {none, none}, mw = none, lw = none;
      const Places<N, P> at;
      {
        bf16x8 ko[NK], qo[NK];
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) {
          ko[ks] = at.keys(sK, w, ks);
          qo[ks] = at.keys(sQ, w, ks);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          __builtin_amdgcn_sched_barrier(0);
          const f32x4 gt = ldf4(sG + 16 * t + 4 * lg), et = ldf4(sE + 16 * t + 4 * lg);
          if (t <= w) {                        // rows j of tile t, column i = own
            f32x4 kk = kZero4, qk = kZero4, m, l;
#pragma unroll
            for (int ks = 0; ks < NK; ++ks) {
              const bf16x8 k = at.keys(sK, t, ks);
              kk = mfma(k, ko[ks], kk);
              qk = mfma(k, qo[ks], qk);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int d = own - (16 * t + 4 * lg + r);
              const float e = d >= 0 ? exp2_fast((gi - gt[r]) + (ei - et[r])) : 0.f;
              m[r] = d >= 0 ? dm[t][r] * e : 0.f;
              const float lk = d > 0 ? -dl[t][r] * e : 0.f;
              l[r] = bi * lk;
              betas += lk * kk[r];
              pairs += m[r] * qk[r] + l[r] * kk[r];
            }
            keep_here(betas), keep_here(pairs);
            set_half(mo[t >> 1], t & 1, m);
            set_half(lo[t >> 1], t & 1, l);
          }
          if (t >= w) {                        // rows i of tile t, column j = own
            f32x4 kk = kZero4, qk = kZero4, m, l;
#pragma unroll
            for (int ks = 0; ks < NK; ++ks) {
              kk = mfma(at.keys(sK, t, ks), ko[ks], kk);
              qk = mfma(at.keys(sQ, t, ks), ko[ks], qk);
            }
            const f32x4 bt = ldf4(sBt + 16 * t + 4 * lg);
            const f32x4 dmt = t == w ? dmw : dm[t], dlt = t == w ? dlw : dl[t];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int i = 16 * t + 4 * lg + r, d = i - own;
              const bool in = d >= 0 && i < len;
              const float e = in ? exp2_fast((gt[r] - gi) + (et[r] - ei)) : 0.f;
              m[r] = in ? dmt[r] * e : 0.f;
              l[r] = in && d > 0 ? -bt[r] * dlt[r] * e : 0.f;
              pairs -= m[r] * qk[r] + l[r] * kk[r];
            }
            keep_here(pairs);
            if (t / 2 == w / 2) {
              set_half(mw, t & 1, m);
              set_half(lw, t & 1, l);
            } else {
              set_half(mo[t >> 1], t & 1, m);
              set_half(lo[t >> 1], t & 1, l);
            }
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < NK; ++nb)
#pragma unroll
        for (int par = 0; par < 2; ++par) {
          __builtin_amdgcn_sched_barrier(0);
          const int n0 = 32 * nb + 16 * par;
          f32x4 q = dQ[nb][par], k = dK[nb][par];
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            const bf16x8 kT = at.columns(sK, kt, n0);
            k = mfma(kT, lo[kt], k);
            if (kt <= w / 2)                   // tokens up to this wave's
              q = mfma(kT, mo[kt], q);
            else                               // and behind them
              k = mfma(at.columns(sQ, kt, n0), mo[kt], k);
            if (kt == w / 2) {
              k = mfma(kT, lw, k);
              k = mfma(at.columns(sQ, kt, n0), mw, k);
            }
          }
          dQ[nb][par] = q;
          dK[nb][par] = k;
        }
    }
    // the states, from the value channels taken last to the first; the next block under way
    for (int pb = last; pb >= 0; pb -= P) {
      bf16x8 yo[PK];
      Split ro[PK], uo[PK];
      {
        const Places<N, P> at;
#pragma unroll
        for (int ps = 0; ps < PK; ++ps) {
          yo[ps] = at.values(sY, w, ps);
          ro[ps] = at.tokens(sR, ps, w);
          uo[ps] = at.tokens(sU, ps, w);
        }
      }
      const auto block = [&](int nb, const bf16 (*A)[P * 32],
                             const bf16 (*B)[P * 32]) __attribute__((always_inline)) {
        const Places<N, P> at;
#pragma unroll
        for (int par = 0; par < 2; ++par) {
          __builtin_amdgcn_sched_barrier(0);
          f32x4 ys = kZero4, rs = kZero4, us = kZero4;
#pragma unroll
          for (int ps = 0; ps < PK; ++ps) {
            const Split s0 = at.state(A, ps, par), s1 = at.state(B, ps, par);
            ys = mfma(s0, yo[ps], ys);
            rs = mfma(s0, ro[ps], rs);
            us = mfma(s1, uo[ps], us);
            if (((2 * nb + par) & 3) == w) ss += dot8(s0, s1);
          }
          __builtin_amdgcn_sched_barrier(0);
          const int o = (at.own4 ^ (32 * nb + 16 * par)) + 16 * w * N;
          const bf16x4 k4 = *reinterpret_cast<const bf16x4 *>(sK + o);
          const bf16x4 q4 = *reinterpret_cast<const bf16x4 *>(sQ + o);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            zq += (float)q4[r] * ys[r];
            zk += (float)k4[r] * rs[r];
            zu += (float)k4[r] * us[r];
          }
          keep_here(zq), keep_here(zk), keep_here(zu), keep_here(ss);
          dQ[nb][par] += ef * ys;
          dK[nb][par] += lf * us - be * rs;
        }
      };
#pragma unroll
      for (int nb = 0; nb < NK; ++nb) {
        if (nb + 1 < NK) {
          if (nb & 1)
            fetch_states(pb, nb + 1, sA0, sB0);
          else
            fetch_states(pb, nb + 1, sA1, sB1);
        } else if (pb > 0) {
          fetch_states(pb - P, 0, sA0, sB0);
        }
        if (nb == 1 && pb > 0) fetch_rows(pb - P);  // (all waves have this pass's)
        if (nb & 1)
          block(nb, sA1, sB1);
        else
          block(nb, sA0, sB0);
        if (nb + 1 < NK || pb > 0) {
          wait_vmem_all();
          __syncthreads();
        }
      }
    }
    // dbeta and dg
    rv = sum_lg(rv);
    betas = sum_lg(betas);
    pairs = sum_lg(pairs);
    zq = sum_lg(zq);
    zk = sum_lg(zk);
    zu = sum_lg(zu);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) ss += __shfl_xor(ss, o);
    if (lg == 0) {
      sZ[own] = live ? ef * zq - be * zk + pairs : 0.f;
      sP[own] = lf * zu;
      if (live) ((bf16 *)a.dbeta)[tok * a.H + h] = (bf16)(rv + betas - ef * zk);
    }
    if (lane == 0) sS[w] = ss;
    __syncthreads();
    if (w == 0) {
      const float z = sZ[lane], p = sP[lane];
      const float upto = wave_inclusive_sum(z), all = __shfl(upto, 63);
      const float before = wave_inclusive_sum(p) - p;
      const float ends = exp2_fast(gc) * (sS[0] + sS[1] + sS[2] + sS[3]);
      if (lane < len)
        ((bf16 *)a.dg)[(size_t)(start + lane) * a.H + h] = (bf16)(all - (upto - z) + before + ends);
    }
  }
  if (!live) return;
#pragma unroll
  for (int nb = 0; nb < NK; ++nb)
#pragma unroll
    for (int par = 0; par < 2; ++par) {
      const int n = 32 * nb + 16 * par + 4 * lg;
      if (n >= a.N) continue;
      const f32x4 k = dK[nb][par], q = dQ[nb][par];
      if (a.hparts == 1) {
        const size_t at = (tok * a.G + grp) * a.N + n;
        *reinterpret_cast<uint2 *>((bf16 *)a.dB + at) = make_uint2(pack2(k[0], k[1]), pack2(k[2], k[3]));
        *reinterpret_cast<uint2 *>((bf16 *)a.dC + at) = make_uint2(pack2(q[0], q[1]), pack2(q[2], q[3]));
      } else {
        const size_t at = ((tok * a.G + grp) * a.hparts + part) * a.N + n;
        stf4(a.part + at, k);
        stf4(a.part + (size_t)a.T * a.G * a.hparts * a.N + at, q);
      }
    }
}

template <int NK>
hipError_t grad(const DeltaArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.nslots * a.G * a.hparts)), block(256);
  hipLaunchKernelGGL(k_delta_grad<NK>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

int delta_grad_parts(const DeltaArgs &a) {
  // workgroups for the card before a workgroup takes more heads of a group
  int64_t parts = a.nslots ? 1024 / ((int64_t)a.nslots * a.G) : 1;
  parts = parts < 1 ? 1 : parts > a.hpg ? a.hpg : parts;
  const int per = (int)((a.hpg + parts - 1) / parts);
  return (a.hpg + per - 1) / per;
}

hipError_t launch_delta_grad(const DeltaArgs &a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  const hipError_t e = a.N <= 64 ? grad<2>(a, s) : a.N <= 128 ? grad<4>(a, s) : grad<8>(a, s);
  if (e != hipSuccess || a.hparts == 1) return e;
  return launch_delta_heads_sum(a, true, s);
}

}  // namespace ssd
