// k_norm.hip -- group norm with SiLU, channels last: what stands between the
// SSD layer's output and the output projection, forward and backward.
//
// Per token and group of n channels, with s(z) = z / (1 + e^-z):
//   u = x s(z) (gate first) or x;  mu = mean(u) if centred, else 0
//   r = 1 / sqrt(mean((u - mu)^2) + eps);  h = (u - mu) r;  v = h w + b
//   out = v (gate first),  v s(z) (gate last)  or  s(v) (no gate)
// and backwards, dv being dout, dout s(z) or dout s'(v):
//   dw += dv h;  db += dv;  g = dv w;  du = r (g - [mean(g)] - h mean(g h))
//   dx = du s(z), dz = du x s'(z) (gate first);  dx = du, dz = dout v s'(z)
//   (gate last);  dx = du (no gate)
//
// A row of a group is read once and held in registers by a team: a power of
// two of lanes inside a wave for groups up to 512 channels (no barrier), one
// workgroup for wider ones. Every lane owns 8 channels (16 bytes of bf16), R
// times, and keeps them over all the rows it walks, so the affine weights are
// loaded once and the gradients of the weights are summed in registers; each
// workgroup writes one row of partial sums. The next row's loads are issued
// before the current row's sums. All sums are fp32, rows side by side in a
// workgroup are joined in fp32 in turn, and the partial rows are added in fp64.
// Squares are summed as they are: |u| above about 1e18 overflows.
//
// Both directions are bound by HBM. Measured, caches cold, bf16, gate first:
// 16384 tokens of one group of 5120 channels forward 86 us for 503 MB (5.8
// TB/s), backward 147 to 155 us for 839 MB (5.4 to 5.7 TB/s); 32768 tokens of 8
// groups of 512 forward 131 us for 805 MB (6.1 TB/s), with both inputs kept in
// 8 bits 190 us for 1082 MB (5.7 TB/s), backward from them 205 to 222 us for
// 1082 MB (4.9 to 5.3 TB/s; 41 vector instructions an element are 140 us of
// it). One token of 5120 channels takes 4.8 us. Furthest from that is the
// backward pass without a gate, which needs the statistics before it has dv and
// so takes one more sum after the others: 8192 tokens of one group of 5120
// channels 90 us in bf16 (252 MB, 2.8 TB/s; vector instructions 42% of the
// waves' time, waits 33%) and 117 us centred, with three sums in turn (34% and
// 46%); in fp32 (503 MB) 116 and 128 us.
#include "norm.h"

namespace ssd {

namespace {

// Where the inputs come from and what is kept of them.
enum : int { kPlain = 0, kCkpt = 1 };

constexpr int kTeamThreads = 256;  // workgroup of the in-wave teams
constexpr int kMaxWaves = 8;

template <int Ctrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(
                 __builtin_amdgcn_update_dpp(0, __float_as_int(v), Ctrl, 0xf, 0xf, true));
}

// Sum over aligned teams of `team` lanes (a power of two up to 64), the same
// bits on every lane: each step adds the two halves in both orders. Inside
// rows of 16 by DPP (quad swaps, then mirrors of values equal per quad or
// half row), across rows by lane exchanges.
__device__ __forceinline__ float team_sum(float v, int team) {
  constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;
  if (team > 1) v = dpp_add<kXor1>(v);
  if (team > 2) v = dpp_add<kXor2>(v);
  if (team > 4) v = dpp_add<kHalfMirror>(v);
  if (team > 8) v = dpp_add<kMirror>(v);
  if (team > 16) v += __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401f));
  if (team > 32) v += __shfl_xor(v, 32);
  return v;
}

// Sums of N values over the team. A workgroup team leaves each wave's sums in
// LDS (two buffers taken in turn, so one barrier suffices) and every thread
// adds the waves' in the same order.
template <bool WIDE, int N>
__device__ __forceinline__ void team_sums(float (&v)[N], int team, float (*lds)[kMaxWaves * 4],
                                          int &turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = team_sum(v[i], WIDE ? 64 : team);
  if (WIDE) {
    const int nw = team >> 6;
    float *buf = lds[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[(threadIdx.x >> 6) * 4 + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < nw; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += buf[w * 4 + i];
  }
}

// The lane's place: its channels for each r and whether they exist. Lanes
// without channels load channel 0's, so that loads need no branch, and store
// nothing; their terms of a sum are replaced, not multiplied, by zero, since
// channel 0 of another group may hold infinities or NaN.
template <bool WIDE, int R>
struct Place {
  int c[R];
  bool live[R];
  int row, step;  // first row, and rows between one of the lane's rows and the next
  __device__ __forceinline__ explicit Place(const NormArgs &a) {
    // in-wave teams of few channels take several rows side by side
    const int need = a.G * a.team;
    const int sub = !WIDE && a.subs > 1 ? threadIdx.x / need : 0;
    row = blockIdx.y * a.subs + sub;
    if (sub >= a.subs) row = a.rows;  // lanes left over
    step = gridDim.y * a.subs;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int g, in;
      if (WIDE) {
        g = blockIdx.x;
        in = (r * a.team + threadIdx.x) * 8;
      } else {
        const int per = blockDim.x / a.team, lane = threadIdx.x - sub * need;
        g = blockIdx.x * per + lane / a.team;
        in = (r * a.team + (lane & (a.team - 1))) * 8;
      }
      live[r] = g < a.G && in < a.gs;
      c[r] = live[r] ? g * a.gs + in : 0;
    }
  }
};

// Weights or biases of the lane's channels (float arrays of any alignment).
template <int R>
__device__ __forceinline__ void load_affine(const float *p, float otherwise, const int (&c)[R],
                                            float (&v)[R][8]) {
  const bool wide = ((uintptr_t)p & 15) == 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (p == nullptr) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[r][k] = otherwise;
    } else if (wide) {
      Row8<float> q;
      q.load(p, c[r]);
      q.widen(v[r]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[r][k] = p[c[r] + k];
    }
  }
}

template <typename T, int MODE, int CK, int R, bool WIDE, int THREADS>
__global__ __launch_bounds__(THREADS) void k_norm(NormArgs a) {
  __shared__ float lds[2][kMaxWaves * 4];
  const Place<WIDE, R> at(a);
  float w[R][8], b[R][8];
  load_affine(a.w, 1.f, at.c, w);
  load_affine(a.b, 0.f, at.c, b);
  constexpr bool kGated = MODE != kNoGate;
  Row8<T> xr[R], zr[R];
  auto fetch = [&](int row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      xr[r].load_once(a.x, (size_t)row * a.x_stride + at.c[r]);
      if (kGated) zr[r].load_once(a.z, (size_t)row * a.z_stride + at.c[r]);
    }
  };
  int turn = 0;
  int row = at.row;
  if (row < a.rows) fetch(row);
  for (; row < a.rows; row += at.step) {
    float x[R][8], z[R][8], u[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      xr[r].widen(x[r]);
      if (kGated) zr[r].widen(z[r]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        u[r][k] = MODE == kGateFirst ? x[r][k] * silu(z[r][k]) : x[r][k];
      }
    }
    if (row + at.step < a.rows) fetch(row + at.step);
    if (CK == kCkpt) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        store_ckpt(a.xk, (size_t)row, a.C, at.c[r], x[r], at.live[r]);
        if (kGated) store_ckpt(a.zk, (size_t)row, a.C, at.c[r], z[r], at.live[r]);
      }
    }
    if (a.center) {
      float m[1] = {0.f};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float part = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) part += u[r][k];
        m[0] += at.live[r] ? part : 0.f;
      }
      team_sums<WIDE>(m, a.team, lds, turn);
      const float mu = m[0] * a.inv_n;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 8; ++k) u[r][k] -= mu;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float part = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) part += u[r][k] * u[r][k];
      q[0] += at.live[r] ? part : 0.f;
    }
    team_sums<WIDE>(q, a.team, lds, turn);
    const float rs = 1.f / sqrtf(q[0] * a.inv_n + a.eps);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = u[r][k] * rs * w[r][k] + b[r][k];
        o[k] = MODE == kGateFirst ? v : MODE == kGateLast ? v * silu(z[r][k]) : silu(v);
      }
      if (at.live[r]) Row8<T>::store(a.out, (size_t)row * a.out_stride + at.c[r], o);
    }
  }
}

template <typename T, int CK> struct NormRowOf { typedef Row8<T> type; };
template <typename T> struct NormRowOf<T, kCkpt> { typedef RowQ8 type; };

template <typename T>
__device__ __forceinline__ void load_row(Row8<T> &r, const void *p, int64_t stride, const Ckpt &,
                                         int, int row, int c) {
  r.load_once(p, (size_t)row * stride + c);
}
__device__ __forceinline__ void load_row(RowQ8 &r, const void *, int64_t, const Ckpt &k, int C,
                                         int row, int c) {
  r.load_once(k, (size_t)row, C, c);
}

// Hide that the raw row still holds what was widened from it: after a barrier
// the fp32 copies are made again (a shift or mask each) instead of held in
// twice the registers.
__device__ __forceinline__ void forget(Row8<bf16> &r) {
  asm volatile("" : "+v"(r.q.x), "+v"(r.q.y), "+v"(r.q.z), "+v"(r.q.w));
}
__device__ __forceinline__ void forget(Row8<float> &) {}
__device__ __forceinline__ void forget(RowQ8 &r) { asm volatile("" : "+v"(r.q.x), "+v"(r.q.y)); }

template <typename T, int MODE, int CK, bool BIAS, int R, bool WIDE, int THREADS>
__global__ __launch_bounds__(THREADS) void k_norm_backward(NormArgs a) {
  __shared__ float lds[2][kMaxWaves * 4];
  const Place<WIDE, R> at(a);
  // With 4 parts a lane there are no registers for a second row, and in fp32
  // or with a bias none for the weights either: those are read again, from
  // L2, for each row. 4096 tokens of 16384 channels, with a bias, from tensors
  // and from 8 bits, against the weights held: fp32 gate first 327 and 244 us
  // (held 427 and 262), gate last 336 and 259 (552 and 481), no gate 241 and 212
  // (236 and 206); bf16 gate first 158 and 145 (152 and 140), gate last 181 and
  // 167 (175 and 173), no gate 167 and 163 (152 and 151). In fp32 with a bias
  // three of these kernels still spill some registers (60 bytes a lane gate
  // first from tensors, 136 gate last, 120 gate last from 8 bits), which the
  // times above include.
  constexpr bool kAhead = R < 4, kRoom = R < 4 || (sizeof(T) == 2 && !BIAS);
  float dw[R][8], db[R][BIAS ? 8 : 1];
  float ws[kRoom ? R : 1][8], bs[kRoom && BIAS ? R : 1][8];
  if constexpr (kRoom) {
    load_affine<R>(a.w, 1.f, at.c, ws);
    if constexpr (BIAS) load_affine<R>(a.b, 0.f, at.c, bs);
  }
  auto weights = [&](int r, float (&w)[8], float (&b)[8]) {
    if constexpr (kRoom) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w[k] = ws[kRoom ? r : 0][k];
        b[k] = BIAS ? bs[kRoom && BIAS ? r : 0][k] : 0.f;
      }
    } else {
      const int c[1] = {at.c[r]};
      float v[1][8];
      load_affine<1>(a.w, 1.f, c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = v[0][k];
      if (BIAS) load_affine<1>(a.b, 0.f, c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = BIAS ? v[0][k] : 0.f;
    }
  };
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      dw[r][k] = 0.f;
      if (BIAS) db[r][BIAS ? k : 0] = 0.f;
    }
  constexpr bool kGated = MODE != kNoGate;
  typedef typename NormRowOf<T, CK>::type In;
  In xr[R], zr[R], xn[R], zn[R];
  Row8<T> dr[R], dn[R];
  auto fetch = [&](int row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      load_row(xn[r], a.x, a.x_stride, a.xk, a.C, row, at.c[r]);
      if (kGated) load_row(zn[r], a.z, a.z_stride, a.zk, a.C, row, at.c[r]);
      dn[r].load_once(a.dout, (size_t)row * a.out_stride + at.c[r]);
    }
  };
  int turn = 0;
  int row = at.row;
  if (kAhead && row < a.rows) fetch(row);
  for (; row < a.rows; row += at.step) {
    if (!kAhead) fetch(row);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      xr[r] = xn[r];
      if (kGated) zr[r] = zn[r];
      dr[r] = dn[r];
    }
    if (kAhead && row + at.step < a.rows) fetch(row + at.step);
    // silu(z) and its derivative are kept over the sums; u and g are made again
    float sz[R][8], dsz[R][8];
    auto widen_u = [&](int r, float (&x)[8], float (&u)[8]) {
      xr[r].widen(x);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = MODE == kGateFirst ? x[k] * sz[r][k] : x[k];
    };
    auto widen_g = [&](int r, float (&d)[8], float (&dv)[8]) {
      dr[r].widen(d);
#pragma unroll
      for (int k = 0; k < 8; ++k) dv[k] = MODE == kGateLast ? d[k] * sz[r][k] : d[k];
    };
    if (kGated) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float z[8];
        zr[r].widen(z);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float s = sigmoid(z[k]);
          sz[r][k] = z[k] * s;
          dsz[r][k] = s + sz[r][k] * (1.f - s);
        }
      }
    }
    float mu = 0.f, mg = 0.f;
    if (a.center) {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x[8], u[8], d[8], dv[8], w[8], b[8];
        widen_u(r, x, u);
        widen_g(r, d, dv);
        weights(r, w, b);
        float p0 = 0.f, p1 = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          p0 += u[k];
          p1 += dv[k] * w[k];
        }
        m[0] += at.live[r] ? p0 : 0.f;
        m[1] += at.live[r] ? p1 : 0.f;
        forget(xr[r]);
        forget(dr[r]);
      }
      team_sums<WIDE>(m, a.team, lds, turn);
      mu = m[0] * a.inv_n;
      if (kGated) mg = m[1] * a.inv_n;
    }
    // with a gate dv does not depend on the statistics, so the sums of
    // (u - mu)^2 and g (u - mu) are one reduction
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x[8], u[8], d[8], dv[8], w[8], b[8];
      widen_u(r, x, u);
      widen_g(r, d, dv);
      if (kGated) weights(r, w, b);
      float p0 = 0.f, p1 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float c = u[k] - mu;
        p0 += c * c;
        if (kGated) p1 += dv[k] * w[k] * c;
      }
      q[0] += at.live[r] ? p0 : 0.f;
      q[1] += at.live[r] ? p1 : 0.f;
      forget(xr[r]);
      forget(dr[r]);
    }
    team_sums<WIDE>(q, a.team, lds, turn);
    const float rs = 1.f / sqrtf(q[0] * a.inv_n + a.eps);
    float mgh = rs * q[1] * a.inv_n;
    if (!kGated) {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x[8], d[8], w[8], b[8];
        xr[r].widen(x);
        dr[r].widen(d);
        weights(r, w, b);
        float p0 = 0.f, p1 = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float h = (x[k] - mu) * rs;
          const float v = h * w[k] + b[k];
          const float s = sigmoid(v);
          const float ds = d[k] * s, dv = ds + ds * (v - v * s);
          sz[r][k] = dv;   // (no gate: the registers hold dv)
          p0 += dv * w[k] * h;
          p1 += dv * w[k];
        }
        m[0] += at.live[r] ? p0 : 0.f;
        m[1] += at.live[r] ? p1 : 0.f;
        forget(xr[r]);
      }
      team_sums<WIDE>(m, a.team, lds, turn);
      mgh = m[0] * a.inv_n;
      mg = a.center ? m[1] * a.inv_n : 0.f;
    }
    // du = r (g - mean(g) - h mean(g h)) with r taken into each term, h = c r
    const float mgr = rs * mg, mghr = rs * rs * mgh;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x[8], u[8], d[8], dv[8], dx[8], dz[8], w[8], b[8];
      widen_u(r, x, u);
      widen_g(r, d, dv);
      weights(r, w, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float c = u[k] - mu;
        const float e = MODE == kNoGate ? sz[r][k] : dv[k];
        const float er = e * rs;
        dw[r][k] += er * c;
        if (BIAS) db[r][BIAS ? k : 0] += e;
        const float du = (er * w[k] - mgr) - c * mghr;
        dx[k] = MODE == kGateFirst ? du * sz[r][k] : du;
        if (MODE == kGateFirst) dz[k] = du * x[k] * dsz[r][k];
        if (MODE == kGateLast) dz[k] = d[k] * (c * rs * w[k] + b[k]) * dsz[r][k];
      }
      if (at.live[r]) {
        Row8<T>::store(a.dx, (size_t)row * a.dx_stride + at.c[r], dx);
        if (kGated) Row8<T>::store(a.dz, (size_t)row * a.dz_stride + at.c[r], dz);
      }
    }
  }
  if (a.part) {
    float *p = a.part + (size_t)blockIdx.y * (BIAS ? 2 : 1) * a.C;
    bool mine = true;
    if constexpr (!WIDE) {
      // rows side by side: joined in the order of the rows
      if (a.subs > 1) {
        __shared__ float join[8][kTeamThreads];
        const int need = a.G * a.team;
        mine = (int)threadIdx.x < need;
        auto joined = [&](float (&v)[8]) {
          __syncthreads();
#pragma unroll
          for (int k = 0; k < 8; ++k) join[k][threadIdx.x] = v[k];
          __syncthreads();
          if (mine)
            for (int i = 1; i < a.subs; ++i)
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] += join[k][threadIdx.x + i * need];
        };
        joined(dw[0]);
        if constexpr (BIAS) joined(db[0]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (mine && at.live[r]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          p[at.c[r] + k] = dw[r][k];
          if (BIAS) p[a.C + at.c[r] + k] = db[r][BIAS ? k : 0];
        }
      }
  }
}

// How the lanes are dealt to the groups. In-wave teams: `size` lanes per
// group. Workgroup teams: `size` threads with R parts of 8 channels each.
struct Team {
  bool wide;
  int r, size, threads, xblocks, subs;
};

// Groups of up to 64 lanes stay inside a wave; up to 512 lanes take a wave per
// 64; wider ones take 4 or 8 waves with 2 to 4 parts a lane. More waves than 8
// a group, or a number that the 4 SIMDs of a compute unit do not share evenly,
// cost more than lanes without channels: 16384 tokens of one group of 5120
// channels (640 lanes) take 97 us forward and 164 us backward with 10 waves of
// one part, 86 us with 4 waves of 3 (forward), 150 us with 8 waves of 2
// (backward).
Team team_of(const NormArgs &a, int r_wide, int threads_wide) {
  Team t{};
  const int lanes = a.gs / 8;
  t.r = 1;
  t.subs = 1;
  if (lanes <= 64) {
    t.size = 1;
    while (t.size < lanes) t.size *= 2;
    const int64_t need = (int64_t)a.G * t.size;
    if (need <= kTeamThreads / 2) {
      // a row takes part of a workgroup: several side by side
      t.threads = kTeamThreads;
      t.subs = (int)(kTeamThreads / need);
      t.xblocks = 1;
    } else {
      // the workgroup size with the fewest lanes left over in the last one
      int64_t best = 0;
      for (int n = kTeamThreads; n >= 64; n -= 64) {
        if (n % t.size) continue;
        const int64_t all = (need + n - 1) / n * n;
        if (!best || all < best) {
          best = all;
          t.threads = n;
        }
      }
      t.xblocks = (int)(best / t.threads);
    }
  } else {
    t.wide = true;
    t.xblocks = a.G;
    if (lanes <= 512) {
      t.threads = (lanes + 63) / 64 * 64;
    } else if (lanes <= r_wide * threads_wide) {
      t.r = r_wide;
      t.threads = threads_wide;
    } else if (lanes <= 1024) {
      t.r = 1024 / threads_wide;
      t.threads = threads_wide;
    } else {
      t.r = 4;
      t.threads = 512;
    }
    t.size = t.threads;
  }
  return t;
}

// Forward: 4 waves of 3 or 4 parts. Backward: 8 waves of 2 parts; from 8-bit
// checkpoints, whose loads are shorter, 4 waves of 3 up to 768 lanes (bf16, gate
// first: 140 us at the shape above against 168 us with 8 waves of 2; 8192 tokens
// of 5632 channels 80 against 84; past 768 lanes 4 waves of 4 lose, 115 us
// against 111 at 8192 x 8192). In fp32 neither wins everywhere: 8192 tokens of
// 5120 channels, without and with a bias, no gate 92 and 108 us with 4 waves of
// 3, 117 and 125 with 8 of 2; gate first 127 and 136 against 132 and 124; gate
// last, whose 4 waves of 3 need so many registers that one wave a SIMD is
// resident, 137 and 151 against 130 and 136 (4104 channels: gated 111 to 142
// against 103 to 123, no gate 87 and 101 against 114 and 121).
Team forward_team(const NormArgs &a) { return team_of(a, 3, 256); }
Team backward_team(const NormArgs &a) {
  const int lanes = a.gs / 8;
  return a.xk.q && lanes <= 768 ? team_of(a, 3, 256) : team_of(a, 2, 512);
}

// Workgroups along the rows: what the card holds at once at `waves` waves per
// compute unit, but no more than `cap`; or where rows are many, so many that
// each lane walks `most` rows. All walk the same number up to one.
int row_blocks(const NormArgs &a, const Team &t, int waves, int cap, int most) {
  constexpr int kUnits = 256;
  int per = waves * 64 / t.threads;
  if (per < 1) per = 1;
  int64_t n = (int64_t)kUnits * per / t.xblocks * t.subs;
  if (n > (int64_t)cap * t.subs) n = (int64_t)cap * t.subs;
  if ((a.rows + (int64_t)most - 1) / most > n) n = (a.rows + (int64_t)most - 1) / most;
  if (n > (int64_t)65535 * t.subs) n = (int64_t)65535 * t.subs;
  if (n < 1) n = 1;
  const int64_t rounds = (a.rows + n - 1) / n;
  n = (a.rows + rounds - 1) / rounds;
  return (int)((n + t.subs - 1) / t.subs);
}

// Forward: in-wave teams run best as many short workgroups (32768 tokens of 8
// groups of 512: 131 us with 3 rows each, 158 us with 32 waves a unit that
// stay), workgroup teams as few that stay (one group of 5120: 86 us with 8
// waves a unit, 92 with 4 rows each; groups of 1024 to 4096: 69 us at 16, 71
// to 72 with 6 rows; in fp32, with twice the bytes a load, 8: 32768 tokens of
// 1024 channels 78 us against 82).
int forward_blocks(const NormArgs &a, const Team &t) {
  if (!t.wide) return row_blocks(a, t, 32, 65535, 3);
  return row_blocks(a, t, t.r == 1 && a.bf16_io ? 16 : 8, 65535, INT32_MAX);
}

// Backward: every workgroup costs a row of partial sums, and more loads in
// flight do not help: 8 waves a unit (16384 tokens of groups of 1024 to 4096:
// 113 to 117 us; 12 waves 119 to 125), from checkpoints of bf16, with half the
// bytes a load, 16 (110 to 111 us; 8 waves 125 to 135; of fp32, whose gradients
// are as wide as ever, 8: 8192 tokens of 8 groups of 512 97 us against 110).
// Lanes of several parts hold twice the loads: 8 (also where the registers leave
// room for 4 only, and the rest wait their turn). No lane adds up more than 256
// rows in fp32 (up to 16 million tokens); where a workgroup takes rows side by
// side, up to 255 more sums are added to a lane's in turn.
int backward_blocks(const NormArgs &a, const Team &t) {
  return row_blocks(a, t, a.xk.q && a.bf16_io && t.r == 1 ? 16 : 8, 2048, 256);
}

template <typename T, int MODE>
hipError_t launch_forward(NormArgs a, hipStream_t s) {
  const Team t = forward_team(a);
  a.team = t.size;
  a.subs = t.subs;
  const dim3 grid(t.xblocks, forward_blocks(a, t)), block(t.threads);
  // fused checkpoints need whole blocks inside a group; others are written by
  // a pass of their own
  const bool fused = a.gs % kCkptBlock == 0;
  if (a.xk.q && !fused) {
    constexpr bool bf = sizeof(T) == 2;
    hipError_t e = launch_ckpt_save(a.x, a.x_stride, a.rows, a.C, bf, a.xk, s);
    if (e == hipSuccess && a.z) e = launch_ckpt_save(a.z, a.z_stride, a.rows, a.C, bf, a.zk, s);
    if (e != hipSuccess) return e;
  }
#define SSD_NORM_K(CK, R, WIDE, THREADS) \
  hipLaunchKernelGGL((k_norm<T, MODE, CK, R, WIDE, THREADS>), grid, block, 0, s, a)
#define SSD_NORM(CK)                       \
  do {                                     \
    if (!t.wide)                           \
      SSD_NORM_K(CK, 1, false, 256);       \
    else if (t.r == 1)                     \
      SSD_NORM_K(CK, 1, true, 512);        \
    else if (t.r == 3)                     \
      SSD_NORM_K(CK, 3, true, 256);        \
    else                                   \
      SSD_NORM_K(CK, 4, true, 512);        \
  } while (0)
  if (a.xk.q && fused)
    SSD_NORM(kCkpt);
  else
    SSD_NORM(kPlain);
#undef SSD_NORM
#undef SSD_NORM_K
  return hipGetLastError();
}

template <typename T, int MODE, int CK, bool BIAS>
hipError_t launch_back(NormArgs a, hipStream_t s) {
  const Team t = backward_team(a);
  a.team = t.size;
  a.subs = t.subs;
  const dim3 grid(t.xblocks, a.nparts), block(t.threads);
#define SSD_NORM(R, WIDE, THREADS) \
  hipLaunchKernelGGL((k_norm_backward<T, MODE, CK, BIAS, R, WIDE, THREADS>), grid, block, 0, s, a)
  if (!t.wide)
    SSD_NORM(1, false, 256);
  else if (t.r == 1)
    SSD_NORM(1, true, 512);
  else if (t.r == 2)
    SSD_NORM(2, true, 512);
  else if (t.r == 4)
    SSD_NORM(4, true, 512);
  else if constexpr (CK == kCkpt)
    SSD_NORM(3, true, 256);
#undef SSD_NORM
  return hipGetLastError();
}

template <typename T, int MODE>
hipError_t launch_back(const NormArgs &a, hipStream_t s) {
  const bool bias = a.b != nullptr || a.sum_b;
  if (a.xk.q)
    return bias ? launch_back<T, MODE, kCkpt, true>(a, s) : launch_back<T, MODE, kCkpt, false>(a, s);
  return bias ? launch_back<T, MODE, kPlain, true>(a, s) : launch_back<T, MODE, kPlain, false>(a, s);
}

}  // namespace

int norm_partial_rows(const NormArgs &a) {
  if (a.rows == 0) return 0;
  const Team t = backward_team(a);
  return backward_blocks(a, t);
}

hipError_t launch_norm(const NormArgs &a, NormMode mode, bool bf16_io, hipStream_t s) {
  switch (mode) {
    case kGateFirst:
      return bf16_io ? launch_forward<bf16, kGateFirst>(a, s) : launch_forward<float, kGateFirst>(a, s);
    case kGateLast:
      return bf16_io ? launch_forward<bf16, kGateLast>(a, s) : launch_forward<float, kGateLast>(a, s);
    default:
      return bf16_io ? launch_forward<bf16, kNoGate>(a, s) : launch_forward<float, kNoGate>(a, s);
  }
}

hipError_t launch_norm_backward(const NormArgs &a, NormMode mode, bool bf16_io, hipStream_t s) {
  switch (mode) {
    case kGateFirst:
      return bf16_io ? launch_back<bf16, kGateFirst>(a, s) : launch_back<float, kGateFirst>(a, s);
    case kGateLast:
      return bf16_io ? launch_back<bf16, kGateLast>(a, s) : launch_back<float, kGateLast>(a, s);
    default:
      return bf16_io ? launch_back<bf16, kNoGate>(a, s) : launch_back<float, kNoGate>(a, s);
  }
}

// ---- column sums of partial rows ------------------------------------------------
// 64 columns per workgroup, 16 slices of the rows, added in fp64.
namespace {
constexpr int kSumSlices = 16;
__global__ __launch_bounds__(1024) void k_column_sums(const float *part, int n, int taps, int ch,
                                                      int64_t cols, float *dw, float *db) {
  __shared__ double lds[kSumSlices][64];
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int64_t j = (int64_t)blockIdx.x * 64 + lane;
  double sum = 0.0;
  if (j < cols) {
#pragma unroll 8
    for (int i = slice; i < n; i += kSumSlices) sum += (double)part[(size_t)i * cols + j];
  }
  lds[slice][lane] = sum;
  __syncthreads();
  if (slice == 0 && j < cols) {
    for (int i = 1; i < kSumSlices; ++i) sum += lds[i][lane];
    const int k = (int)(j / ch), c = (int)(j - (int64_t)k * ch);
    if (k < taps) {
      if (dw) dw[(size_t)c * taps + k] = (float)sum;
    } else if (db) {
      db[c] = (float)sum;
    }
  }
}
}  // namespace

hipError_t launch_column_sums(const float *part, int n, int rows, int taps, int ch, float *dw,
                              float *db, hipStream_t s) {
  const int64_t cols = (int64_t)rows * ch;
  hipLaunchKernelGGL(k_column_sums, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, s, part, n,
                     taps, ch, cols, dw, db);
  return hipGetLastError();
}

}  // namespace ssd
