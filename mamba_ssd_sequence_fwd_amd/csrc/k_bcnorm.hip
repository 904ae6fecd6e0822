// k_bcnorm.hip -- B and C (the recurrences' keys and queries) normalised per
// head and rotated by their positions in one pass, and that pass backwards.
//
// Per token and head, with n = N (or 1 for unit length) and w the side's weight:
//   h = x r,  r = 1 / sqrt(sum x^2 / n + eps),  v = h w
//   out = v with its first `rot` channels turned in pairs (u, v) by
//         angle = position * freq:  (u cos - v sin, u sin + v cos)
// backwards: dv = dout turned back, dw = sum over tokens and heads of dv h,
//   dh = dv w,  dx = r (dh - h sum(dh h) / n).
//
// HBM is the bound (two or three accesses an element). A team of N / 8 lanes
// (rounded up to a power of two) holds a head's row, each lane two groups of 4
// channels: where pairs lie half a rotation apart, the groups c and c + rot / 2,
// so both members of every pair meet in one lane; else 8 channels in a row.
// The angles of a lane's four pairs are the same for all heads of a token, so
// a team walks several heads with one set of sines. They come from the product
// in 64 bits, in turns: a far position keeps its fraction (an fp32 product at
// position 10^6 is off by up to 0.06 rad).
//
// A lone row's way is its memory's latency, so a team has four heads (backwards two)
// on their way at a time. Measured (MI355X), bf16, 32 heads of 128: 16384 tokens 51
// us, 5.3 TB/s (96 us head by head; 68 us with pieces of 8 bytes where 16 do), 16
// tokens 5 us; backwards, 40 heads of 128, all turned, 16384 tokens: 96 us, 5.2 TB/s
// (127 us head by head), and 5 us for the weights' column sums.
#include "bcnorm.h"
#include "rows.h"

namespace ssd {
namespace {

// Four channels as they lie in memory, and their values: the rows of several
// heads are on their way before the first is used.
__device__ __forceinline__ f32x4_t fetch4(const float *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const f32x4_t *>(p));
}
__device__ __forceinline__ u32x2_t fetch4(const bf16 *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x2_t *>(p));
}
__device__ __forceinline__ void values4(f32x4_t q, float *v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = q[k];
}
__device__ __forceinline__ void values4(u32x2_t q, float *v) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    v[2 * k] = __uint_as_float(q[k] << 16);
    v[2 * k + 1] = __uint_as_float(q[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ f32x4_t packed4(const float *, const float *v) {
  return f32x4_t{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ u32x2_t packed4(const bf16 *, const float *v) {
  return u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}
// A lane's eight channels: two fours from c0 and c1, or in bf16 one access where
// they lie in a row for all lanes (`joined`; 68 us for 16384 tokens without it).
template <typename Four>
__device__ __forceinline__ void fetch8(const bf16 *p, int c0, int c1, bool joined, Four *q) {
  if (joined) {
    const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(p + c0));
    q[0] = u32x2_t{v[0], v[1]};
    q[1] = u32x2_t{v[2], v[3]};
  } else {
    q[0] = fetch4(p + c0);
    q[1] = fetch4(p + c1);
  }
}
template <typename Four>
__device__ __forceinline__ void fetch8(const float *p, int c0, int c1, bool, Four *q) {
  q[0] = fetch4(p + c0);
  q[1] = fetch4(p + c1);
}
__device__ __forceinline__ void store8(bf16 *p, int c0, int c1, bool joined, const float *v) {
  const u32x2_t a = packed4(p, v), b = packed4(p, v + 4);
  if (joined) {
    const u32x4_t q = {a[0], a[1], b[0], b[1]};
    __builtin_nontemporal_store(q, reinterpret_cast<u32x4_t *>(p + c0));
  } else {
    __builtin_nontemporal_store(a, reinterpret_cast<u32x2_t *>(p + c0));
    __builtin_nontemporal_store(b, reinterpret_cast<u32x2_t *>(p + c1));
  }
}
__device__ __forceinline__ void store8(float *p, int c0, int c1, bool, const float *v) {
  __builtin_nontemporal_store(packed4(p, v), reinterpret_cast<f32x4_t *>(p + c0));
  __builtin_nontemporal_store(packed4(p, v + 4), reinterpret_cast<f32x4_t *>(p + c1));
}

template <int Ctrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(
                 __builtin_amdgcn_update_dpp(0, __float_as_int(v), Ctrl, 0xf, 0xf, true));
}

// Sum over a team of lanes, in every lane: within quads, then the other quad
// of eight and the other half of a row by mirrors (their lanes agree by then).
template <int TEAM>
__device__ __forceinline__ float team_sum(float v) {
  v = dpp_add<0xb1>(v);                        // quad_perm [1,0,3,2]
  if (TEAM >= 4) v = dpp_add<0x4e>(v);         // quad_perm [2,3,0,1]
  if (TEAM >= 8) v = dpp_add<0x141>(v);        // row_half_mirror
  if (TEAM >= 16) v = dpp_add<0x140>(v);       // row_mirror
  if (TEAM >= 32) v += __shfl_xor(v, 16);
  return v;
}

// Four pairs of a lane's channels v[0..7] turned by (c, s).
__device__ __forceinline__ void turn2(float &x, float &y, float c, float s) {
  const float u = x * c - y * s;
  y = x * s + y * c;
  x = u;
}
__device__ __forceinline__ void turn(float (&v)[8], const float (&c)[4], const float (&s)[4],
                                     bool side_by_side) {
  // (the layout is the same for all lanes: a branch, no selects)
  if (side_by_side) {
#pragma unroll
    for (int p = 0; p < 4; ++p) turn2(v[2 * p], v[2 * p + 1], c[p], s[p]);
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p) turn2(v[p], v[p + 4], c[p], s[p]);
  }
}

template <typename T, int TEAM, bool kBackward>
__global__ __launch_bounds__(256) void k_bc_norm(BcNormArgs a) {
  constexpr int kTeams = 256 / TEAM, kBatch = kBackward ? 2 : 4;  // heads under way
  const int j = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const bool on = 8 * j < a.N;
  const bool rotated = a.pos && 8 * j < a.rot;
  // the lane's two groups of channels
  const bool apart = rotated && !a.interleaved;
  const int c0 = !on ? 0 : apart ? 4 * j : 8 * j;
  const int c1 = !on ? 0 : apart ? 4 * j + a.rot / 2 : 8 * j + 4;
  const bool joined = !a.pos || a.interleaved;
  float w[2][8], dw[2][8];
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w[side][k] = a.w[side] ? a.w[side][(k < 4 ? c0 : c1) + (k & 3)] : 1.f;
      dw[side][k] = 0.f;
    }
  double f[4] = {0.0, 0.0, 0.0, 0.0};
  if (rotated)
#pragma unroll
    for (int p = 0; p < 4; ++p)
      f[p] = (double)a.freqs[4 * j + p] * 0.15915494309189533577;  // turns a position
  const int64_t units = (int64_t)a.tokens * a.parts;
  for (int64_t u = (int64_t)blockIdx.x * kTeams + team; u < units;
       u += (int64_t)gridDim.x * kTeams) {
    const int64_t t = a.parts == 1 ? u : u / a.parts;
    const int part = (int)(u - t * a.parts);
    float cs[4], sn[4];
    if (a.pos) {
      const double p = rotated ? (double)a.pos[t % a.period] : 0.0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const double turns = p * f[q];
        sincospif(2.f * (float)(turns - rint(turns)), &sn[q], &cs[q]);
        if (kBackward) sn[q] = -sn[q];
      }
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      // (the sides' heads in a row, every parts-th of them from the part's own)
      const int heads = a.heads[side];
      int h = side ? part - a.heads[0] % a.parts : part;
      if (h < 0) h += a.parts;
      const T *x = (const T *)a.in[side] + t * a.in_stride[side];
      const T *g = kBackward ? (const T *)a.dout[side] + t * a.out_stride[side] : nullptr;
      T *o = kBackward ? (T *)a.out[side] + t * a.dx_stride[side]
                       : (T *)a.out[side] + t * a.out_stride[side];
      for (; h < heads; h += kBatch * a.parts) {
        decltype(fetch4((const T *)nullptr)) raw[kBatch][kBackward ? 4 : 2];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int64_t at = (int64_t)min(h + b * a.parts, heads - 1) * a.N;
          fetch8(x + at, c0, c1, joined, raw[b]);
          if (kBackward) fetch8(g + at, c0, c1, joined, raw[b] + 2);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (h + b * a.parts >= heads) break;
          const int64_t at = (int64_t)(h + b * a.parts) * a.N;
          float v[8], d[8];
          values4(raw[b][0], v);
          values4(raw[b][1], v + 4);
          float ss = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) ss += v[k] * v[k];
          ss = team_sum<TEAM>(on ? ss : 0.f);
          const float r = rsqrtf(ss * a.inv_n + a.eps);
          if (!kBackward) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= r * w[side][k];
            if (rotated) turn(v, cs, sn, a.interleaved);
            if (on) store8(o + at, c0, c1, joined, v);
          } else {
            values4(raw[b][2], d);
            values4(raw[b][3], d + 4);
            if (rotated) turn(d, cs, sn, a.interleaved);
            float dot = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              v[k] *= r;
              dw[side][k] += d[k] * v[k];
              d[k] *= w[side][k];
              dot += d[k] * v[k];
            }
            dot = team_sum<TEAM>(on ? dot : 0.f) * a.inv_n;
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = r * (d[k] - v[k] * dot);
            if (on) store8(o + at, c0, c1, joined, d);
          }
        }
      }
    }
  }
  if (kBackward && a.part) {
    __shared__ float lds[kTeams][8 * TEAM];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
      if (on)
#pragma unroll
        for (int k = 0; k < 8; ++k) lds[team][(k < 4 ? c0 : c1) + (k & 3)] = dw[side][k];
      __syncthreads();
      for (int c = threadIdx.x; c < a.N; c += 256) {
        float s = 0.f;
        for (int k = 0; k < kTeams; ++k) s += lds[k][c];
        a.part[((int64_t)blockIdx.x * 2 + side) * a.N + c] = s;
      }
    }
  }
}

int team_of(int N) {
  int t = 2;
  while (8 * t < N) t *= 2;
  return t;
}

template <typename T, int TEAM>
hipError_t bc_norm_team(const BcNormArgs &a, bool backward, int blocks, hipStream_t s) {
  if (backward)
    hipLaunchKernelGGL((k_bc_norm<T, TEAM, true>), dim3(blocks), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_bc_norm<T, TEAM, false>), dim3(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t bc_norm_t(const BcNormArgs &a, bool backward, int blocks, hipStream_t s) {
  switch (team_of(a.N)) {
    case 2: return bc_norm_team<T, 2>(a, backward, blocks, s);
    case 4: return bc_norm_team<T, 4>(a, backward, blocks, s);
    case 8: return bc_norm_team<T, 8>(a, backward, blocks, s);
    case 16: return bc_norm_team<T, 16>(a, backward, blocks, s);
    default: return bc_norm_team<T, 32>(a, backward, blocks, s);
  }
}

}  // namespace

int bc_norm_geometry(BcNormArgs &a, bool backward) {
  const int all = a.heads[0] + a.heads[1], teams = 256 / team_of(a.N);
  // teams for 2048 workgroups before a team takes several heads of a token
  const int64_t want = (int64_t)2048 * teams;
  const int64_t parts = a.tokens ? want / a.tokens : 1;
  a.parts = (int)(parts < 1 ? 1 : parts > all ? all : parts);
  const int64_t blocks = ((int64_t)a.tokens * a.parts + teams - 1) / teams;
  const int64_t most = backward ? 1024 : 2048;
  return (int)(blocks < most ? blocks : most);
}

hipError_t launch_bc_norm(const BcNormArgs &a, bool backward, int blocks, bool bf16_io, float *dw0,
                          float *dw1, hipStream_t s) {
  if (blocks > 0) {
    const hipError_t e = bf16_io ? bc_norm_t<bf16>(a, backward, blocks, s)
                                 : bc_norm_t<float>(a, backward, blocks, s);
    if (e != hipSuccess) return e;
  }
  if (!backward || (!dw0 && !dw1)) return hipSuccess;
  return launch_column_sums(a.part, blocks, 2, 1, a.N, dw0, dw1, s);
}

}  // namespace ssd
