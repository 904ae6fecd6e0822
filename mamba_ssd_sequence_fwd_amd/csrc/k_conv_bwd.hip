// k_conv_bwd.hip -- the convolution front backwards: gradients of the packed
// input, the taps, the bias and the history from those of x, B and C.
//
// Per channel of a sequence of L tokens, e = [K - 1 history rows, inputs] and
// pre_t = bias + sum_k w_k e_{t+k} as in the forward pass:
//   g_t  = dout_t silu'(pre_t)
//   de_j = sum_k w_k g_{j-k}     (0 <= j - k < L; + dhistory_out_{j-L}, j >= L)
//   dw_k = sum_t g_t e_{t+k},   dbias = sum_t g_t
// de_j for j < K - 1 is the history's gradient, the rest the inputs'.
//
// Each lane owns 8 channels and walks one tile of tokens of one sequence,
// with the last K - 1 inputs and the last K - 1 values of g in registers: at
// step t it computes g_t, adds to dw and dbias and emits de_t. A tile runs
// K - 1 steps past its end (the next tokens' g, or zeros after the last
// token), and its first K - 1 emissions belong to the tile before it, or to
// the history at a sequence's start. Tiles never cross a sequence: tile slot
// j belongs to the last sequence s with first(s) <= j, where first(s) =
// cu[s] / tile + s leaves every sequence enough slots (at least one) without
// a table; slots past a sequence's end only write zeros to the partial sums.
// The sums of a workgroup's tiles are joined in LDS and written as one row of
// partial sums; k_column_sums adds those rows.
#include "conv.h"

namespace ssd {

namespace {

template <typename T, bool CK> struct BwdRowOf { typedef Row8<T> type; };
template <typename T> struct BwdRowOf<T, true> { typedef RowQ8 type; };

template <typename T>
__device__ __forceinline__ void load_u(Row8<T> &r, const ConvBwdArgs &a, int t, int c0) {
  r.load(a.xbc, (size_t)t * a.in_stride + c0);
}
__device__ __forceinline__ void load_u(RowQ8 &r, const ConvBwdArgs &a, int t, int c0) {
  r.load(a.ck, (size_t)t, a.ch, c0);
}

template <int K, typename T, bool CK>
__global__ __launch_bounds__(64 * kConvBwdWaves) void k_conv_backward(ConvBwdArgs a, int cblocks) {
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
  // one contiguous range of workgroups per XCD: tiles that share halo rows
  // meet in one L2
  const int nb = gridDim.x, bid = blockIdx.x;
  const int xq = nb >> 3, xr = nb & 7, xcd = bid & 7;
  const int lb = xcd * xq + min(xcd, xr) + (bid >> 3);
  const int tb = lb / cblocks;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cg = ((lb - tb * cblocks) * 64 + lane) * 8;
  const bool live = cg < a.ch;
  const int c0 = live ? cg : a.ch - 8;
  const int slot = tb * kConvBwdWaves + wave;

  // The tile [t0, t1) of sequence s = [ss, se); len < 0: nothing to do.
  int s = 0, ss = 0, se = 0, t0 = 0, t1 = 0;
  bool some = slot < a.tiles;
  if (some) {
    int first;
    if (a.cu) {
      int lo = 0, hi = a.nseq - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu[mid] / a.tile + mid <= slot) lo = mid; else hi = mid - 1;
      }
      s = lo;
      ss = a.cu[s];
      se = a.cu[s + 1];
      first = ss / a.tile + s;
      // offsets that are no partition of the tokens must not lead outside them
      if (ss < 0 || se < ss || se > a.T || slot < first) some = false;
    } else {
      s = slot / a.seq_tiles;
      ss = s * a.seqlen;
      se = ss + a.seqlen;
      first = s * a.seq_tiles;
    }
    if (some) {
      const int64_t lt = (int64_t)(slot - first) * a.tile;
      some = lt == 0 || lt < se - ss;
      t0 = ss + (int)(some ? lt : 0);
      t1 = min(t0 + a.tile, se);
    }
  }

  float dw[8][K], db[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    db[c] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[c][k] = 0.f;
  }

  if (some && se > ss) {
    // Array and column of this lane's output gradients.
    const void *src;
    int dcol, dstride;
    if (c0 < a.x_dim) {
      src = a.dx; dcol = c0; dstride = a.x_dim;
    } else if (c0 < a.x_dim + a.bc_dim) {
      src = a.dB; dcol = c0 - a.x_dim; dstride = a.bc_dim;
    } else {
      src = a.dC; dcol = c0 - a.x_dim - a.bc_dim; dstride = a.bc_dim;
    }
    typename BwdRowOf<T, CK>::type u[kBatch], un[kBatch];
    Row8<T> d[kBatch], dn[kBatch];
    const int steps = t1 - t0 + K - 1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int t = min(t0 + j, se - 1);
      load_u(u[j], a, t, c0);
      d[j].load(src, (size_t)t * dstride + dcol);
    }
    float w[8][K], bias[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[c][k] = a.w[(size_t)(c0 + c) * K + k];
      bias[c] = a.bias ? a.bias[c0 + c] : 0.f;
    }
    float win[K - 1][8], gwin[K - 1][8];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int tok = t0 - (K - 1) + j;
#pragma unroll
      for (int c = 0; c < 8; ++c) win[j][c] = gwin[j][c] = 0.f;
      if (tok >= ss) {
        typename BwdRowOf<T, CK>::type r;
        load_u(r, a, tok, c0);
        r.widen(win[j]);
      } else if (a.hist_in) {
        Row8<T> r;
        r.load(a.hist_in, ((size_t)s * (K - 1) + (tok - ss + K - 1)) * a.ch + c0);
        r.widen(win[j]);
      }
    }
    for (int i0 = 0; i0 < steps; i0 += kBatch) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int t = min(t0 + i0 + kBatch + j, se - 1);
        load_u(un[j], a, t, c0);
        dn[j].load(src, (size_t)t * dstride + dcol);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int t = t0 + i0 + j;
        if (i0 + j < steps) {
          float cur[8], dd[8], g[8], de[8];
          u[j].widen(cur);
          d[j].widen(dd);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float pre = bias[c] + w[c][K - 1] * cur[c];
#pragma unroll
            for (int k = 0; k < K - 1; ++k) pre += w[c][k] * win[k][c];
            const float sg = sigmoid(pre);
            g[c] = t < se ? dd[c] * (sg * (1.f + pre * (1.f - sg))) : 0.f;
            de[c] = w[c][0] * g[c];
#pragma unroll
            for (int k = 1; k < K; ++k) de[c] += w[c][k] * gwin[K - 1 - k][c];
          }
          if (t < t1) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              db[c] += g[c];
              dw[c][K - 1] += g[c] * cur[c];
#pragma unroll
              for (int k = 0; k < K - 1; ++k) dw[c][k] += g[c] * win[k][c];
            }
          }
          // de belongs to row t - ss of [history, inputs]
          if (a.dhist_out && t >= se) {
            Row8<T> r;
            float v[8];
            r.load(a.dhist_out, ((size_t)s * (K - 1) + (t - se)) * a.ch + c0);
            r.widen(v);
#pragma unroll
            for (int c = 0; c < 8; ++c) de[c] += v[c];
          }
          if (t - ss >= K - 1) {
            if (live && i0 + j >= K - 1)
              Row8<T>::store(a.dxbc, (size_t)(t - (K - 1)) * a.out_stride + c0, de);
          } else if (live && a.dhist) {
            Row8<T>::store(a.dhist, ((size_t)s * (K - 1) + (t - ss)) * a.ch + c0, de);
          }
#pragma unroll
          for (int k = 0; k + 1 < K - 1; ++k)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              win[k][c] = win[k + 1][c];
              gwin[k][c] = gwin[k + 1][c];
            }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            win[K - 2][c] = cur[c];
            gwin[K - 2][c] = g[c];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        u[j] = un[j];
        d[j] = dn[j];
      }
    }
  } else if (some && a.dhist && live) {
    // no tokens: the history passes through
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const size_t at = ((size_t)s * (K - 1) + j) * a.ch + c0;
      if (a.dhist_out) {
        Row8<T> r;
        r.load(a.dhist_out, at);
        r.widen(v);
      }
      Row8<T>::store(a.dhist, at, v);
    }
  }

  // Join the tiles of the workgroup.
  __shared__ float lds[kConvBwdWaves - 1][K + 1][8][64];
  if (wave > 0) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
#pragma unroll
      for (int k = 0; k < K; ++k) lds[wave - 1][k][c][lane] = dw[c][k];
      lds[wave - 1][K][c][lane] = db[c];
    }
  }
  __syncthreads();
  if (wave == 0 && live) {
#pragma unroll
    for (int k = 0; k <= K; ++k) {
      float *p = a.part + ((size_t)tb * (K + 1) + k) * a.ch + c0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float v = k < K ? dw[c][k < K ? k : 0] : db[c];
#pragma unroll
        for (int o = 0; o < kConvBwdWaves - 1; ++o) v += lds[o][k][c][lane];
        p[c] = v;
      }
    }
  }
}

template <int K, typename T>
hipError_t launch_width(const ConvBwdArgs &a, hipStream_t s) {
  const int cblocks = (a.ch / 8 + 63) / 64;
  const int tblocks = (a.tiles + kConvBwdWaves - 1) / kConvBwdWaves;
  const dim3 grid((unsigned)(cblocks * tblocks)), block(64 * kConvBwdWaves);
  if (a.ck.q)
    hipLaunchKernelGGL((k_conv_backward<K, T, true>), grid, block, 0, s, a, cblocks);
  else
    hipLaunchKernelGGL((k_conv_backward<K, T, false>), grid, block, 0, s, a, cblocks);
  return hipGetLastError();
}

}  // namespace

int conv_bwd_geometry(ConvBwdArgs &a) {
  a.tile = 61;  // with the K - 1 = 3 steps past the end, 64 steps
  if (a.cu) {
    a.seq_tiles = 0;
    a.tiles = a.T / a.tile + a.nseq;
  } else {
    a.seq_tiles = a.seqlen > 0 ? (a.seqlen + a.tile - 1) / a.tile : 1;
    a.tiles = a.nseq * a.seq_tiles;
  }
  return (a.tiles + kConvBwdWaves - 1) / kConvBwdWaves;
}

hipError_t launch_conv_backward(const ConvBwdArgs &a, int width, bool bf16_io, hipStream_t s) {
  if (a.tiles == 0) return hipSuccess;
  switch (width) {
    case 2: return bf16_io ? launch_width<2, bf16>(a, s) : launch_width<2, float>(a, s);
    case 3: return bf16_io ? launch_width<3, bf16>(a, s) : launch_width<3, float>(a, s);
    case 4: return bf16_io ? launch_width<4, bf16>(a, s) : launch_width<4, float>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
