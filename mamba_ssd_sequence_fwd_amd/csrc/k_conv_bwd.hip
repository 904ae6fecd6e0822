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
// Each lane owns 4 channels and walks one tile of tokens of one sequence,
// with the last K - 1 inputs and the last K - 1 values of g in registers: at
// step t it computes g_t, adds to dw and dbias and emits de_t. A tile runs
// K - 1 steps past its end (the next tokens' g, or zeros after the last
// token), and its first K - 1 emissions belong to the tile before it, or to
// the history at a sequence's start. Tiles never cross a sequence (TileMap);
// slots without tokens only write zeros to the partial sums. The sums of a
// workgroup's tiles are joined in LDS and written as one row of partial sums;
// k_column_sums adds those rows.
//
// The taps, their sums, the bias's and the two windows are 16 K - 4 registers a
// lane for 4 channels, which leaves 4 waves a SIMD (8 channels: 2). Steps
// inside a tile run without a branch, kBatch rows in flight, each loaded into
// the registers that the row kBatch before it leaves. Some 26 vector
// instructions an element, two of them at a quarter of the rate, are 80 us at
// 8 x 2048 tokens of 5376 channels, against 85 us of memory from a checkpoint
// at a copy's 5.2 TB/s: both bound it. Measured, K = 4, bf16, caches cold:
// that size from 8 bits 99 to 103 us for 443 MB; 124,399 packed tokens of 5376
// channels 749 to 778 us for 4.01 GB (5.2 to 5.4 TB/s, a copy's rate).
// Three of four tiles taking the g of their last K - 1 steps from the next wave
// through LDS read 5% less and took as long; 8 waves a workgroup halve the
// partial sums and took 2% off that size, 15% onto 8192 tokens from 8 bits.
#include <type_traits>

#include "conv.h"

namespace ssd {

namespace {

constexpr int kLane = 4;  // channels per lane

template <typename T> using Row = Row4<T>;
template <typename T, bool CK> using BwdRow = std::conditional_t<CK, RowQ4, Row<T>>;

template <typename T>
__device__ __forceinline__ void load_u(Row<T> &r, const ConvBwdArgs &a, int t, int c0) {
  r.load(a.xbc, (size_t)t * a.in_stride + c0);
}
template <typename T>
__device__ __forceinline__ void load_u(RowQ4 &r, const ConvBwdArgs &a, int t, int c0) {
  r.load(a.ck, (size_t)t, a.ch, c0);
}

template <int K, typename T, bool CK>
__global__ __launch_bounds__(64 * kConvBwdWaves)
__attribute__((amdgpu_waves_per_eu(4))) void k_conv_backward(ConvBwdArgs a, int cblocks) {
  constexpr int P = K - 1;
  // rows in flight per lane, a multiple of P so that the windows come round to
  // the same registers
  constexpr int kBatch = P == 3 ? 3 : sizeof(T) == 2 ? 4 : 2;
  static_assert(kBatch >= P && kBatch % P == 0, "a first batch covers the steps before the tile's own");
  const int tb = blockIdx.x / cblocks;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cg = ((blockIdx.x - tb * cblocks) * 64 + lane) * kLane;
  const bool live = cg < a.ch;
  const int c0 = live ? cg : a.ch - kLane;
  const int slot = tb * kConvBwdWaves + wave;

  Tile tile{};
  const bool some = tile_of(a.map, slot, tile);
  const int s = tile.s, ss = tile.ss, se = tile.se, t0 = tile.t0, t1 = tile.t1;

  float dw[kLane][K], db[kLane];
#pragma unroll
  for (int c = 0; c < kLane; ++c) {
    db[c] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[c][k] = 0.f;
  }

  if (some && se > ss) {
    // Array and column of this lane's output gradients.
    const char *dsrc;
    int dstride;
    {
      const void *src;
      int dcol;
      if (c0 < a.x_dim) {
        src = a.dx; dcol = c0; dstride = a.x_dim;
      } else if (c0 < a.x_dim + a.bc_dim) {
        src = a.dB; dcol = c0 - a.x_dim; dstride = a.bc_dim;
      } else {
        src = a.dC; dcol = c0 - a.x_dim - a.bc_dim; dstride = a.bc_dim;
      }
      dsrc = static_cast<const char *>(src) + (size_t)dcol * sizeof(T);
      dstride *= (int)sizeof(T);
    }
    BwdRow<T, CK> u[kBatch];
    Row<T> d[kBatch];
    // row t of the inputs and of the gradients, into the registers that the
    // row kBatch before it left (past the walk's last row that one again)
    const int end = t1 + P, last = min(end, se) - 1;
    auto fetch = [&](int j, int t) __attribute__((always_inline)) {
      t = min(t, last);
      load_u<T>(u[j], a, t, c0);
      d[j].load(dsrc + (size_t)t * dstride, 0);
    };
#pragma unroll
    for (int j = 0; j < kBatch; ++j) fetch(j, t0 + j);
    float w[kLane][K], bias[kLane];
#pragma unroll
    for (int c = 0; c < kLane; ++c) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[c][k] = a.w[(size_t)(c0 + c) * K + k];
      bias[c] = a.bias ? a.bias[c0 + c] : 0.f;
    }
    float win[P][kLane], gwin[P][kLane];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int tok = t0 - P + j;
#pragma unroll
      for (int c = 0; c < kLane; ++c) win[j][c] = gwin[j][c] = 0.f;
      if (tok >= ss) {
        BwdRow<T, CK> r;
        load_u<T>(r, a, tok, c0);
        r.widen(win[j]);
      } else if (a.hist_in) {
        Row<T> r;
        r.load(a.hist_in, ((size_t)s * P + (tok - ss + P)) * a.ch + c0);
        r.widen(win[j]);
      }
    }
    // One step; inside: a token of the tile whose de is one of its tokens'.
    auto step = [&](auto inside_, int j, int t) __attribute__((always_inline)) {
      constexpr bool inside = decltype(inside_)::value;
      float cur[kLane], dd[kLane], de[kLane];
      u[j].widen(cur);
      d[j].widen(dd);
      fetch(j, t + kBatch);
#pragma unroll
      for (int c = 0; c < kLane; ++c) {
        float pre = bias[c] + w[c][K - 1] * cur[c];
#pragma unroll
        for (int k = 0; k < P; ++k) pre += w[c][k] * win[k][c];
        // g = d s (1 + pre (1 - s))
        const float sg = sigmoid(pre), ds = dd[c] * sg;
        float g = ds + ds * (pre - pre * sg);
        if (!inside) g = t < se ? g : 0.f;
        de[c] = w[c][0] * g;
#pragma unroll
        for (int k = 1; k < K; ++k) de[c] += w[c][k] * gwin[K - 1 - k][c];
        if (inside || t < t1) {
          db[c] += g;
          dw[c][K - 1] += g * cur[c];
#pragma unroll
          for (int k = 0; k < P; ++k) dw[c][k] += g * win[k][c];
        }
#pragma unroll
        for (int k = 0; k + 1 < P; ++k) {
          win[k][c] = win[k + 1][c];
          gwin[k][c] = gwin[k + 1][c];
        }
        win[P - 1][c] = cur[c];
        gwin[P - 1][c] = g;
      }
      // de belongs to row t - ss of [history, inputs]; lanes past the last
      // channel repeat the last lane's stores
      if (inside) {
        Row<T>::store(a.dxbc, (size_t)(t - P) * a.out_stride + c0, de);
      } else {
        if (a.dhist_out && t >= se) {
          Row<T> r;
          float v[kLane];
          r.load(a.dhist_out, ((size_t)s * P + (t - se)) * a.ch + c0);
          r.widen(v);
#pragma unroll
          for (int c = 0; c < kLane; ++c) de[c] += v[c];
        }
        if (t - ss >= P) {
          if (t - t0 >= P)
            Row<T>::store(a.dxbc, (size_t)(t - P) * a.out_stride + c0, de);
        } else if (a.dhist) {
          Row<T>::store(a.dhist, ((size_t)s * P + (t - ss)) * a.ch + c0, de);
        }
      }
    };
    auto checked = [&](int t) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (t + j < end) step(std::false_type(), j, t + j);
    };
    int t = t0;
    checked(t);
    t += kBatch;
    for (; t + kBatch <= t1; t += kBatch) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) step(std::true_type(), j, t + j);
    }
    for (; t < end; t += kBatch) checked(t);
  } else if (some && a.dhist) {
    // no tokens: the history passes through
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      float v[kLane] = {};
      const size_t at = ((size_t)s * (K - 1) + j) * a.ch + c0;
      if (a.dhist_out) {
        Row<T> r;
        r.load(a.dhist_out, at);
        r.widen(v);
      }
      Row<T>::store(a.dhist, at, v);
    }
  }

  // Join the tiles of the workgroup.
  __shared__ float lds[kConvBwdWaves - 1][K + 1][kLane][64];
  if (wave > 0) {
#pragma unroll
    for (int c = 0; c < kLane; ++c) {
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
      for (int c = 0; c < kLane; ++c) {
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
  const int cblocks = conv_bwd_channel_blocks(a);
  const int tblocks = (a.map.slots + kConvBwdWaves - 1) / kConvBwdWaves;
  const dim3 grid((unsigned)(cblocks * tblocks)), block(64 * kConvBwdWaves);
  if (a.ck.q)
    hipLaunchKernelGGL((k_conv_backward<K, T, true>), grid, block, 0, s, a, cblocks);
  else
    hipLaunchKernelGGL((k_conv_backward<K, T, false>), grid, block, 0, s, a, cblocks);
  return hipGetLastError();
}

// Tokens per tile. Shorter tiles spread the work more evenly, longer ones
// repeat fewer steps at their ends: from a checkpoint the kernel is bound by
// its arithmetic (2 x 16384 tokens, 8192 channels: 288 us with 60 tokens, 298
// with 36), from 16 bits by memory (124,399 packed tokens, 5376 channels: 786
// us with 36, 809 with 60). Few tokens take the shortest, so that there are
// workgroups for every compute unit (5376 channels, bf16 and 8 bits, caches
// warm: 1024 tokens 15 us with 12, 18 and 24 us with the longer; 2048 tokens, 315
// workgroups of 36, 21 and 22 against 24 and 26; 4096 tokens, 609, 37 and 35
// against 32 and 36; 8192 tokens 64 and 60 against 54 and 49).
constexpr int kTile = 36, kCkptTile = 60, kShortTile = 12;
constexpr int kFewBlocks = 480;

}  // namespace

int conv_bwd_channel_blocks(const ConvBwdArgs &a) { return (a.ch / kLane + 63) / 64; }

int conv_bwd_geometry(ConvBwdArgs &a) {
  const int64_t blocks = (tile_slots(a.map, kTile) + kConvBwdWaves - 1) / kConvBwdWaves;
  set_tile(a.map, blocks * conv_bwd_channel_blocks(a) < kFewBlocks ? kShortTile
                  : a.ck.q                                         ? kCkptTile
                                                                   : kTile);
  return (a.map.slots + kConvBwdWaves - 1) / kConvBwdWaves;
}

hipError_t launch_conv_backward(const ConvBwdArgs &a, int width, bool bf16_io, hipStream_t s) {
  if (a.map.slots == 0) return hipSuccess;
  switch (width) {
    case 2: return bf16_io ? launch_width<2, bf16>(a, s) : launch_width<2, float>(a, s);
    case 3: return bf16_io ? launch_width<3, bf16>(a, s) : launch_width<3, float>(a, s);
    case 4: return bf16_io ? launch_width<4, bf16>(a, s) : launch_width<4, float>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
