// k_conv_ckpt.hip -- the convolution front with an 8-bit checkpoint of its
// input: the forward pass that keeps the input on the way, and the
// recomputation of x, B and C from what was kept, for the SSD backward pass.
//
// The mathematics are those of the front (k_conv.hip):
//   pre[t, c] = bias[c] + sum_k w[c, k] u[t - (K - 1) + k, c]
//   out[t, c] = pre / (1 + exp(-pre))
// with the terms of pre added in that kernel's order, so that outputs are equal
// bit for bit, and the checkpoint is that of u (rows.h). Keeping it adds 33
// bytes to write per 32 channels and none to read; from it 33 bytes are read
// instead of 64.
//
// Each lane owns 4 channels and walks one tile of tokens of one sequence
// (TileMap) with the last K - 1 inputs in registers; eight lanes share a block
// of the checkpoint. kBatch token rows are in flight, each loaded into the
// registers that the row kBatch before it leaves, in a loop short enough to
// stay in the instruction cache (4 x 1087 tokens of 1312 channels, kept: 11.7
// us with 8 channels a lane; with the walk unrolled over a tile of 16 tokens 24
// us). With 4 channels instead of 8 the registers hold twice the waves: kept
// 102 -> 90 us at the size below, 1024 tokens 11.8 -> 8.8 us.
//
// Bound by HBM, of which three fifths are writes. Measured at 8 x 2048 tokens
// of 5376 channels, bf16, K = 4: keeping 90 us for 443 MB with cold caches (4.9
// TB/s; the front alone takes 81 us cold for 353 MB) and 73 us with warm ones,
// from 8 bits 48 us warm for 267 MB (5.5 TB/s), where 12 vector instructions an
// element, two of them at a quarter of the rate, take nearly as long as the
// memory.
#include "conv.h"

#include <type_traits>

namespace ssd {

namespace {

constexpr int kConvCkptWaves = 4;  // tiles per workgroup
constexpr int kLane = 4;           // channels per lane

template <typename T>
__device__ __forceinline__ void load_in(Row4<T> &r, const ConvArgs &a, const Ckpt &, int t,
                                        int c0) {
  r.load(a.xbc, (size_t)t * a.in_stride + c0);
}
template <typename T>
__device__ __forceinline__ void load_in(RowQ4 &r, const ConvArgs &a, const Ckpt &ck, int t,
                                        int c0) {
  r.load(ck, (size_t)t, a.ch, c0);
}

// FROM: read the checkpoint in the input's place; else write it.
template <int K, typename T, bool FROM>
__global__ __launch_bounds__(64 * kConvCkptWaves) void k_conv_ckpt(ConvArgs a, Ckpt ck, TileMap map,
                                                               int cblocks) {
  constexpr int P = K - 1;
  // a multiple of P, so that the window comes round to the same registers
  constexpr int kBatch = 6;
  typedef std::conditional_t<FROM, RowQ4, Row4<T>> In;
  const int tb = blockIdx.x / cblocks;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cg = ((blockIdx.x - tb * cblocks) * 64 + lane) * kLane;
  // lanes past the last channel repeat the last lane's, with zeros in the
  // checkpoint's block, of which they store nothing
  const bool live = cg < a.ch;
  const int c0 = live ? cg : a.ch - kLane;
  Tile tile;
  if (!tile_of(map, tb * kConvCkptWaves + wave, tile)) return;
  const int s = tile.s, ss = tile.ss, se = tile.se, t0 = tile.t0, t1 = tile.t1;

  float win[P][kLane];
  if (se > ss) {
    In u[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) load_in<T>(u[j], a, ck, min(t0 + j, t1 - 1), c0);
    // Output array and column of this lane's channels.
    char *dst;
    int dstride;
    {
      void *to;
      int dcol;
      if (c0 < a.x_dim) {
        to = a.x; dcol = c0; dstride = a.x_dim;
      } else if (c0 < a.x_dim + a.bc_dim) {
        to = a.B; dcol = c0 - a.x_dim; dstride = a.bc_dim;
      } else {
        to = a.C; dcol = c0 - a.x_dim - a.bc_dim; dstride = a.bc_dim;
      }
      dst = static_cast<char *>(to) + (size_t)dcol * sizeof(T);
      dstride *= (int)sizeof(T);
    }
    float w[kLane][K], bias[kLane];
#pragma unroll
    for (int c = 0; c < kLane; ++c) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[c][k] = a.w[(size_t)(c0 + c) * K + k];
      bias[c] = a.bias ? a.bias[c0 + c] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int tok = t0 - P + j;
#pragma unroll
      for (int c = 0; c < kLane; ++c) win[j][c] = 0.f;
      if (tok >= ss) {
        In r;
        load_in<T>(r, a, ck, tok, c0);
        r.widen(win[j]);
      } else if (a.hist_in) {
        Row4<T> r;
        r.load(a.hist_in, ((size_t)s * P + (tok - ss + P)) * a.ch + c0);
        r.widen(win[j]);
      }
    }
    auto step = [&](int j, int t) __attribute__((always_inline)) {
      float cur[kLane], out[kLane];
      u[j].widen(cur);
      load_in<T>(u[j], a, ck, min(t + kBatch, t1 - 1), c0);
      if constexpr (!FROM) {
        float v[kLane];
#pragma unroll
        for (int c = 0; c < kLane; ++c) v[c] = live ? cur[c] : 0.f;
        store_ckpt(ck, (size_t)t, a.ch, c0, v, live);
      }
#pragma unroll
      for (int c = 0; c < kLane; ++c) {
        float pre = bias[c] + w[c][K - 1] * cur[c];
#pragma unroll
        for (int k = 0; k < P; ++k) pre += w[c][k] * win[k][c];
        out[c] = silu(pre);
#pragma unroll
        for (int k = 0; k + 1 < P; ++k) win[k][c] = win[k + 1][c];
        win[P - 1][c] = cur[c];
      }
      Row4<T>::store(dst + (size_t)t * dstride, 0, out);
    };
    int t = t0;
    for (; t + kBatch <= t1; t += kBatch) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) step(j, t + j);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (t + j < t1) step(j, t + j);
  } else if (!FROM && a.hist_out) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
#pragma unroll
      for (int c = 0; c < kLane; ++c) win[j][c] = 0.f;
      if (a.hist_in) {
        Row4<T> r;
        r.load(a.hist_in, ((size_t)s * P + j) * a.ch + c0);
        r.widen(win[j]);
      }
    }
  }
  // the last K - 1 inputs of the sequence, oldest first (exact copies)
  if (!FROM && a.hist_out && t1 == se) {
#pragma unroll
    for (int j = 0; j < P; ++j)
      Row4<T>::store(a.hist_out, ((size_t)s * P + j) * a.ch + c0, win[j]);
  }
}

// Tokens per tile: longer ones repeat fewer rows at their ends, shorter ones
// spread the work more evenly (8 x 2048 tokens of 5376 channels, cold, kept: 137
// us with 12 tokens and the read back, 133 with 18, 134 with 24, 137 with 36).
// Few tokens take the short tile, so that there are workgroups for every
// compute unit (5376 channels, kept and from 8 bits, caches warm: 256 tokens 6.5
// and 5.1 us against 7.9 and 5.9 with 18; 1024 tokens 8.8 and 6.5 against 10.6
// and 7.6; 4096 tokens, 1200 workgroups of 18, 23.7 and 15.7 against 22.8 and
// 14.7).
constexpr int kTile = 18, kShortTile = 12;
constexpr int kFewBlocks = 512;

template <int K, typename T>
hipError_t launch_width(const ConvArgs &a, const Ckpt &ck, hipStream_t s) {
  TileMap map{};
  map.cu = a.cu;
  map.T = a.T;
  map.seqlen = a.seqlen;
  map.nseq = a.nseq;
  const int cblocks = (a.ch / kLane + 63) / 64;
  const int64_t blocks =
      (tile_slots(map, kTile) + kConvCkptWaves - 1) / kConvCkptWaves * cblocks;
  set_tile(map, blocks < kFewBlocks ? kShortTile : kTile);
  const int tblocks = (map.slots + kConvCkptWaves - 1) / kConvCkptWaves;
  const dim3 grid((unsigned)(cblocks * tblocks)), block(64 * kConvCkptWaves);
  if (a.xbc)
    hipLaunchKernelGGL((k_conv_ckpt<K, T, false>), grid, block, 0, s, a, ck, map, cblocks);
  else
    hipLaunchKernelGGL((k_conv_ckpt<K, T, true>), grid, block, 0, s, a, ck, map, cblocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_ckpt(const ConvArgs &a, const Ckpt &ck, int width, bool bf16_io,
                            hipStream_t s) {
  switch (width) {
    case 2: return bf16_io ? launch_width<2, bf16>(a, ck, s) : launch_width<2, float>(a, ck, s);
    case 3: return bf16_io ? launch_width<3, bf16>(a, ck, s) : launch_width<3, float>(a, ck, s);
    case 4: return bf16_io ? launch_width<4, bf16>(a, ck, s) : launch_width<4, float>(a, ck, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ssd
