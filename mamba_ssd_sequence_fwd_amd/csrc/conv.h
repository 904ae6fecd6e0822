// conv.h -- device-side view of one ssd_conv1d_silu call (the convolution
// front that produces x, B and C) and its launcher. Not part of the public ABI.
#pragma once

#include "rows.h"

namespace ssd {

struct ConvArgs {
  const void *xbc;       // (T, in_stride) dtype; the channels are [0, ch) of each row
  const float *w;        // (ch, K) taps, tap K-1 on the current token
  const float *bias;     // (ch) or null
  const void *hist_in;   // (nseq, K-1, ch) dtype or null (zeros)
  const int32_t *cu;     // (nseq + 1) packed offsets, or null (dense rows of seqlen)
  void *x;               // (T, x_dim) dtype
  void *B;               // (T, bc_dim) dtype
  void *C;               // (T, bc_dim) dtype
  void *hist_out;        // (nseq, K-1, ch) dtype or null
  int32_t T;             // tokens
  int32_t seqlen;        // dense: tokens per sequence
  int32_t nseq;          // sequences (dense: batch rows)
  int32_t ch, x_dim, bc_dim;
  int32_t in_stride;     // elements between token rows of xbc
  int32_t groups;        // ch / 8: channel groups, one per lane
  int32_t tiles;         // token tiles of kConvTile tokens
};

constexpr int kConvTile = 16;      // tokens per lane
constexpr int kConvThreads = 256;  // threads per workgroup

hipError_t launch_conv(const ConvArgs &a, int width, bool bf16_io, hipStream_t s);

// Tiles of tokens that never cross a sequence: the tokens of tile slot j are
// the (j - first(s))-th `tile` tokens of the last sequence s with first(s) <=
// j. Dense rows have seq_tiles slots each. Packed sequences have first(s) =
// cu[s] / tile + s, which leaves each of them enough slots (one at least)
// without a table. Slots past a sequence's end hold nothing.
struct TileMap {
  const int32_t *cu;   // (nseq + 1) packed offsets, or null (dense rows of seqlen)
  int32_t T, seqlen, nseq;
  int32_t tile;        // tokens per tile
  int32_t seq_tiles;   // dense: slots per sequence
  int32_t slots;
};

inline int64_t tile_slots(const TileMap &m, int tile) {
  return m.cu ? (int64_t)m.T / tile + m.nseq
              : (int64_t)m.nseq * (m.seqlen > 0 ? (m.seqlen + tile - 1) / tile : 1);
}
inline void set_tile(TileMap &m, int tile) {
  m.tile = tile;
  m.seq_tiles = m.cu ? 0 : m.seqlen > 0 ? (m.seqlen + tile - 1) / tile : 1;
  m.slots = (int32_t)tile_slots(m, tile);
}

// A slot's tokens [t0, t1) of sequence s = [ss, se); false if it holds
// nothing (a sequence without tokens has one slot, with t0 == t1). Offsets
// that are no partition of the tokens never lead outside them.
struct Tile { int s, ss, se, t0, t1; };
__device__ __forceinline__ bool tile_of(const TileMap &m, int slot, Tile &k) {
  if (slot >= m.slots) return false;
  int first;
  if (m.cu) {
    int lo = 0, hi = m.nseq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (m.cu[mid] / m.tile + mid <= slot) lo = mid; else hi = mid - 1;
    }
    k.s = lo;
    k.ss = m.cu[k.s];
    k.se = m.cu[k.s + 1];
    first = k.ss / m.tile + k.s;
    if (k.ss < 0 || k.se < k.ss || k.se > m.T || slot < first) return false;
  } else {
    k.s = slot / m.seq_tiles;
    k.ss = k.s * m.seqlen;
    k.se = k.ss + m.seqlen;
    first = k.s * m.seq_tiles;
  }
  const int64_t at = (int64_t)(slot - first) * m.tile;
  if (at != 0 && at >= k.se - k.ss) return false;
  k.t0 = k.ss + (int)at;
  k.t1 = min(k.t0 + m.tile, k.se);
  return true;
}

// ssd_conv1d_silu with an 8-bit checkpoint of its input, written (a.xbc given)
// or read in its place (a.xbc null). Fills in the tiles itself.
hipError_t launch_conv_ckpt(const ConvArgs &a, const Ckpt &ck, int width, bool bf16_io,
                            hipStream_t s);

// Device-side view of one ssd_conv1d_silu_backward call.
struct ConvBwdArgs {
  const void *xbc;        // (T, in_stride) dtype, or null (ck is read)
  const float *w;         // (ch, K)
  const float *bias;      // (ch) or null
  const void *hist_in;    // (nseq, K-1, ch) dtype or null (zeros)
  const void *dx, *dB, *dC;   // gradients of the outputs, dtype
  const void *dhist_out;  // (nseq, K-1, ch) dtype or null (zeros)
  void *dxbc;             // (T, out_stride) dtype
  void *dhist;            // (nseq, K-1, ch) dtype or null (not wanted)
  float *part;            // (tile blocks, K + 1, ch) partial sums of dw and dbias
  Ckpt ck;                // 8-bit checkpoint of xbc, or null
  TileMap map;            // one tile per wave
  int32_t ch, x_dim, bc_dim;
  int32_t in_stride, out_stride;
};
constexpr int kConvBwdWaves = 4;   // tiles per workgroup

// Choose the tiles of a problem whose sizes are set; the workgroups along the
// tokens.
int conv_bwd_geometry(ConvBwdArgs &a);
int conv_bwd_channel_blocks(const ConvBwdArgs &a);  // workgroups along the channels
hipError_t launch_conv_backward(const ConvBwdArgs &a, int width, bool bf16_io, hipStream_t s);

}  // namespace ssd
