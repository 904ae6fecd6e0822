// norm.h -- device-side view of one group-norm call (forward or backward) and
// its launchers, and the sum over partial rows that the backward kernels of
// the layer's surroundings share. Not part of the public ABI.
#pragma once

#include "rows.h"

namespace ssd {

enum NormMode : int {
  kGateFirst = 0,  // out = norm(x silu(z)) w + b
  kGateLast = 1,   // out = (norm(x) w + b) silu(z)
  kNoGate = 2      // out = silu(norm(x) w + b)
};

struct NormArgs {
  const void *x;      // rows at x_stride (null where xk is read)
  const void *z;      // rows at z_stride, or null
  const float *w;     // (C) or null (ones)
  const float *b;     // (C) or null (zeros)
  void *out;          // forward: rows at out_stride
  const void *dout;   // backward: rows at out_stride
  void *dx, *dz;      // backward: rows at dx_stride, dz_stride
  float *part;        // backward: (nparts, 1 or 2, C) partial sums of dw (and db), or null
  Ckpt xk, zk;        // forward: written; backward: read
  int64_t x_stride, z_stride, out_stride, dx_stride, dz_stride;  // elements
  int32_t rows, C, G, gs;
  int32_t center;     // subtract the group's mean
  int32_t team;       // lanes per group (a power of two up to 64), or threads per workgroup
  int32_t subs;       // rows a workgroup takes side by side (in-wave teams)
  int32_t nparts;     // backward: rows of partial sums
  int32_t sum_b;      // backward: db is wanted
  int32_t bf16_io;    // tensors are bf16, else fp32
  float eps, inv_n;   // inv_n = 1 / gs
};

constexpr int kNormMaxGroup = 16384;  // channels of a group the kernels hold on chip
// Rows of partial sums of the backward pass (one per workgroup along the rows).
int norm_partial_rows(const NormArgs &a);
hipError_t launch_norm(const NormArgs &a, NormMode mode, bool bf16_io, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs &a, NormMode mode, bool bf16_io, hipStream_t s);

// Column sums of part (n, rows, ch): column (k, c) goes to dw[c * taps + k] for
// k < taps and to db[c] for k = taps (a null array is not written).
hipError_t launch_column_sums(const float *part, int n, int rows, int taps, int ch, float *dw,
                              float *db, hipStream_t s);

// Whole-tensor checkpoints: rows of T at `stride` to and from a checkpoint.
hipError_t launch_ckpt_save(const void *src, int64_t stride, int64_t rows, int channels,
                            bool bf16_io, const Ckpt &k, hipStream_t s);
hipError_t launch_ckpt_load(const Ckpt &k, int64_t rows, int channels, bool bf16_io, void *dst,
                            int64_t stride, hipStream_t s);

}  // namespace ssd
