// bcnorm.h -- device-side view of one norm-and-rotation call on B and C and its
// launchers. Not part of the public ABI.
#pragma once

#include "norm.h"

namespace ssd {

struct BcNormArgs {
  // side 0 is B, side 1 is C
  const void *in[2];          // rows at in_stride, heads[side] x N each
  const void *dout[2];        // backward: rows at out_stride
  void *out[2];               // forward: rows at out_stride; backward: dx rows at dx_stride
  const float *w[2];          // (N) or null (ones)
  float *part;                // backward: (blocks, 2, N) partial sums of dw, or null
  const int32_t *pos;         // (period) or null (no rotation)
  const float *freqs;         // (rot / 2)
  int64_t in_stride[2], out_stride[2], dx_stride[2];  // elements
  int32_t heads[2];
  int32_t tokens, N, rot, period;
  int32_t interleaved;
  int32_t parts;              // teams that share a token's heads
  float inv_n, eps;           // inv_n = 1 / N, or 1 (unit)
};

// Workgroups (rows of partial sums) of the backward pass; sets parts.
int bc_norm_geometry(BcNormArgs &a, bool backward);
hipError_t launch_bc_norm(const BcNormArgs &a, bool backward, int blocks, bool bf16_io,
                          float *dw0, float *dw1, hipStream_t s);

}  // namespace ssd
