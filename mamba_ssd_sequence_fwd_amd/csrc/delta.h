// delta.h -- device-side view of one gated-delta-rule call and its launchers
// (forward, backward and one-token step). Not part of the public ABI.
//
// Per sequence and head, with state h (P x N), key B, query C, value x:
//   h_t = e^{g_t} h_{t-1} (I - beta_t B_t B_t^T) + beta_t x_t B_t^T,  y_t = h_t C_t
// By chunks of c tokens, with S = h^T (N x P) entering the chunk, gam the
// prefix sums of g inside it and K, Q, V, Y its rows of B, C, x, y:
//   L[i][j] = beta_i (K_i . K_j) e^{gam_i - gam_j}  (i > j),  T = (I + L)^-1
//   M[i][j] = (Q_i . K_j) e^{gam_i - gam_j}         (i >= j)
//   R = beta (V - e^gam K S),   U = T R
//   Y = e^gam Q S + M U,        S <- e^{gam_c} S + K^T (e^{gam_c - gam} U)
// (U_i is what token i writes to the state: the product over the tokens'
// rank-1 updates, unrolled, is the triangular system (I + L) U = R.)
#pragma once

#include "ssd_internal.h"

namespace ssd {

constexpr int kDeltaChunk = 64;

struct DeltaArgs {
  const void *x;       // (T, H, P)
  const void *g;       // (T, H)  log decay
  const void *beta;    // (T, H)
  const void *B, *C;   // (T, G, N)
  const float *h0;     // (S, H, P, N) or null
  const int32_t *cu;   // (nseq + 1) device, packed only
  void *y;             // (T, H, P)
  float *hT;           // (S, H, P, N) or null
  // backward
  const void *dy;      // (T, H, P)
  const float *dhT;    // (S, H, P, N) or null
  void *dx, *dg, *dbeta, *dB, *dC;
  float *dh0;          // (S, H, P, N) or null
  // workspace, per (chunk slot, head)
  void *tri;           // triangular matrices, tri_bytes each
  void *st0, *st1;     // backward: S and dL/dS at the chunk's start and end
  void *u, *dr;        // backward: U and dL/dR, (64, P)
  float *part;         // backward: per-head dK, dQ of fp32 calls, (2, T, H, N)
  int64_t T;           // tokens
  int32_t L, H, P, N, G, hpg;
  int32_t nseq, nc_per, nslots;
};

// Triangular matrices of a (slot, head): what the chunks' own products need.
enum DeltaTri : int {
  kTriForward = 0,   // T, M
  kTriBackward = 1   // T, T^T, M^T
};

// The log decay in base 2, at least -150: 2^-150 is 0 in fp32, so a decay of
// e^-inf resets the state and no difference of two sums is inf - inf.
__device__ __forceinline__ float delta_log2_decay(float g) {
  return fmaxf(g * 1.4426950408889634f, -150.f);
}

// Tokens [lo, hi) of sequence s, within the stream whatever cu holds.
__device__ __forceinline__ void delta_seq(const DeltaArgs &a, int s, int64_t &lo, int64_t &hi) {
  if (!a.cu) {
    lo = (int64_t)s * a.L;
    hi = lo + a.L;
    return;
  }
  lo = min(max((int64_t)a.cu[s], (int64_t)0), a.T);
  hi = min(max((int64_t)a.cu[s + 1], lo), a.T);
}

// First chunk slot of sequence s that starts at token lo. Packed: lo / 64 + s
// leaves every sequence room for its chunks without a table (a sequence of n
// tokens has at most (lo + n) / 64 - lo / 64 + 1 of them).
__device__ __forceinline__ int delta_slot0(const DeltaArgs &a, int s, int64_t lo) {
  return a.cu ? (int)(lo / kDeltaChunk) + s : s * a.nc_per;
}

// First token and length of the chunk in a slot; false if the slot has none.
__device__ __forceinline__ bool delta_chunk(const DeltaArgs &a, int slot, int64_t &start,
                                            int &len) {
  int s;
  if (!a.cu) {
    s = slot / a.nc_per;
  } else {
    int l = 0, r = a.nseq - 1;  // the last sequence whose first slot is not past this one
    while (l < r) {
      const int m = (l + r + 1) / 2;
      const int64_t lo = min(max((int64_t)a.cu[m], (int64_t)0), a.T);
      if (delta_slot0(a, m, lo) <= slot) l = m; else r = m - 1;
    }
    s = l;
  }
  int64_t lo, hi;
  delta_seq(a, s, lo, hi);
  const int64_t at = (int64_t)(slot - delta_slot0(a, s, lo)) * kDeltaChunk;
  if (at < 0 || at >= hi - lo) return false;
  start = lo + at;
  len = (int)min((int64_t)kDeltaChunk, hi - start);
  return true;
}

// Bytes of one (slot, head)'s triangular matrices.
size_t delta_tri_bytes(bool bf16_path, DeltaTri which);

hipError_t launch_delta_prep(const DeltaArgs &a, bool bf16_io, DeltaTri which, hipStream_t s);
hipError_t launch_delta_chain_f32(const DeltaArgs &a, bool bf16_io, bool states, hipStream_t s);
hipError_t launch_delta_reverse_f32(const DeltaArgs &a, bool bf16_io, hipStream_t s);
hipError_t launch_delta_grad_f32(const DeltaArgs &a, bool bf16_io, hipStream_t s);

struct DeltaStepArgs {
  const void *x, *g, *beta, *B, *C;
  float *state;        // (rows, N), rows = batch * H * P
  void *y;
  int64_t rows;
  int32_t H, N, G, heads_per_group, p_shift;
};
hipError_t launch_delta_step(const DeltaStepArgs &a, bool bf16_io, hipStream_t s);

}  // namespace ssd
