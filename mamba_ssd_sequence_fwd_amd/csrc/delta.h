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
  // backward, on the bf16 path in two bf16 each: all rounded, then what that left
  void *st0, *st1;     // S and dL/dS at the chunk's start and end, (P, N)
  void *u, *dr;        // U and dL/dR, (64, P); on the bf16 path (P, 64), tokens in the
                       // order of the operand tiles
  int32_t *order;      // the sequences by their chunks, longest first, or null (delta_unit)
  float *part;         // backward: dK, dQ of parts of a group's heads, (2, T, G parts, N)
  // workspace, per (segment, head)
  float *span;         // rows (P + N, N): first its own state and then the one at
                       // its start; and the columns of its transition
  float *dspan;        // backward: (P, N), the same for dL/dS at its end
  int64_t T;           // tokens
  int32_t L, H, P, N, G, hpg;
  int32_t nseq, nc_per, nslots;
  int32_t seg, nseg_per, nsegs;  // chunks of a segment (0: whole sequences), segments of a
                       // dense sequence, segment slots
  int32_t hparts;      // backward: parts a group's heads are taken in
  int32_t tri_stride;  // bf16 path: elements of a (slot, head)'s triangular matrices
  int64_t st_rest, u_rest;  // bf16 path: elements from st0 and st1, u and dr to their rests
};

// Triangular matrices of a (slot, head): what the chunks' own products need.
enum DeltaTri : int {
  kTriForward = 0,   // T, and in fp32 M
  kTriBackward = 1   // T, T^T, M^T
};

// The log decay in base 2, at least -150: 2^-150 is 0 in fp32, so a decay of
// e^-inf resets the state and no difference of two sums is inf - inf. (A NaN
// stays one.)
__device__ __forceinline__ float delta_log2_decay(float g) {
  const float v = g * 1.4426950408889634f;
  return v < -150.f ? -150.f : v;
}

// Sums of a chunk's log decays, each lane's up to and including its own, in two
// floats: the decay between two tokens is e^(difference of two sums), and behind
// a reset the sums are large and the difference is not (one float at -150 is off
// by 2^-17, 5e-6 of every decay behind it; with the residuals only the difference
// itself is rounded).
struct DecaySum {
  float hi, lo;
};
template <int Ctrl, int RowMask>
__device__ __forceinline__ void decay_sum_step(DecaySum &v) {
  const float h = dpp_or_zero<Ctrl, RowMask>(v.hi), l = dpp_or_zero<Ctrl, RowMask>(v.lo);
  const float sum = v.hi + h, part = sum - v.hi;
  v.lo += l + ((v.hi - (sum - part)) + (h - part));  // what rounding left
  v.hi = sum;
}
__device__ __forceinline__ DecaySum decay_sums(float g) {
  DecaySum v = {g, 0.f};
  decay_sum_step<kDppRowShr1, 0xf>(v);
  decay_sum_step<kDppRowShr2, 0xf>(v);
  decay_sum_step<kDppRowShr4, 0xf>(v);
  decay_sum_step<kDppRowShr8, 0xf>(v);
  decay_sum_step<kDppRowBcast15, 0xa>(v);
  decay_sum_step<kDppRowBcast31, 0xc>(v);
  return v;
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

// The sequence that a unit (a chunk slot, or with `step` chunks a segment) of a
// packed call belongs to: the last whose first unit is not past it.
__device__ __forceinline__ int delta_owner(const DeltaArgs &a, int unit, int64_t step) {
  int l = 0, r = a.nseq - 1;
  while (l < r) {
    const int m = (l + r + 1) / 2;
    const int64_t lo = min(max((int64_t)a.cu[m], (int64_t)0), a.T);
    if (lo / (kDeltaChunk * step) + m <= unit) l = m; else r = m - 1;
  }
  return l;
}

// What a walk over chunks covers: tokens [lo, hi) of sequence s, from chunk
// slot `slot` on; all of a sequence, or one segment of it.
struct DeltaWalk {
  int64_t lo, hi;
  int s, slot;
  bool first, last;  // of its sequence
};
__device__ __forceinline__ bool delta_walk(const DeltaArgs &a, int unit, DeltaWalk &w) {
  int k = 0;
  if (!a.seg) {
    w.s = unit;
  } else if (!a.cu) {
    w.s = unit / a.nseg_per;
    k = unit - w.s * a.nseg_per;
  } else {
    w.s = delta_owner(a, unit, a.seg);
    const int64_t lo = min(max((int64_t)a.cu[w.s], (int64_t)0), a.T);
    k = unit - (int)(lo / (kDeltaChunk * (int64_t)a.seg)) - w.s;
    if (k < 0) return false;
  }
  delta_seq(a, w.s, w.lo, w.hi);
  w.slot = delta_slot0(a, w.s, w.lo);
  w.first = k == 0;
  w.last = true;
  if (a.seg) {
    const int64_t n = (int64_t)kDeltaChunk * a.seg, at = k * n;
    if (k > 0 && at >= w.hi - w.lo) return false;
    w.last = w.hi - w.lo <= at + n;
    w.hi = min(w.hi, w.lo + at + n);
    w.lo += at;
    w.slot += k * a.seg;
  }
  return true;
}

// First token and length of the chunk in a slot; false if the slot has none.
__device__ __forceinline__ bool delta_chunk(const DeltaArgs &a, int slot, int64_t &start,
                                            int &len) {
  const int s = a.cu ? delta_owner(a, slot, 1) : slot / a.nc_per;
  int64_t lo, hi;
  delta_seq(a, s, lo, hi);
  const int64_t at = (int64_t)(slot - delta_slot0(a, s, lo)) * kDeltaChunk;
  if (at < 0 || at >= hi - lo) return false;
  start = lo + at;
  len = (int)min((int64_t)kDeltaChunk, hi - start);
  return true;
}

// Workgroup b's place of n in the order of units: workgroups go round-robin over
// the eight XCDs, and each takes an eighth of the units in a row, so that heads
// that read the same rows of B and C find them in one L2.
__device__ __forceinline__ int xcd_unit(int b, int n) {
  const int q = n / 8, r = n % 8, x = b % 8;
  return x * q + min(x, r) + b / 8;
}
__device__ __forceinline__ int xcd_unit() { return xcd_unit((int)blockIdx.x, (int)gridDim.x); }

// The same for walks of `per` workgroups a sequence. Packed sequences of unequal length
// are dealt to the XCDs in order of their length, there and back (a run of whole
// eighths left the last XCD at work for twice the first's time, and a long sequence
// taken last all others waiting; -1: no sequence is left for this one).
__device__ __forceinline__ int delta_unit(const DeltaArgs &a, int b, int n, int per) {
  if (!a.order) return xcd_unit(b, n);
  const int x = b % 8, i = b / 8, j = i / per, rank = 8 * j + (j & 1 ? 7 - x : x);
  return rank < a.nseq ? a.order[rank] * per + (i - j * per) : -1;
}

// Bytes of one (slot, head)'s triangular matrices.
size_t delta_tri_bytes(bool tiles, DeltaTri which);

hipError_t launch_delta_prep(const DeltaArgs &a, bool bf16_io, DeltaTri which, hipStream_t s);
// Whether a call's sequences are ordered: packed in numbers between where eighths of
// them are too few to deal and where they even out by themselves (and their order, each
// against all others, takes too long). Measured, 24 heads of 64, us a call as they come
// and ordered: 20 sequences up to 2000 tokens 208, 201; 33 up to 2000 260, 228; 48 up to
// 1536 281, 234, backward 1650, 1570; 200 up to 600 504, 453; 512 up to 300 682, 665.
constexpr int kLeastOrdered = 32, kMostOrdered = 512;
inline bool delta_ordered(const DeltaArgs &a, bool packed) {
  return packed && !a.seg && a.T > 0 && a.nseq >= kLeastOrdered && a.nseq <= kMostOrdered;
}

// The bf16 path: segments (sets a.seg, a.nseg_per, a.nsegs), the forward call
// (triangular matrices in place), and the backward call's steps.
void delta_segments(DeltaArgs &a, bool packed, bool backward);
hipError_t launch_delta_forward(const DeltaArgs &a, hipStream_t s);
hipError_t launch_delta_both_ways(const DeltaArgs &a, hipStream_t s);
hipError_t launch_delta_grad(const DeltaArgs &a, hipStream_t s);
// Parts that a group's heads are taken in by the gradients (1: dB and dC are
// written at once).
int delta_grad_parts(const DeltaArgs &a);
hipError_t launch_delta_heads_sum(const DeltaArgs &a, bool bf16_io, hipStream_t s);
// The same in fp32.
hipError_t launch_delta_walk_f32(const DeltaArgs &a, bool both, hipStream_t s);
hipError_t launch_delta_grad_f32(const DeltaArgs &a, hipStream_t s);

struct DeltaStepArgs {
  const void *x, *g, *beta, *B, *C;
  float *state;        // (rows, N), rows = batch * H * P
  void *y;
  int64_t rows;
  int32_t H, N, G, heads_per_group, p_shift;
};
hipError_t launch_delta_step(const DeltaStepArgs &a, bool bf16_io, hipStream_t s);

}  // namespace ssd
