// k_delta_step.hip -- one decode step of the gated delta rule: every sequence
// advances by one token, its fp32 state updated in place (delta.h).
//
// Per sequence, head and state row p (N contiguous floats), with a = e^g:
//   e = beta (x_p - a h_p . B),  h_p <- a h_p + e B,  y_p = a h_p . C + e B . C
// (y from the old row, so that its sum and the write's are taken side by side
// and the row is read once). Every state element is read and written once for
// 7 flops: HBM is the bound. R lanes hold a row, 4 columns each; a wave makes
// two passes with all loads issued first, nontemporal, as in the layer's step.
// Measured (MI355X), 80 heads of 64 x 128: 256 sequences 218 to 223 us, 6.1 TB/s.
#include "delta.h"
#include "mfma_common.h"

namespace ssd {

constexpr int kDeltaStepPasses = 2, kDeltaStepWaves = 4;

__device__ __forceinline__ f32x4 widen_row4(const float *p) {
  return *reinterpret_cast<const f32x4 *>(p);
}
__device__ __forceinline__ f32x4 widen_row4(const bf16 *p) {
  const bf16x4 v = *reinterpret_cast<const bf16x4 *>(p);
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
  return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}

template <int R, typename T>
__global__ __launch_bounds__(kDeltaStepWaves * 64) void k_delta_step(DeltaStepArgs a) {
  constexpr int kRows = 64 / R, kP = kDeltaStepPasses;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = ((int64_t)blockIdx.x * kDeltaStepWaves + wave) * (kRows * kP) + lane / R;
  const int n0 = 4 * (lane % R);
  f32x4 st[kP], k[kP], q[kP];
  float x[kP], b[kP], d[kP];
  bool ok[kP];
#pragma unroll
  for (int it = 0; it < kP; ++it) {
    const int64_t row = row0 + it * kRows;
    ok[it] = row < a.rows;
    st[it] = k[it] = q[it] = f32x4{0.f, 0.f, 0.f, 0.f};
    x[it] = b[it] = d[it] = 0.f;
    if (ok[it]) {
      // row = (s * H + h) * P + p; batch * H fits 32 bits (checked on the host)
      const uint32_t sh = (uint32_t)(row >> a.p_shift);
      const uint32_t s = sh / (uint32_t)a.H, h = sh - s * (uint32_t)a.H;
      const size_t bc = ((size_t)s * a.G + h / (uint32_t)a.heads_per_group) * a.N + n0;
      x[it] = ld<T>(a.x, (size_t)row);
      b[it] = ld<T>(a.beta, (size_t)sh);
      d[it] = ld<T>(a.g, (size_t)sh);
      if (n0 < a.N) {
        st[it] = __builtin_nontemporal_load(
            reinterpret_cast<const f32x4 *>(a.state + (size_t)row * a.N + n0));
        k[it] = widen_row4((const T *)a.B + bc);
        q[it] = widen_row4((const T *)a.C + bc);
      }
    }
  }
#pragma unroll
  for (int it = 0; it < kP; ++it) {
    st[it] *= exp2_fast(delta_log2_decay(d[it]));
    float hk = dot4(st[it], k[it]), hq = dot4(st[it], q[it]), kq = dot4(k[it], q[it]);
#pragma unroll
    for (int off = R / 2; off >= 1; off >>= 1) {
      hk += __shfl_xor(hk, off);
      hq += __shfl_xor(hq, off);
      kq += __shfl_xor(kq, off);
    }
    const float e = b[it] * (x[it] - hk);
    const int64_t row = row0 + it * kRows;
    if (ok[it]) {
      if (n0 < a.N)
        __builtin_nontemporal_store(
            st[it] + e * k[it], reinterpret_cast<f32x4 *>(a.state + (size_t)row * a.N + n0));
      if (n0 == 0) static_cast<T *>(a.y)[row] = from_f32<T>(hq + e * kq);
    }
  }
}

template <int R, typename T>
hipError_t delta_step_r(const DeltaStepArgs &a, hipStream_t s) {
  const int64_t per = (int64_t)kDeltaStepWaves * (64 / R) * kDeltaStepPasses;
  hipLaunchKernelGGL((k_delta_step<R, T>), dim3((unsigned)((a.rows + per - 1) / per)),
                     dim3(kDeltaStepWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t delta_step_t(const DeltaStepArgs &a, hipStream_t s) {
  if (a.N <= 16) return delta_step_r<4, T>(a, s);
  if (a.N <= 32) return delta_step_r<8, T>(a, s);
  if (a.N <= 64) return delta_step_r<16, T>(a, s);
  if (a.N <= 128) return delta_step_r<32, T>(a, s);
  return delta_step_r<64, T>(a, s);
}

hipError_t launch_delta_step(const DeltaStepArgs &a, bool bf16_io, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return bf16_io ? delta_step_t<bf16>(a, s) : delta_step_t<float>(a, s);
}

}  // namespace ssd
