// k_ckpt.hip -- 8-bit checkpoints of whole tensors (the form is described in
// rows.h): save reads each element once and writes 33 bytes per 32 channels,
// load reads those and writes each element once, so both are bound by HBM
// bandwidth. A lane owns 8 channels of kCkptRows rows, whose loads are all
// issued before the first is used; four neighbouring lanes share a block.
// Measured at 16384 rows of 5376 bf16 channels (267 MB): save 48 us (5.6 TB/s),
// load 42 us (6.4 TB/s).
#include "norm.h"

namespace ssd {

namespace {

constexpr int kCkptThreads = 256, kCkptRows = 4;

template <typename T>
__global__ __launch_bounds__(kCkptThreads) void k_ckpt_save(const void *src, int64_t stride,
                                                            int64_t rows, int ch, int groups,
                                                            Ckpt k) {
  const int64_t gid = (int64_t)blockIdx.x * kCkptThreads + threadIdx.x;
  const int64_t r0 = gid / groups * kCkptRows;
  if (r0 >= rows) return;  // the same for all four lanes of a block
  const int cg = (int)(gid % groups) * 8;
  const bool live = cg < ch;
  const int c0 = live ? cg : ch - 8;
  Row8<T> row[kCkptRows];
#pragma unroll
  for (int i = 0; i < kCkptRows; ++i) row[i].load(src, (size_t)(min(r0 + i, rows - 1) * stride + c0));
#pragma unroll
  for (int i = 0; i < kCkptRows; ++i) {
    if (r0 + i < rows) {
      float v[8];
      row[i].widen(v);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = live ? v[c] : 0.f;
      store_ckpt(k, (size_t)(r0 + i), ch, c0, v, live);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kCkptThreads) void k_ckpt_load(Ckpt k, int64_t rows, int ch,
                                                            int groups, void *dst,
                                                            int64_t stride) {
  const int64_t gid = (int64_t)blockIdx.x * kCkptThreads + threadIdx.x;
  const int64_t r0 = gid / groups * kCkptRows;
  if (r0 >= rows) return;
  const int c0 = (int)(gid % groups) * 8;
  RowQ8 row[kCkptRows];
#pragma unroll
  for (int i = 0; i < kCkptRows; ++i) row[i].load(k, (size_t)min(r0 + i, rows - 1), ch, c0);
#pragma unroll
  for (int i = 0; i < kCkptRows; ++i) {
    if (r0 + i < rows) {
      float v[8];
      row[i].widen(v);
      Row8<T>::store(dst, (size_t)((r0 + i) * stride + c0), v);
    }
  }
}

dim3 blocks_for(int64_t rows, int groups) {
  const int64_t threads = (rows + kCkptRows - 1) / kCkptRows * groups;
  return dim3((unsigned)((threads + kCkptThreads - 1) / kCkptThreads));
}

}  // namespace

hipError_t launch_ckpt_save(const void *src, int64_t stride, int64_t rows, int channels,
                            bool bf16_io, const Ckpt &k, hipStream_t s) {
  const int groups = ckpt_blocks(channels) * kCkptLanes;
  const dim3 grid = blocks_for(rows, groups), block(kCkptThreads);
  if (bf16_io)
    hipLaunchKernelGGL(k_ckpt_save<bf16>, grid, block, 0, s, src, stride, rows, channels, groups, k);
  else
    hipLaunchKernelGGL(k_ckpt_save<float>, grid, block, 0, s, src, stride, rows, channels, groups, k);
  return hipGetLastError();
}

hipError_t launch_ckpt_load(const Ckpt &k, int64_t rows, int channels, bool bf16_io, void *dst,
                            int64_t stride, hipStream_t s) {
  const int groups = channels / 8;
  const dim3 grid = blocks_for(rows, groups), block(kCkptThreads);
  if (bf16_io)
    hipLaunchKernelGGL(k_ckpt_load<bf16>, grid, block, 0, s, k, rows, channels, groups, dst, stride);
  else
    hipLaunchKernelGGL(k_ckpt_load<float>, grid, block, 0, s, k, rows, channels, groups, dst, stride);
  return hipGetLastError();
}

}  // namespace ssd
