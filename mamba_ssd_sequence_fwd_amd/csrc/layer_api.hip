// layer_api.hip -- the C ABI of the operators around the SSD layer
// (include/ssd.h): the convolution front and its backward pass, the group norm
// with SiLU and its backward pass, and 8-bit activation checkpoints. Argument
// checks on the host, then launches on the caller's stream; nothing is
// allocated, synchronised or read back.
#include <math.h>

#include "api.h"
#include "conv.h"
#include "norm.h"

namespace {

using ssd::fail;

constexpr size_t kAlign = 256;  // of workspaces
// A launch takes fewer than 2^32 threads along x: workgroups of 256 threads,
// and columns of k_column_sums (1024 threads for 64 of them).
constexpr int64_t kMostBlocks = (1 << 24) - 1, kMostColumns = (1 << 28) - 64;

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

size_t element_bytes(int32_t dtype) { return dtype == SSD_DTYPE_BF16 ? 2 : 4; }

// A checkpoint argument: absent (NULL), or both arrays given and aligned.
ssd_status check_ckpt(const ssd_checkpoint *k, const char *name) {
  if (!k) return SSD_OK;
  if (!k->q || !k->exponents)
    return fail(SSD_ERR_INVALID_ARG, "%s: q and exponents must be non-NULL", name);
  if (((uintptr_t)k->q & 7) != 0)
    return fail(SSD_ERR_INVALID_ARG, "%s: q must be 8-byte aligned", name);
  return SSD_OK;
}

ssd::Ckpt ckpt_of(const ssd_checkpoint *k) {
  ssd::Ckpt c{};
  if (k) {
    c.q = k->q;
    c.e = k->exponents;
  }
  return c;
}

// ---- convolution front ---------------------------------------------------------

// The sizes of a front problem; `T` tokens and `nseq` sequences on success.
// in_stride is that of xbc: looked at unless a checkpoint is read in its place.
ssd_status check_conv(const ssd_conv_problem *p, const int32_t *cu_seqlens, bool strided,
                      int64_t *T, int64_t *nseq) {
  ssd::clear_detail();
  if (!p) return fail(SSD_ERR_INVALID_ARG, "problem is NULL");
  if (p->batch < 0 || p->seqlen < 0 || p->num_seqs < 0 || p->x_dim < 0 || p->bc_dim < 0)
    return fail(SSD_ERR_INVALID_ARG,
                "sizes must be non-negative (batch %d, seqlen %d, num_seqs %d, x_dim %d, "
                "bc_dim %d)", p->batch, p->seqlen, p->num_seqs, p->x_dim, p->bc_dim);
  if (p->flags != 0)
    return fail(SSD_ERR_INVALID_ARG, "the convolution takes no flags (0x%x)", p->flags);
  if (p->dtype != SSD_DTYPE_F32 && p->dtype != SSD_DTYPE_BF16)
    return fail(SSD_ERR_UNSUPPORTED, "dtype %d not supported", p->dtype);
  if (p->width < 2 || p->width > 4)
    return fail(SSD_ERR_UNSUPPORTED, "width %d not in {2, 3, 4}", p->width);
  if (p->x_dim % 8 != 0 || p->bc_dim % 8 != 0)
    return fail(SSD_ERR_UNSUPPORTED, "x_dim %d and bc_dim %d must be multiples of 8", p->x_dim,
                p->bc_dim);
  const int64_t ch = (int64_t)p->x_dim + 2 * (int64_t)p->bc_dim;
  if (ch < 8 || ch > INT32_MAX / 8)
    return fail(SSD_ERR_INVALID_ARG, "channel count %lld out of range",
                (long long)ch);
  const size_t esz = element_bytes(p->dtype);
  if (strided && (p->in_stride < ch || ((size_t)p->in_stride * esz) % 16 != 0))
    return fail(SSD_ERR_INVALID_ARG,
                "in_stride %d must be >= the channel count %lld and a multiple of 16 bytes",
                p->in_stride, (long long)ch);
  const bool varlen = p->num_seqs > 0;
  if (varlen && p->batch != 1)
    return fail(SSD_ERR_INVALID_ARG, "packed sequences take batch 1, got %d", p->batch);
  if (varlen && !cu_seqlens)
    return fail(SSD_ERR_INVALID_ARG, "num_seqs > 0 needs cu_seqlens");
  *T = (int64_t)p->batch * p->seqlen;
  *nseq = varlen ? p->num_seqs : p->batch;
  const int64_t tiles = (*T + ssd::kConvTile - 1) / ssd::kConvTile;
  if (*T > INT32_MAX - ssd::kConvTile ||
      (tiles * (ch / 8) + ssd::kConvThreads - 1) / ssd::kConvThreads > INT32_MAX ||
      (*nseq * (ch / 8) + ssd::kConvThreads - 1) / ssd::kConvThreads > INT32_MAX)
    return fail(SSD_ERR_UNSUPPORTED, "%lld tokens x %lld channels too large for one launch",
                (long long)*T, (long long)ch);
  return SSD_OK;
}

// Bounds of the kernels that walk tiles of at least 12 tokens, 256 channels
// and 4 tiles to a workgroup.
ssd_status check_tiles(const ssd_conv_problem *p, int64_t T, int64_t nseq) {
  const int64_t ch = (int64_t)p->x_dim + 2 * (int64_t)p->bc_dim;
  if (T + 2 * nseq > INT32_MAX / 2 ||
      ((T / 12 + nseq) / 4 + 1) * (ch / 256 + 1) > kMostBlocks)
    return fail(SSD_ERR_UNSUPPORTED, "%lld tokens in %lld sequences x %lld channels too large for "
                "one launch", (long long)T, (long long)nseq, (long long)ch);
  return SSD_OK;
}

ssd_status conv_forward(const ssd_conv_problem *p, const void *xbc, const ssd_checkpoint *ck,
                        const float *weight, const float *bias, const void *history_in,
                        const int32_t *cu_seqlens, void *x, void *B, void *C, void *history_out,
                        void *stream) {
  int64_t T = 0, nseq = 0;
  ssd_status st = check_conv(p, cu_seqlens, xbc || !ck, &T, &nseq);
  if (st != SSD_OK) return st;
  if (ck && (st = check_tiles(p, T, nseq)) != SSD_OK) return st;
  if (nseq == 0 || (T == 0 && !history_out)) return SSD_OK;
  if (!weight) return fail(SSD_ERR_INVALID_ARG, "weight must be non-NULL");
  if (T > 0 && ((!xbc && !ck) || (p->x_dim > 0 && !x) || (p->bc_dim > 0 && (!B || !C))))
    return fail(SSD_ERR_INVALID_ARG, "xbc, and x, B, C for non-empty parts, must be non-NULL");
  if (!aligned16(xbc) || !aligned16(x) || !aligned16(B) || !aligned16(C) ||
      !aligned16(history_in) || !aligned16(history_out))
    return fail(SSD_ERR_INVALID_ARG, "xbc, x, B, C and the histories must be 16-byte aligned");
  ssd::ConvArgs a{};
  a.xbc = xbc;
  a.w = weight;
  a.bias = bias;
  a.hist_in = history_in;
  a.cu = p->num_seqs > 0 ? cu_seqlens : nullptr;
  a.x = x;
  a.B = B;
  a.C = C;
  a.hist_out = history_out;
  a.T = (int32_t)T;
  a.seqlen = p->seqlen;
  a.nseq = (int32_t)nseq;
  a.ch = p->x_dim + 2 * p->bc_dim;
  a.x_dim = p->x_dim;
  a.bc_dim = p->bc_dim;
  a.in_stride = p->in_stride;
  a.groups = a.ch / 8;
  a.tiles = (int32_t)((T + ssd::kConvTile - 1) / ssd::kConvTile);
  const bool bf = p->dtype == SSD_DTYPE_BF16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = ck && T > 0 ? ssd::launch_conv_ckpt(a, ckpt_of(ck), p->width, bf, s)
                                   : ssd::launch_conv(a, p->width, bf, s);
  if (e != hipSuccess)
    return fail(SSD_ERR_HIP, "convolution kernel launch failed: %s", hipGetErrorString(e));
  return SSD_OK;
}

// Geometry of the front's backward pass: tile blocks, or an error.
ssd_status conv_backward_geometry(const ssd_conv_problem *p, const int32_t *cu, int64_t T,
                                  int64_t nseq, ssd::ConvBwdArgs *a, int64_t *tblocks) {
  ssd_status st;
  a->map.cu = p->num_seqs > 0 ? cu : nullptr;
  a->map.T = (int32_t)T;
  a->map.seqlen = p->seqlen;
  a->map.nseq = (int32_t)nseq;
  a->ch = p->x_dim + 2 * p->bc_dim;
  a->x_dim = p->x_dim;
  a->bc_dim = p->bc_dim;
  a->in_stride = p->in_stride;
  if ((st = check_tiles(p, T, nseq)) != SSD_OK) return st;
  if ((int64_t)a->ch * (p->width + 1) > kMostColumns)
    return fail(SSD_ERR_UNSUPPORTED, "%d channels are too many for one launch", a->ch);
  *tblocks = ssd::conv_bwd_geometry(*a);
  return SSD_OK;
}

size_t conv_backward_bytes(const ssd::ConvBwdArgs &a, int width, int64_t tblocks) {
  return (size_t)tblocks * (width + 1) * a.ch * sizeof(float);
}

// ---- group norm ------------------------------------------------------------------

ssd_status check_norm(const ssd_norm_problem *p) {
  ssd::clear_detail();
  if (!p) return fail(SSD_ERR_INVALID_ARG, "problem is NULL");
  if (p->tokens < 0 || p->channels < 1 || p->groups < 1)
    return fail(SSD_ERR_INVALID_ARG, "sizes must be valid (tokens %d >= 0, channels %d, groups %d)",
                p->tokens, p->channels, p->groups);
  if (p->channels % p->groups != 0)
    return fail(SSD_ERR_INVALID_ARG, "channels %d not divisible by groups %d", p->channels,
                p->groups);
  if (p->flags & ~(SSD_NORM_CENTER | SSD_NORM_BEFORE_GATE))
    return fail(SSD_ERR_INVALID_ARG, "unknown flags 0x%x", p->flags);
  if (!(p->eps >= 0.f) || isinf(p->eps))
    return fail(SSD_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (p->dtype != SSD_DTYPE_F32 && p->dtype != SSD_DTYPE_BF16)
    return fail(SSD_ERR_UNSUPPORTED, "dtype %d not supported", p->dtype);
  const int gs = p->channels / p->groups;
  if (gs % 8 != 0 || gs > ssd::kNormMaxGroup)
    return fail(SSD_ERR_UNSUPPORTED, "group size %d is not a multiple of 8 up to %d", gs,
                ssd::kNormMaxGroup);
  if (2 * (int64_t)p->channels > kMostColumns || p->tokens > INT32_MAX / 2)
    return fail(SSD_ERR_UNSUPPORTED, "%d tokens x %d channels too large for 32-bit indexing",
                p->tokens, p->channels);
  return SSD_OK;
}

ssd_status check_stride(const ssd_norm_problem *p, int64_t stride, const char *name) {
  if (stride < p->channels || (stride * (int64_t)element_bytes(p->dtype)) % 16 != 0 ||
      stride > INT32_MAX)
    return fail(SSD_ERR_INVALID_ARG,
                "%s %lld must be >= the channel count %d and a multiple of 16 bytes", name,
                (long long)stride, p->channels);
  return SSD_OK;
}

ssd::NormArgs norm_args(const ssd_norm_problem *p) {
  ssd::NormArgs a{};
  a.rows = p->tokens;
  a.C = p->channels;
  a.G = p->groups;
  a.gs = p->channels / p->groups;
  a.center = (p->flags & SSD_NORM_CENTER) ? 1 : 0;
  a.bf16_io = p->dtype == SSD_DTYPE_BF16;
  a.eps = p->eps;
  a.inv_n = 1.f / (float)a.gs;
  a.x_stride = p->x_stride;
  a.z_stride = p->z_stride;
  a.out_stride = p->out_stride;
  a.dx_stride = p->dx_stride;
  a.dz_stride = p->dz_stride;
  return a;
}

ssd::NormMode norm_mode(const ssd_norm_problem *p, bool gated) {
  if (!gated) return ssd::kNoGate;
  return (p->flags & SSD_NORM_BEFORE_GATE) ? ssd::kGateLast : ssd::kGateFirst;
}

ssd_status check_gate(const ssd_norm_problem *p, bool gated) {
  if (!gated && (p->flags & SSD_NORM_BEFORE_GATE))
    return fail(SSD_ERR_INVALID_ARG, "SSD_NORM_BEFORE_GATE needs z");
  return SSD_OK;
}

// Enough for both sources of the inputs, whose geometries differ.
size_t norm_backward_bytes(ssd::NormArgs a) {
  static int8_t some;
  a.xk.q = nullptr;
  const int plain = ssd::norm_partial_rows(a);
  a.xk.q = &some;
  const int kept = ssd::norm_partial_rows(a);
  return (size_t)(plain > kept ? plain : kept) * 2 * a.C * sizeof(float);
}

ssd_status check_workspace(const void *ws, size_t have, size_t need) {
  if (need == 0) return SSD_OK;
  if (!ws || ((uintptr_t)ws % kAlign) != 0)
    return fail(SSD_ERR_WORKSPACE, "workspace is NULL or not 256-byte aligned");
  if (have < need)
    return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return SSD_OK;
}

// ---- checkpoints -------------------------------------------------------------------

ssd_status check_ckpt_problem(const ssd_checkpoint_problem *p, const void *tensor,
                              const ssd_checkpoint *ck) {
  ssd::clear_detail();
  if (!p) return fail(SSD_ERR_INVALID_ARG, "problem is NULL");
  if (p->rows < 0 || p->channels < 1)
    return fail(SSD_ERR_INVALID_ARG, "sizes must be valid (rows %lld >= 0, channels %d)",
                (long long)p->rows, p->channels);
  if (p->flags != 0)
    return fail(SSD_ERR_INVALID_ARG, "checkpoints take no flags (0x%x)", p->flags);
  if (p->dtype != SSD_DTYPE_F32 && p->dtype != SSD_DTYPE_BF16)
    return fail(SSD_ERR_UNSUPPORTED, "dtype %d not supported", p->dtype);
  if (p->channels % 8 != 0)
    return fail(SSD_ERR_UNSUPPORTED, "channels %d is not a multiple of 8", p->channels);
  if (p->stride < p->channels || p->stride > INT32_MAX ||
      (p->stride * (int64_t)element_bytes(p->dtype)) % 16 != 0)
    return fail(SSD_ERR_INVALID_ARG,
                "stride %lld must be >= the channel count %d and a multiple of 16 bytes",
                (long long)p->stride, p->channels);
  if (p->rows > INT32_MAX ||
      (p->rows + 3) / 4 * (p->channels / 8 + 4) / 256 + 1 > kMostBlocks)
    return fail(SSD_ERR_UNSUPPORTED, "%lld rows x %d channels too large for one launch",
                (long long)p->rows, p->channels);
  if (p->rows == 0) return SSD_OK;
  if (!tensor || !ck)
    return fail(SSD_ERR_INVALID_ARG, "the tensor and the checkpoint must be non-NULL");
  if (!aligned16(tensor))
    return fail(SSD_ERR_INVALID_ARG, "the tensor must be 16-byte aligned");
  return check_ckpt(ck, "checkpoint");
}

}  // namespace

extern "C" {

ssd_status ssd_conv1d_silu(const ssd_conv_problem *p, const void *xbc, const float *weight,
                           const float *bias, const void *history_in,
                           const int32_t *cu_seqlens, void *x, void *B, void *C,
                           void *history_out, void *stream) {
  return conv_forward(p, xbc, nullptr, weight, bias, history_in, cu_seqlens, x, B, C,
                      history_out, stream);
}

ssd_status ssd_conv1d_silu_checkpoint(const ssd_conv_problem *p, const void *xbc,
                                      const ssd_checkpoint *checkpoint, const float *weight,
                                      const float *bias, const void *history_in,
                                      const int32_t *cu_seqlens, void *x, void *B, void *C,
                                      void *history_out, void *stream) {
  ssd::clear_detail();
  if (!checkpoint) return fail(SSD_ERR_INVALID_ARG, "checkpoint must be non-NULL");
  // without tokens xbc is NULL too (an empty tensor's address), and the history passes through
  const bool tokens = p && (int64_t)p->batch * p->seqlen > 0;
  if (tokens && !xbc && history_out)
    return fail(SSD_ERR_INVALID_ARG, "a checkpoint does not hold the exact history");
  ssd_status st = tokens ? check_ckpt(checkpoint, "checkpoint") : SSD_OK;
  if (st != SSD_OK) return st;
  return conv_forward(p, xbc, checkpoint, weight, bias, history_in, cu_seqlens, x, B, C,
                      history_out, stream);
}

ssd_status ssd_conv1d_silu_backward_workspace_size(const ssd_conv_problem *p, size_t *bytes) {
  // only the sizes matter here; any non-NULL offsets stand for the packed form
  static const int32_t some = 0;
  int64_t T = 0, nseq = 0, tblocks = 0;
  ssd_status st = check_conv(p, &some, false, &T, &nseq);
  if (st != SSD_OK) return st;
  if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
  ssd::ConvBwdArgs a{};  // (a checkpoint takes no more tiles than the tensor)
  st = conv_backward_geometry(p, &some, T, nseq, &a, &tblocks);
  if (st != SSD_OK) return st;
  *bytes = conv_backward_bytes(a, p->width, tblocks);
  return SSD_OK;
}

ssd_status ssd_conv1d_silu_backward(const ssd_conv_problem *p, const void *xbc,
                                    const ssd_checkpoint *checkpoint, const float *weight,
                                    const float *bias, const void *history_in,
                                    const int32_t *cu_seqlens, const void *dx, const void *dB,
                                    const void *dC, const void *dhistory_out, void *dxbc,
                                    int32_t dxbc_stride, float *dweight, float *dbias,
                                    void *dhistory, void *workspace, size_t workspace_bytes,
                                    void *stream) {
  int64_t T = 0, nseq = 0, tblocks = 0;
  ssd_status st = check_conv(p, cu_seqlens, xbc || !checkpoint, &T, &nseq);
  if (st != SSD_OK) return st;
  if (!weight || !dweight)
    return fail(SSD_ERR_INVALID_ARG, "weight and dweight must be non-NULL");
  if (T > 0) {
    if (!xbc == !checkpoint)
      return fail(SSD_ERR_INVALID_ARG, "give xbc or a checkpoint of it, and not both");
    if ((p->x_dim > 0 && !dx) || (p->bc_dim > 0 && (!dB || !dC)) || !dxbc)
      return fail(SSD_ERR_INVALID_ARG, "dxbc, and dx, dB, dC for non-empty parts, must be non-NULL");
    st = check_ckpt(checkpoint, "checkpoint");
    if (st != SSD_OK) return st;
  }
  const int64_t ch = (int64_t)p->x_dim + 2 * (int64_t)p->bc_dim;
  if (dxbc_stride < ch || ((size_t)dxbc_stride * element_bytes(p->dtype)) % 16 != 0)
    return fail(SSD_ERR_INVALID_ARG,
                "dxbc_stride %d must be >= the channel count %lld and a multiple of 16 bytes",
                dxbc_stride, (long long)ch);
  if (!aligned16(xbc) || !aligned16(dx) || !aligned16(dB) || !aligned16(dC) ||
      !aligned16(history_in) || !aligned16(dhistory_out) || !aligned16(dxbc) ||
      !aligned16(dhistory))
    return fail(SSD_ERR_INVALID_ARG, "xbc, dx, dB, dC, dxbc and the histories must be 16-byte "
                "aligned");
  ssd::ConvBwdArgs a{};
  a.ck = ckpt_of(checkpoint);
  st = conv_backward_geometry(p, cu_seqlens, T, nseq, &a, &tblocks);
  if (st != SSD_OK) return st;
  st = check_workspace(workspace, workspace_bytes, conv_backward_bytes(a, p->width, tblocks));
  if (st != SSD_OK) return st;
  a.xbc = xbc;
  a.w = weight;
  a.bias = bias;
  a.hist_in = history_in;
  a.dx = dx;
  a.dB = dB;
  a.dC = dC;
  a.dhist_out = dhistory_out;
  a.dxbc = dxbc;
  a.out_stride = dxbc_stride;
  a.dhist = dhistory;
  a.part = static_cast<float *>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = ssd::launch_conv_backward(a, p->width, p->dtype == SSD_DTYPE_BF16, s);
  if (e == hipSuccess)
    e = ssd::launch_column_sums(a.part, (int)tblocks, p->width + 1, p->width, a.ch, dweight, dbias,
                                s);
  if (e != hipSuccess)
    return fail(SSD_ERR_HIP, "convolution backward launch failed: %s", hipGetErrorString(e));
  return SSD_OK;
}

ssd_status ssd_group_norm_silu(const ssd_norm_problem *p, const void *x, const void *z,
                               const float *weight, const float *bias, void *out,
                               const ssd_checkpoint *x_checkpoint,
                               const ssd_checkpoint *z_checkpoint, void *stream) {
  ssd_status st = check_norm(p);
  if (st != SSD_OK) return st;
  if (p->tokens == 0) return SSD_OK;
  if (!x || !out) return fail(SSD_ERR_INVALID_ARG, "x and out must be non-NULL");
  if ((st = check_gate(p, z != nullptr)) != SSD_OK) return st;
  if ((st = check_stride(p, p->x_stride, "x_stride")) != SSD_OK) return st;
  if (z && (st = check_stride(p, p->z_stride, "z_stride")) != SSD_OK) return st;
  if ((st = check_stride(p, p->out_stride, "out_stride")) != SSD_OK) return st;
  if (!aligned16(x) || !aligned16(z) || !aligned16(out))
    return fail(SSD_ERR_INVALID_ARG, "x, z and out must be 16-byte aligned");
  if ((st = check_ckpt(x_checkpoint, "x_checkpoint")) != SSD_OK) return st;
  if ((st = check_ckpt(z_checkpoint, "z_checkpoint")) != SSD_OK) return st;
  if ((z_checkpoint != nullptr) != (x_checkpoint != nullptr && z != nullptr))
    return fail(SSD_ERR_INVALID_ARG, "checkpoints are kept of x and, where it is given, z, or "
                "of neither");
  ssd::NormArgs a = norm_args(p);
  a.x = x;
  a.z = z;
  a.w = weight;
  a.b = bias;
  a.out = out;
  a.xk = ckpt_of(x_checkpoint);
  a.zk = ckpt_of(z_checkpoint);
  const hipError_t e = ssd::launch_norm(a, norm_mode(p, z != nullptr),
                                        p->dtype == SSD_DTYPE_BF16,
                                        static_cast<hipStream_t>(stream));
  if (e != hipSuccess)
    return fail(SSD_ERR_HIP, "group norm launch failed: %s", hipGetErrorString(e));
  return SSD_OK;
}

ssd_status ssd_group_norm_silu_backward_workspace_size(const ssd_norm_problem *p, size_t *bytes) {
  ssd_status st = check_norm(p);
  if (st != SSD_OK) return st;
  if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = norm_backward_bytes(norm_args(p));
  return SSD_OK;
}

ssd_status ssd_group_norm_silu_backward(const ssd_norm_problem *p, const void *dout,
                                        const void *x, const void *z,
                                        const ssd_checkpoint *x_checkpoint,
                                        const ssd_checkpoint *z_checkpoint, const float *weight,
                                        const float *bias, void *dx, void *dz, float *dweight,
                                        float *dbias, void *workspace, size_t workspace_bytes,
                                        void *stream) {
  ssd_status st = check_norm(p);
  if (st != SSD_OK) return st;
  ssd::NormArgs a = norm_args(p);
  const bool gated = z != nullptr || z_checkpoint != nullptr;
  const bool sums = dweight != nullptr || dbias != nullptr;
  a.b = bias;
  a.sum_b = dbias != nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (p->tokens > 0) {
    if ((st = check_gate(p, gated)) != SSD_OK) return st;
    if (!x == !x_checkpoint || (z && z_checkpoint))
      return fail(SSD_ERR_INVALID_ARG, "give x (and z) or checkpoints of them, and not both");
    if (gated && (x == nullptr) != (z == nullptr))
      return fail(SSD_ERR_INVALID_ARG, "x and z must both be tensors or both checkpoints");
    if (!dout || !dx || (gated && !dz))
      return fail(SSD_ERR_INVALID_ARG, "dout, dx, and dz with a gate, must be non-NULL");
    if ((st = check_ckpt(x_checkpoint, "x_checkpoint")) != SSD_OK) return st;
    if ((st = check_ckpt(z_checkpoint, "z_checkpoint")) != SSD_OK) return st;
    if (x && (st = check_stride(p, p->x_stride, "x_stride")) != SSD_OK) return st;
    if (z && (st = check_stride(p, p->z_stride, "z_stride")) != SSD_OK) return st;
    if ((st = check_stride(p, p->out_stride, "out_stride")) != SSD_OK) return st;
    if ((st = check_stride(p, p->dx_stride, "dx_stride")) != SSD_OK) return st;
    if (gated && (st = check_stride(p, p->dz_stride, "dz_stride")) != SSD_OK) return st;
    if (!aligned16(dout) || !aligned16(x) || !aligned16(z) || !aligned16(dx) || !aligned16(dz))
      return fail(SSD_ERR_INVALID_ARG, "dout, x, z, dx and dz must be 16-byte aligned");
    if (sums &&
        (st = check_workspace(workspace, workspace_bytes, norm_backward_bytes(a))) != SSD_OK)
      return st;
    a.x = x;
    a.z = z;
    a.xk = ckpt_of(x_checkpoint);
    a.zk = ckpt_of(z_checkpoint);
    a.w = weight;
    a.dout = dout;
    a.dx = dx;
    a.dz = dz;
    a.nparts = ssd::norm_partial_rows(a);
    a.part = sums ? static_cast<float *>(workspace) : nullptr;
    const hipError_t e = ssd::launch_norm_backward(a, norm_mode(p, gated),
                                                   p->dtype == SSD_DTYPE_BF16, s);
    if (e != hipSuccess)
      return fail(SSD_ERR_HIP, "group norm backward launch failed: %s", hipGetErrorString(e));
  }
  if (sums) {
    const int rows = a.b != nullptr || a.sum_b ? 2 : 1;
    const hipError_t e =
        ssd::launch_column_sums(a.part, a.nparts, rows, 1, a.C, dweight, dbias, s);
    if (e != hipSuccess)
      return fail(SSD_ERR_HIP, "group norm backward launch failed: %s", hipGetErrorString(e));
  }
  return SSD_OK;
}

ssd_status ssd_checkpoint_save(const ssd_checkpoint_problem *p, const void *src,
                               const ssd_checkpoint *checkpoint, void *stream) {
  ssd_status st = check_ckpt_problem(p, src, checkpoint);
  if (st != SSD_OK || p->rows == 0) return st;
  const hipError_t e = ssd::launch_ckpt_save(src, p->stride, p->rows, p->channels,
                                             p->dtype == SSD_DTYPE_BF16, ckpt_of(checkpoint),
                                             static_cast<hipStream_t>(stream));
  if (e != hipSuccess)
    return fail(SSD_ERR_HIP, "checkpoint kernel launch failed: %s", hipGetErrorString(e));
  return SSD_OK;
}

ssd_status ssd_checkpoint_load(const ssd_checkpoint_problem *p, const ssd_checkpoint *checkpoint,
                               void *dst, void *stream) {
  ssd_status st = check_ckpt_problem(p, dst, checkpoint);
  if (st != SSD_OK || p->rows == 0) return st;
  const hipError_t e = ssd::launch_ckpt_load(ckpt_of(checkpoint), p->rows, p->channels,
                                             p->dtype == SSD_DTYPE_BF16, dst, p->stride,
                                             static_cast<hipStream_t>(stream));
  if (e != hipSuccess)
    return fail(SSD_ERR_HIP, "checkpoint kernel launch failed: %s", hipGetErrorString(e));
  return SSD_OK;
}

}  // extern "C"
