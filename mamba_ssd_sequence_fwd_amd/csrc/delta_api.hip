// delta_api.hip -- the C ABI of the gated delta rule and of the norm and
// rotation of its keys and queries (include/ssd.h): argument checks on the
// host, then launches on the caller's stream; nothing is allocated,
// synchronised or read back.
#include <math.h>

#include "api.h"
#include "bcnorm.h"
#include "delta.h"

namespace {

using ssd::fail;

constexpr size_t kAlign = 256;  // of workspaces and of the parts of one
// A launch takes fewer than 2^32 threads along x: workgroups of 256 threads.
constexpr int64_t kMostBlocks = (1 << 24) - 1;
constexpr int64_t kMostTokens = 1 << 30;

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }
size_t padded(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// The sizes of a problem, and the device view's part of them.
ssd_status check_delta(const ssd_problem *p, bool step, ssd::DeltaArgs *a) {
  ssd::clear_detail();
  if (!p) return fail(SSD_ERR_INVALID_ARG, "problem is NULL");
  if (p->batch < 0 || p->seqlen < 0 || p->num_seqs < 0 || p->nheads < 1 || p->headdim < 1 ||
      p->dstate < 1 || p->ngroups < 1)
    return fail(SSD_ERR_INVALID_ARG,
                "sizes must be valid (batch %d >= 0, seqlen %d >= 0, num_seqs %d >= 0, nheads %d, "
                "headdim %d, dstate %d, ngroups %d)", p->batch, p->seqlen, p->num_seqs, p->nheads,
                p->headdim, p->dstate, p->ngroups);
  if (p->nheads % p->ngroups != 0)
    return fail(SSD_ERR_INVALID_ARG, "nheads %d not divisible by ngroups %d", p->nheads,
                p->ngroups);
  if (p->flags != 0)
    return fail(SSD_ERR_INVALID_ARG, "the delta rule takes no flags (0x%x)", p->flags);
  if (step && (p->seqlen != 1 || p->num_seqs != 0))
    return fail(SSD_ERR_INVALID_ARG, "a step takes seqlen 1 and num_seqs 0, got %d and %d",
                p->seqlen, p->num_seqs);
  if (p->num_seqs > 0 && p->batch != 1)
    return fail(SSD_ERR_INVALID_ARG, "packed sequences take batch 1, got %d", p->batch);
  if (p->dtype != SSD_DTYPE_F32 && p->dtype != SSD_DTYPE_BF16)
    return fail(SSD_ERR_UNSUPPORTED, "dtype %d not supported", p->dtype);
  if (p->headdim != 16 && p->headdim != 32 && p->headdim != 64 && p->headdim != 128)
    return fail(SSD_ERR_UNSUPPORTED, "headdim %d not in {16, 32, 64, 128}", p->headdim);
  if (p->dstate % 16 != 0 || p->dstate > 256)
    return fail(SSD_ERR_UNSUPPORTED, "dstate %d not a multiple of 16 in [16, 256]", p->dstate);
  const int64_t T = (int64_t)p->batch * p->seqlen;
  const bool packed = p->num_seqs > 0;
  const int64_t nseq = packed ? p->num_seqs : p->batch;
  const int64_t per = ((int64_t)p->seqlen + ssd::kDeltaChunk - 1) / ssd::kDeltaChunk;
  const int64_t slots = packed ? T / ssd::kDeltaChunk + nseq : nseq * per;
  const int64_t quads = T * p->ngroups * (p->dstate / 4);  // of dB and dC, each
  if (T >= kMostTokens || slots > kMostBlocks || nseq > kMostBlocks ||
      slots * p->nheads > kMostBlocks || nseq * p->nheads * (p->headdim / 16) > kMostBlocks ||
      quads > kMostBlocks * 128 || (int64_t)p->ngroups * p->dstate > (1 << 24) ||
      (int64_t)p->nheads * p->headdim > (1 << 24))
    return fail(SSD_ERR_UNSUPPORTED, "%lld tokens in %lld sequences x %d heads too large for one "
                "launch", (long long)T, (long long)nseq, p->nheads);
  a->T = T;
  a->L = p->seqlen;
  a->H = p->nheads;
  a->P = p->headdim;
  a->N = p->dstate;
  a->G = p->ngroups;
  a->hpg = p->nheads / p->ngroups;
  a->nseq = (int32_t)nseq;
  a->nc_per = (int32_t)per;
  a->nslots = (int32_t)(T ? slots : 0);
  return SSD_OK;
}

ssd_status check_packed(const ssd_problem *p, const int32_t *cu) {
  if (p->num_seqs > 0 && !cu)
    return fail(SSD_ERR_INVALID_ARG, "num_seqs > 0 needs cu_seqlens");
  return SSD_OK;
}

ssd_status check_workspace(const void *ws, size_t have, size_t need) {
  if (need == 0) return SSD_OK;
  if (!ws || ((uintptr_t)ws % kAlign) != 0)
    return fail(SSD_ERR_WORKSPACE, "workspace is NULL or not 256-byte aligned");
  if (have < need)
    return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return SSD_OK;
}

// Parts of a workspace in turn; with a base, their addresses.
struct Carver {
  char *base;
  size_t at = 0;
  void *take(size_t n) {
    void *p = base ? base + at : nullptr;
    at += padded(n);
    return p;
  }
};

// The forward pass's workspace; with a base, its parts are set.
size_t forward_bytes(ssd::DeltaArgs *a, const ssd_problem *p, void *ws) {
  const bool bf = p->dtype == SSD_DTYPE_BF16;
  if (bf) ssd::delta_segments(*a, p->num_seqs > 0, false);
  Carver c{static_cast<char *>(ws)};
  const size_t tri = ssd::delta_tri_bytes(bf, ssd::kTriForward);
  a->tri = c.take((size_t)a->nslots * a->H * tri);
  a->tri_stride = (int32_t)(tri / 2);
  if (bf && ssd::delta_ordered(*a, p->num_seqs > 0))
    a->order = static_cast<int32_t *>(c.take((size_t)a->nseq * sizeof(int32_t)));
  if (a->seg)
    a->span = static_cast<float *>(
        c.take((size_t)a->nsegs * a->H * (a->P + a->N) * a->N * sizeof(float)));
  return c.at;
}

// The backward pass's.
size_t backward_bytes(ssd::DeltaArgs *a, const ssd_problem *p, void *ws) {
  const bool bf = p->dtype == SSD_DTYPE_BF16;
  const size_t es = sizeof(float), sh = (size_t)a->nslots * a->H;  // (bf16: two of them)
  if (bf) ssd::delta_segments(*a, p->num_seqs > 0, true);
  a->hparts = bf ? ssd::delta_grad_parts(*a) : a->hpg;
  Carver c{static_cast<char *>(ws)};
  const size_t tri = ssd::delta_tri_bytes(bf, ssd::kTriBackward);
  a->tri = c.take(sh * tri);
  a->tri_stride = (int32_t)(tri / 2);
  if (bf && ssd::delta_ordered(*a, p->num_seqs > 0))
    a->order = static_cast<int32_t *>(c.take((size_t)a->nseq * sizeof(int32_t)));
  a->st_rest = (int64_t)(sh * a->P * a->N);
  a->u_rest = (int64_t)(sh * ssd::kDeltaChunk * a->P);
  a->st0 = c.take(sh * a->P * a->N * es);
  a->st1 = c.take(sh * a->P * a->N * es);
  a->u = c.take(sh * ssd::kDeltaChunk * a->P * es);
  a->dr = c.take(sh * ssd::kDeltaChunk * a->P * es);
  if (a->hparts > 1)
    a->part = static_cast<float *>(
        c.take(2 * (size_t)a->T * a->G * a->hparts * a->N * sizeof(float)));
  if (a->seg) {
    const size_t seg = (size_t)a->nsegs * a->H * a->N * sizeof(float);
    a->span = static_cast<float *>(c.take(seg * (a->P + a->N)));
    a->dspan = static_cast<float *>(c.take(seg * a->P));
  }
  return c.at;
}

ssd_status hip_result(hipError_t e, const char *what) {
  if (e == hipSuccess) return SSD_OK;
  return fail(SSD_ERR_HIP, "%s kernel launch failed: %s", what, hipGetErrorString(e));
}

// ---- norm and rotation of B and C -------------------------------------------------

ssd_status check_bc_stride(const ssd_bc_norm_problem *p, int64_t stride, int32_t heads,
                           const char *name) {
  const int64_t es = p->dtype == SSD_DTYPE_BF16 ? 2 : 4;
  if (stride < (int64_t)heads * p->dim || (stride * es) % 16 != 0 || stride > INT32_MAX)
    return fail(SSD_ERR_INVALID_ARG, "%s %lld must be >= %d heads x %d channels and a multiple of "
                "16 bytes", name, (long long)stride, heads, p->dim);
  return SSD_OK;
}

ssd_status check_bc_norm(const ssd_bc_norm_problem *p, bool backward, bool rotated,
                         ssd::BcNormArgs *a) {
  ssd::clear_detail();
  if (!p) return fail(SSD_ERR_INVALID_ARG, "problem is NULL");
  if (p->tokens < 0 || p->b_heads < 1 || p->c_heads < 1 || p->dim < 1 || p->rotary_dim < 0 ||
      p->period < 0)
    return fail(SSD_ERR_INVALID_ARG, "sizes must be valid (tokens %d, b_heads %d, c_heads %d, dim "
                "%d, rotary_dim %d, period %d)", p->tokens, p->b_heads, p->c_heads, p->dim,
                p->rotary_dim, p->period);
  if (p->flags & ~(SSD_BC_NORM_UNIT | SSD_BC_NORM_INTERLEAVED))
    return fail(SSD_ERR_INVALID_ARG, "unknown flags 0x%x", p->flags);
  if (!(p->eps >= 0.f) || isinf(p->eps))
    return fail(SSD_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (p->dtype != SSD_DTYPE_F32 && p->dtype != SSD_DTYPE_BF16)
    return fail(SSD_ERR_UNSUPPORTED, "dtype %d not supported", p->dtype);
  if (p->dim % 8 != 0 || p->dim > 256)
    return fail(SSD_ERR_UNSUPPORTED, "dim %d not a multiple of 8 up to 256", p->dim);
  if (p->rotary_dim % 8 != 0 || p->rotary_dim > p->dim)
    return fail(SSD_ERR_INVALID_ARG, "rotary_dim %d must be a multiple of 8 up to dim %d",
                p->rotary_dim, p->dim);
  if (p->tokens > 0 && rotated != (p->rotary_dim > 0))
    return fail(SSD_ERR_INVALID_ARG, "positions and freqs go with rotary_dim > 0");
  if (p->tokens > 0 && rotated && p->period < 1)
    return fail(SSD_ERR_INVALID_ARG, "period must be at least 1");
  if (p->b_heads > (1 << 20) || p->c_heads > (1 << 20) || p->tokens >= kMostTokens)
    return fail(SSD_ERR_UNSUPPORTED, "%d tokens x (%d + %d) heads too large for one launch",
                p->tokens, p->b_heads, p->c_heads);
  ssd_status st = check_bc_stride(p, p->b_out_stride, p->b_heads, "b_out_stride");
  if (st == SSD_OK) st = check_bc_stride(p, p->c_out_stride, p->c_heads, "c_out_stride");
  if (st == SSD_OK) st = check_bc_stride(p, p->b_stride, p->b_heads, "b_stride");
  if (st == SSD_OK) st = check_bc_stride(p, p->c_stride, p->c_heads, "c_stride");
  if (st == SSD_OK && backward) st = check_bc_stride(p, p->db_stride, p->b_heads, "db_stride");
  if (st == SSD_OK && backward) st = check_bc_stride(p, p->dc_stride, p->c_heads, "dc_stride");
  if (st != SSD_OK) return st;
  a->in_stride[0] = p->b_stride;
  a->in_stride[1] = p->c_stride;
  a->out_stride[0] = p->b_out_stride;
  a->out_stride[1] = p->c_out_stride;
  a->dx_stride[0] = p->db_stride;
  a->dx_stride[1] = p->dc_stride;
  a->heads[0] = p->b_heads;
  a->heads[1] = p->c_heads;
  a->tokens = p->tokens;
  a->N = p->dim;
  a->rot = p->rotary_dim;
  a->period = p->period;
  a->interleaved = (p->flags & SSD_BC_NORM_INTERLEAVED) ? 1 : 0;
  a->inv_n = (p->flags & SSD_BC_NORM_UNIT) ? 1.f : 1.f / (float)p->dim;
  a->eps = p->eps;
  return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_delta_workspace_size(const ssd_problem *p, size_t *bytes) {
  ssd::DeltaArgs a{};
  ssd_status st = check_delta(p, false, &a);
  if (st != SSD_OK) return st;
  if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = forward_bytes(&a, p, nullptr);
  return SSD_OK;
}

ssd_status ssd_delta_forward(const ssd_problem *p, const void *x, const void *g, const void *beta,
                             const void *B, const void *C, const float *initial_state,
                             const int32_t *cu_seqlens, void *y, float *final_state,
                             void *workspace, size_t workspace_bytes, void *stream) {
  ssd::DeltaArgs a{};
  ssd_status st = check_delta(p, false, &a);
  if (st != SSD_OK) return st;
  if ((st = check_packed(p, cu_seqlens)) != SSD_OK) return st;
  if (a.nseq == 0 || (a.T == 0 && !final_state)) return SSD_OK;
  if (a.T > 0 && (!x || !g || !beta || !B || !C || !y))
    return fail(SSD_ERR_INVALID_ARG, "x, g, beta, B, C and y must be non-NULL");
  if (!aligned16(x) || !aligned16(B) || !aligned16(C) || !aligned16(y) ||
      !aligned16(initial_state) || !aligned16(final_state))
    return fail(SSD_ERR_INVALID_ARG, "x, B, C, y and the states must be 16-byte aligned");
  const bool bf = p->dtype == SSD_DTYPE_BF16;
  const size_t need = forward_bytes(&a, p, workspace);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != SSD_OK) return st;
  a.x = x;
  a.g = g;
  a.beta = beta;
  a.B = B;
  a.C = C;
  a.h0 = initial_state;
  a.cu = p->num_seqs > 0 ? cu_seqlens : nullptr;
  a.y = y;
  a.hT = final_state;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = hip_result(ssd::launch_delta_prep(a, bf, ssd::kTriForward, s), "delta rule prep")) !=
      SSD_OK)
    return st;
  return hip_result(bf ? ssd::launch_delta_forward(a, s)
                       : ssd::launch_delta_walk_f32(a, false, s), "delta rule");
}

ssd_status ssd_delta_step(const ssd_problem *p, const void *x, const void *g, const void *beta,
                          const void *B, const void *C, float *state, void *y, void *stream) {
  ssd::DeltaArgs d{};
  ssd_status st = check_delta(p, true, &d);
  if (st != SSD_OK) return st;
  ssd::DeltaStepArgs a{};
  a.rows = (int64_t)p->batch * p->nheads * p->headdim;
  a.H = p->nheads;
  a.N = p->dstate;
  a.G = p->ngroups;
  a.heads_per_group = d.hpg;
  a.p_shift = __builtin_ctz((unsigned)p->headdim);
  if (a.rows / 8 > kMostBlocks)  // at least 8 rows to a workgroup
    return fail(SSD_ERR_UNSUPPORTED, "batch %d too large for one launch", p->batch);
  if (p->batch == 0) return SSD_OK;
  if (!x || !g || !beta || !B || !C || !state || !y)
    return fail(SSD_ERR_INVALID_ARG, "x, g, beta, B, C, state and y must be non-NULL");
  if (!aligned16(x) || !aligned16(B) || !aligned16(C) || !aligned16(y) || !aligned16(state))
    return fail(SSD_ERR_INVALID_ARG, "x, B, C, y and state must be 16-byte aligned");
  a.x = x;
  a.g = g;
  a.beta = beta;
  a.B = B;
  a.C = C;
  a.state = state;
  a.y = y;
  return hip_result(ssd::launch_delta_step(a, p->dtype == SSD_DTYPE_BF16,
                                           static_cast<hipStream_t>(stream)), "delta rule step");
}

ssd_status ssd_delta_backward_workspace_size(const ssd_problem *p, size_t *bytes) {
  ssd::DeltaArgs a{};
  ssd_status st = check_delta(p, false, &a);
  if (st != SSD_OK) return st;
  if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = backward_bytes(&a, p, nullptr);
  return SSD_OK;
}

ssd_status ssd_delta_backward(const ssd_problem *p, const void *x, const void *g, const void *beta,
                              const void *B, const void *C, const float *initial_state,
                              const int32_t *cu_seqlens, const void *dy,
                              const float *dfinal_state, void *dx, void *dg, void *dbeta, void *dB,
                              void *dC, float *dinitial_state, void *workspace,
                              size_t workspace_bytes, void *stream) {
  ssd::DeltaArgs a{};
  ssd_status st = check_delta(p, false, &a);
  if (st != SSD_OK) return st;
  if ((st = check_packed(p, cu_seqlens)) != SSD_OK) return st;
  if (a.nseq == 0 || (a.T == 0 && !dinitial_state)) return SSD_OK;
  if (a.T > 0 && (!x || !g || !beta || !B || !C || !dy || !dx || !dg || !dbeta || !dB || !dC))
    return fail(SSD_ERR_INVALID_ARG,
                "x, g, beta, B, C, dy and their gradients must be non-NULL");
  if (!aligned16(x) || !aligned16(B) || !aligned16(C) || !aligned16(dy) || !aligned16(dx) ||
      !aligned16(dB) || !aligned16(dC) || !aligned16(initial_state) ||
      !aligned16(dfinal_state) || !aligned16(dinitial_state))
    return fail(SSD_ERR_INVALID_ARG,
                "x, B, C, dy, dx, dB, dC and the states must be 16-byte aligned");
  const bool bf = p->dtype == SSD_DTYPE_BF16;
  const size_t need = backward_bytes(&a, p, workspace);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != SSD_OK) return st;
  a.x = x;
  a.g = g;
  a.beta = beta;
  a.B = B;
  a.C = C;
  a.h0 = initial_state;
  a.cu = p->num_seqs > 0 ? cu_seqlens : nullptr;
  a.dy = dy;
  a.dhT = dfinal_state;
  a.dx = dx;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dB = dB;
  a.dC = dC;
  a.dh0 = dinitial_state;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = hip_result(ssd::launch_delta_prep(a, bf, ssd::kTriBackward, s), "delta rule prep")) !=
      SSD_OK)
    return st;
  if ((st = hip_result(bf ? ssd::launch_delta_both_ways(a, s)
                          : ssd::launch_delta_walk_f32(a, true, s), "delta rule walks")) != SSD_OK)
    return st;
  return hip_result(bf ? ssd::launch_delta_grad(a, s) : ssd::launch_delta_grad_f32(a, s),
                    "delta rule gradients");
}

ssd_status ssd_bc_norm(const ssd_bc_norm_problem *p, const void *B, const void *C,
                       const float *b_weight, const float *c_weight, const int32_t *positions,
                       const float *freqs, void *b_out, void *c_out, void *stream) {
  ssd::BcNormArgs a{};
  ssd_status st = check_bc_norm(p, false, positions && freqs, &a);
  if (st != SSD_OK) return st;
  if (p->tokens == 0) return SSD_OK;
  if (!B || !C || !b_out || !c_out)
    return fail(SSD_ERR_INVALID_ARG, "B, C and the outputs must be non-NULL");
  if (!aligned16(B) || !aligned16(C) || !aligned16(b_out) || !aligned16(c_out))
    return fail(SSD_ERR_INVALID_ARG, "B, C and the outputs must be 16-byte aligned");
  a.in[0] = B;
  a.in[1] = C;
  a.out[0] = b_out;
  a.out[1] = c_out;
  a.w[0] = b_weight;
  a.w[1] = c_weight;
  a.pos = positions;
  a.freqs = freqs;
  const int blocks = ssd::bc_norm_geometry(a, false);
  return hip_result(ssd::launch_bc_norm(a, false, blocks, p->dtype == SSD_DTYPE_BF16, nullptr,
                                        nullptr, static_cast<hipStream_t>(stream)), "norm");
}

ssd_status ssd_bc_norm_backward_workspace_size(const ssd_bc_norm_problem *p, size_t *bytes) {
  ssd::BcNormArgs a{};
  ssd_status st = check_bc_norm(p, true, p && p->rotary_dim > 0, &a);
  if (st != SSD_OK) return st;
  if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)ssd::bc_norm_geometry(a, true) * 2 * a.N * sizeof(float);
  return SSD_OK;
}

ssd_status ssd_bc_norm_backward(const ssd_bc_norm_problem *p, const void *db_out,
                                const void *dc_out, const void *B, const void *C,
                                const float *b_weight, const float *c_weight,
                                const int32_t *positions, const float *freqs, void *dB, void *dC,
                                float *db_weight, float *dc_weight, void *workspace,
                                size_t workspace_bytes, void *stream) {
  ssd::BcNormArgs a{};
  ssd_status st = check_bc_norm(p, true, positions && freqs, &a);
  if (st != SSD_OK) return st;
  const bool sums = db_weight || dc_weight;
  if (p->tokens == 0 && !sums) return SSD_OK;
  const int blocks = ssd::bc_norm_geometry(a, true);
  if (p->tokens > 0) {
    if (!db_out || !dc_out || !B || !C || !dB || !dC)
      return fail(SSD_ERR_INVALID_ARG, "B, C and the gradients must be non-NULL");
    if (!aligned16(B) || !aligned16(C) || !aligned16(db_out) || !aligned16(dc_out) ||
        !aligned16(dB) || !aligned16(dC))
      return fail(SSD_ERR_INVALID_ARG, "B, C and the gradients must be 16-byte aligned");
  }
  if (sums) {
    st = check_workspace(workspace, workspace_bytes, (size_t)blocks * 2 * a.N * sizeof(float));
    if (st != SSD_OK) return st;
    a.part = static_cast<float *>(workspace);
  }
  a.in[0] = B;
  a.in[1] = C;
  a.dout[0] = db_out;
  a.dout[1] = dc_out;
  a.out[0] = dB;
  a.out[1] = dC;
  a.w[0] = b_weight;
  a.w[1] = c_weight;
  a.pos = positions;
  a.freqs = freqs;
  return hip_result(ssd::launch_bc_norm(a, true, blocks, p->dtype == SSD_DTYPE_BF16, db_weight,
                                        dc_weight, static_cast<hipStream_t>(stream)),
                    "norm backward");
}

}  // extern "C"
