// C ABI of the operators around the layer (declarations and contracts in
// include/moe.h): argument validation and the launch of each entry point.
// No device memory is allocated here.
#include <math.h>

#include "../../include/moe.h"
#include "common.cuh"
#include "kernels.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

using namespace moe;

static int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

static bool type_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }
static int type_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// A buffer that the call uses: present and aligned to its element type.
static bool there(const void *p, int es) { return p && ((uintptr_t)p % es) == 0; }
// One that it uses if it is given.
static bool maybe(const void *p, int es) { return !p || ((uintptr_t)p % es) == 0; }
// A row stride: 0 (dense) or at least the row.
static bool stride_ok(int64_t ld, int64_t n) { return ld == 0 || (ld >= n && ld < ((int64_t)1 << 40)); }

static int workspace_status(const void *ws, size_t have, size_t need) {
  if (!need) return MOE_OK;
  if (have < need) return MOE_ERR_WORKSPACE;
  return ws && ((uintptr_t)ws & 255) == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// ---------------------------------------------------------------- block_norm
// What can be told without the buffers.
static int norm_sizes(const moe_norm_args_t *a) {
  if (!a || a->T < 0 || a->H <= 0 || !type_ok(a->dtype) || !type_ok(a->wdtype) || !type_ok(a->rdtype) || a->reserved)
    return MOE_ERR_INVALID_ARG;
  if (a->rdtype != a->dtype && a->rdtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (a->wdtype != a->dtype && a->wdtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (a->gate_kind < MOE_GATE_NONE || a->gate_kind > MOE_GATE_ELEMENT) return MOE_ERR_INVALID_ARG;
  if (!isfinite(a->scale) || !isfinite(a->weight_offset) || !(a->eps >= 0.f) || !isfinite(a->eps)) return MOE_ERR_INVALID_ARG;
  for (int64_t ld : {a->ld_r, a->ld_y, a->ld_gate, a->ld_r_out, a->ld_h, a->ld_dr_out, a->ld_dh, a->ld_dr, a->ld_dy, a->ld_dgate})
    if (!stride_ok(ld, a->H)) return MOE_ERR_INVALID_ARG;
  return a->H > NORM_MAX_H ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

static int norm_dims(const moe_norm_args_t *a) {
  const int rc = norm_sizes(a);
  if (rc == MOE_ERR_INVALID_ARG) return rc;
  if (a->T > 0 && !a->y && (a->w_post || a->gate_kind != MOE_GATE_NONE || !a->w_pre)) return MOE_ERR_INVALID_ARG;
  return rc;
}

static int norm_inputs(const moe_norm_args_t *a) {
  const int e = type_size(a->dtype), w = type_size(a->wdtype);
  bool ok = maybe(a->y, e) && maybe(a->w_post, w) && maybe(a->w_pre, w);
  if (a->gate_kind != MOE_GATE_NONE)
    ok = ok && there(a->gate, a->gate_kind == MOE_GATE_TOKEN ? 4 : a->gate_kind == MOE_GATE_CHANNEL ? w : e);
  return ok ? MOE_OK : MOE_ERR_INVALID_ARG;
}

static NormArgs norm_args(const moe_norm_args_t *a) {
  auto ld = [&](int64_t v) { return v ? v : (int64_t)a->H; };
  NormArgs r = {};
  r.T = a->T;
  r.H = a->H;
  r.f32 = a->dtype == MOE_F32;
  r.rf32 = a->rdtype == MOE_F32;
  r.wf32 = a->wdtype == MOE_F32;
  r.gate_kind = a->gate_kind;
  r.scale = a->scale;
  r.eps = a->eps;
  r.offset = a->weight_offset;
  r.ld_r = ld(a->ld_r);
  r.ld_y = ld(a->ld_y);
  r.ld_gate = ld(a->ld_gate);
  r.ld_r_out = ld(a->ld_r_out);
  r.ld_h = ld(a->ld_h);
  r.ld_dr_out = ld(a->ld_dr_out);
  r.ld_dh = ld(a->ld_dh);
  r.ld_dr = ld(a->ld_dr);
  r.ld_dy = ld(a->ld_dy);
  r.ld_dgate = ld(a->ld_dgate);
  r.y = a->y;
  r.w_post = a->w_post;
  r.w_pre = a->w_pre;
  r.gate = a->gate_kind == MOE_GATE_NONE ? nullptr : a->gate;
  return r;
}

static NormArgs norm_fwd_args(const moe_norm_args_t *a) {
  NormArgs r = norm_args(a);
  r.r = a->r;
  r.r_out = a->y ? a->r_out : nullptr;
  r.h = a->w_pre ? a->h : nullptr;
  return r;
}

static NormArgs norm_bwd_args(const moe_norm_args_t *a) {
  NormArgs r = norm_args(a);
  r.r_out = a->w_pre ? a->r_out : nullptr;
  r.dr_out = a->dr_out;
  r.dh = a->w_pre ? a->dh : nullptr;
  r.dr = a->w_pre ? a->dr : nullptr;  // without the second norm it is dr_out
  r.dy = a->y ? a->dy : nullptr;
  r.dw_post = a->w_post ? a->dw_post : nullptr;
  r.dw_pre = a->w_pre ? a->dw_pre : nullptr;
  r.dgate = a->gate_kind == MOE_GATE_NONE ? nullptr : a->dgate;
  return r;
}

MOE_API int moe_block_norm(const moe_norm_args_t *a, void *stream) {
  int rc = norm_dims(a);
  if (rc != MOE_OK || a->T == 0) return rc;
  if ((rc = norm_inputs(a)) != MOE_OK) return rc;
  const int e = type_size(a->dtype), r = type_size(a->rdtype);
  if (!there(a->r, r) || (a->y && !there(a->r_out, r)) || (a->w_pre && !there(a->h, e))) return MOE_ERR_INVALID_ARG;
  int *status = device_status_ptr();
  if (!status) return MOE_ERR_CUDA;
  return cuda_status(launch_block_norm(norm_fwd_args(a), status, (cudaStream_t)stream));
}

MOE_API size_t moe_block_norm_workspace_size(const moe_norm_args_t *a) {
  if (norm_sizes(a) != MOE_OK) return 0;
  return (size_t)round_up((int64_t)block_norm_scratch_bytes(norm_args(a)), 256);
}

MOE_API int moe_block_norm_backward(const moe_norm_args_t *a, void *ws, size_t ws_bytes, void *stream) {
  int rc = norm_dims(a);
  if (rc != MOE_OK) return rc;
  const int e = type_size(a->dtype), r = type_size(a->rdtype);
  if ((a->w_post && !there(a->dw_post, 4)) || (a->w_pre && !there(a->dw_pre, 4))) return MOE_ERR_INVALID_ARG;
  if (a->gate_kind == MOE_GATE_CHANNEL && !there(a->dgate, 4)) return MOE_ERR_INVALID_ARG;
  if (a->T > 0) {
    if ((rc = norm_inputs(a)) != MOE_OK) return rc;
    if (!maybe(a->dr_out, r) || (!a->dr_out && !a->w_pre)) return MOE_ERR_INVALID_ARG;
    if (a->w_pre && (!there(a->r_out, r) || !there(a->dh, e) || !there(a->dr, r))) return MOE_ERR_INVALID_ARG;
    if (a->y && !there(a->dy, e)) return MOE_ERR_INVALID_ARG;
    if (a->gate_kind != MOE_GATE_NONE && !there(a->dgate, a->gate_kind == MOE_GATE_ELEMENT ? e : 4))
      return MOE_ERR_INVALID_ARG;
  }
  const NormArgs n = norm_bwd_args(a);
  if ((rc = workspace_status(ws, ws_bytes, (size_t)round_up((int64_t)block_norm_scratch_bytes(n), 256))) != MOE_OK) return rc;
  int *status = device_status_ptr();
  if (!status) return MOE_ERR_CUDA;
  return cuda_status(launch_block_norm_bwd(n, ws, status, (cudaStream_t)stream));
}

// ---------------------------------------------------------------- embed
static int embed_dims(const moe_embed_args_t *a) {
  if (!a || a->T < 0 || a->H <= 0 || a->V <= 0 || !type_ok(a->dtype) || !type_ok(a->odtype)) return MOE_ERR_INVALID_ARG;
  if (a->odtype != a->dtype && a->odtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if ((a->ids64 & ~1) || (a->accumulate & ~1) || !isfinite(a->scale)) return MOE_ERR_INVALID_ARG;
  if (!stride_ok(a->ld_table, a->H) || !stride_ok(a->ld_out, a->H)) return MOE_ERR_INVALID_ARG;
  if (a->T > 0 && !there(a->ids, a->ids64 ? 8 : 4)) return MOE_ERR_INVALID_ARG;
  return a->V < (1 << 20) && a->T < 0x7fffff00 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

static EmbedArgs embed_args(const moe_embed_args_t *a) {
  EmbedArgs r = {};
  r.T = a->T;
  r.H = a->H;
  r.V = a->V;
  r.f32 = a->dtype == MOE_F32;
  r.of32 = a->odtype == MOE_F32;
  r.ids64 = a->ids64;
  r.accumulate = a->accumulate;
  r.scale = a->scale;
  r.padding_id = a->padding_id;
  r.ld_table = a->ld_table ? a->ld_table : a->H;
  r.ld_out = a->ld_out ? a->ld_out : a->H;
  r.ids = a->ids;
  r.table = a->table;
  r.out = a->out;
  r.dout = a->dout;
  r.dtable = a->dtable;
  return r;
}

MOE_API int moe_embed(const moe_embed_args_t *a, void *stream) {
  int rc = embed_dims(a);
  if (rc != MOE_OK || a->T == 0) return rc;
  if (!there(a->table, type_size(a->dtype)) || !there(a->out, type_size(a->odtype))) return MOE_ERR_INVALID_ARG;
  int *status = device_status_ptr();
  if (!status) return MOE_ERR_CUDA;
  return cuda_status(launch_embed(embed_args(a), status, (cudaStream_t)stream));
}

MOE_API size_t moe_embed_workspace_size(const moe_embed_args_t *a) {
  if (!a) return 0;
  moe_embed_args_t b = *a;
  b.ids = (const void *)16;  // sizes do not depend on the buffers
  if (embed_dims(&b) != MOE_OK || b.T == 0) return 0;
  return (size_t)round_up((int64_t)embed_scratch_bytes(embed_args(&b)), 256);
}

MOE_API int moe_embed_backward(const moe_embed_args_t *a, void *ws, size_t ws_bytes, void *stream) {
  int rc = embed_dims(a);
  if (rc != MOE_OK) return rc;
  if (!there(a->dtable, 4) || (a->T > 0 && !there(a->dout, type_size(a->odtype)))) return MOE_ERR_INVALID_ARG;
  if ((rc = workspace_status(ws, ws_bytes, moe_embed_workspace_size(a))) != MOE_OK) return rc;
  int *status = device_status_ptr();
  if (!status) return MOE_ERR_CUDA;
  return cuda_status(launch_embed_bwd(embed_args(a), ws, status, (cudaStream_t)stream));
}

// ---------------------------------------------------------------- distill
static int distill_run(const moe_distill_args_t *a, int mode, void *stream) {
  if (!a || a->T < 0 || a->V <= 0 || a->K <= 0 || !type_ok(a->dtype)) return MOE_ERR_INVALID_ARG;
  if (!(a->temperature > 0.f) || !isfinite(a->temperature) || !isfinite(a->scale)) return MOE_ERR_INVALID_ARG;
  if (!isfinite(1.f / a->temperature) || !stride_ok(a->ld_logits, a->V) || !stride_ok(a->ld_dlogits, a->V))
    return MOE_ERR_INVALID_ARG;
  if (a->K > DISTILL_MAX_K || a->T > DISTILL_MAX_T || a->V > DISTILL_MAX_V) return MOE_ERR_UNSUPPORTED;
  if (a->T == 0) return MOE_OK;
  const int e = type_size(a->dtype);
  if (!there(a->logits, e) || !there(a->t_ids, 4) || !there(a->t_logits, 4) || !maybe(a->t_lse, 4) || !maybe(a->lse, 4))
    return MOE_ERR_INVALID_ARG;
  if ((mode & DISTILL_LOSS) && !there(a->loss, 4)) return MOE_ERR_INVALID_ARG;
  if ((mode & DISTILL_GRAD) && (!there(a->weight, 4) || !there(a->dlogits, e))) return MOE_ERR_INVALID_ARG;
  if (mode != (DISTILL_LOSS | DISTILL_GRAD) && !a->lse) return MOE_ERR_INVALID_ARG;
  DistillArgs r = {};
  r.T = a->T;
  r.V = a->V;
  r.K = a->K;
  r.f32 = a->dtype == MOE_F32;
  r.inv_tau = 1.f / a->temperature;
  r.scale = a->scale;
  r.ld_logits = a->ld_logits ? a->ld_logits : a->V;
  r.ld_dlogits = a->ld_dlogits ? a->ld_dlogits : a->V;
  r.logits = a->logits;
  r.t_ids = a->t_ids;
  r.t_logits = a->t_logits;
  r.t_lse = a->t_lse;
  r.weight = a->weight;
  r.loss = a->loss;
  r.lse = a->lse;
  r.dlogits = a->dlogits;
  if ((mode & DISTILL_GRAD) && r.dlogits == r.logits && r.ld_dlogits != r.ld_logits) return MOE_ERR_INVALID_ARG;
  int *status = device_status_ptr();
  if (!status) return MOE_ERR_CUDA;
  return cuda_status(launch_distill(r, mode, status, (cudaStream_t)stream));
}

MOE_API int moe_distill(const moe_distill_args_t *a, void *stream) { return distill_run(a, DISTILL_LOSS, stream); }
MOE_API int moe_distill_backward(const moe_distill_args_t *a, void *stream) { return distill_run(a, DISTILL_GRAD, stream); }
MOE_API int moe_distill_step(const moe_distill_args_t *a, void *stream) {
  return distill_run(a, DISTILL_LOSS | DISTILL_GRAD, stream);
}
