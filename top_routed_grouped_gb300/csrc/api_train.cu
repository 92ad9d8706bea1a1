// C ABI of the end of a training step (declarations and contracts in
// include/moe.h): argument validation and the launch of each entry point.
// No device memory is allocated here.
#include <math.h>

#include <algorithm>
#include <vector>

#include "../../include/moe.h"
#include "common.cuh"
#include "kernels.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

using namespace moe;

static int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

static bool type_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }
static int type_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
static bool there(const void *p, int es) { return p && ((uintptr_t)p % es) == 0; }
static bool stride_ok(int64_t ld, int64_t n) { return ld == 0 || (ld >= n && ld < ((int64_t)1 << 40)); }

static int workspace_status(const void *ws, size_t have, size_t need) {
  if (!need) return MOE_OK;
  if (have < need) return MOE_ERR_WORKSPACE;
  return ws && ((uintptr_t)ws & 255) == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// ---------------------------------------------------------------- linear_ce
// What can be told without the buffers.
static int ce_sizes(const moe_linear_ce_args_t *a) {
  if (!a || a->T < 0 || a->D <= 0 || a->V <= 0 || !type_ok(a->dtype) || !type_ok(a->dweight_dtype) || a->reserved)
    return MOE_ERR_INVALID_ARG;
  if (a->dweight_dtype != a->dtype && a->dweight_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if ((a->accumulate & ~1) || (a->targets64 & ~1) || (a->accumulate && a->dweight_dtype != MOE_F32)) return MOE_ERR_INVALID_ARG;
  if (!isfinite(a->scale) || !isfinite(a->z_loss) || a->z_loss < 0.f) return MOE_ERR_INVALID_ARG;
  if (!stride_ok(a->ld_hidden, a->D) || !stride_ok(a->ld_weight, a->D) || !stride_ok(a->ld_dhidden, a->D))
    return MOE_ERR_INVALID_ARG;
  return a->T > CE_MAX_T || a->D > CE_MAX_D || a->V > CE_MAX_V ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

static CeArgs ce_args(const moe_linear_ce_args_t *a) {
  CeArgs r = {};
  r.T = a->T;
  r.D = a->D;
  r.V = a->V;
  r.f32 = a->dtype == MOE_F32;
  r.gf32 = a->dweight_dtype == MOE_F32;
  r.accumulate = a->accumulate;
  r.targets64 = a->targets64;
  r.scale = a->scale;
  r.z_loss = a->z_loss;
  r.ignore_index = a->ignore_index;
  r.ld_h = a->ld_hidden ? a->ld_hidden : a->D;
  r.ld_w = a->ld_weight ? a->ld_weight : a->D;
  r.ld_dh = a->ld_dhidden ? a->ld_dhidden : a->D;
  r.hidden = a->hidden;
  r.weight = a->weight;
  r.targets = a->targets;
  r.dloss = a->dloss;
  r.loss = a->loss;
  r.lse = a->lse;
  r.dh = a->dhidden;
  r.dw = a->dweight;
  return r;
}

MOE_API size_t moe_linear_ce_workspace_size(const moe_linear_ce_args_t *a, int32_t call) {
  if (ce_sizes(a) != MOE_OK || call < MOE_CE_LOSS || call > MOE_CE_STEP || a->T == 0) return 0;
  return ce_scratch_bytes(ce_args(a), call);
}

static int ce_run(const moe_linear_ce_args_t *a, int mode, void *ws, size_t ws_bytes, void *stream) {
  int rc = ce_sizes(a);
  if (rc != MOE_OK) return rc;
  const int e = type_size(a->dtype);
  if ((mode & CE_GRAD) && !there(a->dweight, type_size(a->dweight_dtype))) return MOE_ERR_INVALID_ARG;
  if (a->T > 0) {
    if (!there(a->hidden, e) || !there(a->weight, e) || !there(a->targets, a->targets64 ? 8 : 4)) return MOE_ERR_INVALID_ARG;
    if ((mode & CE_LOSS) && !there(a->loss, 4)) return MOE_ERR_INVALID_ARG;
    if ((mode & CE_GRAD) && (!there(a->dhidden, e) || !there(a->dloss, 4))) return MOE_ERR_INVALID_ARG;
    if (mode == (CE_LOSS | CE_GRAD) ? ((uintptr_t)a->lse & 3) != 0 : !there(a->lse, 4)) return MOE_ERR_INVALID_ARG;
  }
  if ((rc = workspace_status(ws, ws_bytes, moe_linear_ce_workspace_size(a, mode))) != MOE_OK) return rc;
  int *status = device_status_ptr();
  if (!status) return MOE_ERR_CUDA;
  return cuda_status(launch_linear_ce(ce_args(a), mode, ws, status, (cudaStream_t)stream));
}

MOE_API int moe_linear_ce(const moe_linear_ce_args_t *a, void *ws, size_t ws_bytes, void *stream) {
  return ce_run(a, CE_LOSS, ws, ws_bytes, stream);
}
MOE_API int moe_linear_ce_backward(const moe_linear_ce_args_t *a, void *ws, size_t ws_bytes, void *stream) {
  return ce_run(a, CE_GRAD, ws, ws_bytes, stream);
}
MOE_API int moe_linear_ce_step(const moe_linear_ce_args_t *a, void *ws, size_t ws_bytes, void *stream) {
  return ce_run(a, CE_LOSS | CE_GRAD, ws, ws_bytes, stream);
}

// ---------------------------------------------------------------- gradients
static int grads_list(const moe_grads_args_t *a) {
  if (!a || a->n < 0 || a->reserved || (a->n > 0 && (!a->in || !a->numel || !a->dtype))) return MOE_ERR_INVALID_ARG;
  if (a->n > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  int64_t total = 0;
  for (int i = 0; i < a->n; ++i) {
    if (a->numel[i] < 0 || !type_ok(a->dtype[i])) return MOE_ERR_INVALID_ARG;
    if (a->numel[i] > ((int64_t)1 << 42) || (total += a->numel[i]) > ((int64_t)1 << 42)) return MOE_ERR_UNSUPPORTED;
    if (a->numel[i] && !there(a->in[i], type_size(a->dtype[i]))) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

// Outputs: there, and none over another one or over another tensor's input.
static int grads_outputs(const moe_grads_args_t *a) {
  if (!(a->max_norm >= 0.f) || !isfinite(a->max_norm) || !(a->eps >= 0.f) || !isfinite(a->eps)) return MOE_ERR_INVALID_ARG;
  if (a->n > 0 && (!a->out || !a->odtype)) return MOE_ERR_INVALID_ARG;
  struct Range {
    uintptr_t from, to;
    bool write;
  };
  try {
    std::vector<Range> r;
    r.reserve(2 * (size_t)a->n);
    for (int i = 0; i < a->n; ++i) {
      if (!type_ok(a->odtype[i])) return MOE_ERR_INVALID_ARG;
      if (!a->numel[i]) continue;
      if (!there(a->out[i], type_size(a->odtype[i]))) return MOE_ERR_INVALID_ARG;
      const uintptr_t o = (uintptr_t)a->out[i], in = (uintptr_t)a->in[i];
      r.push_back({o, o + (uintptr_t)a->numel[i] * type_size(a->odtype[i]), true});
      if (o != in || a->odtype[i] != a->dtype[i])
        r.push_back({in, in + (uintptr_t)a->numel[i] * type_size(a->dtype[i]), false});
    }
    std::sort(r.begin(), r.end(), [](const Range &x, const Range &y) { return x.from < y.from; });
    uintptr_t any = 0, written = 0;  // where the ranges before end
    for (const Range &x : r) {
      if (x.from < (x.write ? any : written)) return MOE_ERR_INVALID_ARG;
      any = std::max(any, x.to);
      if (x.write) written = std::max(written, x.to);
    }
  } catch (...) {  // no host memory for the list
    return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

static GradList grad_list(const moe_grads_args_t *a) {
  return {a->n, a->in, a->out, a->numel, a->dtype, a->odtype, a->max_norm, a->eps, a->norm};
}

MOE_API size_t moe_grad_workspace_size(const moe_grads_args_t *a) {
  if (!a || a->n < 0 || a->n > (1 << 20)) return 0;
  GradList g = {};
  g.n = a->n;
  return (size_t)round_up((int64_t)grad_scratch_bytes(g), 256);
}

static int grads_run(const moe_grads_args_t *a, int mode, void *ws, size_t ws_bytes, void *stream) {
  int rc = grads_list(a);
  if (rc != MOE_OK) return rc;
  if ((mode & GRAD_SCALE) && (rc = grads_outputs(a)) != MOE_OK) return rc;
  if (!there(a->norm, 4)) return MOE_ERR_INVALID_ARG;
  if ((mode & GRAD_NORM) && (rc = workspace_status(ws, ws_bytes, moe_grad_workspace_size(a))) != MOE_OK) return rc;
  return cuda_status(launch_grads(grad_list(a), mode, ws, (cudaStream_t)stream));
}

MOE_API int moe_grad_norm(const moe_grads_args_t *a, void *ws, size_t ws_bytes, void *stream) {
  return grads_run(a, GRAD_NORM, ws, ws_bytes, stream);
}
MOE_API int moe_grad_clip(const moe_grads_args_t *a, void *ws, size_t ws_bytes, void *stream) {
  return grads_run(a, GRAD_NORM | GRAD_SCALE, ws, ws_bytes, stream);
}
MOE_API int moe_grad_scale(const moe_grads_args_t *a, void *stream) {
  return grads_run(a, GRAD_SCALE, nullptr, 0, stream);
}
