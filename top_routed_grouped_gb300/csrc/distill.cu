// Distillation from a teacher's top logits: loss, gradient, and both in one
// call (contracts with moe_distill in moe.h).
//
// One CTA per row.  Loss: one pass over the row with a running maximum and
// sum per thread, joined in a fixed order.  Gradient: one pass that writes
// P q, then the teacher's few places are written again with P q - p.
// Exponents are differences of logits before they are scaled, so that rows at
// the type's lowest value do not overflow.
#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"

namespace moe {

constexpr int DS_THREADS = 512, DS_WARPS = DS_THREADS / 32;
constexpr float DS_LOG2E = 1.4426950408889634f;

__device__ inline float ds_neg_inf() { return __int_as_float(0xff800000); }

// Max of the logits and sum of 2^(k (. - max)); (-inf, 0) is empty.
struct DsStat {
  float m, s;
};
__device__ inline DsStat ds_join(DsStat a, DsStat b, float k) {
  const float m = fmaxf(a.m, b.m);
  if (m == ds_neg_inf()) return {m, a.s + b.s};
  return {m, a.s * exp2f((a.m - m) * k) + b.s * exp2f((b.m - m) * k)};
}
template <typename F, typename T>
__device__ inline T ds_block(T v, T *buf, F op) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  buf[threadIdx.x] = v;
  __syncthreads();
  (void)warp;
  (void)lane;
  for (int n = DS_THREADS / 2; n; n >>= 1) {
    if ((int)threadIdx.x < n) buf[threadIdx.x] = op(buf[threadIdx.x], buf[threadIdx.x + n]);
    __syncthreads();
  }
  return buf[0];
}

template <typename T>
__device__ inline DsStat ds_row_stat(const T *z, int V, float k) {
  DsStat a = {ds_neg_inf(), 0.f};
  for (int i = threadIdx.x; i < V; i += DS_THREADS) {
    const float x = Elem<T>::load(z + i);
    if (x > a.m) {
      a.s = fmaf(a.s, exp2f((a.m - x) * k), 1.f);
      a.m = x;
    } else if (!(x == ds_neg_inf())) {
      a.s += exp2f((x - a.m) * k);  // NaN stays
    }
  }
  return a;
}

// Teacher slot of this thread: p and log p (0 where there is none); returns P.
struct DsTeacher {
  int id;
  float p, logp, total;
};
__device__ inline DsTeacher ds_teacher(const DistillArgs &a, int64_t t, float *buf, int *status) {
  DsTeacher r = {-1, 0.f, 0.f, 0.f};
  float x = ds_neg_inf();
  if ((int)threadIdx.x < a.K) {
    const int id = a.t_ids[t * a.K + threadIdx.x];
    if (id < -1 || id >= a.V) record_status(status, STATUS_BAD_TEACHER_ID);
    if (id >= 0 && id < a.V) {
      x = a.t_logits[t * a.K + threadIdx.x] * a.inv_tau;
      if (!(x == ds_neg_inf())) r.id = id;
    }
  }
  float c;
  if (a.t_lse) {
    c = a.t_lse[t];
  } else {
    const float m = ds_block(x, buf, [](float u, float v) { return fmaxf(u, v); });
    const float e = r.id >= 0 ? expf(x - m) : 0.f;
    const float s = ds_block(e, buf, [](float u, float v) { return u + v; });
    c = m + logf(s);
  }
  if (r.id >= 0) {
    r.logp = x - c;
    r.p = expf(r.logp);
  }
  r.total = ds_block(r.p, buf, [](float u, float v) { return u + v; });
  return r;
}

// mode: 1 loss and lse, 2 gradient from lse, 3 loss and gradient.
template <typename T>
__global__ void __launch_bounds__(DS_THREADS) distill_kernel(const DistillArgs a, int mode, int *status) {
  __shared__ float buf[DS_THREADS];
  __shared__ DsStat sbuf[DS_THREADS];
  __shared__ int ids[256];
  __shared__ float ps[256];
  griddep_launch();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const T *z = (const T *)a.logits + t * a.ld_logits;
  T *dz = (T *)a.dlogits + t * a.ld_dlogits;
  const float k = a.inv_tau * DS_LOG2E;
  const DsTeacher te = ds_teacher(a, t, buf, status);
  const int any = __syncthreads_or(te.id >= 0);
  float lse;
  if (mode & 1) {
    DsStat st = ds_block(ds_row_stat(z, a.V, k), sbuf, [k](DsStat u, DsStat v) { return ds_join(u, v, k); });
    const float logs = logf(st.s);
    lse = fmaf(st.m, a.inv_tau, logs);
    if (threadIdx.x == 0 && a.lse) a.lse[t] = lse;
    float l = 0.f;
    if (te.id >= 0 && te.p != 0.f)
      l = te.p * (te.logp - fmaf(Elem<T>::load(z + te.id) - st.m, a.inv_tau, -logs));
    l = ds_block(l, buf, [](float u, float v) { return u + v; });
    if (lse == ds_neg_inf()) l = -lse;
    if (threadIdx.x == 0) a.loss[t] = any ? a.scale * l : 0.f;
  } else {
    lse = a.lse[t];
  }
  if (!(mode & 2)) return;
  const float w = a.weight[t] * a.scale * a.inv_tau;
  const bool zero = !any || w == 0.f || lse == ds_neg_inf();
  float fix = 0.f;
  if (te.id >= 0) {
    ids[threadIdx.x] = te.id;
    ps[threadIdx.x] = te.p;
  } else if ((int)threadIdx.x < a.K) {
    ids[threadIdx.x] = -1;
  }
  __syncthreads();
  bool first = te.id >= 0;
  if (te.id >= 0 && !zero) {
    float p = 0.f;
    for (int j = 0; j < a.K; ++j)
      if (ids[j] == te.id) {
        p += ps[j];
        if (j < (int)threadIdx.x) first = false;
      }
    fix = w * (te.total * expf(fmaf(Elem<T>::load(z + te.id), a.inv_tau, -lse)) - p);
  }
  __syncthreads();  // dz may be z
  for (int i = threadIdx.x; i < a.V; i += DS_THREADS) {
    float g = 0.f;
    if (!zero) g = w * te.total * expf(fmaf(Elem<T>::load(z + i), a.inv_tau, -lse));
    dz[i] = Elem<T>::from_f32(g);
  }
  __syncthreads();
  if (first && !zero) dz[te.id] = Elem<T>::from_f32(fix);
}

cudaError_t launch_distill(const DistillArgs &a, int mode, int *status, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  if (a.f32) return launch_pdl(distill_kernel<float>, dim3((unsigned)a.T), dim3(DS_THREADS), 0, stream, a, mode, status);
  return launch_pdl(distill_kernel<__nv_bfloat16>, dim3((unsigned)a.T), dim3(DS_THREADS), 0, stream, a, mode, status);
}

}  // namespace moe
