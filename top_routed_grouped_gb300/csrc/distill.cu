// Distillation from a teacher's top logits: loss, gradient, and both in one
// call (contracts with moe_distill in moe.h).
//
//   lse = m / tau + log s,  m = max z,  s = sum exp((z - m) / tau)
//   dz  = w (P exp((z - m) / tau) / s - p at the teacher's ids)
//
// A row belongs to a cluster of CTAs (one, where it is short) and is cut into
// 16-byte units; every thread holds its units in registers, so that the step
// reads a row once and writes its gradient from what it still holds.  The
// maximum is taken before the exponentials, in the thread's own units first,
// and the (max, sum) pairs of threads, warps and CTAs are joined in a fixed
// order; the CTAs exchange theirs through distributed shared memory.  The
// shape of a launch goes by the vocabulary alone, so a row's results do not
// depend on the batch.  Rows too long for the registers of a cluster are read
// in groups of units, twice.  The teacher's places are few: they are written
// again, with their p subtracted, after the dense pass.
//
// Exponents are differences of logits before they are scaled, so that rows at
// the type's lowest value do not overflow.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"
#include "umma.cuh"

namespace moe {

constexpr int DS_MAX_THREADS = 512;
constexpr float DS_LOG2E = 1.4426950408889634f;

__device__ inline float ds_neg_inf() { return __int_as_float(0xff800000); }

// 2^x in hardware (two units in the last place; results below 2^-126 are 0).
__device__ inline float ds_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two FP32 lanes in one instruction.
struct DsPair {
  uint64_t v;
  __device__ inline DsPair() {}
  __device__ inline DsPair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ inline void get(float &a, float &b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ inline DsPair ds_add2(DsPair a, DsPair b) {
  DsPair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ inline DsPair ds_mul2(DsPair a, DsPair b) {
  DsPair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ inline DsPair ds_fma2(DsPair a, DsPair b, DsPair c) {
  DsPair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// Keeps the compiler from holding what was unpacked from `v` beside it.
__device__ inline void ds_opaque(uint4 &v) { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }

__device__ inline float ds_warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, d));
  return v;
}
__device__ inline float ds_warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
  return v;
}

// Max of logits and sum of 2^(k (. - max)); (-inf, 0) is empty.
struct DsStat {
  float m, s;
};
// The pairs of a warp's lanes as one.
__device__ inline DsStat ds_warp_join(DsStat a, float k) {
  const float m = ds_warp_max(a.m);
  const float base = m == ds_neg_inf() ? 0.f : m;
  return {m, ds_warp_sum(a.s * exp2f((a.m - base) * k))};
}

// Elements n.. of the 2 N elements of (lo, hi), sh = n sizeof(T) bytes.
__device__ inline uint4 ds_funnel(const uint4 &lo, const uint4 &hi, int sh) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (sh & 8)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (sh & 4)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  if (sh & 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Units of a row: unit u holds elements u N .. u N + N - 1.  A row may start
// `off` elements past a 16-byte boundary; its units are then put together from
// the two aligned pieces that they lie in, so that what a thread holds does
// not depend on where the row stands.
template <typename T>
struct DsUnit {
  static constexpr int N = 16 / sizeof(T);
  // What is not of the row reads as -inf.
  static __device__ inline uint4 load(const T *row, int off, int u, int V) {
    const int i = u * N;
    const T *p = row + i - off;  // on a boundary
    if (off == 0 && i + N <= V) return __ldcs((const uint4 *)p);
    if (off != 0 && i >= off && i - off + 2 * N <= V)
      return ds_funnel(*(const uint4 *)p, *(const uint4 *)(p + N), off * (int)sizeof(T));
    uint4 v;
    T *e = (T *)&v;
#pragma unroll
    for (int j = 0; j < N; ++j) e[j] = i + j < V ? row[i + j] : Elem<T>::from_f32(ds_neg_inf());
    return v;
  }
  // The whole warp: lane l holds unit u of consecutive ones.
  static __device__ inline void store(T *row, int off, int u, int V, const float (&g)[N]) {
    uint4 v;
    T *e = (T *)&v;
#pragma unroll
    for (int j = 0; j < N; ++j) e[j] = Elem<T>::from_f32(g[j]);
    const int i = u * N, lane = threadIdx.x & 31;
    int from = 0, to = N;  // what is left to write element by element
    if (off == 0) {
      if (i + N <= V) {
        __stcs((uint4 *)(row + i), v);
        from = N;
      }
    } else {
      // The aligned piece that ends in this unit: the tail of the unit before
      // it and N - off of its own elements.
      uint4 b;
      b.x = __shfl_up_sync(FULL_MASK, v.x, 1);
      b.y = __shfl_up_sync(FULL_MASK, v.y, 1);
      b.z = __shfl_up_sync(FULL_MASK, v.z, 1);
      b.w = __shfl_up_sync(FULL_MASK, v.w, 1);
      if (lane > 0 && i - off + N <= V) {
        __stcs((uint4 *)(row + i - off), ds_funnel(b, v, (N - off) * (int)sizeof(T)));
        from = N - off;
      }
      // The next lane writes the rest, where there is one that does.
      if (lane < 31 && i + 2 * N - off <= V) to = N - off;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j >= from && j < to && i + j < V) row[i + j] = e[j];
  }
};

// The largest element of a unit (NaN aside).
template <typename T>
__device__ inline float ds_unit_max(const uint4 &v) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {
    const __nv_bfloat162 *h = (const __nv_bfloat162 *)&v;
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
}

__device__ inline DsStat ds_ld_cluster(uint32_t addr) {
  DsStat r;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(r.m), "=f"(r.s) : "r"(addr) : "memory");
  return r;
}

// MODE: DISTILL_LOSS, DISTILL_GRAD or both.  U: units a thread holds; groups:
// how many times U units each thread takes.
template <typename T, int MODE, int U>
__global__ void __launch_bounds__(DS_MAX_THREADS, 2)
distill_kernel(const DistillArgs a, int ctas, int groups, int *status) {
  constexpr int N = DsUnit<T>::N;
  __shared__ float sx[DISTILL_MAX_K], sz[DISTILL_MAX_K];
  __shared__ int sid[DISTILL_MAX_K];
  __shared__ DsStat wstat[32];
  __shared__ __align__(8) DsStat cstat;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = blockDim.x;
  griddep_launch();
  griddep_wait();
  const int64_t t = blockIdx.x / ctas;
  const int rank = blockIdx.x % ctas;
  const T *z = (const T *)a.logits + t * a.ld_logits;
  const int off = (int)(((uintptr_t)z / sizeof(T)) % N);
  const float k = a.inv_tau * DS_LOG2E;
  // Group g, unit j of a thread is unit first + (g U + j) threads.
  const int first = rank * groups * U * threads + threadIdx.x;

  uint4 raw[U];
  auto load = [&](int g) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      raw[j] = DsUnit<T>::load(z, off, first + (g * U + j) * threads, a.V);
  };

  // The gradient of a row that has none needs no logits.
  const float w = MODE & DISTILL_GRAD ? a.weight[t] * a.scale * a.inv_tau : 0.f;
  if (MODE & DISTILL_LOSS) load(0);

  // ---- the teacher's slots, in shared memory: id (-1: none), t / tau, the student's logit
  const int lo = rank * groups * U * threads * N, hi = lo + groups * U * threads * N;  // elements of this CTA
  int found = 0;
  for (int s = threadIdx.x; s < a.K; s += threads) {
    int id = a.t_ids[t * a.K + s];
    const float x = a.t_logits[t * a.K + s] * a.inv_tau;
    if (id < -1 || id >= a.V) record_status(status, STATUS_BAD_TEACHER_ID);
    if (id < 0 || id >= a.V || x == ds_neg_inf()) id = -1;
    sid[s] = id;
    sx[s] = id < 0 ? ds_neg_inf() : x;
    // (without a loss, logits of other CTAs may have been overwritten)
    const bool read = id >= 0 && (MODE & DISTILL_LOSS ? true : id >= lo && id < hi);
    sz[s] = read ? Elem<T>::load(z + id) : 0.f;
    found |= id >= 0;
  }

  // ---- the student's statistics
  DsStat st = {0.f, 1.f};
  float lse, logs = 0.f;
  if (MODE & DISTILL_LOSS) {
    DsStat mine = {ds_neg_inf(), 0.f};
    for (int g = 0; g < groups; ++g) {
      if (g) load(g);
      float m = mine.m;
#pragma unroll
      for (int j = 0; j < U; ++j) m = fmaxf(m, ds_unit_max<T>(raw[j]));
      const float base = m == ds_neg_inf() ? 0.f : m;
      float s = mine.s * ds_exp2((mine.m - base) * k);
      const DsPair nbase(-base, -base), kk(k, k);
      DsPair sum(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float v[N];
        ds_opaque(raw[j]);
        Vec16<T>::unpack(raw[j], v);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          float x, y;
          ds_mul2(ds_add2(DsPair(v[i], v[i + 1]), nbase), kk).get(x, y);
          sum = ds_add2(sum, DsPair(ds_exp2(x), ds_exp2(y)));
        }
        ds_opaque(raw[j]);
      }
      float s0, s1;
      sum.get(s0, s1);
      s += s0 + s1;
      mine = {m, s};
    }
    mine = ds_warp_join(mine, k);
    if (lane == 0) wstat[warp] = mine;
  }
  const int any = __syncthreads_or(found);
  if (MODE & DISTILL_LOSS) {
    st = ds_warp_join(lane < threads / 32 ? wstat[lane] : DsStat{ds_neg_inf(), 0.f}, k);
    if (ctas > 1) {
      if (threadIdx.x == 0) cstat = st;
      umma::cluster_sync();
      st = ds_warp_join(lane < ctas ? ds_ld_cluster(umma::mapa_shared(&cstat, lane < ctas ? lane : 0)) : DsStat{ds_neg_inf(), 0.f}, k);
    }
    logs = logf(st.s);
    lse = st.m == ds_neg_inf() && !(st.s != st.s) ? ds_neg_inf() : fmaf(st.m, a.inv_tau, logs);
  } else {
    lse = a.lse[t];
  }

  // ---- the teacher's distribution (every warp alike)
  float c, total = 0.f;
  if (a.t_lse) {
    c = a.t_lse[t];
  } else {
    float m = ds_neg_inf(), s = 0.f;
    for (int i = lane; i < a.K; i += 32) m = fmaxf(m, sx[i]);
    m = ds_warp_max(m);
    for (int i = lane; i < a.K; i += 32)
      if (sid[i] >= 0) s += expf(sx[i] - m);
    c = m + logf(ds_warp_sum(s));
  }
  for (int i = lane; i < a.K; i += 32)
    if (sid[i] >= 0) total += expf(sx[i] - c);
  total = ds_warp_sum(total);

  if ((MODE & DISTILL_LOSS) && rank == 0 && warp == 0) {
    float l = 0.f;
    for (int i = lane; i < a.K; i += 32) {
      const float logp = sx[i] - c, p = sid[i] >= 0 ? expf(logp) : 0.f;
      if (p != 0.f) l += p * (logp - fmaf(sz[i] - st.m, a.inv_tau, -logs));
    }
    l = ds_warp_sum(l);
    if (lse == ds_neg_inf()) l = -lse;
    if (lane == 0) {
      a.loss[t] = any ? a.scale * l : 0.f;
      if (a.lse) a.lse[t] = lse;
    }
  }

  if (MODE & DISTILL_GRAD) {
    T *dz = (T *)a.dlogits + t * a.ld_dlogits;
    const int doff = (int)(((uintptr_t)dz / sizeof(T)) % N);
    const bool zero = !any || w == 0.f || lse == ds_neg_inf();
    // exp((z - m) / tau - log s) with the loss's own m and s, exp(z / tau - lse) without them
    const float sub = MODE & DISTILL_LOSS ? st.m : 0.f;
    const float mul = w * total, add = (MODE & DISTILL_LOSS ? logs : lse) * -DS_LOG2E;
    const DsPair sub2(-sub, -sub), k2(k, k), add2(add, add), tau2(a.inv_tau, a.inv_tau), lse2(-lse, -lse),
        log2e2(DS_LOG2E, DS_LOG2E), mul2(mul, mul);
    auto q2 = [&](float &u, float &v) {  // P w q of two logits
      DsPair x(u, v);
      if (MODE & DISTILL_LOSS) x = ds_fma2(ds_add2(x, sub2), k2, add2);
      else x = ds_mul2(ds_fma2(x, tau2, lse2), log2e2);
      x.get(u, v);
      ds_mul2(DsPair(ds_exp2(u), ds_exp2(v)), mul2).get(u, v);
    };
    for (int g = 0; g < groups; ++g) {
      if (!zero && (!(MODE & DISTILL_LOSS) || groups > 1)) load(g);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
        if (!zero) {
          Vec16<T>::unpack(raw[j], v);
#pragma unroll
          for (int i = 0; i < N; i += 2) q2(v[i], v[i + 1]);
        }
        DsUnit<T>::store(dz, doff, first + (g * U + j) * threads, a.V, v);
      }
    }
    __syncthreads();
    if (!zero)
      for (int s = threadIdx.x; s < a.K; s += threads) {
        const int id = sid[s];
        if (id < 0 || id < lo || id >= hi) continue;
        float p = 0.f;
        bool once = true;  // the first slot of an id writes for all of them
        for (int j = 0; j < a.K; ++j)
          if (sid[j] == id) {
            once = once && j >= s;
            p += expf(sx[j] - c);
          }
        if (once) {
          float u = sz[s], v = 0.f;
          q2(u, v);
          dz[id] = Elem<T>::from_f32(fmaf(-w, p, u));
        }
      }
  }
  if ((MODE & DISTILL_LOSS) && ctas > 1) umma::cluster_sync();  // the others have read this CTA's pair
}

// ---------------------------------------------------------------- host
struct DsShape {
  int threads, units, ctas, groups;
};
static DsShape ds_shape(const DistillArgs &a) {
  const int64_t n = ceil_div(a.V, a.f32 ? 4 : 8);
  DsShape s = {128, 2, 1, 1};
  if (n > 256) s.units = 8;
  while (s.threads < DS_MAX_THREADS && (int64_t)s.threads * s.units < n) s.threads *= 2;
  const int64_t one = (int64_t)s.threads * s.units;
  while (s.ctas < 8 && s.ctas * one < n) s.ctas *= 2;
  s.groups = (int)ceil_div(n, s.ctas * one);
  return s;
}

template <typename T, int MODE, int U>
static cudaError_t ds_launch(const DistillArgs &a, const DsShape &s, int *status, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.T * s.ctas));
  cfg.blockDim = dim3(s.threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = s.ctas;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = (MODE & DISTILL_LOSS) && s.ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, distill_kernel<T, MODE, U>, a, s.ctas, s.groups, status);
}

template <typename T>
static cudaError_t ds_dispatch(const DistillArgs &a, int mode, int *status, cudaStream_t stream) {
  const DsShape s = ds_shape(a);
  if (s.units == 2) {
    if (mode == DISTILL_LOSS) return ds_launch<T, DISTILL_LOSS, 2>(a, s, status, stream);
    if (mode == DISTILL_GRAD) return ds_launch<T, DISTILL_GRAD, 2>(a, s, status, stream);
    return ds_launch<T, DISTILL_LOSS | DISTILL_GRAD, 2>(a, s, status, stream);
  }
  if (mode == DISTILL_LOSS) return ds_launch<T, DISTILL_LOSS, 8>(a, s, status, stream);
  if (mode == DISTILL_GRAD) return ds_launch<T, DISTILL_GRAD, 8>(a, s, status, stream);
  return ds_launch<T, DISTILL_LOSS | DISTILL_GRAD, 8>(a, s, status, stream);
}

cudaError_t launch_distill(const DistillArgs &a, int mode, int *status, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return a.f32 ? ds_dispatch<float>(a, mode, status, stream) : ds_dispatch<__nv_bfloat16>(a, mode, status, stream);
}

}  // namespace moe
