// Distillation from a teacher's top logits: loss, gradient, and both in one
// call (contracts with moe_distill in moe.h).
//
//   lse = m / tau + log s,  m = max z,  s = sum exp((z - m) / tau)
//   dz  = w (P exp((z - m) / tau) / s - p at the teacher's ids)
//
// A row belongs to a cluster of CTAs (one, where it is short), every CTA to a
// slice of it, every thread to some 16-byte units of the slice.  Clusters walk
// over the rows; three slices stand in shared memory, one whose gradient is
// written, one whose statistics are taken and one on its way, so that a row is
// read from memory once and nothing waits for it.  The warps of a CTA:
//   loader     starts the bulk copies, half a slice at a time, as soon as the
//              consumers are done with what stood there
//   consumers  statistics of row j + 1, then gradient of row j
//   joiner     joins the warps' statistics and hands them to the other CTAs
//              through distributed shared memory
//   three row warps, a row each in turn: the teacher's slots and their softmax,
//              then the loss, then the teacher's places of the gradient again,
//              p subtracted, behind the dense pass (apart from the joiner: its
//              stores to memory would hold up the hand-over)
// They meet at mbarriers alone; no barrier stops a whole CTA.
// Sums of exponentials stand beside the logit that they are relative to: a
// thread takes the largest of its first unit, and the largest of all it has
// only where that turns out too small (a sum above 2^40) or is -inf.  The
// (reference, sum) pairs of threads, warps and CTAs are joined in a fixed
// order.
// The shape goes by the vocabulary and by whether all rows start on 16-byte
// boundaries, so a row's results do not depend on the batch, and a thread's
// units do not depend on where the row starts.
// Short rows, where those hand-overs cost more than they hide, and rows too
// long for the shared memory of a cluster take a plainer kernel: a cluster
// (one CTA, for the short ones) for every row, many at once on an SM.
//
// An exponent is one fused multiply-add, z k - m k with k = log2(e) / tau, and m k
// rounded alike wherever it is used; where m k would overflow (rows at the
// type's lowest value) the difference is taken first.
//
// The floor is the logits read once and the gradient written once: 593 us for
// the step at 8192 x 131072 (bfloat16, an eighth of the rows without teacher)
// at the measured copy rate, 72 us for the gradient at 4096 x 32000, 9.9 us for
// the loss at 333 x 50257 in float.  Measured: 597 us (99 %), 81 us (89 %) and
// 25.6 us (38 %).  Reached for the step from 3528 us (a CTA a row, two passes
// through L2): rows in the registers of a cluster 1147, roles and a ring of
// slices 986, teacher and joins in warps of their own 752, statistics handed
// over by st.async instead of a released arrival 643, a row warp for each row
// under way 602.  The loss in float on rows of 16 bytes' multiples runs at
// 91 % (5000 x 50256, 162 us); between boundaries the shifts and the few
// elements at a row's ends cost twice the time (324 us at 50257).  Ends taken
// from the copied pieces instead of from memory made every shape slower
// (414 us there, 627 us for the step): more code in the hot loops.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"
#include "umma.cuh"

namespace moe {

constexpr float DS_LOG2E = 1.4426950408889634f, DS_LN2 = 0.6931471805599453f;

__device__ inline float ds_neg_inf() { return __int_as_float(0xff800000); }

// 2^x in hardware (two units in the last place; results below 2^-126 are 0).
__device__ inline float ds_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Keeps the compiler from holding what was unpacked from `v` beside it.
__device__ inline void ds_opaque(uint4 &v) { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }

__device__ inline float ds_warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ inline float ds_warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
  return v;
}

// 2^((z - m) k) for many z: z b + a, or (z + a) b where m k is out of range.
struct DsPower {
  F2 a, b;
  bool far;
  __device__ inline DsPower(float m, float k) {
    const float base = m == ds_neg_inf() ? 0.f : m, mk = __fmul_rn(base, k);
    far = !(fabsf(mk) < 1e37f);
    const float x = far ? -base : -mk;
    a = F2(x, x);
    b = F2(k, k);
  }
  __device__ inline F2 two(F2 z) const {
    float x, y;
    (far ? mul2(add2(z, a), b) : fma2(z, b, a)).get(x, y);
    return F2(ds_exp2(x), ds_exp2(y));
  }
  // 2^((m' - m) k) for another reference m'.
  __device__ inline float of(float m) const {
    float x, k, y;
    a.get(x, y);
    b.get(k, y);
    return ds_exp2(far ? (m + x) * k : __fadd_rn(__fmul_rn(m, k), x));
  }
};

// A logit and the sum of 2^(k (. - it)); (-inf, 0) is empty.
struct DsStat {
  float m, s;
};
// The pairs of a warp's lanes as one.
__device__ inline DsStat ds_warp_join(DsStat a, float k) {
  const float m = ds_warp_max(a.m);
  return {m, ds_warp_sum(a.s * DsPower(m, k).of(a.m))};
}

// M pairs in shared memory as one, by every thread that calls it.
template <int M>
__device__ inline DsStat ds_join(const DsStat *p, float k) {
  float m = ds_neg_inf(), s = 0.f;
#pragma unroll
  for (int i = 0; i < M; ++i) m = fmaxf(m, p[i].m);
  const DsPower power(m, k);
#pragma unroll
  for (int i = 0; i < M; ++i) s = fmaf(p[i].s, power.of(p[i].m), s);
  return {m, s};
}

// Bytes 2 H .. 2 H + 15 of the 32 bytes of (lo, hi).
template <int H>
__device__ inline uint4 ds_funnel(const uint4 &lo, const uint4 &hi) {
  constexpr int W = H / 2;
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = H % 2 ? __funnelshift_r(w[W + i], w[W + i + 1], 16) : w[W + i];
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// f<H>() for a shift of 2 H bytes below 16 that is the same for all.
template <typename T, typename F>
__device__ inline void ds_by_shift(int off, F f) {
  switch (off * (int)sizeof(T) / 2) {
    case 0: f(std::integral_constant<int, 0>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    case 6: f(std::integral_constant<int, 6>()); break;
    default:
      if constexpr (sizeof(T) == 2) {
        switch (off) {
          case 1: f(std::integral_constant<int, 1>()); break;
          case 3: f(std::integral_constant<int, 3>()); break;
          case 5: f(std::integral_constant<int, 5>()); break;
          default: f(std::integral_constant<int, 7>()); break;
        }
      }
  }
}
__device__ inline uint4 ds_funnel(const uint4 &lo, const uint4 &hi, int sh) {
  uint4 r = lo;
  ds_by_shift<uint16_t>(sh / 2, [&](auto h) { r = ds_funnel<h.value>(lo, hi); });
  return r;
}

// Units of a row: unit u holds elements u N .. u N + N - 1.  A row may start
// `off` elements past a 16-byte boundary; its units are then put together from
// the two aligned pieces that they lie in, so that what a thread holds does
// not depend on where the row stands.
template <typename T>
struct DsUnit {
  static constexpr int N = 16 / sizeof(T);
  // Whether the aligned piece c (elements c N - off ...) lies in the row.
  static __device__ inline bool piece_in(int off, int c, int V) {
    const int i = c * N - off;
    return i >= 0 && i + N <= V;
  }
  // Unit u element by element; what is not of the row reads as -inf.
  static __device__ __noinline__ uint4 edge(const T *row, int u, int V) {
    uint4 v;
    T *e = (T *)&v;
#pragma unroll
    for (int j = 0; j < N; ++j) e[j] = u * N + j < V ? row[u * N + j] : Elem<T>::from_f32(ds_neg_inf());
    return v;
  }
  // Whether all units u, u + step, ... u + (n - 1) step of every lane of the
  // warp lie in the row with their pieces.
  template <bool ALIGNED>
  static __device__ inline bool inner(int off, int u, int step, int n, int V) {
    const int last = u + (n - 1) * step;
    const bool in = ALIGNED || off == 0 ? (int64_t)(last + 1) * N <= V : piece_in(off, u, V) && piece_in(off, last + 1, V);
    return __all_sync(FULL_MASK, in);
  }
  template <bool ALIGNED>
  static __device__ inline uint4 load_inner(const uint4 *pieces, int off) {
    if (ALIGNED || off == 0) return *pieces;
    return ds_funnel(pieces[0], pieces[1], off * (int)sizeof(T));
  }
  // Unit u, from its aligned pieces (`pieces` is where piece u stands, in
  // shared memory or in the row itself) where they are of the row.
  template <bool ALIGNED>
  static __device__ inline uint4 load(const uint4 *pieces, const T *row, int off, int u, int V) {
    if (ALIGNED || off == 0) {
      if ((u + 1) * N <= V) return *pieces;
    } else if (piece_in(off, u, V) && piece_in(off, u + 1, V)) {
      return ds_funnel(pieces[0], pieces[1], off * (int)sizeof(T));
    }
    return edge(row, u, V);
  }
  static __device__ __noinline__ void edge_store(T *row, int u, int V, uint4 v, int from, int to) {
    const T *e = (const T *)&v;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j >= from && j < to && u * N + j < V) row[u * N + j] = e[j];
  }
  // The whole warp: lane l holds unit u of consecutive ones.
  template <bool ALIGNED>
  static __device__ inline void store(T *row, int off, int u, int V, const uint4 &v) {
    const int i = u * N, lane = threadIdx.x & 31;
    int from = 0, to = N;  // what is left to write element by element
    if (ALIGNED || off == 0) {
      if (i + N <= V) {
        __stcs((uint4 *)(row + i), v);
        return;
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
    if (from < to && i + from < V) edge_store(row, u, V, v, from, to);
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

// Writes a pair to the shared memory of a CTA of the cluster.
__device__ inline void ds_st_cluster(uint32_t addr, DsStat v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.m), "f"(v.s) : "memory");
}
// The same, counted on a barrier there: it needs no fence, which would wait
// for every store to memory that the SM has under way.
__device__ inline void ds_st_async(uint32_t addr, DsStat v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr),
               "f"(v.m), "f"(v.s), "r"(bar)
               : "memory");
}

constexpr int DS_MAX_CTAS = 8, DS_RING = 3, DS_STATS = 4;

template <typename T>
__device__ inline int ds_offset(const T *p) {
  return (int)(((uintptr_t)p / sizeof(T)) & (DsUnit<T>::N - 1));
}

// The pair of U units.
template <typename T, int U>
__device__ inline DsStat ds_units_stat(uint4 (&raw)[U], float k) {
  constexpr int N = DsUnit<T>::N;
  float m = ds_unit_max<T>(raw[0]), s;
  for (bool all = m == ds_neg_inf();; all = true) {
    if (all)
#pragma unroll
      for (int j = 0; j < U; ++j) m = fmaxf(m, ds_unit_max<T>(raw[j]));
    const DsPower power(m, k);
    F2 sum[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
    auto add = [&](bool far) {
      DsPower p = power;
      p.far = far;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float v[N];
        ds_opaque(raw[j]);
        Vec16<T>::unpack(raw[j], v);
#pragma unroll
        for (int i = 0; i < N; i += 2) sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], p.two(F2(v[i], v[i + 1])));
      }
    };
    if (power.far) add(true);
    else add(false);
    float s0, s1;
    add2(sum[0], sum[1]).get(s0, s1);
    s = s0 + s1;
    if (all || s <= 1099511627776.f) break;  // (NaN goes on, once)
  }
  return {m, s};
}

// The gradient's dense part: w P q of two logits at a time, by
// 2^((z - m) k) * mul with the loss's own pair (mul holds 1 / s), or by
// exp(z / tau - lse) * mul where only lse is known.
template <bool LOSS>
struct DsGrad {
  DsPower power;
  F2 tau, mul;
  __device__ inline DsGrad(float m_or_lse, float k, float inv_tau, float mul_)
      : power(m_or_lse, k), tau(inv_tau, inv_tau), mul(mul_, mul_) {
    if (!LOSS) power.a = F2(-m_or_lse, -m_or_lse);
  }
  __device__ inline void operator()(float &u, float &v) const {
    F2 x(u, v);
    if (LOSS) {
      x = power.two(x);
    } else {
      mul2(fma2(x, tau, power.a), F2(DS_LOG2E, DS_LOG2E)).get(u, v);
      x = F2(ds_exp2(u), ds_exp2(v));
    }
    mul2(x, mul).get(u, v);
  }
};

// What a row's teacher is to a CTA.
constexpr int DS_MARKS = 2048;
struct __align__(16) DsSlots {
  int id[DISTILL_MAX_K];   // -1 where there is no slot
  float x[DISTILL_MAX_K];  // t / tau
  float p[DISTILL_MAX_K];
  float z[DISTILL_MAX_K];  // the student's logit there
  float c, total, w, lse;  // p = exp(x - c), their sum; the row's weight; its lse where that is given
  int any, twice;          // whether there is a slot; whether an id may be there twice
  float m, s;              // the student's statistics (m: lse where that is given)
  float mul;               // what DsGrad takes; 0 where there is no gradient
};

// One warp: the teacher's distribution from its slots, and whether an id is
// there twice.  For that every slot leaves its number at a place of `marks`
// that its id hashes to: one that reads its own number there is alone or the
// one that its copies read; one that reads another's is a copy, or tries again
// with another hash (its copies, if any, do the same).
__device__ inline void ds_teacher(const DistillArgs &a, int64_t t, DsSlots &sl, uint8_t *marks) {
  constexpr int SL = DISTILL_MAX_K / 32;
  const int lane = threadIdx.x & 31;
  int id[SL];
  float x[SL], e[SL], m = ds_neg_inf(), sum = 0.f;
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    if (32 * i >= a.K) break;
    const int s = lane + 32 * i;
    id[i] = s < a.K ? sl.id[s] : -1;
    x[i] = s < a.K ? sl.x[s] : 0.f;
    if (id[i] >= 0) m = fmaxf(m, x[i]);
  }
  float c = 0.f;
  if (a.t_lse) m = c = a.t_lse[t];
  else m = ds_warp_max(m);
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    if (32 * i >= a.K) break;
    e[i] = id[i] >= 0 ? expf(x[i] - m) : 0.f;
    sum += e[i];
  }
  sum = ds_warp_sum(sum);
  const float inv = a.t_lse ? 1.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    if (32 * i >= a.K) break;
    if (lane + 32 * i < a.K) sl.p[lane + 32 * i] = e[i] * inv;
  }
  bool twice = false, again = a.K > 1;
  uint32_t mix = 2654435761u;
  for (int round = 0; again; ++round) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      if (32 * i >= a.K) break;
      if (id[i] >= 0) marks[(uint32_t)(id[i] + 1) * mix >> 21] = (uint8_t)(lane + 32 * i);
    }
    __syncwarp();
    bool open = false;
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      if (32 * i >= a.K) break;
      if (id[i] < 0) continue;
      const int other = marks[(uint32_t)(id[i] + 1) * mix >> 21];
      if (other != lane + 32 * i) {
        if (sl.id[other] == id[i]) twice = true;
        else {
          open = true;
          continue;
        }
      }
      id[i] = -1;  // settled
    }
    again = __any_sync(FULL_MASK, open);
    if (again && round == 7) {  // an odd set of ids: take it that there are copies
      twice = true;
      break;
    }
    mix = mix * 747796405u + 2891336453u | 1u;
  }
  twice = __any_sync(FULL_MASK, twice);
  if (lane == 0) {
    sl.c = a.t_lse ? c : m + logf(sum);
    sl.total = a.t_lse ? sum : 1.f;
    sl.twice = twice;
  }
}

// Nothing but -inf (NaN is something).
__device__ inline bool ds_none(DsStat st) { return st.m == ds_neg_inf() && !(st.s != st.s); }

// One warp: a row's loss and lse from its statistics.
__device__ inline void ds_loss(const DistillArgs &a, int64_t t, const DsSlots &sl, DsStat st, float k) {
  const int lane = threadIdx.x & 31;
  const float logs = logf(st.s), mk = __fmul_rn(st.m, k);
  const bool far = !(fabsf(mk) < 1e37f);
  float l = 0.f;
  for (int s = lane; s < a.K; s += 32) {
    const float p = sl.p[s];
    const float z = sl.z[s];
    const float d = far || !(fabsf(z * k) < 1e37f) ? (z - st.m) * a.inv_tau : fmaf(z, k, -mk) * DS_LN2;
    if (p != 0.f) l += p * (sl.x[s] - sl.c - (d - logs));
  }
  l = ds_warp_sum(l);
  if (ds_none(st)) l = -ds_neg_inf();
  if (lane == 0) {
    a.loss[t] = sl.any ? a.scale * l : 0.f;
    if (a.lse) a.lse[t] = ds_none(st) ? ds_neg_inf() : far ? fmaf(st.m, a.inv_tau, logs) : fmaf(mk, DS_LN2, logs);
  }
}

// The gradient at the teacher's places in [lo, hi), by `n` threads of which this is number `i`.
template <typename T, bool LOSS>
__device__ inline void ds_places(const DistillArgs &a, const DsSlots &sl, T *dz, int lo, int hi, float w,
                                 const DsGrad<LOSS> &grad, int i, int n) {
  for (int s = i; s < a.K; s += n) {
    const int id = sl.id[s];
    if (id < 0 || id < lo || id >= hi) continue;
    float p = sl.p[s];
    bool once = true;
    if (sl.twice) {  // the first slot of an id writes for all of them
      p = 0.f;
      for (int j = 0; j < a.K; ++j)
        if (sl.id[j] == id) {
          once = once && j >= s;
          p += sl.p[j];
        }
    }
    if (once) {
      float u = sl.z[s], v = 0.f;
      grad(u, v);
      dz[id] = Elem<T>::from_f32(fmaf(-w, p, u));
    }
  }
}

// The dense part of the gradient of U units a thread: load(j, inner) gives
// unit j, half() is called between the halves of them.  The first `inner` (U,
// U - 1 or none) lie in the row for the whole warp and run without a branch
// between them, so that one's exponentials overlap the next one's loads; the
// others one after the other.
template <typename T, bool ALIGNED, bool LOSS, int U, typename Load, typename Half>
__device__ inline void ds_dense(T *dz, int V, int u0, int step, bool zero, int inner, DsGrad<LOSS> grad, Load load, Half half) {
  constexpr int N = DsUnit<T>::N;
  const int off = ALIGNED ? 0 : ds_offset(dz);
  auto unit = [&](const uint4 &raw) {
    float v[N];
    Vec16<T>::unpack(raw, v);
#pragma unroll
    for (int i = 0; i < N; i += 2) grad(v[i], v[i + 1]);
    uint4 o;
    Vec16<T>::store((T *)&o, v);
    return o;
  };
  int done = 0;
  if (!zero && inner && !(LOSS && grad.power.far)) {
    grad.power.far = false;  // known to the compiler
    auto fast = [&](int j) {
      const uint4 o = unit(load(j, true));
      if (ALIGNED) __stcs((uint4 *)dz + u0 + j * step, o);
      else DsUnit<T>::template store<ALIGNED>(dz, off, u0 + j * step, V, o);
      if (j == U / 2 - 1) half();
    };
#pragma unroll
    for (int j = 0; j < U - 1; ++j) fast(j);
    if (inner == U) {
      fast(U - 1);
      return;
    }
    done = U - 1;
  }
  {
#pragma unroll 1
    for (int j = done; j < U; ++j) {
      DsUnit<T>::template store<ALIGNED>(dz, off, u0 + j * step, V, zero ? uint4{} : unit(load(j, false)));
      if (j == U / 2 - 1) half();
    }
  }
}

// The same by aligned pieces of the row, where the gradient's row starts like
// the logits' between 16-byte boundaries (`off` elements past one): piece c of
// the one is written from piece c of the other, nothing is shifted.  load(j)
// gives piece c0 + j step; pieces from `end` on are not this CTA's.
template <typename T, bool LOSS, int U, typename Load, typename Half>
__device__ inline void ds_dense_pieces(const T *z, T *dz, int off, int V, int c0, int step, int end, bool zero,
                                       DsGrad<LOSS> grad, Load load, Half half) {
  constexpr int N = DsUnit<T>::N;
  auto unit = [&](const uint4 &raw) {
    float v[N];
    Vec16<T>::unpack(raw, v);
#pragma unroll
    for (int i = 0; i < N; i += 2) grad(v[i], v[i + 1]);
    uint4 o;
    Vec16<T>::store((T *)&o, v);
    return o;
  };
  uint4 *out = (uint4 *)(dz - off) + c0;
  auto in = [&](int c) { return DsUnit<T>::piece_in(off, c, V) && c < end; };
  const bool most = __all_sync(FULL_MASK, in(c0) && in(c0 + (U - 2) * step)), all = __all_sync(FULL_MASK, in(c0 + (U - 1) * step));
  int done = 0;
  if (!zero && most && !(LOSS && grad.power.far)) {
    grad.power.far = false;
    auto fast = [&](int j) {
      __stcs(out + j * step, unit(load(j)));
      if (j == U / 2 - 1) half();
    };
#pragma unroll
    for (int j = 0; j < U - 1; ++j) fast(j);
    if (all) {
      fast(U - 1);
      return;
    }
    done = U - 1;
  }
#pragma unroll 1
  for (int j = done; j < U; ++j) {
    const int c = c0 + j * step;
    if (in(c)) {
      __stcs(out + j * step, zero ? uint4{} : unit(load(j)));
    } else if (c < end) {
#pragma unroll 1
      for (int e = max(c * N - off, 0); e < min((c + 1) * N - off, V); ++e) {
        float u = 0.f, v = 0.f;
        if (!zero) {
          u = Elem<T>::load(z + e);
          grad(u, v);
        }
        dz[e] = Elem<T>::from_f32(u);
      }
    }
    if (j == U / 2 - 1) half();
  }
}

struct DsShared {
  DsSlots slots[DS_RING];
  __align__(16) DsStat warp[DS_RING][16];
  __align__(16) DsStat cta[DS_STATS][DS_MAX_CTAS];
  uint8_t marks[DS_RING][DS_MARKS];
  uint64_t full[DS_RING], empty[DS_RING][2];      // a slice has arrived; the consumers are done with its halves
  uint64_t ready[DS_RING];                        // a teacher is there
  uint64_t taken[DS_RING], stats[DS_STATS];       // the warps' pairs are there; all CTAs' pairs are there
  uint64_t go[DS_RING];                           // the row's gradient can be written
  int read[DS_RING];                              // whether a slice was loaded (written by the loader before `full`)
  int abort_flag;
};

// U: units a thread; 1 << shift: CTAs of a cluster; span: units of a CTA, above
// (U - 1) 32 DS_WARPS and up to U 32 DS_WARPS.
// ALIGNED: all rows start on 16-byte boundaries.
constexpr int DS_WARPS = 16;  // consumers
template <typename T, bool ALIGNED, int MODE, int U>
__global__ void __launch_bounds__(32 * (DS_WARPS + 2 + DS_RING), 1)
distill_kernel(const DistillArgs a, int shift, int span, int *status) {
  using namespace umma;
  constexpr int N = DsUnit<T>::N, W = DS_WARPS, SPAN = U * W * 32;
  constexpr bool LOSS = (MODE & DISTILL_LOSS) != 0, GRAD = (MODE & DISTILL_GRAD) != 0;
  extern __shared__ __align__(128) uint4 slices[];  // DS_RING x (SPAN + 1) aligned pieces
  __shared__ DsShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ctas = 1 << shift;
  const int rank = blockIdx.x & (ctas - 1), stride = gridDim.x >> shift;
  const float k = a.inv_tau * DS_LOG2E;
  const int u_first = rank * span;  // units, or aligned pieces, of this CTA: span from here
  const int V = min(a.V, (u_first + span) * N);  // where its units end
  // Where the gradient's row starts like the logits', a CTA writes pieces, else units.
  auto by_pieces = [&](const T *z, const T *dz) { return !ALIGNED && ds_offset(z) == ds_offset(dz); };
  auto first_of = [&](const T *z, const T *dz) { return u_first * N - (by_pieces(z, dz) ? ds_offset(z) : 0); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < DS_RING; ++i) {
      mbar_init(&sh.full[i], 2);
      mbar_init(&sh.empty[i][0], W);
      mbar_init(&sh.empty[i][1], W);
      mbar_init(&sh.ready[i], 1);
      mbar_init(&sh.taken[i], W);
      mbar_init(&sh.go[i], 1);
    }
    for (int i = 0; i < DS_STATS; ++i) mbar_init(&sh.stats[i], 1);
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < DS_STATS * DS_MAX_CTAS) sh.cta[0][threadIdx.x] = {ds_neg_inf(), 0.f};  // CTAs that the cluster lacks
  __syncthreads();
  // The barriers of the whole cluster are there before anyone arrives at them.
  if (LOSS && ctas > 1) cluster_sync();
  griddep_launch();
  griddep_wait();

  const int64_t t0 = blockIdx.x >> shift;
  const int rows = t0 < a.T ? (int)((a.T - 1 - t0) / stride) + 1 : 0;  // of this cluster
  auto row_of = [&](int j) { return (const T *)a.logits + (t0 + (int64_t)j * stride) * a.ld_logits; };
  auto out_of = [&](int j) { return (T *)a.dlogits + (t0 + (int64_t)j * stride) * a.ld_dlogits; };
  auto wait = [&](uint64_t *bar, int phase) { return mbar_wait(bar, phase & 1, &sh.abort_flag, status); };

  // Rows that have no gradient and whose loss is 0 or not asked for are not read.
  auto needed = [&](bool any, float w) { return (LOSS && (!GRAD || a.lse)) || (any && (LOSS || w != 0.f)); };
  constexpr int SL = DISTILL_MAX_K / 32;
  auto slot_id = [&](int64_t t, int i) { return lane + 32 * i < a.K ? a.t_ids[t * a.K + lane + 32 * i] : -1; };
  auto slot_x = [&](int64_t t, int i) { return lane + 32 * i < a.K ? a.t_logits[t * a.K + lane + 32 * i] : 0.f; };
  auto counts = [&](int id, float x) { return id >= 0 && id < a.V && x * a.inv_tau != ds_neg_inf(); };

  if (warp == W) {
    // ------------------------------------------------------------ loader
    // Slots two rows ahead (memory under load answers late).
    int id[2][SL];
    float x[2][SL], w[2] = {0.f, 0.f};
    auto fetch = [&](int j, int b) {
      if (!GRAD || j >= rows) return;  // (without a gradient every row is read)
      const int64_t t = t0 + (int64_t)j * stride;
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        if (32 * i >= a.K) break;
        id[b][i] = slot_id(t, i);
        x[b][i] = slot_x(t, i);
      }
      w[b] = a.weight[t];
    };
    int started = 0;  // rows
    auto turn = [&](int j, int b) {
      started = j + 1;
      const int r = j % DS_RING, round = j / DS_RING;
      const T *z = row_of(j);
      bool found = false;
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        if (!GRAD || 32 * i >= a.K) break;
        found |= counts(id[b][i], x[b][i]);
      }
      const bool read = needed(__any_sync(FULL_MASK, found), w[b]);
      fetch(j + 2, b);
      // The aligned pieces that lie in the row (none of a row that is not read).
      const int off = ALIGNED ? 0 : ds_offset(z);
      const int last = read ? (a.V + off) / N : 0;
      uint4 *slice = slices + r * (SPAN + 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!wait(&sh.empty[r][h], round + 1)) return false;
        if (lane == 0) {
          if (h == 1) sh.read[r] = read;
          constexpr int HALF = U / 2 * W * 32;
          const int from = u_first + (h ? HALF : 0) + (off && u_first == 0 && h == 0 ? 1 : 0);
          const int to = min(u_first + (h ? span + (off ? 1 : 0) : HALF), last);
          if (to > from) {
            mbar_arrive_expect_tx(&sh.full[r], (uint32_t)(to - from) * 16);
            bulk_load(slice + (from - u_first), z - off + (int64_t)from * N, (uint32_t)(to - from) * 16, &sh.full[r]);
          } else {
            mbar_arrive(&sh.full[r]);
          }
        }
        __syncwarp();
      }
      return true;
    };
    fetch(0, 0);
    fetch(1, 1);
    for (int j = 0; j < rows; j += 2) {
      if (!turn(j, 0)) break;
      if (j + 1 < rows && !turn(j + 1, 1)) break;
    }
    // The copies land before the CTA ends, even where the others have given up.
    for (int j = max(started - DS_RING, 0); j < started; ++j) mbar_drain(&sh.full[j % DS_RING], (j / DS_RING) & 1);
  } else if (warp > W + 1) {
    // ------------------------------------------------------------ row warps
    const int r = warp - (W + 2);
    DsSlots &sl = sh.slots[r];
    int id[SL];
    float x[SL], w = 0.f, lse = 0.f;
    auto fetch = [&](int j) {
      if (j >= rows) return;
      const int64_t t = t0 + (int64_t)j * stride;
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        if (32 * i >= a.K) break;
        id[i] = slot_id(t, i);
        x[i] = slot_x(t, i);
      }
      if (GRAD) w = a.weight[t];
      if (!LOSS) lse = a.lse[t];
    };
    // The student's logits at the slots of row j go on their way as well.
    bool any = false;
    T zk[SL];
    auto gather = [&](int j) {
      if (j >= rows) return;
      const T *z = row_of(j);
      const int lo = first_of(z, out_of(j)), hi = lo + span * N;
      bool found = false;
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        if (32 * i >= a.K) break;
        if (id[i] < -1 || id[i] >= a.V) record_status(status, STATUS_BAD_TEACHER_ID);
        if (!counts(id[i], x[i])) id[i] = -1;
        found |= id[i] >= 0;
        // without a loss, only this CTA's places matter (others may have been written)
        if (id[i] >= 0 && (LOSS || (id[i] >= lo && id[i] < hi))) zk[i] = z[id[i]];
        else zk[i] = T(0.f);
      }
      any = __any_sync(FULL_MASK, found);
    };
    fetch(r);
    gather(r);
    for (int j = r; j < rows; j += DS_RING) {
      const int round = j / DS_RING;
      const int64_t t = t0 + (int64_t)j * stride;
      const T *z = row_of(j);
      T *dz = out_of(j);
      const int lo = first_of(z, dz), hi = lo + span * N;  // elements of this CTA
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        if (32 * i >= a.K) break;
        const int s = lane + 32 * i;
        if (s < a.K) {
          sl.id[s] = id[i];
          sl.x[s] = x[i] * a.inv_tau;
          sl.z[s] = Elem<T>::to_f32(zk[i]);
        }
      }
      if (lane == 0) {
        sl.w = w * a.scale * a.inv_tau;
        sl.lse = lse;
        sl.any = any;
      }
      __syncwarp();
      fetch(j + DS_RING);
      ds_teacher(a, t, sl, sh.marks[r]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.ready[r]);
      gather(j + DS_RING);
      if (!wait(&sh.go[r], round)) return;
      if (LOSS && rank == 0) ds_loss(a, t, sl, DsStat{sl.m, sl.s}, k);
      if (GRAD) {
        if (!wait(&sh.empty[r][1], round)) return;
        if (sl.mul != 0.f)
          ds_places<T, LOSS>(a, sl, dz, lo, hi, sl.w,
                             DsGrad<LOSS>(sl.m, k, a.inv_tau, sl.mul), lane, 32);
      }
      __syncwarp();
    }
  } else if (warp == W + 1) {
    // ------------------------------------------------------------ joiner
    // One lane: what it does for a row is a chain, and it alone decides whether
    // a wait ran out.
    bool on = lane == 0;
    for (int j = 0; on && j < rows; ++j) {
      const int r = j % DS_RING, q = j % DS_STATS;
      DsSlots &sl = sh.slots[r];
      on = (!LOSS || wait(&sh.taken[r], j / DS_RING)) && wait(&sh.ready[r], j / DS_RING);
      if (!on) break;
      DsStat st = {sl.lse, 1.f};
      if (LOSS) {
        st = ds_join<W>(sh.warp[r], k);
        if (ctas > 1) {
          mbar_arrive_expect_tx(&sh.stats[q], ctas * (uint32_t)sizeof(DsStat));
          for (int c = 0; c < ctas; ++c) ds_st_async(mapa_shared(&sh.cta[q][rank], c), st, mapa_shared(&sh.stats[q], c));
          on = mbar_wait_cluster(&sh.stats[q], (j / DS_STATS) & 1, &sh.abort_flag, status);
          if (!on) break;
          st = ds_join<DS_MAX_CTAS>(sh.cta[q], k);
        }
      }
      const bool none = LOSS ? ds_none(st) : st.m == ds_neg_inf();
      sl.m = st.m;
      sl.s = st.s;
      sl.mul = !sl.any || sl.w == 0.f || none ? 0.f : sl.w * sl.total / st.s;
      mbar_arrive(&sh.go[r]);
    }
    // Where a wait ran out the CTA stays until all of its cluster have ended or
    // given up too: until then they may write to it.
    if (LOSS && ctas > 1 && lane == 0 && !on) cluster_sync();
  } else {
    // ------------------------------------------------------------ consumers
    constexpr int STEP = W * 32;
    const int u0 = u_first + threadIdx.x;
    auto release = [&](int r) {
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.empty[r][0]);
        mbar_arrive(&sh.empty[r][1]);
      }
    };
    // Statistics of row j.
    auto statistics = [&](int j) {
      const int r = j % DS_RING;
      if (!wait(&sh.full[r], j / DS_RING)) return false;
      DsStat mine = {ds_neg_inf(), 0.f};
      if (sh.read[r]) {
        const uint4 *slice = slices + r * (SPAN + 1) + threadIdx.x;
        const T *z = row_of(j);
        const int off = ALIGNED ? 0 : ds_offset(z);
        uint4 raw[U];
        if (DsUnit<T>::template inner<ALIGNED>(off, u0, STEP, U - 1, V)) {
          // (the last unit may be past the CTA's end; its pieces are in the slice all the same)
          const bool all = (int64_t)(u0 + (U - 1) * STEP + 1) * N <= V && (ALIGNED || DsUnit<T>::piece_in(off, u0 + (U - 1) * STEP + 1, a.V));
          if (ALIGNED) {
#pragma unroll
            for (int i = 0; i < U - 1; ++i) raw[i] = slice[i * STEP];
            if (all) raw[U - 1] = slice[(U - 1) * STEP];
          } else {
            ds_by_shift<T>(off, [&](auto h) {
              auto get = [&](int i) { return ds_funnel<h.value>(slice[i * STEP], slice[i * STEP + (h.value ? 1 : 0)]); };
#pragma unroll
              for (int i = 0; i < U - 1; ++i) raw[i] = get(i);
              if (all) raw[U - 1] = get(U - 1);
            });
          }
          if (!all) raw[U - 1] = DsUnit<T>::template load<ALIGNED>(slice + (U - 1) * STEP, z, off, u0 + (U - 1) * STEP, V);
        } else {
#pragma unroll
          for (int i = 0; i < U; ++i) raw[i] = DsUnit<T>::template load<ALIGNED>(slice + i * STEP, z, off, u0 + i * STEP, V);
        }
        if (!GRAD) release(r);  // the slice is in registers
        mine = ds_warp_join(ds_units_stat<T, U>(raw, k), k);
      } else if (!GRAD) {
        release(r);
      }
      // (with a gradient the joiner has been done with row j - DS_RING since that was written)
      if (!GRAD && j >= DS_RING && !wait(&sh.go[r], j / DS_RING - 1)) return false;
      if (lane == 0) {
        sh.warp[r][warp] = mine;
        mbar_arrive(&sh.taken[r]);
      }
      return true;
    };
    // Gradient of row j.
    auto gradient = [&](int j) {
      const int r = j % DS_RING;
      const DsSlots &sl = sh.slots[r];
      if (!wait(&sh.go[r], j / DS_RING)) return false;
      if (!LOSS && !wait(&sh.full[r], j / DS_RING)) return false;
      const T *z = row_of(j);
      const uint4 *slice = slices + r * (SPAN + 1) + threadIdx.x;
      const int off = ALIGNED ? 0 : ds_offset(z);
      T *dz = out_of(j);
      const DsGrad<LOSS> grad(sl.m, k, a.inv_tau, sl.mul);
      const bool zero = sl.mul == 0.f;
      auto half = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[r][0]);
      };
      if (by_pieces(z, dz)) {
        ds_dense_pieces<T, LOSS, U>(z, dz, off, a.V, u0, STEP, u_first + span, zero, grad, [&](int i) { return slice[i * STEP]; }, half);
      } else {
        // (rows that start differently go unit by unit)
        int inner = 0;
        if (ALIGNED && DsUnit<T>::template inner<ALIGNED>(off, u0, STEP, U - 1, V))
          inner = DsUnit<T>::template inner<ALIGNED>(off, u0, STEP, U, V) ? U : U - 1;
        ds_dense<T, ALIGNED, LOSS, U>(dz, V, u0, STEP, zero, inner, grad, [&](int i, bool in) {
          if (in) return DsUnit<T>::template load_inner<ALIGNED>(slice + i * STEP, off);
          return DsUnit<T>::template load<ALIGNED>(slice + i * STEP, z, off, u0 + i * STEP, V);
        }, half);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[r][1]);
      return true;
    };
    if (LOSS && rows > 0 && !statistics(0)) return;
    for (int j = 0; j < rows; ++j) {
      if (LOSS && j + 1 < rows && !statistics(j + 1)) return;
      if (GRAD && !gradient(j)) return;
    }
  }
}

// Rows of any length: a cluster for each row, U units a thread at a time
// straight from memory, for the gradient a second time where there are several
// groups of them.
template <typename T, int MODE, int THREADS, int U>
__global__ void __launch_bounds__(THREADS, THREADS == 128 ? 10 : 1024 / THREADS)
distill_plain_kernel(const DistillArgs a, int shift, int groups, int *status) {
  using namespace umma;
  constexpr int N = DsUnit<T>::N;
  constexpr bool LOSS = (MODE & DISTILL_LOSS) != 0, GRAD = (MODE & DISTILL_GRAD) != 0;
  __shared__ DsSlots sl;
  __shared__ uint8_t marks[DS_MARKS];
  __shared__ DsStat wstat[THREADS / 32], cstat[DS_MAX_CTAS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ctas = 1 << shift;
  const int64_t t = blockIdx.x >> shift;
  const int rank = blockIdx.x & (ctas - 1);
  const float k = a.inv_tau * DS_LOG2E;
  griddep_launch();
  griddep_wait();
  if (LOSS && ctas > 1) cluster_sync();  // all CTAs run
  const T *z = (const T *)a.logits + t * a.ld_logits;
  T *dz = (T *)a.dlogits + t * a.ld_dlogits;
  const int off = ds_offset(z), u_first = rank * groups * U * THREADS;
  const bool by_pieces = off != 0 && off == ds_offset(dz);
  const int lo = u_first * N - (by_pieces ? off : 0), hi = lo + groups * U * THREADS * N;
  auto piece = [&](int u) { return (const uint4 *)(z - off) + u; };
  // The first group's units are on their way while the teacher is worked out.
  uint4 raw[U];
  bool inner = false;
  auto load = [&](int g) {
    const int u0 = u_first + g * U * THREADS + threadIdx.x;
    inner = DsUnit<T>::template inner<false>(off, u0, THREADS, U, a.V);
    if (inner) {
#pragma unroll
      for (int i = 0; i < U; ++i) raw[i] = DsUnit<T>::template load_inner<false>(piece(u0 + i * THREADS), off);
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i)
        raw[i] = DsUnit<T>::template load<false>(piece(u0 + i * THREADS), z, off, u0 + i * THREADS, a.V);
    }
  };
  if (LOSS) load(0);
  if (warp == 0) {
    bool found = false;
    for (int s = lane; s < a.K; s += 32) {
      int id = a.t_ids[t * a.K + s];
      const float x = a.t_logits[t * a.K + s] * a.inv_tau;
      if (id < -1 || id >= a.V) record_status(status, STATUS_BAD_TEACHER_ID);
      if (id < 0 || id >= a.V || x == ds_neg_inf()) id = -1;
      sl.id[s] = id;
      sl.x[s] = x;
      sl.z[s] = id >= 0 && (LOSS || (id >= lo && id < hi)) ? Elem<T>::load(z + id) : 0.f;
      found |= id >= 0;
    }
    found = __any_sync(FULL_MASK, found);
    if (lane == 0) {
      sl.any = found;
      sl.w = GRAD ? a.weight[t] * a.scale * a.inv_tau : 0.f;
      sl.lse = LOSS ? 0.f : a.lse[t];
    }
    __syncwarp();
    ds_teacher(a, t, sl, marks);
  }
  DsStat st = {ds_neg_inf(), 0.f};
  if (LOSS) {
    for (int g = 0; g < groups; ++g) {
      if (g) load(g);
      const DsStat one = ds_units_stat<T, U>(raw, k);
      const DsPower power(fmaxf(st.m, one.m), k);
      st = {fmaxf(st.m, one.m), st.s * power.of(st.m) + one.s * power.of(one.m)};
    }
    st = ds_warp_join(st, k);
    if (lane == 0) wstat[warp] = st;
  }
  __syncthreads();
  if (LOSS) {
    st = ds_join<THREADS / 32>(wstat, k);
    if (ctas > 1) {
      if (warp == 0 && lane < ctas) ds_st_cluster(mapa_shared(&cstat[rank], lane), st);
      cluster_sync();
      st = ds_warp_join(lane < ctas ? cstat[lane] : DsStat{ds_neg_inf(), 0.f}, k);
    }
    if (rank == 0 && warp == 0) ds_loss(a, t, sl, st, k);
  } else {
    st = {sl.lse, 1.f};
  }
  if (!GRAD) return;
  const bool zero = !sl.any || sl.w == 0.f || (LOSS ? ds_none(st) : sl.lse == ds_neg_inf());
  const DsGrad<LOSS> grad(st.m, k, a.inv_tau, sl.w * sl.total / st.s);
  for (int g = 0; g < groups; ++g) {
    const int u0 = u_first + g * U * THREADS + threadIdx.x;
    if (by_pieces) {
      ds_dense_pieces<T, LOSS, U>(z, dz, off, a.V, u0, THREADS, u_first + groups * U * THREADS, zero, grad, [&](int i) { return *piece(u0 + i * THREADS); }, [] {});
      continue;
    }
    if (!zero && (!LOSS || groups > 1)) load(g);
    ds_dense<T, false, LOSS, U>(dz, a.V, u0, THREADS, zero, inner ? U : 0, grad, [&](int i, bool in) {
      if (in) return raw[i];
      return DsUnit<T>::template load<false>(piece(u0 + i * THREADS), z, off, u0 + i * THREADS, a.V);
    }, [] {});
  }
  __syncthreads();
  if (!zero) ds_places<T, LOSS>(a, sl, dz, lo, hi, sl.w, grad, threadIdx.x, THREADS);
}

// ---------------------------------------------------------------- host
template <typename T, bool ALIGNED, int MODE, int THREADS, int U>
static cudaError_t ds_launch_plain(const DistillArgs &a, int shift, int *status, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.T << shift);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 1u << shift;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = shift ? 2 : 1;
  // (a row that starts between boundaries has one piece more than units)
  const int groups = (int)ceil_div(ceil_div(a.V, 16 / (int)sizeof(T)) + (ALIGNED ? 0 : 1), (int64_t)(THREADS * U) << shift);
  return cudaLaunchKernelEx(&cfg, distill_plain_kernel<T, MODE, THREADS, U>, a, shift, groups, status);
}

template <typename T, bool ALIGNED, int MODE, int U>
static cudaError_t ds_launch(const DistillArgs &a, int shift, int span, int *status, cudaStream_t stream) {
  constexpr int W = DS_WARPS;
  const auto kernel = distill_kernel<T, ALIGNED, MODE, U>;
  const int smem = DS_RING * (U * W * 32 + 1) * 16;
  cudaError_t e = ensure_smem((const void *)kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1u << shift);
  cfg.blockDim = dim3(32 * (W + 2 + DS_RING));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1u << shift;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  // Clusters that run at once, asked for once for each shape and device.
  static std::mutex mu;
  static int known[64][4];
  int dev = 0;
  cudaGetDevice(&dev);
  int clusters;
  {
    std::lock_guard<std::mutex> lock(mu);
    int &n = known[dev & 63][shift];
    if (!n) {
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (n < 1) return cudaErrorInvalidConfiguration;
    }
    clusters = n;
  }
  cfg.gridDim = dim3((unsigned)std::min(a.T, clusters) << shift);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, shift, span, status);
}

// The shape of a launch, by the row's 16-byte units (or pieces: one more where
// rows start between boundaries) alone.
template <typename T, bool ALIGNED, int MODE>
static cudaError_t ds_shape(const DistillArgs &a, int *status, cudaStream_t stream) {
  const int64_t n = ceil_div(a.V, 16 / (int)sizeof(T)) + (ALIGNED ? 0 : 1);
  if (n <= 1024) return ds_launch_plain<T, ALIGNED, MODE, 128, 4>(a, 0, status, stream);
  // Up to 2048 units the two kernels are near one another (us, this one / the
  // plain one, 16384 rows: step at V = 16000 248 / 239 and at 12000 236 / 260,
  // gradient 156 / 281, loss 125 / 195; between boundaries, V = 16001: step
  // 418 / 381, loss 262 / 227, gradient 188 / 260).
  if (!ALIGNED && n <= 2048 && (MODE & DISTILL_LOSS)) return ds_launch_plain<T, ALIGNED, MODE, 256, 8>(a, 0, status, stream);
  // As few CTAs as hold the row in slices of 4096 units, alike in size.
  for (int shift = 0; 1 << shift <= DS_MAX_CTAS; ++shift)
    if (n <= (int64_t)4096 << shift) {
      const int span = (int)ceil_div(n, 1 << shift);
      switch (ceil_div(span, DS_WARPS * 32)) {
        case 8: return ds_launch<T, ALIGNED, MODE, 8>(a, shift, span, status, stream);
        case 7: return ds_launch<T, ALIGNED, MODE, 7>(a, shift, span, status, stream);
        case 6: return ds_launch<T, ALIGNED, MODE, 6>(a, shift, span, status, stream);
        case 5: return ds_launch<T, ALIGNED, MODE, 5>(a, shift, span, status, stream);
        case 4: return ds_launch<T, ALIGNED, MODE, 4>(a, shift, span, status, stream);
        default: return ds_launch<T, ALIGNED, MODE, 3>(a, shift, span, status, stream);
      }
    }
  return ds_launch_plain<T, ALIGNED, MODE, 512, 4>(a, 3, status, stream);
}

template <typename T, bool ALIGNED>
cudaError_t ds_mode(const DistillArgs &a, int mode, int *status, cudaStream_t stream) {
  if (mode == DISTILL_LOSS) return ds_shape<T, ALIGNED, DISTILL_LOSS>(a, status, stream);
  if (mode == DISTILL_GRAD) return ds_shape<T, ALIGNED, DISTILL_GRAD>(a, status, stream);
  return ds_shape<T, ALIGNED, DISTILL_LOSS | DISTILL_GRAD>(a, status, stream);
}


}  // namespace moe
