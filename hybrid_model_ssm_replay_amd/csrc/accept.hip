// Acceptance of drafted tokens and the token drawn after them.
//
// Draft i is kept while u_i q_i(x_i) < p_i(x_i).  The refused draft's residual
// max(p - q, 0), or p after the last draft, is sampled by inverse CDF.  One row
// of p and one of q per sequence have to be read: HBM bound for many sequences,
// latency bound for one.
//
// Two launches.  sums_k cuts every row into slices, a workgroup each, so that one
// sequence's vocabulary still fills the card; a workgroup finds the sequence's
// accepted count for itself (T values, read by T lanes at once) and leaves its
// slice's two sums, of the residual and of p, the one to fall back on.  pick_k
// adds the slices up in their order, takes the one that holds the sampling
// number, and looks for the token in it: the rows of 64 within a slice, then the
// lane.  Every sum has a fixed order: no atomics.
//
// Sums are float64: p - q of float32 or bf16 values is exact or nearly so there,
// and the order of a sum over a large vocabulary then moves a sampling border by
// about 1e-13 of the total instead of 1e-4.
#include "ops.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kStep = 8 * kThreads;  // values a workgroup reads at a time, 8 a thread

struct Slices {
  int size, n;         // values of a slice (a multiple of kStep), slices of a row
  double2 *sums;       // [batch][n]: residual, p
  FastDiv fn;
};

__device__ __forceinline__ float at(const void *p, int dtype, int64_t i) {
  return dtype == REPLAY_DT_BF16 ? ldr<bf16_t>((const bf16_t *)p + i) : ldr<float>((const float *)p + i);
}

// Drafts accepted: the first one that fails its test.
__device__ __forceinline__ int accepted(const replay_accept_args &a, int b, int n, int lane) {
  for (int i0 = 0; i0 < n; i0 += kWave) {
    const int i = i0 + lane;
    bool ok = true;
    if (i < n) {
      const int x = a.tokens[(int64_t)b * a.drafts + i];
      ok = x >= 0 && x < a.vocab;
      if (ok) {
        const double p = at(a.target, a.target_dtype, b * a.target_seq_stride + i * a.target_row_stride + x);
        double q = a.draft ? (double)at(a.draft, a.draft_dtype, b * a.draft_seq_stride + i * a.draft_row_stride + x) : 1.0;
        if (!(q > 0.0)) q = 0.0;
        ok = (double)a.uniforms[(int64_t)b * (a.drafts + 1) + i] * q < p;
      }
    }
    const uint64_t bad = __ballot(!ok);
    if (bad) return i0 + __ffsll((unsigned long long)bad) - 1;
  }
  return n;
}
__device__ __forceinline__ int drafts_of(const replay_accept_args &a, int b) {
  return a.lengths ? min(max(a.lengths[b], 0), a.drafts) : a.drafts;
}

// The row to draw from and what it loses.
struct Row {
  int64_t p, q;  // offsets
  int x;         // a certain draft that was refused loses its own token; else -1
  bool less;     // a residual: q is subtracted
};
__device__ __forceinline__ Row row_of(const replay_accept_args &a, int b, int acc, int n) {
  Row r;
  r.less = acc < n;
  r.p = b * a.target_seq_stride + acc * a.target_row_stride;
  r.q = b * a.draft_seq_stride + acc * a.draft_row_stride;
  r.x = r.less && !a.draft ? a.tokens[(int64_t)b * a.drafts + acc] : -1;
  return r;
}
__device__ __forceinline__ double plain(float p) { return p > 0.f ? (double)p : 0.0; }
__device__ __forceinline__ double residual(float p, float q) { return p > fmaxf(q, 0.f) ? (double)p - (double)fmaxf(q, 0.f) : 0.0; }

__device__ __forceinline__ double sum64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// TP, TQ: types; V: values of one load (8 where every row starts on 16 bytes, else 1);
// HAS_Q: draft probabilities are given.
template <typename TP, typename TQ, int V, bool HAS_Q>
__global__ __launch_bounds__(kThreads) void sums_k(replay_accept_args a, Slices sl) {
  __shared__ double part[2][kWaves];
  const int b = fdiv(blockIdx.x, sl.fn), slice = blockIdx.x - b * sl.n;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int n = drafts_of(a, b), acc = accepted(a, b, n, lane);
  if (slice == 0 && threadIdx.x == 0) a.accepted[b] = acc;
  const Row row = row_of(a, b, acc, n);
  const TP *p = (const TP *)a.target + row.p;
  const TQ *q = (const TQ *)a.draft + row.q;
  double sr = 0.0, sp = 0.0;
  const int v0 = slice * sl.size, v1 = min(a.vocab, v0 + sl.size);
  for (int v = v0; v < v1; v += kStep) {
    float pv[8], qv[8];
    int at0, step;
    if constexpr (V == 8) {
      at0 = v + threadIdx.x * 8, step = 1;
      if (at0 + 8 <= v1) {
        load_vec<TP, 8>(p + at0, pv);
        if (HAS_Q && row.less) load_vec<TQ, 8>(q + at0, qv);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          pv[i] = at0 + i < v1 ? ldr<TP>(p + at0 + i) : 0.f;
          if (HAS_Q && row.less) qv[i] = at0 + i < v1 ? ldr<TQ>(q + at0 + i) : 0.f;
        }
      }
    } else {
      at0 = v + threadIdx.x, step = kThreads;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pv[i] = at0 + i * kThreads < v1 ? ldr<TP>(p + at0 + i * kThreads) : 0.f;
        if (HAS_Q && row.less) qv[i] = at0 + i * kThreads < v1 ? ldr<TQ>(q + at0 + i * kThreads) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double w = plain(pv[i]);
      sp += w;
      if (HAS_Q)
        sr += row.less ? residual(pv[i], qv[i]) : w;
      else
        sr += at0 + i * step == row.x ? 0.0 : w;
    }
  }
  sr = sum64(sr), sp = sum64(sp);
  if (lane == 0) part[0][wave] = sr, part[1][wave] = sp;
  __syncthreads();
  if (threadIdx.x == 0) {
    sr = sp = 0.0;
    for (int i = 0; i < kWaves; ++i) sr += part[0][i], sp += part[1][i];
    sl.sums[(int64_t)b * sl.n + slice] = make_double2(sr, sp);
  }
}

__device__ __forceinline__ double scan64(double v, int lane) {  // inclusive prefix sum of a wave
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const double o = __shfl_up(v, d, kWave);
    if (lane >= d) v += o;
  }
  return v;
}

// The first of a wave's values whose running sum from `run` exceeds want, else the last
// with any weight; -1 if none has.  run becomes the sum before it.
__device__ __forceinline__ int find64(double w, double want, double &run, int lane) {
  const double s = run + scan64(w, lane);
  const uint64_t over = __ballot(w > 0.0 && s > want), any = __ballot(w > 0.0);
  if (!any) return -1;
  const int i = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll(any);
  const double before = __shfl_up(s, 1, kWave);
  run = i ? __shfl(before, i, kWave) : run;
  return i;
}

constexpr int kRows = kStep / kWave;  // rows of 64 that the workgroup sums at a time

__global__ __launch_bounds__(kThreads) void pick_k(replay_accept_args a, Slices sl) {
  __shared__ double rows[kRows];
  const int b = blockIdx.x, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int acc = a.accepted[b], n = drafts_of(a, b);
  Row row = row_of(a, b, acc, n);
  const double2 *sums = sl.sums + (int64_t)b * sl.n;
  // Every wave adds the slices up; the totals say whether the residual has any weight.
  double tr = 0.0, tp = 0.0;
  for (int i = lane; i < sl.n; i += kWave) tr += sums[i].x, tp += sums[i].y;
  tr = sum64(tr), tp = sum64(tp);
  if (!(tr > 0.0)) row.less = false, row.x = -1, tr = tp;
  const bool by_p = !(row.less || row.x >= 0);
  if (!(tr > 0.0)) {  // also where p has a NaN sum: none, since NaN has no weight
    if (threadIdx.x == 0) a.next[b] = -1;
    return;
  }
  const double want = (double)a.uniforms[(int64_t)b * (a.drafts + 1) + a.drafts] * tr;
  // The slice: in turns of 64, keeping the last with weight in case rounding leaves none beyond want.
  int slice = -1;
  double run = 0.0, base = 0.0;
  for (int i0 = 0; i0 < sl.n; i0 += kWave) {
    const double2 s2 = i0 + lane < sl.n ? sums[i0 + lane] : make_double2(0.0, 0.0);
    const double w = by_p ? s2.y : s2.x;
    const double s = run + scan64(w, lane);
    const uint64_t over = __ballot(w > 0.0 && s > want), any = __ballot(w > 0.0);
    if (any) {
      const int i = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll(any);
      const double before = __shfl_up(s, 1, kWave);
      slice = i0 + i;
      base = i ? __shfl(before, i, kWave) : run;
    }
    if (over) break;
    run = __shfl(s, kWave - 1, kWave);
  }
  // The rows of 64 of the slice, kRows at a time, then the lane.
  const int v0 = slice * sl.size, v1 = min(a.vocab, v0 + sl.size);
  auto weight = [&](int v) -> double {
    if (v >= v1 || v == row.x) return 0.0;
    const float p = at(a.target, a.target_dtype, row.p + v);
    return row.less && a.draft ? residual(p, at(a.draft, a.draft_dtype, row.q + v)) : plain(p);
  };
  int token = -1;
  for (int v = v0; v < v1; v += kStep) {
    double w[kRows / kWaves];
#pragma unroll
    for (int i = 0; i < kRows / kWaves; ++i) w[i] = weight(v + (wave * (kRows / kWaves) + i) * kWave + lane);
    __syncthreads();  // the last turn's rows are read
#pragma unroll
    for (int i = 0; i < kRows / kWaves; ++i) {
      const double s = sum64(w[i]);
      if (lane == 0) rows[wave * (kRows / kWaves) + i] = s;
    }
    __syncthreads();
    const double rw = lane < kRows ? rows[lane] : 0.0;
    const double s = base + scan64(rw, lane);
    const uint64_t over = __ballot(rw > 0.0 && s > want), any = __ballot(rw > 0.0);
    if (any) {
      const int i = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll(any);
      const double before = __shfl_up(s, 1, kWave);
      double from = i ? __shfl(before, i, kWave) : base;
      const int lane_at = find64(weight(v + i * kWave + lane), want, from, lane);
      if (lane_at >= 0) token = v + i * kWave + lane_at;
    }
    if (over) break;  // the same for every wave
    base = __shfl(s, kWave - 1, kWave);
  }
  if (threadIdx.x == 0) a.next[b] = token;
}

// Slices of 2048 values, longer where there would be more than 4096 workgroups: those fill the card.
Slices slices_of(int batch, int vocab) {
  Slices s{};
  s.size = kStep;
  while ((int64_t)batch * ((vocab + (int64_t)s.size - 1) / s.size) > 4096 && s.size < vocab) s.size *= 2;
  s.n = (int)((vocab + (int64_t)s.size - 1) / s.size);
  s.fn = make_fastdiv((uint32_t)s.n);
  return s;
}

template <typename TP, typename TQ, bool HAS_Q>
void launch_sums(const replay_accept_args &a, const Slices &s, bool wide, hipStream_t st) {
  const dim3 grid((uint32_t)a.batch * s.n), block(kThreads);
  if (wide)
    hipLaunchKernelGGL((sums_k<TP, TQ, 8, HAS_Q>), grid, block, 0, st, a, s);
  else
    hipLaunchKernelGGL((sums_k<TP, TQ, 1, HAS_Q>), grid, block, 0, st, a, s);
}

template <typename TP>
void launch_q(const replay_accept_args &a, const Slices &s, bool wide, hipStream_t st) {
  if (!a.draft)
    launch_sums<TP, float, false>(a, s, wide, st);
  else if (a.draft_dtype == REPLAY_DT_BF16)
    launch_sums<TP, bf16_t, true>(a, s, wide, st);
  else
    launch_sums<TP, float, true>(a, s, wide, st);
}

}  // namespace

size_t accept_workspace(int batch, int vocab) {
  const Slices s = slices_of(batch, vocab);
  return (size_t)batch * s.n * sizeof(double2);
}

int launch_accept(const replay_accept_args &a, void *workspace, hipStream_t st) {
  Slices s = slices_of(a.batch, a.vocab);
  if ((int64_t)a.batch * s.n > 0x7fffffffLL) return (int)hipErrorInvalidValue;
  s.sums = (double2 *)workspace;
  const bool wide = !(((uintptr_t)a.target | (uintptr_t)a.draft) & 15u) &&
                    !((a.target_seq_stride | a.target_row_stride | a.draft_seq_stride | a.draft_row_stride) & 7);
  if (a.target_dtype == REPLAY_DT_BF16)
    launch_q<bf16_t>(a, s, wide, st);
  else
    launch_q<float>(a, s, wide, st);
  hipLaunchKernelGGL(pick_k, dim3(a.batch), dim3(kThreads), 0, st, a, s);
  return (int)hipGetLastError();
}

}  // namespace rssm
