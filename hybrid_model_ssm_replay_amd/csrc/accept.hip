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
// 128 sequences of 50021, bf16: sums_k reads 26 MB in 9.1 us, pick_k takes 7.4 (a chain of
// loads and scans, each waiting for the one before); one of 131072: 3.5 and 4.0 us.
//
// Sums are float64: p - q of float32 or bf16 values is exact or nearly so there,
// and the order of a sum over a large vocabulary then moves a sampling border by
// about 1e-13 of the total instead of 1e-4.
#include "ops.h"
#include "pieces.h"

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

__device__ __forceinline__ double sum64(double v) { return lane_value(scan64(v), kWave - 1); }

// The first lane whose running sum from `run` exceeds want, else the last with any
// weight, else -1.  over: the first kind.  run becomes the sum before that lane, or
// after all of them where there is none beyond want.
__device__ __forceinline__ int find64(double w, double want, double &run, bool &over) {
  const double s = run + scan64(w);
  const uint64_t beyond = __ballot(w > 0.0 && s > want), any = __ballot(w > 0.0);
  over = beyond != 0;
  const int i = over ? __builtin_ctzll(beyond) : any ? 63 - __builtin_clzll(any) : -1;
  run = over ? (i ? lane_value(s, i - 1) : run) : lane_value(s, kWave - 1);
  return i;
}

// TP, TQ: types; HAS_Q: draft probabilities are given.
template <typename TP, typename TQ, bool HAS_Q>
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
    const int at0 = v + threadIdx.x * 8, there = v1 - at0;
    float pv[8], qv[8];
    load_part<TP, 8>(p + at0, there, pv);
    if (HAS_Q && row.less) load_part<TQ, 8>(q + at0, there, qv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double w = plain(pv[i]);
      sp += w;
      if (HAS_Q)
        sr += row.less ? residual(pv[i], qv[i]) : w;
      else
        sr += at0 + i == row.x ? 0.0 : w;
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

constexpr int kRows = kStep / kWave;  // rows of 64 that the workgroup sums at a time

__global__ __launch_bounds__(kThreads) void pick_k(replay_accept_args a, Slices sl) {
  __shared__ double rows[kRows];
  const int b = blockIdx.x, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int acc = a.accepted[b], n = drafts_of(a, b);
  Row row = row_of(a, b, acc, n);
  const double2 *sums = sl.sums + (int64_t)b * sl.n;
  const double u = (double)a.uniforms[(int64_t)b * (a.drafts + 1) + a.drafts];
  // Every wave adds the slices up, a lane a run of neighbours; the totals say whether
  // the residual has any weight.
  const int per = (sl.n + kWave - 1) / kWave;
  double wr = 0.0, wp = 0.0;
  for (int i = lane * per; i < min(sl.n, (lane + 1) * per); ++i) wr += sums[i].x, wp += sums[i].y;
  double total = sum64(wr);
  const bool by_p = !(total > 0.0) || !row.less;
  if (by_p) row.less = false, row.x = -1, total = sum64(wp);
  if (!(total > 0.0)) {
    if (threadIdx.x == 0) a.next[b] = -1;
    return;
  }
  const double want = u * total;
  // The lane's run, the slice in it, the rows of 64 of the slice, the lane.  Where
  // rounding leaves nothing beyond want, the last with any weight.
  double run = 0.0;
  bool over;
  const int l = find64(by_p ? wp : wr, want, run, over);
  if (!over) {  // the sum before that lane
    const double s = scan64(by_p ? wp : wr);
    run = l ? lane_value(s, l - 1) : 0.0;
  }
  int slice = -1;
  double base = run;
  for (int i = l * per; i < min(sl.n, (l + 1) * per); ++i) {
    const double w = by_p ? sums[i].y : sums[i].x;
    if (w > 0.0) {
      slice = i, base = run;
      if (run + w > want) break;
    }
    run += w;
  }
  const int v0 = slice * sl.size, v1 = min(a.vocab, v0 + sl.size);
  constexpr int MINE = kRows / kWaves;  // rows of a wave
  // All loads of a turn are under way together: no branch stands between them.
  auto values = [&](const void *p, int dtype, int64_t at, int v, float (&w)[MINE]) {
    const int last = v1 - 1;
    if (dtype == REPLAY_DT_BF16) {
#pragma unroll
      for (int i = 0; i < MINE; ++i) w[i] = ldr<bf16_t>((const bf16_t *)p + at + min(v + i * kWave, last));
    } else {
#pragma unroll
      for (int i = 0; i < MINE; ++i) w[i] = ldr<float>((const float *)p + at + min(v + i * kWave, last));
    }
  };
  int token = -1;
  for (int v = v0; v < v1; v += kStep) {
    const int mine = v + wave * MINE * kWave + lane;
    float pw[MINE], qw[MINE] = {};
    values(a.target, a.target_dtype, row.p, mine, pw);
    if (row.less && a.draft) values(a.draft, a.draft_dtype, row.q, mine, qw);
    double w[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int vi = mine + i * kWave;
      w[i] = vi >= v1 || vi == row.x ? 0.0 : residual(pw[i], qw[i]);  // without q: p itself
    }
    __syncthreads();  // the last turn's rows are read
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const double s = scan64(w[i]);
      if (lane == kWave - 1) rows[wave * MINE + i] = s;
    }
    __syncthreads();
    const double rw = lane < kRows ? rows[lane] : 0.0, start = base;
    const int i = find64(rw, want, base, over);
    if (i >= 0 && i / MINE == wave) {
      double from = over ? base : start + (i ? lane_value(scan64(rw), i - 1) : 0.0);
      bool hit;
      double wi = 0.0;
#pragma unroll
      for (int k = 0; k < MINE; ++k) wi = k == i % MINE ? w[k] : wi;
      const int at_lane = find64(wi, want, from, hit);
      if (at_lane >= 0) token = v + i * kWave + at_lane;
    }
    if (over) break;  // the same for every wave
  }
  // The wave whose rows held it; of several turns' last ones, the latest.
  __shared__ int found[kWaves];
  if (lane == 0) found[wave] = token;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kWaves; ++i) token = max(token, found[i]);
    a.next[b] = token;
  }
}

// Slices of 2048 values, longer where there would be more than 2048 workgroups: those
// fill the card at once (128 sequences of 50021, bf16: sums_k 9.1 us, with 2048 values
// 12.7).
Slices slices_of(int batch, int vocab) {
  Slices s{};
  s.size = kStep;
  while ((int64_t)batch * ((vocab + (int64_t)s.size - 1) / s.size) > 2048 && s.size < vocab) s.size *= 2;
  s.n = (int)((vocab + (int64_t)s.size - 1) / s.size);
  s.fn = make_fastdiv((uint32_t)s.n);
  return s;
}

template <typename TP, typename TQ, bool HAS_Q>
void launch_sums(const replay_accept_args &a, const Slices &s, hipStream_t st) {
  const dim3 grid((uint32_t)a.batch * s.n), block(kThreads);
  hipLaunchKernelGGL((sums_k<TP, TQ, HAS_Q>), grid, block, 0, st, a, s);
}

template <typename TP>
void launch_q(const replay_accept_args &a, const Slices &s, hipStream_t st) {
  if (!a.draft)
    launch_sums<TP, float, false>(a, s, st);
  else if (a.draft_dtype == REPLAY_DT_BF16)
    launch_sums<TP, bf16_t, true>(a, s, st);
  else
    launch_sums<TP, float, true>(a, s, st);
}

}  // namespace

size_t accept_workspace(int batch, int vocab) {
  const Slices s = slices_of(batch, vocab);
  return (size_t)batch * s.n * sizeof(double2);
}

int launch_accept(const replay_accept_args &a, void *workspace, hipStream_t st) {
  Slices s = slices_of(a.batch, a.vocab);
  if ((int64_t)a.batch * s.n > kMostBlocks) return kTooLarge;
  s.sums = (double2 *)workspace;
  if (a.target_dtype == REPLAY_DT_BF16)
    launch_q<bf16_t>(a, s, st);
  else
    launch_q<float>(a, s, st);
  hipLaunchKernelGGL(pick_k, dim3(a.batch), dim3(kThreads), 0, st, a, s);
  return (int)hipGetLastError();
}

}  // namespace rssm
