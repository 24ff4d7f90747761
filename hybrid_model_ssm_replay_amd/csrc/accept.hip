// Acceptance of drafted tokens and the token drawn after them.
//
// Draft i is kept while u_i q_i(x_i) < p_i(x_i).  The refused draft's residual
// max(p - q, 0), or p after the last draft, is sampled by inverse CDF.  One row
// of p and one of q per sequence have to be read: HBM bound for many sequences,
// latency bound for one.
//
// Sums are float64: p - q of float32 or bf16 values is exact or nearly so there,
// and the order of a sum over a large vocabulary then moves a sampling border by
// about 1e-13 of the total instead of 1e-4.
#include "ops.h"

namespace rssm {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;

template <typename T>
__device__ __forceinline__ float at(const void *p, int64_t i) {
  return ldr<T>(reinterpret_cast<const T *>(p) + i);
}
__device__ __forceinline__ float at(const void *p, int dtype, int64_t i) {
  return dtype == REPLAY_DT_BF16 ? at<bf16_t>(p, i) : at<float>(p, i);
}

__device__ __forceinline__ double shfl_up_d(double v, int d) { return __shfl_up(v, d, kWave); }

__device__ __forceinline__ double scan64(double v, int lane) {  // inclusive prefix sum of a wave
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const double o = shfl_up_d(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__global__ __launch_bounds__(kThreads) void accept_k(replay_accept_args a) {
  __shared__ double part[kWaves];
  __shared__ int found[kWaves], last[kWaves];
  const int b = blockIdx.x, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int V = a.vocab, T = a.drafts;
  int n = T;
  if (a.lengths) n = min(max(a.lengths[b], 0), T);
  int acc = 0;
  for (; acc < n; ++acc) {
    const int x = a.tokens[(int64_t)b * T + acc];
    if (x < 0 || x >= V) break;
    const double p = at(a.target, a.target_dtype, b * a.target_seq_stride + acc * a.target_row_stride + x);
    double q = a.draft ? (double)at(a.draft, a.draft_dtype, b * a.draft_seq_stride + acc * a.draft_row_stride + x) : 1.0;
    if (!(q > 0.0)) q = 0.0;
    if (!((double)a.uniforms[(int64_t)b * (T + 1) + acc] * q < p)) break;
  }
  bool less = acc < n;
  const int xr = less ? a.tokens[(int64_t)b * T + acc] : -1;
  const int64_t p0 = b * a.target_seq_stride + acc * a.target_row_stride;
  const int64_t q0 = b * a.draft_seq_stride + acc * a.draft_row_stride;
  auto weight = [&](int v) -> double {
    const double p = at(a.target, a.target_dtype, p0 + v);
    double q = 0.0;
    if (less) {
      if (a.draft)
        q = at(a.draft, a.draft_dtype, q0 + v);
      else if (v == xr)
        return 0.0;
    }
    if (!(q > 0.0)) q = 0.0;
    return p > q ? p - q : 0.0;
  };
  const int step = ((V + kWaves - 1) / kWaves + kWave - 1) / kWave * kWave;  // a wave's stretch of the vocabulary
  const int v0 = min(V, wave * step), v1 = min(V, v0 + step);
  double total = 0.0;
  for (int pass = 0; pass < 2; ++pass) {
    double s = 0.0;
    for (int v = v0 + lane; v < v1; v += kWave) s += weight(v);
    s = scan64(s, lane);
    if (lane == kWave - 1) part[wave] = s;
    __syncthreads();
    total = 0.0;
    for (int i = 0; i < kWaves; ++i) total += part[i];
    __syncthreads();
    if (total > 0.0 || !less) break;
    less = false;
  }
  double run = 0.0;
  for (int i = 0; i < wave; ++i) run += part[i];
  const double want = (double)a.uniforms[(int64_t)b * (T + 1) + T] * total;
  int hit = -1, end = -1;
  for (int v = v0; v < v1; v += kWave) {
    const double w = v + lane < v1 ? weight(v + lane) : 0.0;
    const double s = run + scan64(w, lane);
    const uint64_t over = __ballot(w > 0.0 && s > want), any = __ballot(w > 0.0);
    if (any) end = v + 63 - __clzll(any);
    if (hit < 0 && over) hit = v + __ffsll((unsigned long long)over) - 1;
    run = __shfl(s, kWave - 1, kWave);
  }
  if (lane == 0) found[wave] = hit, last[wave] = end;
  __syncthreads();
  if (threadIdx.x == 0) {
    int token = -1, l = -1;
    for (int i = 0; i < kWaves; ++i) {
      if (token < 0 && found[i] >= 0) token = found[i];
      if (last[i] >= 0) l = last[i];
    }
    a.accepted[b] = acc;
    a.next[b] = token >= 0 ? token : l;
  }
}

}  // namespace

size_t accept_workspace(int, int) { return 16; }

int launch_accept(const replay_accept_args &a, void *, hipStream_t st) {
  hipLaunchKernelGGL(accept_k, dim3(a.batch), dim3(kThreads), 0, st, a);
  return (int)hipGetLastError();
}

}  // namespace rssm
