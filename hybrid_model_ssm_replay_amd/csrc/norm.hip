// Gated norm over groups of channels, per token.
//
//   gate first:  h = y silu(z),  out = w h / sqrt(mean(h^2) + eps)
//   norm first:  out = w y / sqrt(mean(y^2) + eps) silu(z)
//
// HBM bound: read y and z, write out.  Both orders end in y silu(z) w times the
// root, so a lane keeps that product of its eight values (or up to four times
// eight) while the squares are added up: one pass over the data.  Groups of up to
// 128 values share a wave four at a time, longer ones have a wave; a wave takes
// several tokens of one group, which share the weights in its registers.
#include "ops.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

__device__ __forceinline__ float sum64(float v) { return sum_quarters(sum16(v)); }
template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
  v = sum16(v);
  if constexpr (LANES == 32) v += __shfl_xor(v, 16, kWave);
  if constexpr (LANES == 64) v = sum_quarters(v);
  return v;
}

// LANES lanes a group, IT steps of eight values a lane; TOK tokens a wave.
template <typename TY, typename TZ, typename TO, int LANES, int IT>
__global__ __launch_bounds__(kThreads) void gated_norm_k(replay_gated_norm_args a, int sets, FastDiv fsets, int tok) {
  constexpr int PER = kWave / LANES;  // groups of a wave
  const int lane = threadIdx.x % LANES, sub = threadIdx.x % kWave / LANES;
  const int64_t item = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
  const int64_t run = fdiv((int)item, fsets);  // a run of tok tokens, and PER neighbouring groups
  const int g = (int)(item - run * sets) * PER + sub, t0 = (int)run * tok;
  if (t0 >= a.tokens) return;
  const int t1 = min(a.tokens, t0 + tok);
  const bool group_there = g * a.group < a.channels;
  const int c0 = group_there ? g * a.group : 0;
  const float inv = 1.f / (float)a.group;
  float w[IT][8];
  bool in[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * LANES + lane) * 8;
    in[i] = group_there && c < a.group;
    if (in[i]) load_vec<float, 8>(a.weight + (a.weight_len == a.channels ? c0 : 0) + c, w[i]);
  }
  for (int t = t0; t < t1; ++t) {
    const TY *y = (const TY *)a.y + t * a.y_stride + c0 + lane * 8;
    const TZ *z = (const TZ *)a.z + t * a.z_stride + c0 + lane * 8;
    float h[IT][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      float zv[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) h[i][v] = 0.f, zv[v] = 0.f;
      if (in[i]) {
        load_vec<TY, 8>(y + i * LANES * 8, h[i]);
        load_vec<TZ, 8>(z + i * LANES * 8, zv);
      }
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const float g8 = silu(zv[v]);
        if (a.norm_first) ss = fmaf(h[i][v], h[i][v], ss);
        h[i][v] *= g8;
        if (!a.norm_first) ss = fmaf(h[i][v], h[i][v], ss);
      }
    }
    const float r = rsqrtf(sum_lanes<LANES>(ss) * inv + a.eps);
    TO *out = (TO *)a.out + t * a.out_stride + c0 + lane * 8;
#pragma unroll
    for (int i = 0; i < IT; ++i)
      if (in[i]) {
#pragma unroll
        for (int v = 0; v < 8; ++v) h[i][v] *= r * w[i][v];
        store_vec<TO, 8>(out + i * LANES * 8, h[i]);
      }
  }
}

// Any group, any alignment: one wave a group of one token, two passes.
template <typename TY, typename TZ, typename TO, int V>
__global__ __launch_bounds__(kThreads) void gated_norm_any_k(replay_gated_norm_args a, FastDiv groups, int items) {
  const int lane = threadIdx.x % kWave;
  const int64_t i64 = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
  if (i64 >= items) return;
  const int t = fdiv((int)i64, groups), g = (int)i64 - t * (int)groups.d;
  const int c0 = g * a.group;
  const TY *y = (const TY *)a.y + t * a.y_stride + c0;
  const TZ *z = (const TZ *)a.z + t * a.z_stride + c0;
  const float *w = a.weight + (a.weight_len == a.channels ? c0 : 0);
  TO *out = (TO *)a.out + t * a.out_stride + c0;
  float ss = 0.f;
  for (int c = lane * V; c < a.group; c += kWave * V) {
    float yv[V], zv[V];
    load_vec<TY, V>(y + c, yv);
    load_vec<TZ, V>(z + c, zv);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float h = a.norm_first ? yv[v] : yv[v] * silu(zv[v]);
      ss = fmaf(h, h, ss);
    }
  }
  const float r = rsqrtf(sum64(ss) / (float)a.group + a.eps);
  for (int c = lane * V; c < a.group; c += kWave * V) {
    float yv[V], zv[V], wv[V], o[V];
    load_vec<TY, V>(y + c, yv);
    load_vec<TZ, V>(z + c, zv);
    load_vec<float, V>(w + c, wv);
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = yv[v] * silu(zv[v]) * r * wv[v];
    store_vec<TO, V>(out + c, o);
  }
}

template <typename TY, typename TZ, typename TO, int LANES, int IT>
int launch_fast(const replay_gated_norm_args &a, hipStream_t st) {
  constexpr int PER = kWave / LANES;
  const int groups = a.channels / a.group, sets = (groups + PER - 1) / PER;
  // Four tokens a wave once that still leaves sixteen waves a CU.
  const int tok = (int64_t)a.tokens * sets >= 4 * 16 * 256 ? 4 : 1;
  const int64_t items = (int64_t)((a.tokens + tok - 1) / tok) * sets;
  hipLaunchKernelGGL((gated_norm_k<TY, TZ, TO, LANES, IT>), dim3((uint32_t)((items + kWaves - 1) / kWaves)), dim3(kThreads), 0,
                     st, a, sets, make_fastdiv((uint32_t)sets), tok);
  return (int)hipGetLastError();
}

template <typename TY, typename TZ, typename TO>
int launch(const replay_gated_norm_args &a, hipStream_t st) {
  const uintptr_t bits = (uintptr_t)a.y | (uintptr_t)a.z | (uintptr_t)a.out | (uintptr_t)a.weight;
  const int64_t steps = a.group | a.y_stride | a.z_stride | a.out_stride;
  if (!(bits & 15u) && steps % 8 == 0) {
    if (a.group <= 128) return launch_fast<TY, TZ, TO, 16, 1>(a, st);
    if (a.group <= 256) return launch_fast<TY, TZ, TO, 32, 1>(a, st);
    if (a.group <= 512) return launch_fast<TY, TZ, TO, 64, 1>(a, st);
    if (a.group <= 1024) return launch_fast<TY, TZ, TO, 64, 2>(a, st);
    if (a.group <= 2048) return launch_fast<TY, TZ, TO, 64, 4>(a, st);
  }
  const int groups = a.channels / a.group;
  const int items = a.tokens * groups;
  const dim3 grid((items + kWaves - 1) / kWaves), block(kThreads);
  const FastDiv f = make_fastdiv((uint32_t)groups);
  if (!(bits & 15u) && steps % 8 == 0)
    hipLaunchKernelGGL((gated_norm_any_k<TY, TZ, TO, 8>), grid, block, 0, st, a, f, items);
  else if (!(bits & 7u) && steps % 2 == 0)  // pairs
    hipLaunchKernelGGL((gated_norm_any_k<TY, TZ, TO, 2>), grid, block, 0, st, a, f, items);
  else
    hipLaunchKernelGGL((gated_norm_any_k<TY, TZ, TO, 1>), grid, block, 0, st, a, f, items);
  return (int)hipGetLastError();
}

template <typename TY, typename TZ>
int launch_o(const replay_gated_norm_args &a, hipStream_t st) {
  return a.out_dtype == REPLAY_DT_BF16 ? launch<TY, TZ, bf16_t>(a, st) : launch<TY, TZ, float>(a, st);
}
template <typename TY>
int launch_z(const replay_gated_norm_args &a, hipStream_t st) {
  return a.z_dtype == REPLAY_DT_BF16 ? launch_o<TY, bf16_t>(a, st) : launch_o<TY, float>(a, st);
}

}  // namespace

int launch_gated_norm(const replay_gated_norm_args &a, hipStream_t st) {
  return a.y_dtype == REPLAY_DT_BF16 ? launch_z<bf16_t>(a, st) : launch_z<float>(a, st);
}

}  // namespace rssm
