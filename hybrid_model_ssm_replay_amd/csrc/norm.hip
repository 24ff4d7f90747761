// Gated norm over groups of channels, per token.
//
//   gate first:  h = y silu(z),  out = w h / sqrt(mean(h^2) + eps)
//   norm first:  out = w y / sqrt(mean(y^2) + eps) silu(z)
//
// HBM bound: read y and z, write out.  One wave a group of one token.
#include "ops.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sum64(float v) { return sum_quarters(sum16(v)); }

template <typename TY, typename TZ, typename TO, int V>
__global__ __launch_bounds__(kThreads) void gated_norm_k(replay_gated_norm_args a, FastDiv groups, int items) {
  const int lane = threadIdx.x % kWave;
  const int64_t i64 = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
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

template <typename TY, typename TZ, typename TO>
int launch(const replay_gated_norm_args &a, hipStream_t st) {
  const int groups = a.channels / a.group;
  const int items = a.tokens * groups;
  const dim3 grid((items + kThreads / kWave - 1) / (kThreads / kWave)), block(kThreads);
  const uintptr_t bits = (uintptr_t)a.y | (uintptr_t)a.z | (uintptr_t)a.out | (uintptr_t)a.weight;
  const bool wide = !(bits & 15u) && a.group % 8 == 0 && a.y_stride % 8 == 0 && a.z_stride % 8 == 0 && a.out_stride % 8 == 0;
  const FastDiv f = make_fastdiv((uint32_t)groups);
  if (wide)
    hipLaunchKernelGGL((gated_norm_k<TY, TZ, TO, 8>), grid, block, 0, st, a, f, items);
  else
    hipLaunchKernelGGL((gated_norm_k<TY, TZ, TO, 1>), grid, block, 0, st, a, f, items);
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
