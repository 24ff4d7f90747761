// Short causal depthwise convolution: prompts (packed) and tokens or drafts (ring).
//
//   y[t][c] = act(bias[c] + sum_k w[c][k] x[t - K + 1 + k][c]),  K = 2..4 taps
//
// A few operations per element: HBM bound.  A thread owns V neighbouring
// channels (16 bytes) and walks along the tokens with the last K - 1 inputs in
// registers, so each input is read once (a prompt tile re-reads K - 1 rows).  It
// issues the loads of several tokens (a prompt) or batch rows (a step) at a time:
// that is what keeps enough bytes under way, and in a step it also shares the
// weights, which are as large as a row's inputs and outputs together.
#include "ops.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;   // tokens of a prompt tile
constexpr int kAhead = 8;   // tokens of a tile whose loads are under way together

template <int V, int K>
struct Taps {
  float w[K][V], b[V];
};

template <int V, int K>
__device__ __forceinline__ Taps<V, K> load_taps(const ShortConvArgs &a, int c) {
  Taps<V, K> t;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < K; ++k) t.w[k][v] = a.weight[(size_t)(c + v) * K + k];
    t.b[v] = a.bias ? a.bias[c + v] : 0.f;
  }
  return t;
}

template <int V, int K>
__device__ __forceinline__ void taps_out(const Taps<V, K> &t, const float (&h)[K - 1][V], const float (&x)[V], int silu_on,
                                         float (&y)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float s = t.b[v];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) s = fmaf(t.w[k][v], h[k][v], s);
    s = fmaf(t.w[K - 1][v], x[v], s);
    y[v] = silu_on ? silu(s) : s;
  }
}

template <int V, int K>
__device__ __forceinline__ void push(float (&h)[K - 1][V], const float (&x)[V]) {
#pragma unroll
  for (int k = 0; k < K - 2; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) h[k][v] = h[k + 1][v];
#pragma unroll
  for (int v = 0; v < V; ++v) h[K - 2][v] = x[v];
}

// Where channel c of output row r goes, and the distance between rows.
template <typename T>
__device__ __forceinline__ T *out_of(const ShortConvArgs &a, int c, int *width) {
  const int f = c < a.w[0] ? 0 : c < a.w[0] + a.w[1] ? 1 : 2;
  *width = a.w[f];
  return reinterpret_cast<T *>(a.out[f]) + (c - (f == 0 ? 0 : f == 1 ? a.w[0] : a.w[0] + a.w[1]));
}

// ROWS batch rows a thread.
template <typename T, int V, int K, int ROWS>
__global__ __launch_bounds__(kThreads) void short_conv_step_k(ShortConvArgs a, FastDiv per_row) {
  const int blk = blockIdx.x;
  const int b0 = fdiv(blk, per_row) * ROWS;
  const int c = ((blk - b0 / ROWS * (int)per_row.d) * kThreads + threadIdx.x) * V;
  if (c >= a.C) return;
  const size_t slot_elems = (size_t)a.batch * a.C;
  const T *x = reinterpret_cast<const T *>(a.x) + c;
  int slot[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int pos = b0 + i < a.batch ? a.pos[b0 + i] : -1;
    if (pos < 0 && b0 + i < a.batch && c == 0 && a.status) atomicOr(a.status, REPLAY_STATUS_BAD_POINTERS);
    slot[i] = pos < 0 ? -1 : pos % a.slots;  // -1: nothing to do
  }
  float h[ROWS][K - 1][V], v[ROWS][V];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    if (slot[i] >= 0) {
      const T *ring = reinterpret_cast<const T *>(a.ring) + (size_t)(b0 + i) * a.C + c;
#pragma unroll
      for (int k = 0; k < K - 1; ++k) {
        int s = slot[i] - (K - 1) + k;
        if (s < 0) s += a.slots;
        load_vec<T, V>(ring + s * slot_elems, h[i][k]);
      }
      load_vec<T, V>(x + (b0 + i) * a.seq_stride, v[i]);
    }
  const Taps<V, K> taps = load_taps<V, K>(a, c);
  int width;
  T *out = out_of<T>(a, c, &width);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (slot[i] < 0) continue;
    T *ring = reinterpret_cast<T *>(a.ring) + (size_t)(b0 + i) * a.C + c;
    T *to = out + (size_t)(b0 + i) * a.T * width;
    int s = slot[i];
    for (int t = 0; t < a.T; ++t) {
      float y[V], next[V];
      if (t + 1 < a.T) load_vec<T, V>(x + (b0 + i) * a.seq_stride + (t + 1) * a.row_stride, next);
      taps_out<V, K>(taps, h[i], v[i], a.silu, y);
      store_vec<T, V>(to + (size_t)t * width, y);
      store_vec<T, V>(ring + s * slot_elems, v[i]);
      s = s + 1 == a.slots ? 0 : s + 1;
      push<V, K>(h[i], v[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = next[e];
    }
  }
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void short_conv_prompt_k(ShortConvArgs a, FastDiv per_item) {
  const int item = fdiv(blockIdx.x, per_item);
  const int c = ((blockIdx.x - item * (int)per_item.d) * kThreads + threadIdx.x) * V;
  const Item it = find_item(a.p, item, kTile);
  const int t0 = it.index * kTile;
  if (c >= a.C || it.index < 0 || (t0 >= it.len && it.index > 0)) return;
  const int row = batch_row(a.p, it.seq, it.index == 0 && c == 0);
  if (row < 0) return;
  const T *x = reinterpret_cast<const T *>(a.x) + (size_t)it.begin * a.row_stride + c;
  float h[K - 1][V];
  if (t0 == 0) {
    // The first tile also replaces the ring's history by the sequence's last
    // inputs: the same thread reads the old slots before it writes them.
    const size_t slot_elems = (size_t)a.batch * a.C;
    T *ring = reinterpret_cast<T *>(a.ring) + (size_t)row * a.C + c;
    int pos = a.pos ? a.pos[row] : 0;
    if (pos < 0) {
      if (c == 0 && a.status) atomicOr(a.status, REPLAY_STATUS_BAD_POINTERS);
      pos = 0;
    }
    const int slot = pos % a.slots;
    const bool known = a.p.resume && a.p.resume[it.seq];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      int s = slot - (K - 1) + k;
      if (s < 0) s += a.slots;
      if (known) {
        load_vec<T, V>(ring + s * slot_elems, h[k]);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) h[k][v] = 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      int s = slot - (K - 1) + k;
      if (s < 0) s += a.slots;
      const int t = it.len - (K - 1) + k;  // negative: that far into the old history
      float v[V];
      if (t >= 0) {
        load_vec<T, V>(x + (size_t)t * a.row_stride, v);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = j == K - 1 + t ? h[j][i] : v[i];
      }
      store_vec<T, V>(ring + s * slot_elems, v);
    }
  } else {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) load_vec<T, V>(x + (size_t)(t0 - (K - 1) + k) * a.row_stride, h[k]);
  }
  const Taps<V, K> taps = load_taps<V, K>(a, c);
  int width;
  T *out = out_of<T>(a, c, &width) + (size_t)it.begin * width;
  const int t1 = min(it.len, t0 + kTile);
  for (int t = t0; t < t1; t += kAhead) {
    float v[kAhead][V];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_vec<T, V>(x + (size_t)min(t + i, t1 - 1) * a.row_stride, v[i]);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float y[V];
      taps_out<V, K>(taps, h, v[i], a.silu, y);
      if (t + i < t1) store_vec<T, V>(out + (size_t)(t + i) * width, y);
      push<V, K>(h, v[i]);
    }
  }
}

// Sixteen bytes a thread where every row, field and pointer allows it.
template <typename T>
bool wide(const ShortConvArgs &a, int v) {
  uintptr_t bits = (uintptr_t)a.x | (uintptr_t)a.ring;
  for (int i = 0; i < 3; ++i) {
    if (a.w[i] % v) return false;
    if (a.w[i]) bits |= (uintptr_t)a.out[i];
  }
  return !(bits & 15u) && a.row_stride % v == 0 && a.seq_stride % v == 0;
}

template <typename T, int V, int K, int ROWS>
void launch_step(const ShortConvArgs &a, int per, hipStream_t st) {
  hipLaunchKernelGGL((short_conv_step_k<T, V, K, ROWS>), dim3((uint32_t)((a.batch + ROWS - 1) / ROWS * per)), dim3(kThreads), 0,
                     st, a, make_fastdiv((uint32_t)per));
}

template <typename T, int V, int K>
int launch(const ShortConvArgs &a, bool prompt, hipStream_t st) {
  const int per = (a.C + kThreads * V - 1) / (kThreads * V);
  const int64_t rows = prompt ? items_of(a.p.tokens, a.p.n, kTile) : a.batch;
  if (rows * per > 0x7fffffffLL) return (int)hipErrorInvalidValue;
  if (prompt) {
    hipLaunchKernelGGL((short_conv_prompt_k<T, V, K>), dim3((uint32_t)(rows * per)), dim3(kThreads), 0, st, a,
                       make_fastdiv((uint32_t)per));
  } else if (rows * per >= 2 * 4 * 256 / 2) {  // two rows a thread still leave two workgroups a CU
    launch_step<T, V, K, 2>(a, per, st);
  } else {
    launch_step<T, V, K, 1>(a, per, st);
  }
  return (int)hipGetLastError();
}

template <typename T>
int dispatch(const ShortConvArgs &a, bool prompt, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(T);
  if (wide<T>(a, W)) {
    if (a.K == 2) return launch<T, W, 2>(a, prompt, st);
    if (a.K == 3) return launch<T, W, 3>(a, prompt, st);
    return launch<T, W, 4>(a, prompt, st);
  }
  if (a.K == 2) return launch<T, 1, 2>(a, prompt, st);
  if (a.K == 3) return launch<T, 1, 3>(a, prompt, st);
  return launch<T, 1, 4>(a, prompt, st);
}

int any(const ShortConvArgs &a, bool prompt, hipStream_t st) {
  return a.dtype == REPLAY_DT_BF16 ? dispatch<bf16_t>(a, prompt, st) : dispatch<float>(a, prompt, st);
}

}  // namespace

int launch_short_conv_step(const ShortConvArgs &a, hipStream_t st) { return any(a, false, st); }
int launch_short_conv_prompt(const ShortConvArgs &a, hipStream_t st) { return any(a, true, st); }

}  // namespace rssm
