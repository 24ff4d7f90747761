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
// With 10240 channels, 4 taps, bf16: a prompt of 8192 tokens moves 336 MB in 74 us (4.5
// TB/s; a large copy reaches 5.1), a step of 256 rows 31 MB in 11 us.  Rows of odd
// length cost more, all accesses being unaligned and the threads at a field's border
// going element by element: 4096 tokens of 10235 channels 168 MB in 108 us, a step of
// 256 rows 20 us.
#include "ops.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // tokens of a tile whose loads are under way while as many are computed

template <int V, int K>
struct Taps {
  float w[K][V], b[V];
};

// The workgroup's taps go through LDS: a thread's own lie 16 V K bytes from its
// neighbour's, so reading them directly would touch eight times the lines (a step
// of 256 rows: 12.1 us so, 14.5 directly).  Granules of 16 bytes are permuted so that
// neither side meets a bank twice.  Every thread of the workgroup takes part.
template <int V, int K>
struct TapsLds {
  static constexpr int kGranules = kThreads * V * K / 4;
  float4 at[kGranules];
  __device__ __forceinline__ static int place(int e) { return e ^ (e >> 3 & 15); }
  // c0: the workgroup's first channel.
  __device__ __forceinline__ void stage(const ShortConvArgs &a, int c0) {
    const float *w = a.weight + (size_t)c0 * K;
    const int64_t n = (int64_t)(a.C - c0) * K;  // values there are
#pragma unroll
    for (int i = 0; i < kGranules / kThreads; ++i) {
      const int e = i * kThreads + threadIdx.x;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (4 * e + 4 <= n)
        v = ld4(w + 4 * e);
      else if (4 * e < n)
        v = make_float4(w[4 * e], 4 * e + 1 < n ? w[4 * e + 1] : 0.f, 4 * e + 2 < n ? w[4 * e + 2] : 0.f, 0.f);
      at[place(e)] = v;
    }
  }
  __device__ __forceinline__ Taps<V, K> get(const ShortConvArgs &a, int c, int n) const {
    Taps<V, K> t;
    float f[V * K];
#pragma unroll
    for (int i = 0; i < V * K / 4; ++i) {
      const float4 v = at[place(threadIdx.x * (V * K / 4) + i)];
      f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int k = 0; k < K; ++k) t.w[k][v] = f[v * K + k];
      t.b[v] = 0.f;
    }
    if (a.bias) load_part<float, V>(a.bias + c, n, t.b);
    return t;
  }
};

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

// Where channels c .. c + V - 1 go: element (row, v) at base + row width + v, all in
// one field, or each in its own.
template <typename T, int V>
struct Out {
  T *base;
  int width, n;        // n of the V channels exist
  bool one;            // in one field
  int c;

  __device__ __forceinline__ static int field(const ShortConvArgs &a, int c) { return c < a.w[0] ? 0 : c < a.w[0] + a.w[1] ? 1 : 2; }
  __device__ __forceinline__ Out(const ShortConvArgs &a, int c0) : c(c0) {
    n = min(V, a.C - c0);
    const int f = field(a, c0);
    one = field(a, c0 + n - 1) == f;
    width = a.w[f];
    base = reinterpret_cast<T *>(a.out[f]) + (c0 - (f == 0 ? 0 : f == 1 ? a.w[0] : a.w[0] + a.w[1]));
  }
  __device__ __forceinline__ void store(const ShortConvArgs &a, size_t row, const float (&y)[V]) const {
    if (one) {
      store_part<T, V>(base + row * width, n, y);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < n) {
          const int f = field(a, c + v);
          const float y1[1] = {y[v]};
          store_vec<T, 1>(reinterpret_cast<T *>(a.out[f]) + row * a.w[f] + (c + v - (f == 0 ? 0 : f == 1 ? a.w[0] : a.w[0] + a.w[1])), y1);
        }
    }
  }
};

// V elements as they lie in memory: what a thread holds of loads under way.
template <typename T, int V, bool WHOLE>
struct Held {
  typename Elems<T, V>::words w;
  __device__ __forceinline__ void load(const T *p, int n) {
    if constexpr (WHOLE) {
      w = *reinterpret_cast<const typename Elems<T, V>::loose *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t u = i < n ? (sizeof(T) == 4 ? __float_as_uint(ldr<T>(p + i)) : __float_as_uint(ldr<T>(p + i)) >> 16) : 0u;
        if constexpr (sizeof(T) == 4)
          w[i] = u;
        else
          w[i / 2] = i % 2 ? w[i / 2] | u << 16 : u;
      }
    }
  }
  __device__ __forceinline__ void store(T *p, int n) const {
    if constexpr (WHOLE) {
      *reinterpret_cast<typename Elems<T, V>::loose *>(p) = w;
    } else {
      float v[V];
      get(v);
      store_part<T, V>(p, n, v);
    }
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4)
        v[i] = __uint_as_float(w[i]);
      else
        v[i] = i % 2 ? __uint_as_float(w[i / 2] & 0xFFFF0000u) : __uint_as_float(w[i / 2] << 16);
    }
  }
};

// ROWS batch rows a thread.  WHOLE: its V channels exist and are in one field.
template <typename T, int V, int K, int ROWS, bool WHOLE>
__device__ __forceinline__ void step_body(const ShortConvArgs &a, const TapsLds<V, K> &lds, const Out<T, V> &out, int c, int b0) {
  const size_t slot_elems = (size_t)a.batch * a.C;
  const T *x = reinterpret_cast<const T *>(a.x) + c;
  int slot[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int pos = b0 + i < a.batch ? a.pos[b0 + i] : -1;
    if (pos < 0 && b0 + i < a.batch && c == 0 && a.status) atomicOr(a.status, REPLAY_STATUS_BAD_POINTERS);
    slot[i] = pos < 0 ? -1 : pos % a.slots;  // -1: nothing to do
  }
  Held<T, V, WHOLE> old[ROWS][K - 1], in[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (slot[i] < 0) continue;
    const T *ring = reinterpret_cast<const T *>(a.ring) + (size_t)(b0 + i) * a.C + c;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      int s = slot[i] - (K - 1) + k;
      if (s < 0) s += a.slots;
      old[i][k].load(ring + s * slot_elems, out.n);
    }
    in[i].load(x + (b0 + i) * a.seq_stride, out.n);
  }
  const Taps<V, K> taps = lds.get(a, c, out.n);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (slot[i] < 0) continue;
    T *ring = reinterpret_cast<T *>(a.ring) + (size_t)(b0 + i) * a.C + c;
    float h[K - 1][V];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) old[i][k].get(h[k]);
    int s = slot[i];
    for (int t = 0; t < a.T; ++t) {
      Held<T, V, WHOLE> next = in[i];
      if (t + 1 < a.T) next.load(x + (b0 + i) * a.seq_stride + (t + 1) * a.row_stride, out.n);
      float v[V], y[V];
      in[i].get(v);
      taps_out<V, K>(taps, h, v, a.silu, y);
      if constexpr (WHOLE)
        store_vec<T, V>(out.base + ((size_t)(b0 + i) * a.T + t) * out.width, y);
      else
        out.store(a, (size_t)(b0 + i) * a.T + t, y);
      in[i].store(ring + s * slot_elems, out.n);
      s = s + 1 == a.slots ? 0 : s + 1;
      push<V, K>(h, v);
      in[i] = next;
    }
  }
}

template <typename T, int V, int K, int ROWS>
__global__ __launch_bounds__(kThreads) void short_conv_step_k(ShortConvArgs a, FastDiv per_row) {
  const int blk = blockIdx.x, set = fdiv(blk, per_row);
  const int c0 = (blk - set * (int)per_row.d) * kThreads * V, c = c0 + threadIdx.x * V;
  __shared__ TapsLds<V, K> lds;
  lds.stage(a, c0);
  __syncthreads();
  if (c >= a.C) return;
  const Out<T, V> out(a, c);
  if (out.n == V && out.one)
    step_body<T, V, K, ROWS, true>(a, lds, out, c, set * ROWS);
  else
    step_body<T, V, K, ROWS, false>(a, lds, out, c, set * ROWS);
}

template <typename T, int V, int K, bool WHOLE>
__device__ __forceinline__ void prompt_body(const ShortConvArgs &a, const TapsLds<V, K> &lds, const Out<T, V> &out, int c, const Item &it, int row) {
  const int t0 = it.index * a.T;
  const T *x = reinterpret_cast<const T *>(a.x) + (size_t)it.begin * a.row_stride + c;
  const int t1 = min(it.len, t0 + a.T);
  constexpr int AHEAD = WHOLE ? kAhead : 1;  // the few threads at a border take no registers from the others
  Held<T, V, WHOLE> in[2][AHEAD], old[K - 1];
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
      if (known)
        old[k].load(ring + s * slot_elems, out.n);
      else
        old[k].w = typename Elems<T, V>::words{};
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      int s = slot - (K - 1) + k;
      if (s < 0) s += a.slots;
      const int t = it.len - (K - 1) + k;  // negative: that far into the old history
      Held<T, V, WHOLE> last;
      if (t >= 0) {
        last.load(x + (size_t)t * a.row_stride, out.n);
      } else {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
          if (j == K - 1 + t) last = old[j];
      }
      last.store(ring + s * slot_elems, out.n);
    }
  } else {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) old[k].load(x + (size_t)(t0 - (K - 1) + k) * a.row_stride, out.n);
  }
  if (t0 >= t1) return;  // an empty sequence had only its ring to do
  auto fetch = [&](int t, int half) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) in[half][i].load(x + (size_t)min(t + i, t1 - 1) * a.row_stride, out.n);
  };
  fetch(t0, 0);
  const Taps<V, K> taps = lds.get(a, c, out.n);
  float h[K - 1][V];
#pragma unroll
  for (int k = 0; k < K - 1; ++k) old[k].get(h[k]);
  auto emit = [&](int t, int half) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      float v[V], y[V];
      in[half][i].get(v);
      taps_out<V, K>(taps, h, v, a.silu, y);
      if (t + i < t1) {
        if constexpr (WHOLE)
          store_vec<T, V>(out.base + ((size_t)it.begin + t + i) * out.width, y);
        else
          out.store(a, (size_t)it.begin + t + i, y);
      }
      push<V, K>(h, v);
    }
  };
  // The loads of the next AHEAD tokens are under way while these are computed.
  for (int t = t0; t < t1; t += 2 * AHEAD) {
    fetch(t + AHEAD, 1);
    emit(t, 0);
    fetch(t + 2 * AHEAD, 0);
    emit(t + AHEAD, 1);
  }
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads, 4) void short_conv_prompt_k(ShortConvArgs a, FastDiv per_item) {
  const int item = fdiv(blockIdx.x, per_item);
  const int c0 = (blockIdx.x - item * (int)per_item.d) * kThreads * V, c = c0 + threadIdx.x * V;
  const Item it = find_item(a.p, item, a.T);
  if (it.index < 0 || (it.index * a.T >= it.len && it.index > 0)) return;
  const int row = batch_row(a.p, it.seq, it.index == 0 && c == 0);
  if (row < 0) return;
  __shared__ TapsLds<V, K> lds;
  lds.stage(a, c0);
  __syncthreads();
  if (c >= a.C) return;
  const Out<T, V> out(a, c);
  if (out.n == V && out.one)
    prompt_body<T, V, K, true>(a, lds, out, c, it, row);
  else
    prompt_body<T, V, K, false>(a, lds, out, c, it, row);
}

template <typename T, int V, int K, int ROWS>
void launch_step(const ShortConvArgs &a, int per, hipStream_t st) {
  hipLaunchKernelGGL((short_conv_step_k<T, V, K, ROWS>), dim3((uint32_t)((a.batch + ROWS - 1) / ROWS * per)), dim3(kThreads), 0,
                     st, a, make_fastdiv((uint32_t)per));
}

// Tokens of a prompt tile: short enough for many workgroups, so that those of uneven
// sequences end together; a tile reads K - 1 of its predecessor's rows once more, from
// HBM: neighbouring tiles of a channel block are on other XCDs (8192 tokens of 10240
// channels, bf16: 197 MB read for 168; 16384 tokens: 142 us with 12 to 24, 156 with 64).
constexpr int kTile = 24;

template <typename T, int V, int K>
int launch(ShortConvArgs a, bool prompt, hipStream_t st) {
  const int per = (a.C + kThreads * V - 1) / (kThreads * V);
  if (prompt) a.T = kTile;
  const int64_t rows = prompt ? items_of(a.p.tokens, a.p.n, a.T) : a.batch;
  // Two rows a thread still leave two workgroups a CU (256 rows: 11.0 us, one by one 12.4).
  const bool two = !prompt && rows * per >= 1024;
  if ((two ? (rows + 1) / 2 : rows) * per > kMostBlocks) return kTooLarge;
  if (prompt) {
    hipLaunchKernelGGL((short_conv_prompt_k<T, V, K>), dim3((uint32_t)(rows * per)), dim3(kThreads), 0, st, a,
                       make_fastdiv((uint32_t)per));
  } else if (two) {
    launch_step<T, V, K, 2>(a, per, st);
  } else {
    launch_step<T, V, K, 1>(a, per, st);
  }
  return (int)hipGetLastError();
}

template <typename T>
int dispatch(const ShortConvArgs &a, bool prompt, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(T);
  if (a.K == 2) return launch<T, W, 2>(a, prompt, st);
  if (a.K == 3) return launch<T, W, 3>(a, prompt, st);
  return launch<T, W, 4>(a, prompt, st);
}

int any(const ShortConvArgs &a, bool prompt, hipStream_t st) {
  return a.dtype == REPLAY_DT_BF16 ? dispatch<bf16_t>(a, prompt, st) : dispatch<float>(a, prompt, st);
}

}  // namespace

int launch_short_conv_step(const ShortConvArgs &a, hipStream_t st) { return any(a, false, st); }
int launch_short_conv_prompt(const ShortConvArgs &a, hipStream_t st) { return any(a, true, st); }

}  // namespace rssm
