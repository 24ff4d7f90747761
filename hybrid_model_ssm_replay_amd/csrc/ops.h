// Shared parts of the operators around the recurrence (short convolution,
// prompts of both families, norms, draft acceptance, log probabilities): packed
// sequences, element types, launch declarations.
#pragma once

#include "common.h"
#include "internal.h"

namespace rssm {

// ---- element types ------------------------------------------------------------
// V consecutive elements of type T (float, or bf16_t: the upper half of a
// float32) as float32.  The pointer is aligned to its element only: global memory
// takes 16-byte accesses at any address, whole lines of a wave at nearly full speed.
template <typename T, int V>
struct Elems {
  typedef uint32_t words __attribute__((ext_vector_type(sizeof(T) * V / 4)));
  typedef words loose __attribute__((aligned(sizeof(T))));
};
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[V]) {
  if constexpr (sizeof(T) * V < 8) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = ldr<T>(p + i);
  } else {
    constexpr int S = sizeof(T) * V > 16 ? V / 2 : V;  // 16 bytes at a time
#pragma unroll
    for (int o = 0; o < V; o += S) {
      const typename Elems<T, S>::words w = *reinterpret_cast<const typename Elems<T, S>::loose *>(p + o);
#pragma unroll
      for (int i = 0; i < S; ++i) {
        if constexpr (sizeof(T) == 4)
          v[o + i] = __uint_as_float(w[i]);
        else
          v[o + i] = i % 2 ? __uint_as_float(w[i / 2] & 0xFFFF0000u) : __uint_as_float(w[i / 2] << 16);
      }
    }
  }
}

// Two float32 values as bf16, rounded to nearest even, the first in the low
// half (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 h2 __attribute__((ext_vector_type(2)));
  const f2 v = {a, b};
  const h2 h = __builtin_convertvector(v, h2);
  return __builtin_bit_cast(uint32_t, h);
}

// The store that goes with load_vec; bf16 rounds to nearest even (half a step,
// at most 2^-8 of the value): the array's type asks for it.
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[V]) {
  if constexpr (sizeof(T) * V < 8) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4)
        p[i] = v[i];
      else
        p[i] = (bf16_t)pack_bf16(v[i], 0.f);
    }
  } else {
    constexpr int S = sizeof(T) * V > 16 ? V / 2 : V;
#pragma unroll
    for (int o = 0; o < V; o += S) {
      typename Elems<T, S>::words w;
#pragma unroll
      for (int i = 0; i < S * (int)sizeof(T) / 4; ++i) {
        if constexpr (sizeof(T) == 4)
          w[i] = __float_as_uint(v[o + i]);
        else
          w[i] = pack_bf16(v[o + 2 * i], v[o + 2 * i + 1]);
      }
      *reinterpret_cast<typename Elems<T, S>::loose *>(p + o) = w;
    }
  }
}

// The first n of V elements; the others are zero, or not written.
template <typename T, int V>
__device__ __forceinline__ void load_part(const T *p, int n, float (&v)[V]) {
  if (n >= V) {
    load_vec<T, V>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < n ? ldr<T>(p + i) : 0.f;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_part(T *p, int n, const float (&v)[V]) {
  if (n >= V) {
    store_vec<T, V>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) {
        const float one[1] = {v[i]};
        store_vec<T, 1>(p + i, one);
      }
  }
}

// v / (1 + exp(-v)) by the hardware exponential and reciprocal: a few 2^-24 relative,
// and about |v| 2^-24 from rounding the exponential's argument.  exp(-v) overflows to infinity for v < -88, where the result is -0.
__device__ __forceinline__ float silu(float v) { return v * __builtin_amdgcn_rcpf(1.f + __expf(-v)); }

// ---- packed sequences -----------------------------------------------------------
struct Packed {
  int tokens, n, batch;
  const int32_t *start;   // [n + 1]
  const int32_t *rows;    // [n] or NULL
  const uint8_t *resume;  // [n] or NULL
  int32_t *status;        // or NULL
};

__device__ __forceinline__ int clamp_start(const Packed &p, int i) {
  const int s = p.start[i];
  return s < 0 ? 0 : s > p.tokens ? p.tokens : s;
}

// Work items of `size` tokens without knowing the lengths on the host: sequence
// i owns the items base_i .. base_{i+1} - 1 with base_i = start_i / size + i,
// which are at least ceil(length_i / size) and at least one; tokens / size + n
// items cover every sequence, and those past a sequence's end do nothing.
__host__ __device__ inline int items_of(int tokens, int n, int size) { return tokens / size + n; }
struct Item {
  int seq, index, begin, len;  // sequence, item within it, its first row and length
};
__device__ __forceinline__ Item find_item(const Packed &p, int item, int size) {
  int lo = 0, hi = p.n - 1;  // the last i with base_i <= item
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (clamp_start(p, mid) / size + mid <= item)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int b = clamp_start(p, lo), e = clamp_start(p, lo + 1);
  return Item{lo, item - (b / size + lo), b, e > b ? e - b : 0};
}

// Batch row of sequence i; -1 (and the status bit) if it is out of range.
__device__ __forceinline__ int batch_row(const Packed &p, int i, bool report) {
  const int r = p.rows ? p.rows[i] : i;
  if (r >= 0 && r < p.batch) return r;
  if (report && p.status) atomicOr(p.status, REPLAY_STATUS_BAD_PROMPT);
  return -1;
}

// ---- launches -------------------------------------------------------------------
// A launch holds fewer than 2^32 work-items.  A launch function returns kTooLarge before
// anything is enqueued where its workgroups of 256 are more.
constexpr int64_t kMostBlocks = (1 << 24) - 1;
constexpr int kTooLarge = -1;
struct ShortConvArgs {
  int C, K, slots, batch, dtype, silu;
  int w[3];
  const float *weight, *bias;
  void *ring;
  const int32_t *pos;
  int32_t *status;
  const void *x;
  int64_t seq_stride, row_stride;
  int T;       // step: tokens a row; prompt: tokens of a tile
  Packed p;    // prompt
  void *out[3];
};
int launch_short_conv_step(const ShortConvArgs &a, hipStream_t st);
int launch_short_conv_prompt(const ShortConvArgs &a, hipStream_t st);

struct ScanArgs {
  int H, G, P, N, bf16, y_bf16;
  Packed p;
  const void *x, *Bm, *Cm;
  const float *dt, *A, *D, *initial;
  float *state;
  void *y;
  void *workspace;
};
size_t scan_workspace(const ScanArgs &a);
int launch_scan(const ScanArgs &a, hipStream_t st);
void scan_plan(const ScanArgs &a, int32_t (&plan)[4]);  // see replay_scan_plan

struct DeltaArgs {
  int H, P, N, bf16, y_bf16;  // P rows (v), N columns (k, q) of a head's state
  Packed p;
  const void *q, *k, *v;
  const float *alpha, *beta, *initial;
  float *state;
  void *y;
  void *workspace;
};
size_t delta_workspace(const DeltaArgs &a);
int launch_delta(const DeltaArgs &a, hipStream_t st);

int launch_renew_read_copy(const Shape &s, const FormatBufs &f, const uint8_t *mask, hipStream_t st);

int launch_gated_norm(const replay_gated_norm_args &a, hipStream_t st);

int launch_residual_norm(const replay_residual_norm_args &a, hipStream_t st);

size_t logprobs_workspace(int rows, int vocab, int top);
int launch_logprobs(const replay_token_logprobs_args &a, void *workspace, hipStream_t st);

size_t accept_workspace(int batch, int vocab);
int launch_accept(const replay_accept_args &a, void *workspace, hipStream_t st);

}  // namespace rssm
