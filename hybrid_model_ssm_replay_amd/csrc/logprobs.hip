// Log probabilities of given tokens, the entropy of each row, its largest words.
//
//   m = max x,  s = sum e^{x - m},  t = sum e^{x - m} (x - m),
//   logprob = x[token] - m - log s,   entropy = log s - t / s.
//
// One pass over the logits: a lane carries a running maximum with the two sums, scaled
// down when the maximum grows.  Few rows are cut into
// slices, a workgroup each, whose sums and words a second launch joins in their order:
// no atomics, and the same result every time.
//
// The largest words: a wave keeps a sorted list, a lane an entry, and puts in what is
// larger than the list's last; of equal words the lower comes first.  Before a long run
// of insertions (the first words, or rows that rise) the last entry is raised to the
// list's size-th largest of the lanes' own maxima, which as many words reach.
//
// -infinity and NaN have no weight; +infinity counts as the largest float32.
#include "ops.h"
#include "pieces.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kStep = 8 * kThreads;  // values a workgroup reads at a time, 8 a thread
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.4028234663852886e38f, kNone = -__builtin_inff();
// Exponents below this are no weight at all; a product with it stays finite.
constexpr float kLeast = -1e4f;

struct Slices {
  int size, n;    // values of a slice (a multiple of kStep), slices of a row
  FastDiv fn;
  float4 *sums;   // [rows][n]: m, s, t
  float *values;  // [rows][n][top]
  int *words;
};

struct Sums {  // m is finite: kLowest before any weight
  float m, s, t;
  __device__ __forceinline__ void scale_to(float to) {  // to >= m
    const float d = fmaxf(m - to, kLeast), c = __builtin_amdgcn_exp2f(d * kLog2e);
    t = (t + s * d) * c, s *= c, m = to;
  }
  __device__ __forceinline__ void join(Sums o) {
    const float to = fmaxf(m, o.m);
    scale_to(to), o.scale_to(to);
    s += o.s, t += o.t;
  }
};

// NaN as -infinity, +infinity as the largest number.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, kNone), -kLowest); }

// Whether a word comes before another: larger, or as large and lower.
__device__ __forceinline__ bool before(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

// A wave's list of `top` words, lane l the l-th.
struct List {
  float v;
  int i;
  float last;  // of the last entry, the same in every lane
  int last_i;
  __device__ __forceinline__ void clear() { v = last = kNone, i = last_i = 0x7fffffff; }
  __device__ __forceinline__ void put(float x, int word, int top, int lane) {  // x, word: the same in every lane
    const int at = __popcll(__ballot(before(v, i, x, word)));
    const float v1 = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x138, 0xF, 0xF, false));
    const int i1 = __builtin_amdgcn_update_dpp(0, i, 0x138, 0xF, 0xF, false);  // from the lane before
    v = lane > at ? v1 : lane == at ? x : v;
    i = lane > at ? i1 : lane == at ? word : i;
    last = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), top - 1));
    last_i = __builtin_amdgcn_readlane(i, top - 1);
  }
  // One candidate of each lane where `is`, none of -infinity.
  __device__ __forceinline__ void offer(float x, int word, bool is, int top, int lane) {
    uint64_t left = __ballot(is && x > kNone && before(x, word, last, last_i));
    while (left) {
      const int l = __builtin_ctzll(left);
      left &= left - 1;
      const float xl = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), l));
      const int wl = __builtin_amdgcn_readlane(word, l);
      if (before(xl, wl, last, last_i)) put(xl, wl, top, lane);
    }
  }
};

// The n-th largest of the lanes' values (n from 1), the same in every lane.
__device__ __forceinline__ float nth(float v, int n, int lane) {
#pragma unroll
  for (int k = 2; k <= kWave; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2) {
      const float o = __shfl_xor(v, j, kWave);
      const bool larger = (lane & j) == 0 ? (lane & k) == 0 || k == kWave : !((lane & k) == 0 || k == kWave);
      v = larger ? fmaxf(v, o) : fminf(v, o);
    }
  return __shfl(v, n - 1, kWave);
}

template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, float (&v)[8]) {  // places past n: no weight
  if (n >= 8) {
    load_vec<T, 8>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? ldr<T>(p + i) : kNone;
  }
}

__device__ __forceinline__ float at(const void *p, int dtype, int64_t i) {
  return dtype == REPLAY_DT_BF16 ? ldr<bf16_t>((const bf16_t *)p + i) : ldr<float>((const float *)p + i);
}

// A row's results from its sums and list.
__device__ __forceinline__ void finish(const replay_token_logprobs_args &a, int row, Sums z, const List &list, int lane) {
  const bool any = z.s > 0.f;
  const float log_s = __builtin_amdgcn_logf(z.s) * kLn2;  // s is at least 1 where there is any weight
  if (lane == 0) {
    const int tok = a.tokens[row];
    float lp = kNone;
    if (any && tok >= 0 && tok < a.vocab) {
      const float x = clean(at(a.logits, a.dtype, (int64_t)row * a.stride + tok));
      if (x > kNone) lp = (x - z.m) - log_s;
    }
    a.logprobs[row] = lp;
    a.entropy[row] = any ? log_s - z.t / z.s : 0.f;
  }
  if (lane < a.top) {
    const bool there = list.v > kNone;
    a.top_logprobs[(int64_t)row * a.top + lane] = there ? (list.v - z.m) - log_s : kNone;
    a.top_tokens[(int64_t)row * a.top + lane] = there ? list.i : -1;
  }
}

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_k(replay_token_logprobs_args a, Slices sl) {
  __shared__ float4 part[kWaves];
  __shared__ float sv[kWaves][REPLAY_MAX_TOP];
  __shared__ int si[kWaves][REPLAY_MAX_TOP];
  const int row = fdiv(blockIdx.x, sl.fn), slice = blockIdx.x - row * sl.n;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const T *x = (const T *)a.logits + (int64_t)row * a.stride;
  const int v0 = slice * sl.size, v1 = min(a.vocab, v0 + sl.size);
  Sums z{kLowest, 0.f, 0.f};
  List list;
  list.clear();
  for (int v = v0; v < v1; v += kStep) {
    const int at0 = v + threadIdx.x * 8;
    float xv[8];
    load8<T>(x + at0, v1 - at0, xv);
    float largest = kNone;
#pragma unroll
    for (int i = 0; i < 8; ++i) xv[i] = clean(xv[i]), largest = fmaxf(largest, xv[i]);
    z.scale_to(fmaxf(z.m, largest));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = fmaxf(xv[i] - z.m, kLeast), e = __builtin_amdgcn_exp2f(d * kLog2e);
      z.s += e, z.t = fmaf(e, d, z.t);
    }
    if constexpr (TOP) {
      const uint64_t some = __ballot(largest > list.last);
      if (some) {
        // At least `top` words of these are as large as the top-th of the lanes' maxima.
        float least = list.last;
        if (__popcll(some) > a.top) least = fmaxf(least, nth(largest, a.top, lane));
#pragma unroll
        for (int i = 0; i < 8; ++i) list.offer(xv[i], at0 + i, xv[i] >= least, a.top, lane);
      }
    }
  }
  // The waves in their order.
#pragma unroll
  for (int o = 1; o < kWave; o *= 2) z.join(Sums{__shfl_xor(z.m, o, kWave), __shfl_xor(z.s, o, kWave), __shfl_xor(z.t, o, kWave)});
  if (lane == 0) part[wave] = make_float4(z.m, z.s, z.t, 0.f);
  if (TOP && lane < a.top) sv[wave][lane] = list.v, si[wave][lane] = list.i;
  __syncthreads();
  if (wave) return;
  for (int w = 1; w < kWaves; ++w) {
    z.join(Sums{part[w].x, part[w].y, part[w].z});
    if constexpr (TOP) list.offer(lane < a.top ? sv[w][lane] : kNone, lane < a.top ? si[w][lane] : 0, lane < a.top, a.top, lane);
  }
  if (sl.n == 1) {
    finish(a, row, z, list, lane);
    return;
  }
  const int64_t to = (int64_t)row * sl.n + slice;
  if (lane == 0) sl.sums[to] = make_float4(z.m, z.s, z.t, 0.f);
  if (TOP && lane < a.top) sl.values[to * a.top + lane] = list.v, sl.words[to * a.top + lane] = list.i;
}

// Joins the slices of a row, a wave each: a lane's run of neighbours, then the lanes.
__global__ __launch_bounds__(kWave) void join_k(replay_token_logprobs_args a, Slices sl) {
  const int row = blockIdx.x, lane = threadIdx.x;
  const float4 *const sums = sl.sums + (int64_t)row * sl.n;
  const int per = (sl.n + kWave - 1) / kWave;
  Sums z{kLowest, 0.f, 0.f};
  for (int i = lane * per; i < min(sl.n, (lane + 1) * per); ++i) z.join(Sums{sums[i].x, sums[i].y, sums[i].z});
#pragma unroll
  for (int o = 1; o < kWave; o *= 2) z.join(Sums{__shfl_xor(z.m, o, kWave), __shfl_xor(z.s, o, kWave), __shfl_xor(z.t, o, kWave)});
  List list;
  list.clear();
  // The slices' first words, then their second ones, and so on: the list is soon full of large ones.
  const float *const values = sl.values + (int64_t)row * sl.n * a.top;
  const int *const words = sl.words + (int64_t)row * sl.n * a.top;
  for (int k = 0; k < a.top; ++k)
    for (int s = 0; s < sl.n; s += kWave) {
      const bool is = s + lane < sl.n;
      const int64_t at = (int64_t)(is ? s + lane : 0) * a.top + k;
      list.offer(values[at], words[at], is, a.top, lane);
    }
  finish(a, row, z, list, lane);
}

// Slices of 2048 values, longer where there would be more than 2048 workgroups.
Slices slices_of(int rows, int vocab) {
  Slices s{};
  s.size = kStep;
  while ((int64_t)rows * ((vocab + (int64_t)s.size - 1) / s.size) > 2048 && s.size < vocab) s.size *= 2;
  s.n = (int)((vocab + (int64_t)s.size - 1) / s.size);
  s.fn = make_fastdiv((uint32_t)s.n);
  return s;
}

size_t sums_bytes(int rows, const Slices &s) { return ((size_t)rows * s.n * sizeof(float4) + 255) / 256 * 256; }
size_t words_bytes(int rows, const Slices &s, int top) { return ((size_t)rows * s.n * top * 4 + 255) / 256 * 256; }

template <typename T>
void launch(const replay_token_logprobs_args &a, const Slices &s, hipStream_t st) {
  const dim3 grid((uint32_t)(a.rows * s.n)), block(kThreads);
  if (a.top)
    hipLaunchKernelGGL((logprobs_k<T, true>), grid, block, 0, st, a, s);
  else
    hipLaunchKernelGGL((logprobs_k<T, false>), grid, block, 0, st, a, s);
}

}  // namespace

size_t logprobs_workspace(int rows, int vocab, int top) {
  const Slices s = slices_of(rows, vocab);
  return s.n == 1 ? 0 : sums_bytes(rows, s) + 2 * words_bytes(rows, s, top);
}

int launch_logprobs(const replay_token_logprobs_args &a, void *workspace, hipStream_t st) {
  Slices s = slices_of(a.rows, a.vocab);
  if ((int64_t)a.rows * s.n > kMostBlocks) return kTooLarge;
  s.sums = (float4 *)workspace;
  s.values = (float *)((char *)workspace + sums_bytes(a.rows, s));
  s.words = (int *)((char *)s.values + words_bytes(a.rows, s, a.top));
  if (a.dtype == REPLAY_DT_BF16)
    launch<bf16_t>(a, s, st);
  else
    launch<float>(a, s, st);
  if (s.n > 1) hipLaunchKernelGGL(join_k, dim3((uint32_t)a.rows), dim3(kWave), 0, st, a, s);
  return (int)hipGetLastError();
}

}  // namespace rssm
