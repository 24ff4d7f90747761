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
// The largest words: a wave keeps a sorted list, a lane an entry, of keys whose order is
// that of the words (falling, of equal ones the lower first).  A few words beyond the
// list's last are put in one by one, more are sorted into it 32 at a time.  Where many
// are beyond it (the first words, or rows that rise), only those count that reach the
// list's size-th largest of the lanes' own maxima: as many words do.
//
// -infinity and NaN have no weight; +infinity counts as the largest float32.
//
// Bound by HBM where rows are many and no words are asked for: 4096 rows of 131072 (bf16) 190
// us, 5.6 TB/s; by the exponentials and the words' comparisons beside it: 1152 rows of 50021 (bf16),
// five words, 35 us, 3.3 TB/s (32 where a third of the words is masked), none 29; of float32 50 and 47,
// 4.6 and 4.9 TB/s; by latency for one row: 131072 of float32, twenty words, 6.3 us and 5.0 for the join.
#include "ops.h"
#include "pieces.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kStep = 8 * kThreads;  // values a workgroup reads at a time, 8 a thread
constexpr int kTurn = 2;             // such reads worked on together: 64 rows of 131072, five words, 20 us, 23 with one
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.4028234663852886e38f, kNone = -__builtin_inff();
// Exponents below this are no weight at all; a product with it stays finite.
constexpr float kLeast = -1e4f;

typedef unsigned long long Key;

struct Slices {
  int size, n;   // values of a slice (a multiple of kStep), slices of a row
  FastDiv fn;
  float4 *sums;  // [rows][n]: m, s, t
  Key *keys;     // [rows][top][n]
};

struct Sums {  // m is finite: kLowest before any weight; t has exponents of 2
  float m, s, t;
  __device__ __forceinline__ void scale_to(float to) {  // to >= m
    const float d = fmaxf((m - to) * kLog2e, kLeast), c = __builtin_amdgcn_exp2f(d);
    t = (t + s * d) * c, s *= c, m = to;
  }
  __device__ __forceinline__ void join(Sums o) {
    const float to = fmaxf(m, o.m);
    scale_to(to), o.scale_to(to);
    s += o.s, t += o.t;
  }
};

// +infinity as the largest number, NaN as -infinity.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, kNone), -kLowest); }

// A word as a number that is larger where the word comes first; 0 for none and -infinity.
__device__ __forceinline__ Key key_of(float x, int word) {
  const uint32_t b = bits(x + 0.f), up = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);  // -0 as 0
  return x > kNone ? (Key)up << 32 | ~(uint32_t)word : 0;
}
__device__ __forceinline__ float value_of(Key k) {
  const uint32_t up = (uint32_t)(k >> 32);
  return k ? __uint_as_float(up & 0x80000000u ? up ^ 0x80000000u : ~up) : kNone;
}
__device__ __forceinline__ int word_of(Key k) { return k ? (int)~(uint32_t)k : -1; }

// The value of lane l ^ J.
template <int J>
__device__ __forceinline__ uint32_t other(uint32_t v, int lane) {
  if constexpr (J == 1) return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false);
  if constexpr (J == 2) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false);
  if constexpr (J == 4)  // 7 - l within eight lanes, then 3 - l within four
    return __builtin_amdgcn_update_dpp(0, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false), 0x1B, 0xF, 0xF, false);
  if constexpr (J == 8) return __builtin_amdgcn_update_dpp(0, v, 0x128, 0xF, 0xF, false);
  if constexpr (J == 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return lane & 16 ? a[0] : a[1];
  }
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return lane & 32 ? a[0] : a[1];
}
template <int J>
__device__ __forceinline__ Key other(Key k, int lane) {
  return (Key)other<J>((uint32_t)(k >> 32), lane) << 32 | other<J>((uint32_t)k, lane);
}
template <int J>
__device__ __forceinline__ float other(float v, int lane) { return __uint_as_float(other<J>(bits(v), lane)); }

// One turn of a bitonic sort, falling over the wave: runs of K lanes, partners J apart.
template <int K, int J, typename V>
__device__ __forceinline__ void turn(V &v, int lane) {
  const bool larger = ((lane & J) == 0) == ((lane & K) == 0 || K == kWave);
  const V o = other<J>(v, lane);
  v = (v > o) == larger ? v : o;
  if constexpr (J > 1) turn<K, J / 2>(v, lane);
}
template <typename V>
__device__ __forceinline__ void sort64(V &v, int lane) {
  turn<2, 1>(v, lane), turn<4, 2>(v, lane), turn<8, 4>(v, lane), turn<16, 8>(v, lane), turn<32, 16>(v, lane);
  turn<64, 32>(v, lane);
}
// The n-th largest of the lanes' values (n from 1), the same in every lane.
__device__ __forceinline__ float nth(float v, int n, int lane) {
  sort64(v, lane);
  return __uint_as_float(__builtin_amdgcn_readlane(bits(v), n - 1));
}

// A wave's list: lanes 0 to 31 hold the largest keys seen, falling.
struct List {
  Key k;
  float last;  // value of the top-th, the same in every lane
  __device__ __forceinline__ void clear() { k = 0, last = kNone; }
  __device__ __forceinline__ void close(int top) {
    last = value_of((Key)__builtin_amdgcn_readlane((uint32_t)(k >> 32), top - 1) << 32 |
                    (uint32_t)__builtin_amdgcn_readlane((uint32_t)k, top - 1));
  }
  __device__ __forceinline__ void put(Key x, int lane) {  // x: the same in every lane
    const int at = __popcll(__ballot(k > x));
    const Key up = (Key)(uint32_t)__builtin_amdgcn_update_dpp(0, (uint32_t)(k >> 32), 0x138, 0xF, 0xF, false) << 32 |
                   (uint32_t)__builtin_amdgcn_update_dpp(0, (uint32_t)k, 0x138, 0xF, 0xF, false);  // of the lane before
    k = lane > at ? up : lane == at ? x : k;
  }
  // n keys in `some`, 32 at a time.
  __device__ __forceinline__ void sort_in(const Key *some, int n, int lane) {
    for (int c = 0; c < n; c += 32) {
      const int i = c + lane - 32;
      if (lane >= 32) k = i < n ? some[i] : 0;
      sort64(k, lane);
    }
  }
};
constexpr int kFew = 12;  // put in one by one: about as long as sorting them in (one row: 12.7 us, 14.0 with 24, 12.8 with 4)

constexpr int kSpread = kWave / (8 * kTurn);  // lanes whose values of a turn are one for each lane of a wave

// Eight neighbouring values as loaded; places past the n-th: no weight.
template <typename T>
struct Eight {
  static constexpr int W = sizeof(T) * 2;
  typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));  // of its element only
  uint32_t w[W];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const loose v = *reinterpret_cast<const loose *>((const char *)p + 4 * i);
      w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
    }
  }
  __device__ __forceinline__ void load(const T *p, int n) {
    if (n >= 8) return load(p);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? ldr<T>(p + i) : kNone;
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = sizeof(T) == 4 ? bits(v[i]) : __builtin_amdgcn_perm(bits(v[2 * i + 1]), bits(v[2 * i]), 0x07060302u);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    return i % 2 ? upper(w[i / 2]) : lower(w[i / 2]);
  }
};

__device__ __forceinline__ float at(const void *p, int dtype, int64_t i) {
  return dtype == REPLAY_DT_BF16 ? ldr<bf16_t>((const bf16_t *)p + i) : ldr<float>((const float *)p + i);
}

// The logit of a row's token, -infinity for one outside the vocabulary: loaded early.
__device__ __forceinline__ float chosen_of(const replay_token_logprobs_args &a, int row) {
  const int tok = a.tokens[row];
  return tok >= 0 && tok < a.vocab ? at(a.logits, a.dtype, (int64_t)row * a.stride + tok) : kNone;
}

// A row's results from its sums and list.
__device__ __forceinline__ void finish(const replay_token_logprobs_args &a, int row, Sums z, const List &list, float chosen, int lane) {
  const bool any = z.s > 0.f;
  const float log2_s = __builtin_amdgcn_logf(z.s), log_s = log2_s * kLn2;  // s is at least 1 where there is any weight
  if (lane == 0) {
    const float x = clean(chosen);
    a.logprobs[row] = x > kNone ? (x - z.m) - log_s : kNone;
    a.entropy[row] = any ? (log2_s - z.t / z.s) * kLn2 : 0.f;
  }
  if (lane < a.top) {
    a.top_logprobs[(int64_t)row * a.top + lane] = list.k ? (value_of(list.k) - z.m) - log_s : kNone;
    a.top_tokens[(int64_t)row * a.top + lane] = word_of(list.k);
  }
}

// Every lane's sums joined.
__device__ __forceinline__ void join_lanes(Sums &z, int lane) {
  z.join(Sums{other<1>(z.m, lane), other<1>(z.s, lane), other<1>(z.t, lane)});
  z.join(Sums{other<2>(z.m, lane), other<2>(z.s, lane), other<2>(z.t, lane)});
  z.join(Sums{other<4>(z.m, lane), other<4>(z.s, lane), other<4>(z.t, lane)});
  z.join(Sums{other<8>(z.m, lane), other<8>(z.s, lane), other<8>(z.t, lane)});
  z.join(Sums{other<16>(z.m, lane), other<16>(z.s, lane), other<16>(z.t, lane)});
  z.join(Sums{other<32>(z.m, lane), other<32>(z.s, lane), other<32>(z.t, lane)});
}

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_k(replay_token_logprobs_args a, Slices sl) {
  __shared__ float4 part[kWaves];
  __shared__ float lasts[kWaves];
  __shared__ Key some[kWaves][TOP ? kStep / kWaves : 1];  // a wave's words of one step beyond its list's last
  const int row = fdiv(blockIdx.x, sl.fn), slice = blockIdx.x - row * sl.n;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const T *x = (const T *)a.logits + (int64_t)row * a.stride;
  // A row of bf16 between two words starts with the value before it, which counts for nothing:
  // loads off a word's bounds are slower (1152 rows of 50021: 36.2 us, 29.6 so, 29.4 of 50016).
  // The first row, and rows that repeat it (stride 0), have none of the logits before them.
  const int odd = sizeof(T) == 2 && row > 0 && a.stride > 0 && ((uintptr_t)x & 2) ? 1 : 0;
  x -= odd;
  const int v0 = slice * sl.size, v1 = slice + 1 == sl.n ? a.vocab + odd : v0 + sl.size;
  Sums z{kLowest, 0.f, 0.f};
  List list;
  list.clear();
  const float chosen = sl.n == 1 ? chosen_of(a, row) : 0.f;
  // The next turn's loads are under way while this one is worked on.  No branch stands
  // between the loads of a turn: each would wait for the one before.
  Eight<T> raw[kTurn];
  auto fetch = [&](int v) {
    const T *const p = x + v + threadIdx.x * 8;
    if (v + kTurn * kStep <= v1) {
#pragma unroll
      for (int u = 0; u < kTurn; ++u) raw[u].load(p + u * kStep);
    } else {
#pragma unroll
      for (int u = 0; u < kTurn; ++u) raw[u].load(p + u * kStep, v1 - (v + (int)threadIdx.x * 8 + u * kStep));
    }
  };
  if constexpr (TOP) {
    if (lane == 0) lasts[wave] = kNone;
    __syncthreads();
  }
  fetch(v0);
  for (int v = v0; v < v1; v += kTurn * kStep) {
    const int at0 = v + threadIdx.x * 8;
    float xv[kTurn][8], largest = kNone;
#pragma unroll
    for (int u = 0; u < kTurn; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xv[u][i] = raw[u].get(i);
        if (u == 0 && i == 0) xv[u][i] = at0 < odd ? kNone : xv[u][i];
        largest = fmaxf(largest, xv[u][i]);
      }
    if (v + kTurn * kStep < v1) fetch(v + kTurn * kStep);
    if (largest > -kLowest) {  // +infinity
      largest = kNone;
#pragma unroll
      for (int u = 0; u < kTurn; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) xv[u][i] = clean(xv[u][i]), largest = fmaxf(largest, xv[u][i]);
    }
    z.scale_to(fmaxf(z.m, largest));
    // The difference first: a product of m alone would be off by |m| 2^-24.
#pragma unroll
    for (int u = 0; u < kTurn; ++u) {
      if (v + u * kStep >= v1) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = fmaxf((xv[u][i] - z.m) * kLog2e, kLeast), e = __builtin_amdgcn_exp2f(d);
        z.s += e, z.t = fmaf(e, d, z.t);
      }
    }
    if constexpr (TOP) {
      // As many words as the list holds reach the last entry of any wave's list.
      float least = list.last;
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        least = fmaxf(least, __hip_atomic_load(&lasts[w], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP));
      const uint64_t beyond = __ballot(largest > list.last && largest >= least);
      if (beyond) {
        const int lanes = __popcll(beyond);
        if (lanes > a.top) least = fmaxf(least, nth(largest, a.top, lane));
        // A few lanes' words: one to a lane, all at once, and not by the place in the lanes (1152 rows
        // of 50021, five words: 36 us, 39; 1024 of 131072, twenty: 74, 84).
        if (lanes <= kSpread) {
          float *const values = reinterpret_cast<float *>(some[wave]);
          int *const first = reinterpret_cast<int *>(values + kWave);
          if (beyond >> lane & 1) {
            const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(beyond >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)beyond, 0));
#pragma unroll
            for (int i = 0; i < 8 * kTurn; i += 4)
              st4(values + rank * 8 * kTurn + i, make_float4(xv[i / 8][i % 8], xv[i / 8][i % 8 + 1], xv[i / 8][i % 8 + 2], xv[i / 8][i % 8 + 3]));
            first[rank] = at0 - odd;
          }
          wave_lds_sync();
          const int from = lane / (8 * kTurn), i = lane % (8 * kTurn);
          const float value = from < lanes ? values[lane] : kNone;
          const int word = first[from < lanes ? from : 0] + i / 8 * kStep + i % 8;
          wave_lds_sync();
          const bool is = value >= least && value > kNone;
          const Key key = is ? key_of(value, word) : 0;
          uint64_t mask = __ballot(is);
          if (__popcll(mask) <= kFew) {
            for (; mask; mask &= mask - 1) {
              const int l = __builtin_ctzll(mask);
              list.put((Key)__builtin_amdgcn_readlane((uint32_t)(key >> 32), l) << 32 | (uint32_t)__builtin_amdgcn_readlane((uint32_t)key, l), lane);
            }
          } else {
            some[wave][lane] = key;
            wave_lds_sync();
            list.sort_in(some[wave], kWave, lane);
            wave_lds_sync();
          }
        } else {
#pragma unroll
          for (int u = 0; u < kTurn; ++u) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const bool is = xv[u][i] >= least && xv[u][i] > kNone;
              const uint64_t mask = __ballot(is);
              if (is) some[wave][n + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] =
                  key_of(xv[u][i], at0 + u * kStep + i - odd);
              n += __popcll(mask);
            }
            if (!n) continue;
            wave_lds_sync();
            if (n <= kFew)
              for (int i = 0; i < n; ++i) list.put(some[wave][i], lane);
            else
              list.sort_in(some[wave], n, lane);
            wave_lds_sync();
          }
        }
        list.close(a.top);
        if (lane == 0) __hip_atomic_store(&lasts[wave], list.last, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      }
    }
  }
  // The waves in their order.
  join_lanes(z, lane);
  if (lane == 0) part[wave] = make_float4(z.m, z.s, z.t, 0.f);
  if (TOP && lane < 32) some[wave][lane] = list.k;
  __syncthreads();
  if (wave) return;
  for (int w = 1; w < kWaves; ++w) {
    z.join(Sums{part[w].x, part[w].y, part[w].z});
    if constexpr (TOP) {  // two falling lists, one of them turned round
      if (lane >= 32) list.k = some[w][63 - lane];
      turn<64, 32>(list.k, lane);
    }
  }
  if (sl.n == 1) {
    finish(a, row, z, list, chosen, lane);
    return;
  }
  if (lane == 0) sl.sums[(int64_t)row * sl.n + slice] = make_float4(z.m, z.s, z.t, 0.f);
  if (TOP && lane < a.top) sl.keys[((int64_t)row * a.top + lane) * sl.n + slice] = list.k;
}

// Joins the slices of a row, a wave each: a lane's slices, then the lanes.
constexpr int kAhead = 8;  // entries of the lists loaded together
__global__ __launch_bounds__(kWave) void join_k(replay_token_logprobs_args a, Slices sl) {
  __shared__ Key some[kAhead * kWave];
  const int row = blockIdx.x, lane = threadIdx.x;
  const float4 *const sums = sl.sums + (int64_t)row * sl.n;
  const Key *const keys = sl.keys + (int64_t)row * sl.n * a.top;
  const float chosen = chosen_of(a, row);
  Sums z{kLowest, 0.f, 0.f};
  List list;
  list.clear();
  for (int s0 = 0; s0 < sl.n; s0 += kWave) {
    const bool is = s0 + lane < sl.n;
    const int s = is ? s0 + lane : 0;
    const float4 v = sums[s];
    for (int k0 = 0; k0 < a.top; k0 += kAhead) {
      Key k[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const Key x = keys[(int64_t)min(k0 + i, a.top - 1) * sl.n + s];
        k[i] = is && k0 + i < a.top ? x : 0;
      }
      float least = list.last;
      const float first = value_of(k[0]);
      const uint64_t beyond = __ballot(first > least);
      if (!beyond && !__ballot(first == least && first > kNone)) break;  // the lists fall: nothing further down either
      if (__popcll(beyond) > a.top) least = fmaxf(least, nth(first, a.top, lane));
      int n = 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const bool in = k[i] && value_of(k[i]) >= least;
        const uint64_t mask = __ballot(in);
        if (in) some[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] = k[i];
        n += __popcll(mask);
      }
      wave_lds_sync();
      list.sort_in(some, n, lane);
      list.close(a.top);
      wave_lds_sync();
      const float next = value_of(k[kAhead - 1]);  // at least what follows
      if (!__ballot(next >= list.last && next > kNone)) break;
    }
    if (is) z.join(Sums{v.x, v.y, v.z});
  }
  join_lanes(z, lane);
  finish(a, row, z, list, chosen, lane);
}

// Slices of 2048 values, longer where there would be more than 1024 workgroups: each slice
// starts its words anew (1024 rows of 131072, bf16, twenty alternatives: 77 us, 91 with up to
// 2048 and 76 with up to 512; 600 rows of 32000, float32, five: 21.4, 28.7 and 21.4; 256 rows of 50016,
// bf16, five: 21.1, 23.3 and 21.3).
Slices slices_of(int rows, int vocab) {
  Slices s{};
  s.size = kStep;
  while ((int64_t)rows * ((vocab + (int64_t)s.size - 1) / s.size) > 1024 && s.size < vocab) s.size *= 2;
  s.n = (int)((vocab + (int64_t)s.size - 1) / s.size);
  s.fn = make_fastdiv((uint32_t)s.n);
  return s;
}

size_t sums_bytes(int rows, const Slices &s) { return ((size_t)rows * s.n * sizeof(float4) + 255) / 256 * 256; }
size_t keys_bytes(int rows, const Slices &s, int top) { return (size_t)rows * s.n * top * sizeof(Key); }

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
  return s.n == 1 ? 0 : sums_bytes(rows, s) + keys_bytes(rows, s, top);
}

int launch_logprobs(const replay_token_logprobs_args &a, void *workspace, hipStream_t st) {
  Slices s = slices_of(a.rows, a.vocab);
  if ((int64_t)a.rows * s.n > kMostBlocks) return kTooLarge;
  s.sums = (float4 *)workspace;
  s.keys = (Key *)((char *)workspace + sums_bytes(a.rows, s));
  if (a.dtype == REPLAY_DT_BF16)
    launch<bf16_t>(a, s, st);
  else
    launch<float>(a, s, st);
  if (s.n > 1) hipLaunchKernelGGL(join_k, dim3((uint32_t)a.rows), dim3(kWave), 0, st, a, s);
  return (int)hipGetLastError();
}

}  // namespace rssm
