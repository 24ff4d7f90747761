// Norm of the residual stream, with the addition that leads to it.
//
//   h = x + residual,   out = w h / sqrt(mean(h^2) + eps)
//
// h is float32; the stream's copy of it is rounded once, in the residual's type, and
// the norm is of h itself.  In 8 bits a group of values shares a scale: out = scale
// times an e4m3 code, scale = max(largest |out| / 448, 2^-126).  Since w h / sqrt(..) is
// one rounded product with the root, the largest |out| of a group is that of w h times
// the root, and one turn through the row's lanes adds up the squares and finds it.
//
// HBM bound: a row stays in registers from its one read to its writes.  8192 rows of 8192
// (bf16): 98.7 us, 5.4 TB/s; 8192 rows of 4096 in e4m3 with scales of 128: 46 us, 5.1 TB/s; 256
// rows of 4096: 4.9 us with its launch, the latency of one read, one sum and one write.
#include "codecs.h"
#include "ops.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kCus = 256, kResident = 8;  // compute units, and workgroups of kThreads that one holds
struct e4m3_t {};  // an output of codes and scales

struct NormArgs {
  replay_residual_norm_args a;
  int lanes;       // lanes of a scale's group, or 0: the whole row shares one
  FastDiv fgroup;  // by the group's channels
};

template <int LANES>
__device__ __forceinline__ float max_lanes(float v) {  // over aligned groups of LANES lanes
  if constexpr (LANES >= 2) v = fmaxf(v, dpp_f<0xB1>(v));
  if constexpr (LANES >= 4) v = fmaxf(v, dpp_f<0x4E>(v));
  if constexpr (LANES >= 8) v = fmaxf(v, dpp_f<0x141>(v));
  if constexpr (LANES >= 16) v = fmaxf(v, dpp_f<0x140>(v));
  if constexpr (LANES >= 32) v = fmaxf(v, __shfl_xor(v, 16, kWave));
  if constexpr (LANES >= 64) v = fmaxf(v, __shfl_xor(v, 32, kWave));
  return v;
}
__device__ __forceinline__ float group_max(float v, int lanes) {
  switch (lanes) {  // the same for the whole launch
    case 2: return max_lanes<2>(v);
    case 4: return max_lanes<4>(v);
    case 8: return max_lanes<8>(v);
    case 16: return max_lanes<16>(v);
    case 32: return max_lanes<32>(v);
    default: return max_lanes<64>(v);
  }
}

__device__ __forceinline__ float scale_of(float largest) { return fmaxf(largest / 448.f, 0x1p-126f); }
// The codes of eight values over their scale; NaN stays NaN.
__device__ __forceinline__ void store_codes(uint8_t *p, int n, const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = e4m3_encode4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float u = v[4 * i + k] * inv;
      if (u != u) w[i] |= 0x7Fu << 8 * k;
    }
  }
  if (n >= 8) {
    typedef uint32_t words __attribute__((ext_vector_type(2)));
    typedef words loose __attribute__((aligned(1)));
    *reinterpret_cast<loose *>(p) = words{w[0], w[1]};
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = (uint8_t)(w[k / 4] >> 8 * (k % 4));
  }
}

// LANES threads a row (a wave, or the workgroup), IT steps of eight values each.
template <typename TX, typename TR, typename TO, int LANES, int IT>
__global__ __launch_bounds__(LANES == kWave ? kThreads : LANES) void residual_norm_k(NormArgs n) {
  constexpr bool CODES = std::is_same<TO, e4m3_t>::value;
  constexpr int ROWS = LANES == kWave ? kThreads / kWave : 1, WAVES = LANES / kWave;
  __shared__ float part[2][WAVES];
  const replay_residual_norm_args &a = n.a;
  const int lane = threadIdx.x % LANES, wave = threadIdx.x / kWave;
  const int t = blockIdx.x * ROWS + (LANES == kWave ? wave : 0), C = a.channels;
  if (t >= a.tokens) return;  // LANES == kWave: no barrier follows
  const TX *x = (const TX *)a.x + t * a.x_stride + lane * 8;
  const TR *res = (const TR *)a.residual + t * a.residual_stride + lane * 8;
  float h[IT][8], ss = 0.f, top[IT], largest = 0.f;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int in = C - (i * LANES + lane) * 8;
#pragma unroll
    for (int v = 0; v < 8; ++v) h[i][v] = 0.f;
    if (in > 0) {
      load_part<TX, 8>(x + i * LANES * 8, in, h[i]);
      if (a.residual) {
        float rv[8];
        load_part<TR, 8>(res + i * LANES * 8, in, rv);
#pragma unroll
        for (int v = 0; v < 8; ++v) h[i][v] += rv[v];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * LANES + lane) * 8, in = C - c;
    if (in > 0) {
      if (a.residual) store_part<TR, 8>((TR *)a.sum + t * a.sum_stride + c, in, h[i]);
      float w[8];
      if (a.weight) load_part<float, 8>(a.weight + c, in, w);
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        ss = fmaf(h[i][v], h[i][v], ss);
        if (a.weight) h[i][v] *= w[v];
      }
    }
    if constexpr (CODES) {
      float m = 0.f;
#pragma unroll
      for (int v = 0; v < 8; ++v) m = fmaxf(m, fabsf(h[i][v]));
      if (n.lanes)
        top[i] = group_max(m, n.lanes);
      else
        largest = fmaxf(largest, m);
    }
  }
  ss = sum_quarters(sum16(ss));
  if constexpr (CODES) largest = max_lanes<64>(largest);
  if constexpr (LANES > kWave) {
    if (threadIdx.x % kWave == 0) part[0][wave] = ss, part[1][wave] = largest;
    __syncthreads();
    ss = part[0][0], largest = part[1][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) ss += part[0][w], largest = fmaxf(largest, part[1][w]);
  }
  const float r = rsqrtf(ss / (float)C + a.eps);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * LANES + lane) * 8, in = C - c;
    if (in <= 0) continue;
#pragma unroll
    for (int v = 0; v < 8; ++v) h[i][v] *= r;
    if constexpr (CODES) {
      const float scale = scale_of((n.lanes ? top[i] : largest) * r);
      const int g = fdiv(c, n.fgroup);
      if (c == g * a.group) a.scales[(int64_t)t * (C / a.group) + g] = scale;
      store_codes((uint8_t *)a.out + t * a.out_stride + c, in, h[i], 1.f / scale);
    } else {
      store_part<TO, 8>((TO *)a.out + t * a.out_stride + c, in, h[i]);
    }
  }
}

// Rows of more than 16384: a workgroup each, two passes (the second reads what the first left
// in L2): 4096 rows of 24576 231 us, 3.5 TB/s of the one read and the writes; 4096 of 16384 146
// where one pass takes 101.
// Nothing is written in the first, so the sum may take the place of an input.
template <typename TX, typename TR, typename TO>
__global__ __launch_bounds__(kThreads) void residual_norm_long_k(NormArgs n) {
  constexpr bool CODES = std::is_same<TO, e4m3_t>::value;
  __shared__ float part[2][kWaves];
  const replay_residual_norm_args &a = n.a;
  const int t = blockIdx.x, C = a.channels, wave = threadIdx.x / kWave;
  const TX *x = (const TX *)a.x + t * a.x_stride;
  const TR *res = (const TR *)a.residual + t * a.residual_stride;
  auto load = [&](int c, float (&h)[8]) {
#pragma unroll
    for (int v = 0; v < 8; ++v) h[v] = 0.f;
    if (c >= C) return;
    load_part<TX, 8>(x + c, C - c, h);
    if (a.residual) {
      float rv[8];
      load_part<TR, 8>(res + c, C - c, rv);
#pragma unroll
      for (int v = 0; v < 8; ++v) h[v] += rv[v];
    }
  };
  auto weigh = [&](int c, float (&h)[8]) {
    float w[8];
    if (!a.weight || c >= C) return;
    load_part<float, 8>(a.weight + c, C - c, w);
#pragma unroll
    for (int v = 0; v < 8; ++v) h[v] *= w[v];
  };
  auto top = [](const float (&h)[8]) {
    float m = 0.f;
#pragma unroll
    for (int v = 0; v < 8; ++v) m = fmaxf(m, fabsf(h[v]));
    return m;
  };
  float ss = 0.f, largest = 0.f;
  for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
    float h[8];
    load(c, h);
#pragma unroll
    for (int v = 0; v < 8; ++v) ss = fmaf(h[v], h[v], ss);
    if (CODES && !n.lanes) {
      weigh(c, h);
      largest = fmaxf(largest, top(h));
    }
  }
  ss = sum_quarters(sum16(ss));
  if constexpr (CODES) largest = max_lanes<64>(largest);
  if (threadIdx.x % kWave == 0) part[0][wave] = ss, part[1][wave] = largest;
  __syncthreads();
  ss = part[0][0] + part[0][1] + part[0][2] + part[0][3];
  largest = fmaxf(fmaxf(part[1][0], part[1][1]), fmaxf(part[1][2], part[1][3]));
  const float r = rsqrtf(ss / (float)C + a.eps);
  for (int c0 = 0; c0 < C; c0 += kThreads * 8) {  // all lanes together: group_max reads its neighbours
    const int c = c0 + threadIdx.x * 8, in = C - c;
    float h[8];
    load(c, h);
    if (in > 0 && a.residual) store_part<TR, 8>((TR *)a.sum + t * a.sum_stride + c, in, h);
    weigh(c, h);
    float m = largest;
    if constexpr (CODES) {
      if (n.lanes) m = group_max(top(h), n.lanes);
    }
    if (in <= 0) continue;
#pragma unroll
    for (int v = 0; v < 8; ++v) h[v] *= r;
    if constexpr (CODES) {
      const float scale = scale_of(m * r);
      const int g = fdiv(c, n.fgroup);
      if (c == g * a.group) a.scales[(int64_t)t * (C / a.group) + g] = scale;
      store_codes((uint8_t *)a.out + t * a.out_stride + c, in, h, 1.f / scale);
    } else {
      store_part<TO, 8>((TO *)a.out + t * a.out_stride + c, in, h);
    }
  }
}

template <typename TX, typename TR, typename TO, int LANES, int IT>
int launch_fast(const NormArgs &n, hipStream_t st) {
  constexpr int PER = LANES == kWave ? kThreads / kWave : 1, THREADS = LANES == kWave ? kThreads : LANES;
  const int64_t blocks = ((int64_t)n.a.tokens + PER - 1) / PER;
  if (blocks * THREADS >= (int64_t)1 << 32) return kTooLarge;
  hipLaunchKernelGGL((residual_norm_k<TX, TR, TO, LANES, IT>), dim3((uint32_t)blocks), dim3(THREADS), 0, st, n);
  return (int)hipGetLastError();
}

// A row's threads.  More than 256, and so fewer steps, where a CU has two rows at most, whose
// latency counts (256 rows of 4096: 4.9 us, 5.7 with 256; of 8192: 6.1 and 8.2; of 16384: 9.1
// and 13.3), and where the rows are more than are resident at once with 256 threads each
// (16384 rows of 8192: 184 and 205 us, 5.8 TB/s; of 4096: 95.8 and 101), but not between
// (2048 rows of 8192: 27.4 and 23.8) nor for rows that start at odd places (16384 of 5003: 218
// and 165).  Up to 1024 channels a wave each and no barrier (65536 rows of 512: 46.6 us, 85.5
// with a workgroup; 8192 of 1024: 13.6 and 17.3).  Rows too many for a launch of so many
// threads each (2^23 with 512, 2^22 with 1024) have 256.
bool wide(const NormArgs &n, int threads) {
  const replay_residual_norm_args &a = n.a;
  if ((int64_t)a.tokens * threads >= (int64_t)1 << 32) return false;
  if (a.tokens <= 2 * kCus) return true;
  return a.tokens > kResident * kCus && ((a.channels | a.x_stride | a.residual_stride) & 7) == 0;
}

template <typename TX, typename TR, typename TO>
int launch(const NormArgs &n, hipStream_t st) {
  const int C = n.a.channels;
  const bool w = wide(n, C <= 4096 ? 512 : 1024);
  if (C <= 512) return launch_fast<TX, TR, TO, kWave, 1>(n, st);
  if (C <= 1024) return launch_fast<TX, TR, TO, kWave, 2>(n, st);
  if (C <= 2048) return launch_fast<TX, TR, TO, kThreads, 1>(n, st);
  if (C <= 4096) return w ? launch_fast<TX, TR, TO, 512, 1>(n, st) : launch_fast<TX, TR, TO, kThreads, 2>(n, st);
  if (C <= 8192) return w ? launch_fast<TX, TR, TO, 1024, 1>(n, st) : launch_fast<TX, TR, TO, kThreads, 4>(n, st);
  if (C <= 16384) return w ? launch_fast<TX, TR, TO, 1024, 2>(n, st) : launch_fast<TX, TR, TO, kThreads, 8>(n, st);
  if (n.a.tokens > kMostBlocks) return kTooLarge;
  hipLaunchKernelGGL((residual_norm_long_k<TX, TR, TO>), dim3((uint32_t)n.a.tokens), dim3(kThreads), 0, st, n);
  return (int)hipGetLastError();
}

template <typename TX, typename TR>
int launch_o(const NormArgs &n, hipStream_t st) {
  if (n.a.out_dtype == REPLAY_DT_E4M3) return launch<TX, TR, e4m3_t>(n, st);
  return n.a.out_dtype == REPLAY_DT_BF16 ? launch<TX, TR, bf16_t>(n, st) : launch<TX, TR, float>(n, st);
}
template <typename TX>
int launch_r(const NormArgs &n, hipStream_t st) {
  return n.a.residual_dtype == REPLAY_DT_BF16 ? launch_o<TX, bf16_t>(n, st) : launch_o<TX, float>(n, st);
}

}  // namespace

int launch_residual_norm(const replay_residual_norm_args &a, hipStream_t st) {
  NormArgs n{};
  n.a = a;
  if (a.out_dtype == REPLAY_DT_E4M3) {
    n.lanes = a.group == a.channels ? 0 : a.group / 8;
    n.fgroup = make_fastdiv((uint32_t)a.group);
  }
  return a.x_dtype == REPLAY_DT_BF16 ? launch_r<bf16_t>(n, st) : launch_r<float>(n, st);
}

}  // namespace rssm
