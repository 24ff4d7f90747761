// Mamba-2 recurrence over packed prompts: S <- exp(dt A) S + dt x B^T, y = S C + D x.
//
// One workgroup per (sequence, head) walks its tokens in order with the state
// in registers: thread (p, j) holds columns 16 j .. 16 j + 15 of row p.
#include "ops.h"

namespace rssm {
namespace {

template <typename R, typename Y>
__global__ __launch_bounds__(1024) void scan_k(ScanArgs a) {
  const int seq = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int row = batch_row(a.p, seq, h == 0 && threadIdx.x == 0);
  if (row < 0) return;
  const int b = clamp_start(a.p, seq), e = max(b, clamp_start(a.p, seq + 1));
  const int J = a.N / 16;
  const int p = threadIdx.x / J, j = threadIdx.x % J;
  const int g = h / (a.H / a.G);
  float s[16];
  const size_t at = (((size_t)row * a.H + h) * a.P + p) * a.N + 16 * j;
  const bool known = a.initial && (!a.p.resume || a.p.resume[seq]);
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = known ? a.initial[at + i] : 0.f;
  const float A = a.A[h], D = a.D[h];
  for (int t = b; t < e; ++t) {
    const float dt = a.dt[(size_t)t * a.H + h];
    const float x = ldr<R>((const R *)a.x + ((size_t)t * a.H + h) * a.P + p);
    const R *Bp = (const R *)a.Bm + ((size_t)t * a.G + g) * a.N + 16 * j;
    const R *Cp = (const R *)a.Cm + ((size_t)t * a.G + g) * a.N + 16 * j;
    const float dec = expf(dt * A), dx = dt * x;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 bv = ldr4<R>(Bp + i), cv = ldr4<R>(Cp + i);
      s[i] = fmaf(dec, s[i], dx * bv.x), s[i + 1] = fmaf(dec, s[i + 1], dx * bv.y);
      s[i + 2] = fmaf(dec, s[i + 2], dx * bv.z), s[i + 3] = fmaf(dec, s[i + 3], dx * bv.w);
      y = fmaf(s[i], cv.x, fmaf(s[i + 1], cv.y, fmaf(s[i + 2], cv.z, fmaf(s[i + 3], cv.w, y))));
    }
    for (int d = 1; d < J; d <<= 1) y += __shfl_xor(y, d, kWave);
    if (j == 0) {
      float o[1] = {fmaf(D, x, y)};
      store_vec<Y, 1>((Y *)a.y + ((size_t)t * a.H + h) * a.P + p, o);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; i += 4) st4(a.state + at + i, make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]));
}

}  // namespace

size_t scan_workspace(const ScanArgs &) { return 0; }

int launch_scan(const ScanArgs &a, hipStream_t st) {
  const int64_t blocks = (int64_t)a.p.n * a.H;
  if (blocks > 0x7fffffffLL) return (int)hipErrorInvalidValue;
  const dim3 grid((uint32_t)blocks), block(a.P * (a.N / 16));
  if (!a.bf16)
    hipLaunchKernelGGL((scan_k<float, float>), grid, block, 0, st, a);
  else if (a.y_bf16)
    hipLaunchKernelGGL((scan_k<bf16_t, bf16_t>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((scan_k<bf16_t, float>), grid, block, 0, st, a);
  return (int)hipGetLastError();
}

}  // namespace rssm
