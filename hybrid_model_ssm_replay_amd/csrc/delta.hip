// Gated delta rule over packed prompts: S <- a S (I - b k k^T) + b v k^T, o = S q.
//
// Chunks of 64 tokens turn it into matrix products.  With g_t the sum of log a over
// the chunk's tokens up to t and S0 the state before it:
//   T[t][j] = b_t e^{g_t - g_j} k_t.k_j  (j < t, else 0),   A = (I + T)^-1 diag(b),
//   P[t][j] = e^{g_t - g_j} q_t.k_j      (j <= t, else 0),
//   U = A (V - diag(e^g) K S0^T),   O = diag(e^g) Q S0^T + P U,
//   S1 = e^{g_C} S0 + sum_j e^{g_C - g_j} u_j k_j^T.
//
// Two launches.  cells_k makes A and P of every chunk and head (a cell), all at once:
// they do not depend on the state.  chain_k walks a sequence's chunks, a workgroup for
// 16 (or 32) rows of a head's state, which evolve independently of the others; its four
// waves take a quarter of the chunk's tokens each for V - K S0^T, U and O, and a quarter
// of the state's columns for S1, and hand each other S, V - K S0^T and U through LDS.
//
// The inverse is a forward substitution inside the diagonal blocks of 16 tokens, joined
// block by block below them in float32 matrix products; no power of T is formed, whose
// entries would grow where keys are alike.  Differences g_t - g_j are taken in float64.
#include <algorithm>

#include "ops.h"
#include "pieces.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int Q = 64;                 // tokens of a chunk
constexpr int kSteps = 6;             // 32-token steps of the lower triangle, by rows of 16 tokens: 1, 1, 2, 2
constexpr int kFrag = kWave * 16;     // bytes of an operand, a lane's 16 bytes each
constexpr int kNowhere = 0x7fffff00;  // past the end of every buffer

__device__ __forceinline__ int step_of(int w, int s) { return w < 2 ? w : 2 * w - 2 + s; }

// What cells_k leaves for chain_k of one chunk and head: operands as the lanes hold
// them.  Operands with tokens along the sum take them in the order of an accumulator
// pair: slot 8 q + 4 h + i of step s is token 32 s + 16 h + 4 q + i.
template <typename R, typename Y, int NK>
struct Cell {
  static constexpr int IP = sizeof(R) == 4 ? 3 : 1;  // pieces of an input
  static constexpr int MP = sizeof(Y) == 4 ? 3 : 2;  // pieces of P, U and S in the output products
  static constexpr int A0 = 0;                       // [3][kSteps]
  static constexpr int P0 = A0 + 3 * kSteps * kFrag;     // [MP][kSteps]
  static constexpr int ROW = sizeof(R) / 2 * kFrag;      // a record's rows, as loaded
  static constexpr int K0 = P0 + MP * kSteps * kFrag;    // [4 tiles of 16 tokens][NK]
  static constexpr int Q0 = K0 + 4 * NK * ROW;
  static constexpr int G0 = Q0 + 4 * NK * ROW;           // e^{g_t} [64], e^{g_C - g_t} [64]
  static constexpr int BYTES = G0 + 2 * Q * 4;
};

struct DeltaPlan {
  int lo, hi;      // the chunks of this pass: places start / 64 + sequence + chunk
  int ny;          // slices of a head's rows
  int units;       // sequences x heads of the pass at most
  FastDiv fH, fny;
  char *cells;     // [hi - lo][H] of Cell
};

// Eight neighbouring columns of a record's row: as loaded, and as an operand in IP pieces.
template <typename R>
struct Rows {
  typedef uint16_t bits;
  uint4 v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int at, int plus) { v = buffer_load16(b, at, plus); }
  __device__ __forceinline__ void get(__amdgpu_buffer_rsrc_t b, int lane, int plus) { v = buffer_load16(b, lane * 16, plus); }
  // The first or second four alone.
  __device__ __forceinline__ void get_half(__amdgpu_buffer_rsrc_t b, int lane, int half, int plus) {
    const i32x2 x = __builtin_bit_cast(i32x2, __builtin_amdgcn_raw_buffer_load_b64(b, lane * 16 + 8 * half, plus, 0));
    v = make_uint4(x[0], x[1], 0, 0);
  }
  __device__ __forceinline__ void put(char *to, int lane) const { reinterpret_cast<uint4 *>(to)[lane] = v; }
  __device__ __forceinline__ void stage(char *to, int) const { *reinterpret_cast<uint4 *>(to) = v; }
  __device__ __forceinline__ void staged(const char *from, int) { v = *reinterpret_cast<const uint4 *>(from); }
  __device__ __forceinline__ void cut(Frag (&f)[1]) const { f[0].v = __builtin_bit_cast(s16x8, v); }
};
template <>
struct Rows<float> {
  typedef uint32_t bits;
  uint4 v, w;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int at, int plus) {
    v = buffer_load16(b, at, plus), w = buffer_load16(b, at, plus + 16);
  }
  __device__ __forceinline__ void get(__amdgpu_buffer_rsrc_t b, int lane, int plus) {
    v = buffer_load16(b, lane * 16, plus), w = buffer_load16(b, lane * 16, plus + kFrag);
  }
  __device__ __forceinline__ void get_half(__amdgpu_buffer_rsrc_t b, int lane, int half, int plus) {
    v = buffer_load16(b, lane * 16 + half * kFrag, plus), w = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void put(char *to, int lane) const {
    reinterpret_cast<uint4 *>(to)[lane] = v, reinterpret_cast<uint4 *>(to + kFrag)[lane] = w;
  }
  __device__ __forceinline__ void stage(char *to, int plane) const {
    *reinterpret_cast<uint4 *>(to) = v, *reinterpret_cast<uint4 *>(to + plane) = w;
  }
  __device__ __forceinline__ void staged(const char *from, int plane) {
    v = *reinterpret_cast<const uint4 *>(from), w = *reinterpret_cast<const uint4 *>(from + plane);
  }
  __device__ __forceinline__ void cut(Frag (&f)[3]) const {
    const uint32_t e[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t p[3];
      pieces<3>(__uint_as_float(e[2 * i]), __uint_as_float(e[2 * i + 1]), p);
#pragma unroll
      for (int u = 0; u < 3; ++u) f[u].w[i] = p[u];
    }
  }
};

__device__ __forceinline__ void put(char *to, int lane, const Frag &f) { *reinterpret_cast<s16x8 *>(to + lane * 16) = f.v; }
__device__ __forceinline__ Frag get(const char *from, int lane) {
  Frag f;
  f.v = *reinterpret_cast<const s16x8 *>(from + lane * 16);
  return f;
}

constexpr int kT = Q + 4;  // floats of a row of T and A in LDS

// Place of granule g of a row of K or Q in LDS, permuted so that 16 rows at one granule
// meet in no bank.
template <int NK>
__device__ __forceinline__ int place_of(int row, int g) {
  return row * 64 * NK + (g ^ (NK == 4 ? row & 15 : NK == 2 ? row >> 1 & 7 : row >> 2 & 3)) * 16;
}

// v where `keep`, else 0: a mask, since a condition would become a branch around v.
__device__ __forceinline__ float only(float v, bool keep) { return __uint_as_float(bits(v) & (keep ? ~0u : 0u)); }

template <typename R, typename Y, int NK>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(sizeof(R) == 4 ? 2 : 4)))
void cells_k(DeltaArgs a, DeltaPlan plan) {
  typedef Cell<R, Y, NK> C;
  constexpr int IP = C::IP, MP = C::MP;
  constexpr int NV = 4 * NK, RB = kThreads / NV;           // granules of eight columns in a row, rows a load
  constexpr int PL = sizeof(R) / 2, ROWS = Q * 16 * NV;    // planes of 16 bytes a granule, bytes of one
  constexpr int TA = 2 * Q * kT * 4, KQ = 2 * PL * ROWS;
  // K and Q, then (they are in registers) T and A.
  __shared__ __attribute__((aligned(16))) char pool[TA > KQ ? TA : KQ];
  float *const sT = reinterpret_cast<float *>(pool), *const sA = sT + Q * kT;
  __shared__ __attribute__((aligned(16))) float sD[kWaves][16][20], sB[Q];
  __shared__ __attribute__((aligned(16))) double sG[Q];
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r = lane % 16, q = lane / 16;
  const int place = fdiv(blockIdx.x, plan.fH), h = blockIdx.x - place * a.H;
  const Item it = find_item(a.p, plan.lo + place, Q);
  const int t0 = it.index * Q;
  if (it.index < 0 || t0 >= it.len) return;
  const int rem = min(Q, it.len - t0), N = a.N;
  const int64_t row0 = (int64_t)it.begin + t0;
  char *const cell = plan.cells + ((int64_t)place * a.H + h) * C::BYTES;

  // Decays: lane = token; past the end a = 1 and b = 0.  A decay of zero forgets everything.
  const int tl = min(lane, rem - 1);
  const float al = a.alpha[(row0 + tl) * a.H + h], be = a.beta[(row0 + tl) * a.H + h];
  const int64_t rK = (int64_t)a.H * N;
  const size_t nK = (size_t)((rem - 1) * rK + N) * sizeof(R);
  const auto bK = buffer_of((const R *)a.k + row0 * rK + (int64_t)h * N, nK);
  const auto bQ = buffer_of((const R *)a.q + row0 * rK + (int64_t)h * N, nK);
  // Whole rows of K and Q, as neighbouring lanes read them, into LDS.
  {
    const int trow = tid / NV, g = tid % NV;
    const int at = 8 * g < N && trow < Q ? (int)((trow * rK + 8 * g) * sizeof(R)) : kNowhere;
    Rows<R> k[Q / RB > 0 ? Q / RB : 1], x[Q / RB > 0 ? Q / RB : 1];
#pragma unroll
    for (int i = 0; i < Q / RB; ++i) k[i].load(bK, at, (int)(i * RB * rK * sizeof(R)));
#pragma unroll
    for (int i = 0; i < Q / RB; ++i) x[i].load(bQ, at, (int)(i * RB * rK * sizeof(R)));
#pragma unroll
    for (int i = 0; i < Q / RB; ++i) {
      k[i].stage(pool + place_of<NK>(trow + i * RB, g), ROWS);
      x[i].stage(pool + PL * ROWS + place_of<NK>(trow + i * RB, g), ROWS);
    }
  }
  if (wave == 0) {
    double g = lane < rem ? (double)log2f(al) : 0.0;
    g = scan64(g < -4096.0 ? -4096.0 : g);
    sG[lane] = g;
    sB[lane] = lane < rem ? be : 0.f;
    float *const e = reinterpret_cast<float *>(cell + C::G0);
    e[lane] = __builtin_amdgcn_exp2f((float)g);
    e[Q + lane] = __builtin_amdgcn_exp2f((float)(lane_value(g, kWave - 1) - g));
  }
  __syncthreads();

  // P^T of this wave's rows of 16 tokens, G^T = (K K^T)^T of the rows 3 - wave; all four
  // tiles of a row, of which those right of the diagonal are masked away.
  const int wg = 3 - wave;
  floatx4 aP[4], aG[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) aP[j] = aG[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll IP == 1 ? NK : 1
  for (int s = 0; s < NK; ++s) {
    Rows<R> row;
    Frag k[4][IP], qf[IP], kg[IP];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      row.staged(pool + place_of<NK>(16 * j + r, 4 * s + q), ROWS);
      row.cut(k[j]);
    }
    row.staged(pool + PL * ROWS + place_of<NK>(16 * wave + r, 4 * s + q), ROWS);
    row.put(cell + C::Q0 + (wave * NK + s) * C::ROW, lane);
    row.cut(qf);
    row.staged(pool + place_of<NK>(16 * wg + r, 4 * s + q), ROWS);
    row.put(cell + C::K0 + (wg * NK + s) * C::ROW, lane);
    row.cut(kg);
#pragma unroll
    for (int u = IP - 1; u >= 0; --u)
#pragma unroll
      for (int v = IP - 1 - u; v >= 0; --v)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          aP[j] = mfma32(k[j][u], qf[v], aP[j]);
          aG[j] = mfma32(k[j][u], kg[v], aG[j]);
        }
  }
  __syncthreads();
  {
    const double gt = sG[16 * wave + r], gg = sG[16 * wg + r];
    const float bt = sB[16 * wg + r];
    char *const to = cell + C::P0 + step_of(wave, 0) * kFrag;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Frag f[MP];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 2 * s + e;
        float p[4], t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 16 * j + 4 * q + i;
          const double gj = sG[tok];
          p[i] = only(aP[j][i] * __builtin_amdgcn_exp2f((float)(gt - gj)), tok <= 16 * wave + r);
          t[i] = only(bt * (aG[j][i] * __builtin_amdgcn_exp2f((float)(gg - gj))), tok < 16 * wg + r);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[MP];
          pieces<MP>(p[2 * i], p[2 * i + 1], w);
#pragma unroll
          for (int u = 0; u < MP; ++u) f[u].w[2 * e + i] = w[u];
        }
        st4(sT + (16 * wg + r) * kT + 16 * j + 4 * q, make_float4(t[0], t[1], t[2], t[3]));
      }
      if (s <= wave / 2) {
#pragma unroll
        for (int u = 0; u < MP; ++u) put(to + (u * kSteps + s) * kFrag, lane, f[u]);
      }
    }
  }
  __syncthreads();

  // Column r of the inverse of the diagonal block `wave`, by substitution, in every 16 lanes.
  {
    float x[16];
    const float *const T = sT + 16 * wave * kT + 16 * wave;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      x[t] = t == r ? 1.f : 0.f;
      if (t % 4 == 0) __builtin_amdgcn_sched_barrier(0);  // not all rows' loads at once
#pragma unroll
      for (int s4 = 0; s4 < t; s4 += 4) {
        const float4 tv = ld4(T + t * kT + s4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (s4 + i < t) x[t] = fmaf(-f4get(tv, i), x[s4 + i], x[t]);
      }
    }
    if (q == 0) {
#pragma unroll
      for (int t = 0; t < 16; ++t) sD[wave][t][r] = x[t];
    }
  }
  __syncthreads();
  // Block column `wave` of the inverse, tile d below the diagonal: rows 16 (wave + d) + 4 q + e, column r.
  floatx4 X[4];
  const float bj = sB[16 * wave + r];
#pragma unroll
  for (int e = 0; e < 4; ++e) X[0][e] = sD[wave][4 * q + e][r];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if (wave + d >= 4) break;
    if (d > 0) {
      floatx4 acc = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < d; ++m) {
        const float4 tv = ld4(sT + (16 * (wave + d) + r) * kT + 16 * (wave + m) + 4 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = mfma_16x16x4(f4get(tv, e), X[m][e], acc);
      }
      const float4 dv = ld4(&sD[wave + d][r][4 * q]);
      X[d] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) X[d] = mfma_16x16x4(-f4get(dv, e), acc[e], X[d]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sA[(16 * (wave + d) + 4 * q + e) * kT + 16 * wave + r] = X[d][e] * bj;
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > wave / 2) break;
    Frag f[3];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (2 * s + e <= wave) v = ld4(sA + (16 * wave + r) * kT + 32 * s + 16 * e + 4 * q);
      uint32_t w0[3], w1[3];
      pieces<3>(v.x, v.y, w0);
      pieces<3>(v.z, v.w, w1);
#pragma unroll
      for (int u = 0; u < 3; ++u) f[u].w[2 * e] = w0[u], f[u].w[2 * e + 1] = w1[u];
    }
#pragma unroll
    for (int u = 0; u < 3; ++u) put(cell + C::A0 + (u * kSteps + step_of(wave, 0) + s) * kFrag, lane, f[u]);
  }
}

// Four float32 values in a row of 16-bit places, NP pieces `gap` bytes apart.
template <int NP>
__device__ __forceinline__ void hand(char *to, int gap, const floatx4 &v) {
  uint32_t a[NP], b[NP];
  pieces<NP>(v[0], v[1], a);
  pieces<NP>(v[2], v[3], b);
#pragma unroll
  for (int u = 0; u < NP; ++u) *reinterpret_cast<uint2 *>(to + u * gap) = make_uint2(a[u], b[u]);
}

// Waves 0 to 3 carry the state, waves 4 to 7 make the outputs; wave w of either has the
// chunk's tokens 16 w .. + 15, and of the former the state's columns 32 w .. + 31 too, in
// two tiles: row 4 q + i of tile m is column 8 q + 4 m + i.  Where there are 64 or fewer
// columns a wave has one of two such tiles.
template <typename R, typename Y, int NK, int CT>
__global__ __launch_bounds__(2 * kThreads) void chain_k(DeltaArgs a, DeltaPlan plan) {
  typedef Cell<R, Y, NK> C;
  constexpr int IP = C::IP, MP = C::MP, COLS = 16 * CT;
  constexpr int MT = NK == 4 ? 2 : 1;                // tiles of the state's columns that a wave has
  constexpr int CW = NK == 1 ? 2 : 4;                // waves that have any
  constexpr int SR = 64 * NK + 16, TR = 2 * Q + 16;  // bytes of a row of S, and of 64 tokens, in LDS
  constexpr int KR = 64;                             // bytes of a row of a wave's columns of K in LDS
  __shared__ __attribute__((aligned(16))) char sS[MP][COLS * SR], sR[3][COLS * TR], sW[3][COLS * TR], sU[MP][COLS * TR];
  __shared__ __attribute__((aligned(16))) char sK[kWaves][IP][Q * KR];
  __shared__ float4 sX[CW][kWaves][CT][kWave];
  const int tid = threadIdx.x, lane = tid % kWave, eighth = __builtin_amdgcn_readfirstlane(tid / kWave), wave = eighth % 4;
  const int r = lane % 16, q = lane / 16;
  // Unit u, a sequence's head, on XCD u % 8: its slices share what cells_k left in an L2.
  const int k8 = blockIdx.x / kXcds, u8 = fdiv(k8, plan.fny);
  const int unit = u8 * kXcds + blockIdx.x % kXcds, slice = k8 - u8 * plan.ny;
  if (unit >= plan.units) return;
  const int n = fdiv(unit, plan.fH), h = unit - n * a.H, P = a.P, N = a.N;
  const int seq = find_item(a.p, plan.lo, Q).seq + n;
  if (seq >= a.p.n) return;
  const int begin = clamp_start(a.p, seq), len = max(0, clamp_start(a.p, seq + 1) - begin);
  const int base = begin / Q + seq, chunks = (len + Q - 1) / Q;  // the sequence's places
  if (base >= plan.hi || base + max(chunks, 1) <= plan.lo) return;
  const int c0 = max(0, plan.lo - base), c1 = min(chunks, plan.hi - base);
  const int row = batch_row(a.p, seq, h == 0 && slice == 0 && tid == 0 && c0 == 0);
  if (row < 0) return;

  // Everything that a chunk reads from memory is loaded a chunk ahead, right behind the use
  // of the chunk before; behind the last one the loads repeat it, or read nothing.
  const int64_t rV = (int64_t)a.H * P, cells = (int64_t)a.H * C::BYTES;
  const char *cell = plan.cells + ((int64_t)(base + c0 - plan.lo) * a.H + h) * C::BYTES;
  const int64_t row0 = (int64_t)begin + c0 * Q;
  int rem = len - c0 * Q;  // of the chunk to be loaded next
  const int most = wave / 2;  // the last step of the wave's rows of the lower triangle
  const int oF0 = step_of(wave, 0) * kFrag + lane * 16, oF1 = step_of(wave, min(1, most)) * kFrag + lane * 16;
  auto rows_v = [&](const void *p, int esize) {
    const int m = min(rem, Q);
    return buffer_of(p, m > 0 ? (size_t)((m - 1) * rV + COLS) * esize : 0);
  };
  auto operand = [&](__amdgpu_buffer_rsrc_t b, int at, int plus) {
    Frag f;
    f.v = __builtin_bit_cast(s16x8, buffer_load16(b, at, plus));
    return f;
  };
  const int oF = r * TR + 16 * q;  // of 64 tokens' row r, slots 8 q .. + 7

  if (eighth < 4) {
    // The state, transposed: columns s0 + 4 m + i of k, row r of the slice's tile.
    floatx4 S[MT][CT];
    const int s0 = (MT == 2 ? 32 * wave : 32 * (wave / 2) + 4 * (wave % 2)) + 8 * q;
    const bool any = CW == 4 || wave < CW;
    const size_t tile0 = ((size_t)row * a.H + h) * P * N + (size_t)(slice * COLS + r) * N + s0;
    const bool known = a.initial && (!a.p.resume || a.p.resume[seq]);
    const float *const from = c0 ? a.state : known ? a.initial : nullptr;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        S[m][ct] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (from && s0 < N) {
          const float4 v = ld4(from + tile0 + (size_t)16 * ct * N + 4 * m);
          S[m][ct] = floatx4{v.x, v.y, v.z, v.w};
        }
      }
    const char *pV = (const char *)((const R *)a.v + row0 * rV + (int64_t)h * P + slice * COLS);
    int oV[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) oV[i] = (int)(((16 * wave + 4 * q + i) * rV + r) * sizeof(R));
    Rows<R> kr[4];
    Frag af[2][3];
    typename Rows<R>::bits v[CT][4];  // as loaded: a conversion would wait for it
    float4 eg4, left4;
    float whole;
    auto load_k = [&]() {
      const auto b = buffer_of(cell, C::BYTES);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if constexpr (MT == 2)
          kr[t].get(b, lane, C::K0 + (t * NK + wave) * C::ROW);
        else
          kr[t].get_half(b, lane, wave % 2, C::K0 + (t * NK + (any ? wave / 2 : 0)) * C::ROW);
      }
    };
    auto load_v = [&]() {
      const auto b = rows_v(pV, sizeof(R));
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (IP == 1)
            v[ct][i] = __builtin_amdgcn_raw_buffer_load_b16(b, oV[i] + 32 * ct, 0, 0);
          else
            v[ct][i] = __builtin_amdgcn_raw_buffer_load_b32(b, oV[i] + 64 * ct, 0, 0);
        }
    };
    auto load_eg = [&]() { eg4 = __builtin_bit_cast(float4, buffer_load16(buffer_of(cell, C::BYTES), 64 * wave + 16 * q, C::G0)); };
    auto load_left = [&]() {
      left4 = __builtin_bit_cast(float4, buffer_load16(buffer_of(cell, C::BYTES), 64 * wave + 16 * q, C::G0 + 4 * Q));
    };
    auto load_whole = [&]() {
      whole = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buffer_of(cell, C::BYTES), 4 * (Q - 1), C::G0, 0));
    };
    auto load_a = [&]() {
      const auto b = buffer_of(cell, C::BYTES);
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        af[0][u] = operand(b, oF0, C::A0 + u * kSteps * kFrag);
        af[1][u] = operand(b, oF1, C::A0 + u * kSteps * kFrag);
      }
    };
    // K in LDS, the wave's own columns: rows of eight 8-byte granules, permuted so that
    // neither the writes (16 rows at two granules) nor the transposing reads (eight rows at
    // every second granule) meet in a bank.  Those leave four rows 4 q .. + 3 of the column
    // that is row r of a tile in a lane.
    auto turned = [](int g) { return (g & 1) | (g >> 1) * 4; };
    char *const toK = sK[wave][0] + r * KR;
    const char *const fromK = sK[wave][0] + (4 * q + r / 4) * KR;
    int gw[2], gr[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) gw[m] = ((2 * q + m) ^ turned(r >> 2)) * 8, gr[m] = ((2 * (r % 4) + m) ^ turned(q)) * 8;
    if (c0 < c1) {  // in the loop's order: what waits for the first must not wait for the last
      load_k();
      __builtin_amdgcn_sched_barrier(0);
      load_v();
      load_eg();
      __builtin_amdgcn_sched_barrier(0);
      load_a();
      load_left();
      __builtin_amdgcn_sched_barrier(0);
      load_whole();
      __builtin_amdgcn_sched_barrier(0);
    }
    // Place of the wave's tokens 4 q + i in a row of 64: step wave / 2, half wave % 2.
    const int oT = r * TR + (32 * (wave / 2) + 8 * q + 4 * (wave % 2)) * 2;
    for (int c = c0; c < c1; ++c) {
      rem -= Q;
      pV += Q * rV * sizeof(R);
      if (c + 1 < c1) cell += cells;
      // K S^T summed over the wave's columns, all tokens; S goes to the output waves.
      if (any) {
        Frag kf[4][IP];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          kr[t].cut(kf[t]);
#pragma unroll
          for (int u = 0; u < IP; ++u)
#pragma unroll
            for (int m = 0; m < MT; ++m) *reinterpret_cast<s16x4 *>(toK + (u * Q + 16 * t) * KR + gw[m]) = kf[t][u].h[m];
        }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          Frag sf[3];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t w0[3] = {0, 0, 0}, w1[3] = {0, 0, 0};
            if (m < MT) {
              pieces<3>(S[m < MT ? m : 0][ct][0], S[m < MT ? m : 0][ct][1], w0);
              pieces<3>(S[m < MT ? m : 0][ct][2], S[m < MT ? m : 0][ct][3], w1);
            }
#pragma unroll
            for (int u = 0; u < 3; ++u) sf[u].w[2 * m] = w0[u], sf[u].w[2 * m + 1] = w1[u];
          }
#pragma unroll
          for (int u = 0; u < MP; ++u) {
            if constexpr (MT == 2)
              *reinterpret_cast<s16x8 *>(sS[u] + (16 * ct + r) * SR + (32 * wave + 8 * q) * 2) = sf[u].v;
            else
              *reinterpret_cast<s16x4 *>(sS[u] + (16 * ct + r) * SR + (32 * (wave / 2) + 8 * q + 4 * (wave % 2)) * 2) = sf[u].h[0];
          }
          floatx4 X[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) X[t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int u = 2; u >= 0; --u)
#pragma unroll
            for (int w = IP - 1; w >= 0; --w)
              if (u + w < 3) {
#pragma unroll
                for (int t = 0; t < 4; ++t) X[t] = mfma32(kf[t][w], sf[u], X[t]);
              }
#pragma unroll
          for (int t = 0; t < 4; ++t) sX[wave][t][ct][lane] = make_float4(X[t][0], X[t][1], X[t][2], X[t][3]);
        }
      }
      load_k();
      lds_barrier();  // the waves' sums are there, and S
      Frag kt[MT][2][IP];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float4 x = sX[0][wave][ct][lane];
#pragma unroll
        for (int w = 1; w < CW; ++w) {
          const float4 y = sX[w][wave][ct][lane];
          x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        const float egv[4] = {eg4.x, eg4.y, eg4.z, eg4.w}, xv[4] = {x.x, x.y, x.z, x.w};
        floatx4 d;
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = fmaf(-egv[i], xv[i], IP == 1 ? lower((uint32_t)v[ct][i]) : __uint_as_float(v[ct][i]));
        hand<3>(sR[0] + 16 * ct * TR + oT, COLS * TR, d);
      }
      load_v();
      load_eg();
      lds_barrier();  // V - K S^T is there
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int ts = 0; ts < 2; ++ts)
#pragma unroll
          for (int u = 0; u < IP; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) kt[m][ts][u].h[e] = read_tr(fromK + (u * Q + 32 * ts + 16 * e) * KR + gr[m]);
      const float lev[4] = {left4.x, left4.y, left4.z, left4.w};
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        floatx4 U = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (s <= most) {
            Frag rf[3];
#pragma unroll
            for (int u = 0; u < 3; ++u) rf[u].v = *reinterpret_cast<const s16x8 *>(sR[u] + 16 * ct * TR + oF + 64 * s);
#pragma unroll
            for (int u = 2; u >= 0; --u)
#pragma unroll
              for (int w = 2 - u; w >= 0; --w) U = mfma32(af[s][u], rf[w], U);
          }
        hand<MP>(sU[0] + 16 * ct * TR + oT, COLS * TR, U);
#pragma unroll
        for (int i = 0; i < 4; ++i) U[i] *= lev[i];
        hand<3>(sW[0] + 16 * ct * TR + oT, COLS * TR, U);
      }
      load_a();
      load_left();
      lds_barrier();  // U is there
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          S[m][ct] *= whole;
          asm volatile("" : "+v"(S[m][ct]));  // before the next value is loaded: a copy of it would wait for the load
        }
      load_whole();
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int ts = 0; ts < 2; ++ts) {
          Frag wf[3];
#pragma unroll
          for (int u = 0; u < 3; ++u) wf[u].v = *reinterpret_cast<const s16x8 *>(sW[u] + 16 * ct * TR + oF + 64 * ts);
#pragma unroll
          for (int u = 2; u >= 0; --u)
#pragma unroll
            for (int w = IP - 1; w >= 0; --w)
              if (u + w < 3) {
#pragma unroll
                for (int m = 0; m < MT; ++m) S[m][ct] = mfma32(kt[m][ts][w], wf[u], S[m][ct]);
              }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        if (s0 < N)
          st4(a.state + tile0 + (size_t)16 * ct * N + 4 * m, make_float4(S[m][ct][0], S[m][ct][1], S[m][ct][2], S[m][ct][3]));
  } else {
    char *pY = (char *)((Y *)a.y + row0 * rV + (int64_t)h * P + slice * COLS);
    const int oY = (int)(((16 * wave + r) * rV + 4 * q) * sizeof(Y));
    Rows<R> qr[NK];
    Frag pf[2][MP];
    float eg;
    auto load_q = [&]() {
      const auto b = buffer_of(cell, C::BYTES);
#pragma unroll
      for (int s = 0; s < NK; ++s) qr[s].get(b, lane, C::Q0 + (wave * NK + s) * C::ROW);
    };
    auto load_g = [&]() {
      eg = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buffer_of(cell, C::BYTES), 64 * wave + 4 * r, C::G0, 0));
    };
    auto load_p = [&]() {
      const auto b = buffer_of(cell, C::BYTES);
#pragma unroll
      for (int u = 0; u < MP; ++u) {
        pf[0][u] = operand(b, oF0, C::P0 + u * kSteps * kFrag);
        pf[1][u] = operand(b, oF1, C::P0 + u * kSteps * kFrag);
      }
    };
    if (c0 < c1) {
      load_q();
      __builtin_amdgcn_sched_barrier(0);
      load_g();
      __builtin_amdgcn_sched_barrier(0);
      load_p();
      __builtin_amdgcn_sched_barrier(0);
    }
    uint32_t far = 0;
    for (int c = c0; c < c1; ++c) {
      // A line a lane of the cell two chunks on, a part of it in every slice: then it is in the
      // L2 that the slices share when they load it (8192 tokens: 199 us, 187 with it).
      asm volatile("" ::"v"(far));
      if (eighth == 4 && c + 2 < c1)
        far = __builtin_amdgcn_raw_buffer_load_b32(buffer_of(cell + 2 * cells, C::BYTES), (slice * kWave + lane) * 128, 0, 0);
      const auto bY = rows_v(pY, sizeof(Y));  // rows past the end are not written
      rem -= Q;
      pY += Q * rV * sizeof(Y);
      if (c + 1 < c1) cell += cells;
      lds_barrier();  // S is there
      floatx4 O[CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) O[ct] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        Frag qf[IP];
        qr[s].cut(qf);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          Frag sf[MP];
#pragma unroll
          for (int u = 0; u < MP; ++u) sf[u].v = *reinterpret_cast<const s16x8 *>(sS[u] + (16 * ct + r) * SR + (32 * s + 8 * q) * 2);
#pragma unroll
          for (int u = MP - 1; u >= 0; --u)
#pragma unroll
            for (int w = IP - 1; w >= 0; --w)
              if (u + w < 3) O[ct] = mfma32(sf[u], qf[w], O[ct]);
        }
      }
      load_q();
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) O[ct] *= eg;
      load_g();
      lds_barrier();  // V - K S^T is there
      lds_barrier();  // U is there
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (s <= most) {
            Frag uf[MP];
#pragma unroll
            for (int u = 0; u < MP; ++u) uf[u].v = *reinterpret_cast<const s16x8 *>(sU[u] + 16 * ct * TR + oF + 64 * s);
#pragma unroll
            for (int u = MP - 1; u >= 0; --u)
#pragma unroll
              for (int w = MP - 1 - u; w >= 0; --w) O[ct] = mfma32(uf[u], pf[s][w], O[ct]);
          }
      }
      load_p();
      // This lane holds four neighbouring rows of the state's output for token 16 wave + r.
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const floatx4 o = O[ct];
        const int at = oY + 16 * ct * (int)sizeof(Y);
        if constexpr (sizeof(Y) == 2)
          __builtin_amdgcn_raw_buffer_store_b64(i32x2{(int)pack_bf16(o[0], o[1]), (int)pack_bf16(o[2], o[3])}, bY, at, 0, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b128(
              i32x4{__float_as_int(o[0]), __float_as_int(o[1]), __float_as_int(o[2]), __float_as_int(o[3])}, bY, at, 0, 0);
      }
    }
  }
}

// Cells of one pass: at most 256 MB of them, so that long prompts need no more than that.
constexpr size_t kCells = 256u << 20;

template <typename R, typename Y, int NK>
int places_of(const DeltaArgs &a) {
  const int all = items_of(a.p.tokens, a.p.n, Q);
  const size_t most = kCells / ((size_t)a.H * Cell<R, Y, NK>::BYTES);
  return most < 8 ? std::min(all, 8) : most < (size_t)all ? (int)most : all;
}

template <typename R, typename Y, int NK, int CT>
int launch(const DeltaArgs &a, hipStream_t st) {
  const int all = items_of(a.p.tokens, a.p.n, Q), most = places_of<R, Y, NK>(a);
  DeltaPlan p{};
  p.fH = make_fastdiv((uint32_t)a.H);
  p.ny = a.P / (16 * CT);
  p.fny = make_fastdiv((uint32_t)p.ny);
  p.cells = (char *)a.workspace;
  for (int64_t lo = 0; lo < all; lo += most) {
    p.lo = (int)lo, p.hi = (int)std::min<int64_t>(all, lo + most);
    const int64_t places = p.hi - p.lo, units = std::min<int64_t>(a.p.n, places) * a.H;
    const int64_t blocks = (units + kXcds - 1) / kXcds * kXcds * p.ny;
    if (places * a.H > kMostBlocks || 2 * blocks > kMostBlocks) return kTooLarge;
    p.units = (int)units;
    if (a.p.tokens) hipLaunchKernelGGL((cells_k<R, Y, NK>), dim3((uint32_t)(places * a.H)), dim3(kThreads), 0, st, a, p);
    hipLaunchKernelGGL((chain_k<R, Y, NK, CT>), dim3((uint32_t)blocks), dim3(2 * kThreads), 0, st, a, p);
  }
  return (int)hipGetLastError();
}

template <typename R, typename Y>
size_t workspace_n(const DeltaArgs &a) {
  if (!a.p.tokens) return 0;
  if (a.N <= 32) return (size_t)places_of<R, Y, 1>(a) * a.H * Cell<R, Y, 1>::BYTES;
  if (a.N == 64) return (size_t)places_of<R, Y, 2>(a) * a.H * Cell<R, Y, 2>::BYTES;
  return (size_t)places_of<R, Y, 4>(a) * a.H * Cell<R, Y, 4>::BYTES;
}

template <typename R, typename Y>
int launch_n(const DeltaArgs &a, hipStream_t st) {
  if (a.N <= 32) return launch<R, Y, 1, 1>(a, st);
  if (a.N == 64) return launch<R, Y, 2, 1>(a, st);
  return launch<R, Y, 4, 1>(a, st);
}

}  // namespace

size_t delta_workspace(const DeltaArgs &a) {
  if (!a.bf16) return workspace_n<float, float>(a);
  return a.y_bf16 ? workspace_n<bf16_t, bf16_t>(a) : workspace_n<bf16_t, float>(a);
}

int launch_delta(const DeltaArgs &a, hipStream_t st) {
  if (!a.bf16) return launch_n<float, float>(a, st);
  return a.y_bf16 ? launch_n<bf16_t, bf16_t>(a, st) : launch_n<bf16_t, float>(a, st);
}

}  // namespace rssm
