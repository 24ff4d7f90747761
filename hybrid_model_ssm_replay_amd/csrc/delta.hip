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
  static constexpr int KT0 = P0 + MP * kSteps * kFrag;   // [IP][2 NK tiles of k's columns][2 steps]
  static constexpr int K0 = KT0 + IP * 4 * NK * kFrag;   // [IP][4 token tiles][NK], float32 records only
  static constexpr int Q0 = K0 + (IP == 3 ? IP * 4 * NK * kFrag : 0);
  static constexpr int G0 = Q0 + (IP == 3 ? IP * 4 * NK * kFrag : 0);  // e^{g_t} [64], e^{g_C - g_t} [64]
  static constexpr int BYTES = G0 + 2 * Q * 4;
};

struct DeltaPlan {
  int lo, hi;      // the chunks of this pass: places start / 64 + sequence + chunk
  int ny;          // slices of a head's rows
  int units;       // sequences x heads of the pass at most
  FastDiv fH, fny;
  char *cells;     // [hi - lo][H] of Cell
};

// Rows of a record, eight neighbouring columns a lane, as an operand in IP pieces.
template <typename R>
struct Rows;
template <>
struct Rows<bf16_t> {
  static __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int at, Frag (&f)[1]) {
    f[0].v = __builtin_bit_cast(s16x8, buffer_load16(b, at, 0));
  }
};
template <>
struct Rows<float> {
  static __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int at, Frag (&f)[3]) {
    const uint4 v = buffer_load16(b, at, 0), w = buffer_load16(b, at, 16);
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

template <typename R, typename Y, int NK>
__global__ __launch_bounds__(kThreads) void cells_k(DeltaArgs a, DeltaPlan plan) {
  typedef Cell<R, Y, NK> C;
  constexpr int IP = C::IP, MP = C::MP;
  __shared__ __attribute__((aligned(16))) float sT[Q * kT], sA[Q * kT], sD[kWaves][16][20], sB[Q];
  __shared__ double sG[Q];
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
  double g = lane < rem ? log2((double)al) : 0.0;
  g = scan64(g < -4096.0 ? -4096.0 : g);
  const double gC = lane_value(g, kWave - 1);
  if (wave == 0) {
    sG[lane] = g;
    sB[lane] = lane < rem ? be : 0.f;
    float *const e = reinterpret_cast<float *>(cell + C::G0);
    e[lane] = __builtin_amdgcn_exp2f((float)g);
    e[Q + lane] = __builtin_amdgcn_exp2f((float)(gC - g));
  }
  __syncthreads();

  // P^T of this wave's rows of 16 tokens, G^T = (K K^T)^T of the rows 3 - wave.
  const int wg = 3 - wave;
  const int64_t rK = (int64_t)a.H * N;
  const size_t nK = (size_t)((rem - 1) * rK + N) * sizeof(R);
  const auto bK = buffer_of((const R *)a.k + row0 * rK + (int64_t)h * N, nK);
  const auto bQ = buffer_of((const R *)a.q + row0 * rK + (int64_t)h * N, nK);
  floatx4 aP[4], aG[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) aP[j] = aG[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int s = 0; s < NK; ++s) {
    const int c = 32 * s + 8 * q;
    auto at = [&](int tile) { return c < N ? (int)(((16 * tile + r) * rK + c) * sizeof(R)) : kNowhere; };
    Frag k[4][IP], qf[IP], kg[IP];
#pragma unroll
    for (int j = 0; j < 4; ++j) Rows<R>::load(bK, at(j), k[j]);
    Rows<R>::load(bQ, at(wave), qf);
    Rows<R>::load(bK, at(wg), kg);
#pragma unroll
    for (int u = IP - 1; u >= 0; --u)
#pragma unroll
      for (int v = IP - 1 - u; v >= 0; --v)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j <= wave) aP[j] = mfma32(k[j][u], qf[v], aP[j]);
          if (j <= wg) aG[j] = mfma32(k[j][u], kg[v], aG[j]);
        }
    // K^T of column tile 2 s + half: the products of K's rows with the unit vectors give
    // its values (one factor is 1, the others 0) with a column a lane.
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if ((2 * s + half) % kWaves != wave) continue;
      Frag one;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c0 = 8 * q + 2 * i - 16 * half;
        one.w[i] = (c0 == r ? 0x3F80u : 0u) | (c0 + 1 == r ? 0x3F800000u : 0u);
      }
#pragma unroll
      for (int u = 0; u < IP; ++u)
#pragma unroll
        for (int ts = 0; ts < 2; ++ts) {
          Frag f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const floatx4 x = mfma32(k[2 * ts + e][u], one, floatx4{0.f, 0.f, 0.f, 0.f});
            f.w[2 * e] = __builtin_amdgcn_perm(bits(x[1]), bits(x[0]), 0x07060302u);
            f.w[2 * e + 1] = __builtin_amdgcn_perm(bits(x[3]), bits(x[2]), 0x07060302u);
          }
          put(cell + C::KT0 + ((u * 2 * NK + 2 * s + half) * 2 + ts) * kFrag, lane, f);
        }
    }
    if constexpr (IP == 3) {
#pragma unroll
      for (int u = 0; u < IP; ++u) {
        put(cell + C::Q0 + ((u * 4 + wave) * NK + s) * kFrag, lane, qf[u]);
        put(cell + C::K0 + ((u * 4 + wg) * NK + s) * kFrag, lane, kg[u]);
      }
    }
  }
  {
    const double gt = sG[16 * wave + r], gg = sG[16 * wg + r];
    const float bt = sB[16 * wg + r];
    Frag f[2][MP];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float p[4], t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 16 * j + 4 * q + i;
        const double gj = sG[tok];
        p[i] = tok <= 16 * wave + r ? aP[j][i] * __builtin_amdgcn_exp2f((float)(gt - gj)) : 0.f;
        t[i] = tok < 16 * wg + r ? bt * (aG[j][i] * __builtin_amdgcn_exp2f((float)(gg - gj))) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[MP];
        pieces<MP>(p[2 * i], p[2 * i + 1], w);
#pragma unroll
        for (int u = 0; u < MP; ++u) f[j / 2][u].w[j % 2 * 2 + i] = w[u];
      }
      st4(sT + (16 * wg + r) * kT + 16 * j + 4 * q, make_float4(t[0], t[1], t[2], t[3]));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s <= wave / 2) {
#pragma unroll
        for (int u = 0; u < MP; ++u) put(cell + C::P0 + (u * kSteps + step_of(wave, s)) * kFrag, lane, f[s][u]);
      }
  }
  __syncthreads();

  // Column r of the inverse of the diagonal block `wave`, by substitution.
  float x[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    x[t] = t == r ? 1.f : 0.f;
    const float *const row = sT + (16 * wave + t) * kT + 16 * wave;
#pragma unroll
    for (int s4 = 0; s4 < t; s4 += 4) {
      const float4 tv = ld4(row + s4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (s4 + i < t) x[t] = fmaf(-f4get(tv, i), x[s4 + i], x[t]);
    }
  }
  floatx4 X[4];  // block column `wave` of the inverse: rows 16 i + 4 q + e, column r
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    X[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i == wave) X[i][e] = q == 0 ? x[e] : q == 1 ? x[4 + e] : q == 2 ? x[8 + e] : x[12 + e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sD[wave][4 * q + e][r] = q == 0 ? x[e] : q == 1 ? x[4 + e] : q == 2 ? x[8 + e] : x[12 + e];
  __syncthreads();
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    if (i <= wave) continue;
    floatx4 acc = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < i; ++m) {
      if (m < wave) continue;
      const float4 tv = ld4(sT + (16 * i + r) * kT + 16 * m + 4 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = mfma_16x16x4(f4get(tv, e), X[m][e], acc);
    }
    const float4 dv = ld4(&sD[i][r][4 * q]);
#pragma unroll
    for (int e = 0; e < 4; ++e) X[i] = mfma_16x16x4(-f4get(dv, e), acc[e], X[i]);
  }
  const float bj = sB[16 * wave + r];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sA[(16 * i + 4 * q + e) * kT + 16 * wave + r] = X[i][e] * bj;
  __syncthreads();
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (s <= wave / 2) {
      Frag f[3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 v = ld4(sA + (16 * wave + r) * kT + 32 * s + 16 * e + 4 * q);
        uint32_t w0[3], w1[3];
        pieces<3>(v.x, v.y, w0);
        pieces<3>(v.z, v.w, w1);
#pragma unroll
        for (int u = 0; u < 3; ++u) f[u].w[2 * e] = w0[u], f[u].w[2 * e + 1] = w1[u];
      }
#pragma unroll
      for (int u = 0; u < 3; ++u) put(cell + C::A0 + (u * kSteps + step_of(wave, s)) * kFrag, lane, f[u]);
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

template <typename R, typename Y, int NK, int CT>
__global__ __launch_bounds__(kThreads) void chain_k(DeltaArgs a, DeltaPlan plan) {
  typedef Cell<R, Y, NK> C;
  constexpr int IP = C::IP, MP = C::MP, COLS = 16 * CT;
  constexpr int MT = NK == 4 ? 2 : 1;            // tiles of the state's columns that a wave has
  constexpr int SR = 64 * NK + 16, TR = 2 * Q + 16;  // bytes of a row of S, and of 64 tokens, in LDS
  __shared__ __attribute__((aligned(16))) char sS[3][COLS * SR], sR[3][COLS * TR], sW[3][COLS * TR], sU[MP][COLS * TR];
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
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

  // The state, transposed: tile m of this wave, columns 16 (wave + 4 m) + 4 q + i of k, row r of the slice's tile.
  floatx4 S[MT][CT];
  auto there = [&](int m) { return wave + 4 * m < 2 * NK; };
  const size_t tile0 = ((size_t)row * a.H + h) * P * N + (size_t)(slice * COLS + r) * N + 16 * wave + 4 * q;
  const bool known = a.initial && (!a.p.resume || a.p.resume[seq]);
  const float *const from = c0 ? a.state : known ? a.initial : nullptr;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      S[m][ct] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (from && 16 * (wave + 4 * m) < N) {
        const float4 v = ld4(from + tile0 + (size_t)16 * ct * N + 64 * m);
        S[m][ct] = floatx4{v.x, v.y, v.z, v.w};
      }
    }
  auto hand_state = [&]() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        if (there(m)) hand<3>(sS[0] + (16 * ct + r) * SR + (16 * (wave + 4 * m) + 4 * q) * 2, COLS * SR, S[m][ct]);
  };
  hand_state();

  const int64_t rK = (int64_t)a.H * N, rV = (int64_t)a.H * P;
  const char *cell = plan.cells + ((int64_t)(base + c0 - plan.lo) * a.H + h) * C::BYTES;
  const int64_t cells = (int64_t)a.H * C::BYTES;
  // Place of the wave's tokens 4 q + i in a row of 64: step wave / 2, half wave % 2.
  const int oT = r * TR + (32 * (wave / 2) + 8 * q + 4 * (wave % 2)) * 2;

  for (int c = c0; c < c1; ++c, cell += cells) {
    const int rem = min(Q, len - c * Q);
    const int64_t row0 = (int64_t)begin + c * Q;
    Frag kf[NK][IP], qf[NK][IP];
    if constexpr (IP == 1) {
      const size_t nK = (size_t)((rem - 1) * rK + N) * sizeof(R);
      const auto bK = buffer_of((const R *)a.k + row0 * rK + (int64_t)h * N, nK);
      const auto bQ = buffer_of((const R *)a.q + row0 * rK + (int64_t)h * N, nK);
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        const int col = 32 * s + 8 * q, at = col < N ? (int)(((16 * wave + r) * rK + col) * sizeof(R)) : kNowhere;
        Rows<R>::load(bK, at, kf[s]);
        Rows<R>::load(bQ, at, qf[s]);
      }
    } else {
#pragma unroll
      for (int s = 0; s < NK; ++s)
#pragma unroll
        for (int u = 0; u < IP; ++u) {
          kf[s][u] = get(cell + C::K0 + ((u * 4 + wave) * NK + s) * kFrag, lane);
          qf[s][u] = get(cell + C::Q0 + ((u * 4 + wave) * NK + s) * kFrag, lane);
        }
    }
    float v[CT][4];
    {
      const auto bV = buffer_of((const R *)a.v + row0 * rV + (int64_t)h * P + slice * COLS,
                                (size_t)((rem - 1) * rV + COLS) * sizeof(R));
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = (int)(((16 * wave + 4 * q + i) * rV + 16 * ct + r) * sizeof(R));
          if constexpr (IP == 1)
            v[ct][i] = lower((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(bV, at, 0, 0));
          else
            v[ct][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(bV, at, 0, 0));
        }
    }
    const float *const e = reinterpret_cast<const float *>(cell + C::G0);
    const float4 eg4 = ld4(e + 16 * wave + 4 * q), left4 = ld4(e + Q + 16 * wave + 4 * q);
    const float eg = e[16 * wave + r], whole = e[Q - 1];

    lds_barrier();  // S is there
    floatx4 X[CT], O[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) X[ct] = O[ct] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < NK; ++s)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        Frag sf[3];
#pragma unroll
        for (int u = 0; u < 3; ++u) sf[u].v = *reinterpret_cast<const s16x8 *>(sS[u] + (16 * ct + r) * SR + (32 * s + 8 * q) * 2);
#pragma unroll
        for (int u = 2; u >= 0; --u)
#pragma unroll
          for (int w = IP - 1; w >= 0; --w)
            if (u + w < 3) {
              X[ct] = mfma32(kf[s][w], sf[u], X[ct]);
              if (u < MP) O[ct] = mfma32(sf[u], qf[s][w], O[ct]);
            }
      }
    const float egv[4] = {eg4.x, eg4.y, eg4.z, eg4.w}, lev[4] = {left4.x, left4.y, left4.z, left4.w};
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      floatx4 d;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = fmaf(-egv[i], X[ct][i], v[ct][i]);
      hand<3>(sR[0] + 16 * ct * TR + oT, COLS * TR, d);
      O[ct] *= eg;
    }
    Frag af[2][3], pf[2][MP];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s <= wave / 2) {
#pragma unroll
        for (int u = 0; u < 3; ++u) af[s][u] = get(cell + C::A0 + (u * kSteps + step_of(wave, s)) * kFrag, lane);
#pragma unroll
        for (int u = 0; u < MP; ++u) pf[s][u] = get(cell + C::P0 + (u * kSteps + step_of(wave, s)) * kFrag, lane);
      }
    Frag kt[MT][2][IP];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (there(m)) {
#pragma unroll
        for (int ts = 0; ts < 2; ++ts)
#pragma unroll
          for (int u = 0; u < IP; ++u) kt[m][ts][u] = get(cell + C::KT0 + ((u * 2 * NK + wave + 4 * m) * 2 + ts) * kFrag, lane);
      }
    lds_barrier();  // V - K S^T is there
    const int oF = r * TR + 16 * q;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      floatx4 U = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= wave / 2) {
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
    lds_barrier();  // U is there
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
      for (int m = 0; m < MT; ++m) S[m][ct] *= whole;
#pragma unroll
      for (int ts = 0; ts < 2; ++ts) {
        Frag wf[3];
#pragma unroll
        for (int u = 0; u < 3; ++u) wf[u].v = *reinterpret_cast<const s16x8 *>(sW[u] + 16 * ct * TR + oF + 64 * ts);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (there(m)) {
#pragma unroll
            for (int u = 2; u >= 0; --u)
#pragma unroll
              for (int w = IP - 1; w >= 0; --w)
                if (u + w < 3) S[m][ct] = mfma32(kt[m][ts][w], wf[u], S[m][ct]);
          }
      }
    }
    hand_state();
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= wave / 2) {
          Frag uf[MP];
#pragma unroll
          for (int u = 0; u < MP; ++u) uf[u].v = *reinterpret_cast<const s16x8 *>(sU[u] + 16 * ct * TR + oF + 64 * s);
#pragma unroll
          for (int u = MP - 1; u >= 0; --u)
#pragma unroll
            for (int w = MP - 1 - u; w >= 0; --w) O[ct] = mfma32(uf[u], pf[s][w], O[ct]);
        }
      // This lane holds four neighbouring rows of the state's output for token 16 wave + r.
      const auto bY = buffer_of((Y *)a.y + row0 * rV + (int64_t)h * P + slice * COLS,
                                (size_t)((rem - 1) * rV + COLS) * sizeof(Y));  // rows past the end are not written
      const int at = (int)(((16 * wave + r) * rV + 16 * ct + 4 * q) * sizeof(Y));
      const floatx4 o = O[ct];
      if constexpr (sizeof(Y) == 2)
        __builtin_amdgcn_raw_buffer_store_b64(i32x2{(int)pack_bf16(o[0], o[1]), (int)pack_bf16(o[2], o[3])}, bY, at, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b128(
            i32x4{__float_as_int(o[0]), __float_as_int(o[1]), __float_as_int(o[2]), __float_as_int(o[3])}, bY, at, 0, 0);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
      if (16 * (wave + 4 * m) < N)
        st4(a.state + tile0 + (size_t)16 * ct * N + 64 * m, make_float4(S[m][ct][0], S[m][ct][1], S[m][ct][2], S[m][ct][3]));
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
    if (places * a.H > kMostBlocks || blocks > kMostBlocks) return kTooLarge;
    p.units = (int)units;
    if (a.p.tokens) hipLaunchKernelGGL((cells_k<R, Y, NK>), dim3((uint32_t)(places * a.H)), dim3(kThreads), 0, st, a, p);
    hipLaunchKernelGGL((chain_k<R, Y, NK, CT>), dim3((uint32_t)blocks), dim3(kThreads), 0, st, a, p);
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
