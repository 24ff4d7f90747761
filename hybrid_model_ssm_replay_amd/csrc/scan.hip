// Mamba-2 recurrence over packed prompts: S <- exp(dt A) S + dt x B^T, y = S C + D x.
//
// Chunks of Q tokens (64; 32 with float32 records) turn it into matrix products.
// With a_t the sum of dt A over the chunk's tokens up to t and S0 the state before it:
//   G = C B^T,   M[t][j] = G[t][j] e^{a_t - a_j} dt_j  (j <= t, else 0),
//   y_t = e^{a_t} S0 C_t + sum_j M[t][j] x_j + D x_t,
//   S1  = e^{a_Q} S0 + sum_j (e^{a_Q - a_j} dt_j x_j) B_j^T.
//
// Decays are never differences of long sums: a chunk is cut into blocks of 16
// tokens, and e^{a_t - a_j} is e^{(sum inside t's block up to t)} times the
// whole blocks' decays between times e^{(sum inside j's block after j)}, three
// factors of at most 1; only inside one block is it the exponential of a
// difference, of running sums held as two float32 (the float64 sum and what
// rounding left of it), so that the difference is good to float32 itself.
//
// A workgroup takes up to 128 columns of x (heads of one group, which share
// B, C and G) of one sequence, and walks its chunks; a wave owns 32 columns of
// one head with their whole state in registers (S^T as accumulators of
// v_mfma_f32_16x16x32_bf16: lane l holds rows n = 4 (l / 16) + i of column p =
// l % 16).  That layout is at once the operand layout of S C^T with the sum
// over n taken in the order n = 32 k + 16 (i / 4) + 4 (l / 16) + i % 4, so the
// state never leaves its wave, and G^T as accumulators is in the same way the
// operand M of M x.  B^T and x^T operands come from row-major LDS tiles by the
// transposing LDS read (lane l gets column l % 16 of rows 4 (l / 16) .. + 3).
//
// Precision.  bf16 records enter the products as they are, float32 records as
// three bf16 pieces (their sum is the value; products of pieces below 2^-24 are
// dropped).  The weighted inputs of the state update are always three pieces:
// the state stays float32.  M and S in the output products are three pieces for
// float32 outputs, and one bf16 for bf16 outputs: 2^-9 of each term on average
// next to the output's own 2^-9.
#include "ops.h"

namespace rssm {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kCols = 128;        // x columns of a workgroup
constexpr int kXs = kCols + 16;   // row strides of the LDS tiles in elements: no bank twice in a read
constexpr float kLog2e = 1.4426950408889634f;

union Frag {  // eight bf16 of one lane: an operand of the 16x16x32 product
  s16x8 v;
  s16x4 h[2];
  uint32_t w[4];
};

__device__ __forceinline__ floatx4 mfma32(const Frag &a, const Frag &b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
}

__device__ __forceinline__ s16x4 read_tr(const bf16_t *p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p); }

// The upper halves of two words: b's in the upper half.
__device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }
__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ float cut(float v) { return __uint_as_float(bits(v) & 0xFFFF0000u); }

// Two values as MP words of bf16 pairs: one piece rounds to nearest, three
// pieces cut (8 bits each: together the 24 bits of the value).
template <int MP>
__device__ __forceinline__ void pieces(float a, float b, uint32_t (&w)[MP]) {
  if constexpr (MP == 1) {
    w[0] = pack_bf16(a, b);
  } else {
    w[0] = upper(bits(a), bits(b));
    a -= cut(a), b -= cut(b);
    w[1] = upper(bits(a), bits(b));
    a -= cut(a), b -= cut(b);
    w[2] = upper(bits(a), bits(b));
  }
}

template <int CTRL>
__device__ __forceinline__ float row_shift(float v) {  // within 16 lanes, zeros shifted in
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double row_shift(double v) {
  const int2 w = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_update_dpp(0, w.x, CTRL, 0xF, 0xF, true),
                                              __builtin_amdgcn_update_dpp(0, w.y, CTRL, 0xF, 0xF, true)));
}

// Four entries of M of one lane: rounded to bf16, or float32 to be cut in pieces when used.
template <int MP>
struct MTile {
  typedef float4 type;
};
template <>
struct MTile<1> {
  typedef uint2 type;
};

struct ScanPlan {
  int seg;        // tokens of a segment (a multiple of 64), or 0: sequences are not split
  int items;      // segments of all sequences
  int hw, wph;    // heads of a workgroup, waves of a head
  int nb;         // workgroups of a group
  int units;      // items x groups: the workgroups of a unit share B and C
  FastDiv fnb, fG;
  float *state;   // [items][H][P N]: a segment's own state, then its start
  float *decay;   // [items][H]
};

// The parts of one launch.  kAll: sequences in one piece.  kOwn: every segment but
// the last of a sequence leaves the state it would build from zero, and its
// decay.  kFrom: segments start from the states that combine_k left.
enum { kAll = 0, kOwn = 1, kFrom = 2 };

template <typename R, typename Y, int NK, int MODE>
__global__ __launch_bounds__(kThreads, sizeof(R) == 4 && NK == 4 ? 1 : 2) void scan_k(ScanArgs a, ScanPlan plan) {
  constexpr int IP = sizeof(R) == 4 ? 3 : 1;             // pieces of an input
  constexpr int MP = sizeof(Y) == 4 ? 3 : 1;             // pieces of M and S
  constexpr int QB = IP == 3 ? 2 : 4, Q = 16 * QB;       // blocks and tokens of a chunk
  constexpr int KB = QB / 2;                             // 32-token steps
  constexpr int NT = 2 * NK, Ns = 32 * NK + 8;
  constexpr int V = 16 / (int)sizeof(R);                 // elements of a 16-byte load
  constexpr int NV = 32 * NK / V, XV = kCols / V;        // loads of a row
  constexpr int LB = Q * NV / kThreads > 0 ? Q * NV / kThreads : 1, LX = Q * XV / kThreads;
  constexpr bool OUT = MODE != kOwn;
  constexpr int TILES = QB * (QB + 1) / 2;
  __shared__ __attribute__((aligned(16))) bf16_t sB[IP][Q][Ns];
  __shared__ __attribute__((aligned(16))) bf16_t sC[OUT ? IP : 1][OUT ? Q : 1][Ns];
  __shared__ __attribute__((aligned(16))) bf16_t sX[IP][Q][kXs];
  typedef typename MTile<MP>::type mtile;
  __shared__ mtile sM[OUT ? kWaves : 1][OUT ? TILES : 1][kWave];            // per head of the workgroup
  __shared__ __attribute__((aligned(16))) float sc[kWaves][5][kWave];     // per head and token, see below

  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int r = lane % 16, q = lane / 16;
  // Unit u on XCD u % 8 (workgroup i runs on XCD i % 8): a unit's workgroups share an
  // L2, and items without work, which come at the end of each sequence, spread over the XCDs.
  const int k8 = blockIdx.x / kXcds, u8 = fdiv(k8, plan.fnb);
  const int unit = u8 * kXcds + blockIdx.x % kXcds, blk = k8 - u8 * plan.nb;
  if (unit >= plan.units) return;
  const int item = fdiv(unit, plan.fG), g = unit - item * a.G;
  const int Hg = a.H / a.G, P = a.P, N = a.N;

  int seq, begin, len, t_first = 0, t_end;
  if constexpr (MODE == kAll) {
    seq = item;
    begin = clamp_start(a.p, seq);
    len = max(0, clamp_start(a.p, seq + 1) - begin);
    t_end = len;
  } else {
    const Item it = find_item(a.p, item, plan.seg);
    seq = it.seq, begin = it.begin, len = it.len;
    t_first = it.index * plan.seg;
    if (it.index < 0 || (it.index > 0 && t_first >= len)) return;
    t_end = min(len, t_first + plan.seg);
    if (MODE == kOwn && t_end == len) return;  // nothing starts from the last segment's state
  }
  const int row = batch_row(a.p, seq, g == 0 && blk == 0 && tid == 0 && MODE != kOwn && t_first == 0);
  if (row < 0) return;

  const int hi = wave / plan.wph;
  const int h0 = g * Hg + blk * plan.hw;                       // the workgroup's first head
  const int nh = min(plan.hw, Hg - blk * plan.hw);
  const bool active = hi < nh;
  const int h = h0 + (active ? hi : 0);
  const int pt0 = (wave % plan.wph) * 2;
  const int np = active ? min(2, P / 16 - pt0) : 0;            // this wave's 16-column tiles
  const int xcol = (active ? hi : 0) * P + (np > 0 ? 16 * pt0 : 0);
  const int ncols = nh * P;
  const float Al = a.A[h] * kLog2e;

  // The state: S^T tile nt of column tile pt.
  floatx4 S[NT][2];
  const size_t tile0 = (size_t)h * P * N + (size_t)(16 * pt0 + r) * N + 4 * q;
  const size_t states = (size_t)a.H * P * N;
  bool split = false;
  if constexpr (MODE == kFrom) split = len > plan.seg;
  const bool known = a.initial && (!a.p.resume || a.p.resume[seq]);
  const float *from = nullptr;
  if constexpr (MODE != kOwn) from = split ? plan.state + item * states : known ? a.initial + row * states : nullptr;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) {
      S[nt][pt] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (from && pt < np && 16 * nt < N) {
        const float4 v = ld4(from + tile0 + (size_t)16 * pt * N + 16 * nt);
        S[nt][pt] = floatx4{v.x, v.y, v.z, v.w};
      }
    }

  // Global to registers, and registers to LDS.  Rows are uniform, a thread adds
  // its place in them; whole chunks of full width need no checks.
  uint4 pB[LB], pC[OUT ? LB : 1], pX[LX];
  const size_t rB = (size_t)a.G * N, rX = (size_t)a.H * P;
  const R *Bg = (const R *)a.Bm + (size_t)begin * rB + (size_t)g * N;
  const R *Cg = (const R *)a.Cm + (size_t)begin * rB + (size_t)g * N;
  const R *Xg = (const R *)a.x + (size_t)begin * rX + (size_t)h0 * P;
  constexpr int RB = kThreads / NV, RX = kThreads / XV;  // rows of one load
  const int tB = tid / NV, cB = tid % NV * V, tX = tid / XV, cX = tid % XV * V;
  const uint32_t oB = (uint32_t)(tB * rB + cB) * sizeof(R), oX = (uint32_t)(tX * rX + cX) * sizeof(R);
  const bool full_width = N == 32 * NK && ncols == kCols;
  auto load16 = [](const void *base, uint32_t off) {
    return *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(base) + off);
  };
  auto fetch = [&](int t0) {
    const R *Bt = Bg + t0 * rB, *Ct = Cg + t0 * rB, *Xt = Xg + t0 * rX;
    if (full_width && t0 + Q <= t_end) {
#pragma unroll
      for (int i = 0; i < LB; ++i) {
        pB[i] = load16(Bt + i * RB * rB, oB);
        if constexpr (OUT) pC[i] = load16(Ct + i * RB * rB, oB);
      }
#pragma unroll
      for (int i = 0; i < LX; ++i) pX[i] = load16(Xt + i * RX * rX, oX);
    } else {
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < LB; ++i) {
        const bool in = t0 + i * RB + tB < t_end && cB < N;
        pB[i] = in ? load16(Bt + i * RB * rB, oB) : zero;
        if constexpr (OUT) pC[i] = in ? load16(Ct + i * RB * rB, oB) : zero;
      }
#pragma unroll
      for (int i = 0; i < LX; ++i)
        pX[i] = t0 + i * RX + tX < t_end && cX < ncols ? load16(Xt + i * RX * rX, oX) : zero;
    }
  };
  auto put = [&](uint4 v, bf16_t *at, int piece) {  // at: the first piece's place; piece: elements between pieces
    if constexpr (IP == 1) {
      *reinterpret_cast<uint4 *>(at) = v;
    } else {
      uint32_t lo[3], hi3[3];
      pieces<3>(__uint_as_float(v.x), __uint_as_float(v.y), lo);
      pieces<3>(__uint_as_float(v.z), __uint_as_float(v.w), hi3);
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2 *>(at + k * piece) = make_uint2(lo[k], hi3[k]);
    }
  };
  auto spill = [&]() {
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      put(pB[i], &sB[0][i * RB + tB][cB], Q * Ns);
      if constexpr (OUT) put(pC[i], &sC[0][i * RB + tB][cB], Q * Ns);
    }
#pragma unroll
    for (int i = 0; i < LX; ++i) put(pX[i], &sX[0][i * RX + tX][cX], Q * kXs);
  };
  const float *dtg = a.dt + (size_t)begin * a.H + h;
  auto fetch_dt = [&](int t0) {
    const int t = t0 + lane;
    return lane < Q && t < t_end && active ? dtg[(size_t)t * a.H] : 0.f;
  };

  // Operand of 32 columns of a row-major tile: row r of block b, columns in the order of an accumulator pair.
  auto rows = [&](const bf16_t *tile, int stride, int b, int k) {
    Frag f;
    const bf16_t *p = tile + (16 * b + r) * stride + 32 * k + 4 * q;
    f.h[0] = *reinterpret_cast<const s16x4 *>(p);
    f.h[1] = *reinterpret_cast<const s16x4 *>(p + 16);
    return f;
  };
  // Operand of 32 tokens: column c0 + r, tokens in the same order.
  auto cols = [&](const bf16_t *tile, int stride, int c0, int k) {
    Frag f;
    const bf16_t *p = tile + (32 * k + 4 * q + r / 4) * stride + c0 + 4 * (r % 4);
    f.h[0] = read_tr(p);
    f.h[1] = read_tr(p + 16 * stride);
    return f;
  };

  float decay = 1.f;
  fetch(t_first);
  float dtv = fetch_dt(t_first);
  for (int t0 = t_first; t0 < t_end; t0 += Q) {
    lds_barrier();  // every wave is done with the last chunk's tiles
    spill();
    const float dt = dtv;
    if (t0 + Q < t_end) {
      fetch(t0 + Q);
      dtv = fetch_dt(t0 + Q);
    }
    // Decays: lane = token.
    double sum = dt;
    float suf = dt;
    sum += row_shift<0x111>(sum), suf += row_shift<0x101>(suf);
    sum += row_shift<0x112>(sum), suf += row_shift<0x102>(suf);
    sum += row_shift<0x114>(sum), suf += row_shift<0x104>(suf);
    sum += row_shift<0x118>(sum), suf += row_shift<0x108>(suf);
    suf = row_shift<0x101>(suf);  // the tokens after this one
    const float pre = (float)sum;
    const float epre = __builtin_amdgcn_exp2f(Al * pre);
    if (active && pt0 == 0) {
      sc[hi][0][lane] = pre;
      sc[hi][1][lane] = epre;
      sc[hi][2][lane] = __builtin_amdgcn_exp2f(Al * suf) * dt;
      if constexpr (OUT) {
        sc[hi][3][lane] = dt;
        sc[hi][4][lane] = (float)(sum - (double)pre);
      }
    }
    float E[QB];  // the blocks' decays
#pragma unroll
    for (int b = 0; b < QB; ++b) E[b] = __uint_as_float(__builtin_amdgcn_readlane(bits(epre), 16 * b + 15));
    lds_barrier();

    floatx4 Yt[QB][2];
    if constexpr (OUT) {
      // G^T tiles (rows j, columns t), and M^T from them for each of the workgroup's heads.
      for (int i = wave; i < TILES; i += kWaves) {
        int tb = 0;
        while ((tb + 1) * (tb + 2) / 2 <= i) ++tb;
        const int jb = i - tb * (tb + 1) / 2;
        floatx4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          Frag bf[IP], cf[IP];
#pragma unroll
          for (int u = 0; u < IP; ++u) bf[u] = rows(&sB[u][0][0], Ns, jb, k), cf[u] = rows(&sC[u][0][0], Ns, tb, k);
#pragma unroll
          for (int u = IP - 1; u >= 0; --u)
#pragma unroll
            for (int v = IP - 1 - u; v >= 0; --v) acc = mfma32(bf[u], cf[v], acc);
        }
        for (int hd = 0; hd < nh; ++hd) {
          const float ah = a.A[h0 + hd] * kLog2e;
          float m[4];
          if (jb < tb) {
            float f = sc[hd][1][16 * tb + r];  // t's block up to t, and the whole blocks between
            for (int b = jb + 1; b < tb; ++b) f *= sc[hd][1][16 * b + 15];
            const float4 w = *reinterpret_cast<const float4 *>(&sc[hd][2][16 * jb + 4 * q]);
            m[0] = acc[0] * (f * w.x), m[1] = acc[1] * (f * w.y), m[2] = acc[2] * (f * w.z), m[3] = acc[3] * (f * w.w);
          } else {
            const float p1 = sc[hd][0][16 * tb + r], l1 = sc[hd][4][16 * tb + r];
            const float4 p4 = *reinterpret_cast<const float4 *>(&sc[hd][0][16 * jb + 4 * q]);
            const float4 d4 = *reinterpret_cast<const float4 *>(&sc[hd][3][16 * jb + 4 * q]);
            const float4 l4 = *reinterpret_cast<const float4 *>(&sc[hd][4][16 * jb + 4 * q]);
            const float pj[4] = {p4.x, p4.y, p4.z, p4.w}, dj[4] = {d4.x, d4.y, d4.z, d4.w};
            const float lj[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v = acc[e] * (__builtin_amdgcn_exp2f(ah * ((p1 - pj[e]) + (l1 - lj[e]))) * dj[e]);
              m[e] = 4 * q + e <= r ? v : 0.f;
            }
          }
          if constexpr (MP == 1)
            sM[hd][i][lane] = make_uint2(pack_bf16(m[0], m[1]), pack_bf16(m[2], m[3]));
          else
            sM[hd][i][lane] = make_float4(m[0], m[1], m[2], m[3]);
        }
      }
      // S0 C^T, transposed: rows p, columns t.
#pragma unroll
      for (int tb = 0; tb < QB; ++tb)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) Yt[tb][pt] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (np > 0) {
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          Frag sp[2][MP];
#pragma unroll
          for (int pt = 0; pt < 2; ++pt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const floatx4 &s = S[2 * k + i / 2][pt];
              uint32_t w[MP];
              pieces<MP>(s[i % 2 * 2], s[i % 2 * 2 + 1], w);
#pragma unroll
              for (int u = 0; u < MP; ++u) sp[pt][u].w[i] = w[u];
            }
#pragma unroll
          for (int tb = 0; tb < QB; ++tb) {
            Frag cf[IP];
#pragma unroll
            for (int u = 0; u < IP; ++u) cf[u] = rows(&sC[u][0][0], Ns, tb, k);
#pragma unroll
            for (int pt = 0; pt < 2; ++pt)
#pragma unroll
              for (int u = MP - 1; u >= 0; --u)
#pragma unroll
                for (int v = 0; v < IP; ++v)
                  if (u + v < 3) Yt[tb][pt] = mfma32(sp[pt][u], cf[v], Yt[tb][pt]);
          }
        }
        float f = 1.f;
#pragma unroll
        for (int tb = 0; tb < QB; ++tb) {
          const float e = f * sc[hi][1][16 * tb + r];
          Yt[tb][0] *= e;
          Yt[tb][1] *= e;
          f *= E[tb];
        }
      }
      lds_barrier();  // M is complete
    }

    if (np > 0) {
      Frag xf[KB][2][IP];
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
#pragma unroll
          for (int u = 0; u < IP; ++u) xf[k][pt][u] = cols(&sX[u][0][0], kXs, xcol + (pt < np ? 16 * pt : 0), k);
      if constexpr (OUT) {
#pragma unroll
        for (int tb = 0; tb < QB; ++tb) {
#pragma unroll
          for (int k = 0; k <= tb / 2; ++k) {
            Frag mf[MP];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int jb = 2 * k + half;
              if (jb > tb) {
#pragma unroll
                for (int u = 0; u < MP; ++u) mf[u].h[half] = s16x4{0, 0, 0, 0};
                continue;
              }
              const mtile m = sM[hi][tb * (tb + 1) / 2 + jb][lane];
              if constexpr (MP == 1) {
                mf[0].w[2 * half] = m.x, mf[0].w[2 * half + 1] = m.y;
              } else {
                uint32_t w0[MP], w1[MP];
                pieces<MP>(m.x, m.y, w0);
                pieces<MP>(m.z, m.w, w1);
#pragma unroll
                for (int u = 0; u < MP; ++u) mf[u].w[2 * half] = w0[u], mf[u].w[2 * half + 1] = w1[u];
              }
            }
#pragma unroll
            for (int pt = 0; pt < 2; ++pt)
#pragma unroll
              for (int u = MP - 1; u >= 0; --u)
#pragma unroll
                for (int v = 0; v < IP; ++v)
                  if (u + v < 3) Yt[tb][pt] = mfma32(xf[k][pt][v], mf[u], Yt[tb][pt]);
          }
        }
        // y: this lane holds four neighbouring channels of token 16 tb + r.
        const float D = a.D[h];
#pragma unroll
        for (int tb = 0; tb < QB; ++tb) {
          const int t = t0 + 16 * tb + r;
          if (t < t_end) {
#pragma unroll
            for (int pt = 0; pt < 2; ++pt)
              if (pt < np) {
                float o[4];
                float x4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = IP - 1; u >= 0; --u) {
                  float v[4];
                  load_vec<bf16_t, 4>(&sX[u][16 * tb + r][xcol + 16 * pt + 4 * q], v);
#pragma unroll
                  for (int i = 0; i < 4; ++i) x4[i] += v[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = fmaf(D, x4[i], Yt[tb][pt][i]);
                store_vec<Y, 4>((Y *)a.y + ((size_t)(begin + t) * a.H + h) * P + 16 * (pt0 + pt) + 4 * q, o);
              }
          }
        }
      }
      // The state after the chunk.
      float all = 1.f;
#pragma unroll
      for (int b = 0; b < QB; ++b) all *= E[b];
      decay *= all;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) S[nt][pt] *= all;
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        float f1 = 1.f;
#pragma unroll
        for (int b = 0; b < QB; ++b)
          if (b > 2 * k + 1) f1 *= E[b];
        const float f0 = f1 * E[2 * k + 1];
        const float4 w0 = *reinterpret_cast<const float4 *>(&sc[hi][2][32 * k + 4 * q]);
        const float4 w1 = *reinterpret_cast<const float4 *>(&sc[hi][2][32 * k + 16 + 4 * q]);
        const float w[8] = {f0 * w0.x, f0 * w0.y, f0 * w0.z, f0 * w0.w, f1 * w1.x, f1 * w1.y, f1 * w1.z, f1 * w1.w};
        Frag xw[2][3];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float lo = 0.f, hi2 = 0.f;
#pragma unroll
            for (int u = IP - 1; u >= 0; --u) {
              lo += __uint_as_float(xf[k][pt][u].w[i] << 16);
              hi2 += __uint_as_float(xf[k][pt][u].w[i] & 0xFFFF0000u);
            }
            uint32_t pw[3];
            pieces<3>(lo * w[2 * i], hi2 * w[2 * i + 1], pw);
#pragma unroll
            for (int u = 0; u < 3; ++u) xw[pt][u].w[i] = pw[u];
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Frag bf[IP];
#pragma unroll
          for (int u = 0; u < IP; ++u) bf[u] = cols(&sB[u][0][0], Ns, 16 * nt, k);
#pragma unroll
          for (int pt = 0; pt < 2; ++pt)
#pragma unroll
            for (int u = 2; u >= 0; --u)
#pragma unroll
              for (int v = 0; v < IP; ++v)
                if (u + v < 3) S[nt][pt] = mfma32(bf[v], xw[pt][u], S[nt][pt]);
        }
      }
    }
  }

  float *to = MODE == kOwn ? plan.state + item * states : t_end == len ? a.state + row * states : nullptr;
  if (to) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
        if (pt < np && 16 * nt < N)
          st4(to + tile0 + (size_t)16 * pt * N + 16 * nt, make_float4(S[nt][pt][0], S[nt][pt][1], S[nt][pt][2], S[nt][pt][3]));
  }
  if (MODE == kOwn && np > 0 && wave % plan.wph == 0 && lane == 0) plan.decay[(size_t)item * a.H + h] = decay;
}

// Where each segment of a split sequence starts: the segment before it decays
// that one's start and adds its own state.  One thread, four state elements.
__global__ __launch_bounds__(kThreads) void combine_k(ScanArgs a, ScanPlan plan, FastDiv blocks) {
  const int seq = fdiv(blockIdx.x, blocks);
  const int begin = clamp_start(a.p, seq), len = clamp_start(a.p, seq + 1) - begin;
  const int row = batch_row(a.p, seq, false);
  const int e = ((blockIdx.x - seq * (int)blocks.d) * kThreads + threadIdx.x) * 4;
  const int PN = a.P * a.N;
  if (len <= plan.seg || row < 0 || e >= a.H * PN) return;
  const int item0 = begin / plan.seg + seq, n = (len + plan.seg - 1) / plan.seg, h = e / PN;
  const size_t states = (size_t)a.H * PN;
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.initial && (!a.p.resume || a.p.resume[seq])) run = ld4(a.initial + row * states + e);
  for (int i = 0; i < n; ++i) {
    float *at = plan.state + (item0 + i) * states + e;
    const float d = i + 1 < n ? plan.decay[(size_t)(item0 + i) * a.H + h] : 0.f;
    const float4 own = i + 1 < n ? ld4(at) : make_float4(0.f, 0.f, 0.f, 0.f);
    st4(at, run);
    run = make_float4(fmaf(run.x, d, own.x), fmaf(run.y, d, own.y), fmaf(run.z, d, own.z), fmaf(run.w, d, own.w));
  }
}

ScanPlan make_plan(const ScanArgs &a) {
  ScanPlan p{};
  p.wph = (a.P + 31) / 32;
  p.hw = kWaves / p.wph;
  const int Hg = a.H / a.G;
  p.nb = (Hg + p.hw - 1) / p.hw;
  const int per = a.G * p.nb;
  p.fnb = make_fastdiv((uint32_t)p.nb);
  p.fG = make_fastdiv((uint32_t)a.G);
  // Split sequences along the length when there are too few to fill the card.
  const int want = (512 + per - 1) / per;
  const int seg = ((a.p.tokens + want - 1) / want + 63) / 64 * 64;
  p.seg = a.p.n >= want || seg >= a.p.tokens ? 0 : seg < 256 ? 256 : seg;
  if (p.seg >= a.p.tokens) p.seg = 0;
  p.items = p.seg ? items_of(a.p.tokens, a.p.n, p.seg) : a.p.n;
  p.units = p.items * a.G;
  return p;
}

size_t decay_bytes(const ScanArgs &a, const ScanPlan &p) { return ((size_t)p.items * a.H * 4 + 255) / 256 * 256; }

template <typename R, typename Y, int NK>
int launch(const ScanArgs &a, const ScanPlan &p, hipStream_t st) {
  const int64_t blocks = ((int64_t)p.items * a.G + kXcds - 1) / kXcds * kXcds * p.nb;
  const int per_seq = (a.H * a.P * a.N / 4 + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL || (int64_t)a.p.n * per_seq > 0x7fffffffLL) return (int)hipErrorInvalidValue;
  const dim3 grid((uint32_t)blocks), block(kThreads);
  if (!p.seg) {
    hipLaunchKernelGGL((scan_k<R, Y, NK, kAll>), grid, block, 0, st, a, p);
  } else {
    hipLaunchKernelGGL((scan_k<R, Y, NK, kOwn>), grid, block, 0, st, a, p);
    hipLaunchKernelGGL(combine_k, dim3((uint32_t)(a.p.n * per_seq)), block, 0, st, a, p, make_fastdiv((uint32_t)per_seq));
    hipLaunchKernelGGL((scan_k<R, Y, NK, kFrom>), grid, block, 0, st, a, p);
  }
  return (int)hipGetLastError();
}

template <typename R, typename Y>
int launch_n(const ScanArgs &a, const ScanPlan &p, hipStream_t st) {
  if (a.N <= 32) return launch<R, Y, 1>(a, p, st);
  if (a.N == 64) return launch<R, Y, 2>(a, p, st);
  return launch<R, Y, 4>(a, p, st);
}

}  // namespace

size_t scan_workspace(const ScanArgs &a) {
  const ScanPlan p = make_plan(a);
  return p.seg ? decay_bytes(a, p) + (size_t)p.items * a.H * a.P * a.N * 4 : 0;
}

int launch_scan(const ScanArgs &a, hipStream_t st) {
  ScanPlan p = make_plan(a);
  p.decay = (float *)a.workspace;
  p.state = p.seg ? (float *)((char *)a.workspace + decay_bytes(a, p)) : nullptr;
  if (!a.bf16) return launch_n<float, float>(a, p, st);
  return a.y_bf16 ? launch_n<bf16_t, bf16_t>(a, p, st) : launch_n<bf16_t, float>(a, p, st);
}

}  // namespace rssm
