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
// one head (16, and a workgroup 64, in calls of few workgroups and for the own
// states of float32 records) with their whole state in registers (S^T as accumulators of
// v_mfma_f32_16x16x32_bf16: lane l holds rows n = 4 (l / 16) + i of column p =
// l % 16).  That layout is at once the operand layout of S C^T with the sum
// over n taken in the order n = 32 k + 16 (i / 4) + 4 (l / 16) + i % 4, so the
// state never leaves its wave, and G^T as accumulators is in the same way the
// operand M of M x.  B^T and x^T operands come from row-major LDS tiles by the
// transposing LDS read (lane l gets column l % 16 of rows 4 (l / 16) .. + 3).
//
// Few long sequences are cut into segments that fill the card, in three steps:
// each segment's own state from zero (scan_k, kOwn), the states that segments
// start from (combine_k, or the segments themselves), the outputs (kFrom).
//
// Precision.  bf16 records enter the products as they are, float32 records as
// three bf16 pieces (their sum is the value; products of pieces below 2^-24 are
// dropped).  The weighted inputs of the state update are always three pieces:
// the state stays float32.  M and S in the output products are three pieces for
// float32 outputs and two for bf16 outputs, whatever the launch: within 2^-16 of
// each term, next to the output's own 2^-8.  One piece there is 3 to 10 % faster and
// leaves the outputs of a resumed batch at an error of 0.0021 where their rounding
// is 0.0017; three pieces are up to 10 % slower than two and leave the same 0.0017.
//
// What bounds it is instruction issue.  A chunk of 64 tokens costs a wave 196
// matrix products (240 with float32 outputs) and 1140 (1400) other vector
// operations, and two waves a SIMD, all that the registers hold, issue one of
// those about every six cycles; the matrix pipe is busy 38 % of the time, the clock
// near 2.0 GHz under this load.  128 heads of 64, states of 128, bf16: one prompt of
// 8192 tokens 204 to 210 us (own states 61, combine_k 10, outputs 133; 0.3 GB would
// take 60), 24 prompts of 16384 tokens with float32 outputs 398 to 403
// us (1.1 GB, 211 us).
#include "ops.h"
#include "pieces.h"

namespace rssm {
namespace {


constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr float kLog2e = 1.4426950408889634f;

// LDS tiles are rows of 256 bytes, a token each, in 16-byte granules of eight
// bf16.  A read serves 256 bytes at a time, so its lanes' granules must differ in
// their low four bits; the granules of a row are permuted by an exclusive or that
// does that for the reads at hand (measured: no conflicts).
constexpr int kRow = 256;
// B and x: 4 rows at 16 neighbouring columns (the transposing read), and 16 rows
// at one column; 32 lanes of 8 bytes at a time each.
__device__ __forceinline__ int in_row(int row, int c) {  // byte of column c (a multiple of 4) in its row
  return ((c >> 3 ^ (2 * (row & 7) | (row >> 3 & 1))) << 4) + (c >> 2 & 1) * 8;
}
// x in rows of 128 bytes, two of which meet the banks that one of 256 does: the transposing read only.
template <int BYTES>
__device__ __forceinline__ int in_row_x(int row, int c) {
  return BYTES == kRow ? in_row(row, c) : ((c >> 3 ^ (row & 6)) << 4) + (c >> 2 & 1) * 8;
}
// C: a granule holds a lane's operand of one 32-column step k, columns 32 k + 4 q
// .. + 3 and 32 k + 16 + 4 q .. + 3, and is read whole by 16 rows at a time.
__device__ __forceinline__ int in_row_c(int row, int k, int q) { return ((4 * k + q) ^ (row & 15)) << 4; }

// A value all lanes share, in a scalar register.
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(bits(v)));
}

// v, but not known to the compiler to be what it was before.
__device__ __forceinline__ int again(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Eight neighbouring elements of a record on their way to a granule of LDS: as
// they are, or float32 cut in three bf16 pieces, a tile each.
template <typename R>
struct Granule {
  uint4 v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int at, int plus) { v = buffer_load16(b, at, plus); }
  __device__ __forceinline__ void load2(__amdgpu_buffer_rsrc_t b, int at0, int at1, int plus) {  // four and four
    const i32x2 x = __builtin_bit_cast(i32x2, __builtin_amdgcn_raw_buffer_load_b64(b, at0, plus, 0));
    const i32x2 y = __builtin_bit_cast(i32x2, __builtin_amdgcn_raw_buffer_load_b64(b, at1, plus, 0));
    v = make_uint4(x[0], x[1], y[0], y[1]);
  }
  __device__ __forceinline__ void put(char *to, int) const { *reinterpret_cast<uint4 *>(to) = v; }
};
template <>
struct Granule<float> {
  uint4 v, w;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int at, int plus) { load2(b, at, at + 16, plus); }
  __device__ __forceinline__ void load2(__amdgpu_buffer_rsrc_t b, int at0, int at1, int plus) {
    v = buffer_load16(b, at0, plus);
    w = buffer_load16(b, at1, plus);
  }
  __device__ __forceinline__ void put(char *to, int piece) const {
    uint32_t a[3], b[3], c[3], d[3];
    pieces<3>(__uint_as_float(v.x), __uint_as_float(v.y), a);
    pieces<3>(__uint_as_float(v.z), __uint_as_float(v.w), b);
    pieces<3>(__uint_as_float(w.x), __uint_as_float(w.y), c);
    pieces<3>(__uint_as_float(w.z), __uint_as_float(w.w), d);
#pragma unroll
    for (int u = 0; u < 3; ++u) *reinterpret_cast<uint4 *>(to + u * piece) = make_uint4(a[u], b[u], c[u], d[u]);
  }
};

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

// Tile i of the lower triangle, row by row.
__device__ __forceinline__ int tile_row(int i) { return 0x3333222110ull >> 4 * i & 15; }
__device__ __forceinline__ int tile_col(int i) { return 0x3210210100ull >> 4 * i & 15; }

// Asks the compiler to issue N matrix products with V other vector operations behind each.
template <int N, int V>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x2, V, 0);
  }
}

struct ScanPlan {
  int seg;        // tokens of a segment (a multiple of 64), or 0: sequences are not split
  int items;      // segments of all sequences
  int hw, wph;    // heads of a workgroup, waves of a head in it
  int parts;      // workgroups a head's columns are spread over (then hw is 1)
  int nb;         // workgroups of a group
  int adds;       // segments add up the own states before them themselves; 0: combine_k does
  int64_t units;  // items x groups: the workgroups of a unit share B and C
  FastDiv fnb, fG, fparts;
  float *state;   // [items][H][P N]: a segment's own state, then its start
  float *decay;   // [items][H]
};

// The parts of one launch.  kAll: sequences in one piece.  kOwn: every segment but
// the last of a sequence leaves the state it would build from zero, and its
// decay.  kFrom: segments start from the states that combine_k left.
enum { kAll = 0, kOwn = 1, kFrom = 2 };

// Compile-time shape of a kernel: R records, Y outputs, NK 32-column steps of the
// state, CT 16-column tiles of x a wave.
template <typename R, typename Y, int NK, int CT, int MODE>
struct Shape_ {
  static constexpr int COLS = 16 * CT * kWaves;            // x columns of a workgroup
  static constexpr bool OUT = MODE != kOwn;
  static constexpr int IP = sizeof(R) == 4 ? 3 : 1;        // pieces of an input
  static constexpr int MP = sizeof(Y) == 4 ? 3 : 2;        // pieces of M and S in the output products
  static constexpr int QB = IP == 3 ? 2 : 4, Q = 16 * QB;  // blocks and tokens of a chunk
  static constexpr int TILES = QB * (QB + 1) / 2;
  static constexpr int RS = kRow, XS = 2 * COLS;           // bytes of a row of B and C, and of x
  static constexpr int B0 = 0, C0 = B0 + IP * Q * RS, X0 = C0 + (OUT ? IP * Q * RS : 0), SC0 = X0 + IP * Q * XS;
  static constexpr int SC = 6 * Q * 4;  // per head: six values a token
  static constexpr int G0 = SC0, SC1 = G0 + (OUT ? TILES * kWave * 16 : 0);
  static constexpr int lds(int heads) { return SC1 + heads * SC; }
  // Waves a SIMD: as many as registers (outputs, 32 columns) and tiles allow; kernels of 16
  // columns with outputs run where there are few workgroups.
  static constexpr int WAVES = CT == 2 || OUT ? 2 : 4;
};

template <typename R, typename Y, int NK, int CT, int MODE>
__global__ __launch_bounds__(kThreads)
__attribute__((amdgpu_waves_per_eu(Shape_<R, Y, NK, CT, MODE>::WAVES, Shape_<R, Y, NK, CT, MODE>::WAVES)))
void scan_k(ScanArgs a, ScanPlan plan) {
  typedef Shape_<R, Y, NK, CT, MODE> Z;
  constexpr int kCols = Z::COLS;
  constexpr int IP = Z::IP, MP = Z::MP, QB = Z::QB, Q = Z::Q, TILES = Z::TILES, RS = Z::RS, XS = Z::XS;
  constexpr int KB = QB / 2, NT = 2 * NK;                // 32-token steps, 16-column tiles of the state
  constexpr int NV = 4 * NK, XV = kCols / 8;             // granules of a row
  constexpr int RB = kThreads / NV, RX = kThreads / XV;  // rows of one granule a thread
  constexpr int LB = Q > RB ? Q / RB : 1, LX = Q / RX;
  static_assert(RX % 16 == 0 && RB % 16 == 0, "a thread's rows share their permutation");
  constexpr bool OUT = Z::OUT;
  extern __shared__ __attribute__((aligned(16))) char lds[];

  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r = lane % 16, q = lane / 16;
  // Unit u on XCD u % 8 (workgroup i runs on XCD i % 8): a unit's workgroups share an
  // L2, and with eight groups (or a multiple) so do a group's segments and their states.
  const int k8 = blockIdx.x / kXcds, u8 = fdiv(k8, plan.fnb);
  const int unit = u8 * kXcds + blockIdx.x % kXcds, blk = k8 - u8 * plan.nb;
  if (unit >= plan.units) return;
  const int item = fdiv(unit, plan.fG), g = unit - item * a.G;
  const int Hg = a.H / a.G, P = a.P, N = a.N;

  int seq, begin, len, t_first = 0, t_end, before = 0;  // before: own states to add up first
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
    if (MODE == kFrom && plan.adds) before = it.index;
    t_end = min(len, t_first + plan.seg);
    // Nothing starts from the last segment's state.  Its place keeps where the sequence
    // starts if segments add up for themselves: kFrom may write over `initial`.
    if (MODE == kOwn && t_end == len) {
      if (!plan.adds || it.index == 0) return;
      t_end = t_first;
    }
  }
  const int row = batch_row(a.p, seq, g == 0 && blk == 0 && tid == 0 && MODE != kOwn && t_first == 0);
  if (row < 0) return;

  // The workgroup's heads, or its part of one head's columns.
  const int bh = fdiv(blk, plan.fparts), part = blk - bh * plan.parts;
  const int h0 = g * Hg + bh * plan.hw;                        // the first head
  const int nh = min(plan.hw, Hg - bh * plan.hw);
  const int hw_ = wave / plan.wph, pw = wave - hw_ * plan.wph;
  const int c0 = part * plan.wph * 16 * CT;                    // the head's first column here
  const bool active = hw_ < nh && c0 + 16 * CT * pw < P;       // this wave has tiles of x columns
  const int hi = active ? hw_ : 0, pt0 = active ? c0 / 16 + pw * CT : c0 / 16;
  const int np = min(CT, P / 16 - pt0);                        // a head's last wave may have a tile less
  const int h = h0 + hi;
  const int xcol = hi * P + 16 * pt0 - c0;
  const int ncols = plan.parts > 1 ? min(plan.wph * 16 * CT, P - c0) : nh * P;
  const bool first = active && pw == 0;                        // the head's first wave here
  const float Al = uniform(a.A[h] * kLog2e), D = OUT ? uniform(a.D[h]) : 0.f;
  float *const my = reinterpret_cast<float *>(lds + Z::SC1) + hi * 6 * Q;  // the head's values a token
  float4 *const sG = reinterpret_cast<float4 *>(lds + Z::G0) + lane;

  // The state: S^T tile nt, rows n = 16 nt + 4 q + i, column p = r of each of the wave's tiles.
  floatx4 S[NT][CT];
  const size_t tile0 = (size_t)h * P * N + (size_t)(16 * pt0 + r) * N + 4 * q;
  const size_t states = (size_t)a.H * P * N;
  const bool known = a.initial && (!a.p.resume || a.p.resume[seq]);
  const float *from = known && (MODE != kOwn || t_end == t_first) ? a.initial + row * states : nullptr;
  if constexpr (MODE == kFrom) {
    if (len > plan.seg) from = plan.state + (plan.adds ? item - before + (len - 1) / plan.seg : item) * states;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int pt = 0; pt < CT; ++pt) {
      S[nt][pt] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (from && 16 * nt < N && pt < np) {
        const float4 v = ld4(from + tile0 + (size_t)16 * pt * N + 16 * nt);
        S[nt][pt] = floatx4{v.x, v.y, v.z, v.w};
      }
    }

  if constexpr (MODE == kFrom) {
    for (int j = item - before; j < item; ++j) {
      const float d = plan.decay[(size_t)j * a.H + h];
      const float *own = plan.state + j * states + tile0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int pt = 0; pt < CT; ++pt)
          if (16 * nt < N && pt < np) {
            const float4 v = ld4(own + (size_t)16 * pt * N + 16 * nt);
            floatx4 &s = S[nt][pt];
            s = floatx4{fmaf(s[0], d, v.x), fmaf(s[1], d, v.y), fmaf(s[2], d, v.z), fmaf(s[3], d, v.w)};
          }
    }
  }

  // Global to registers through buffers that end with the chunk's last row: rows
  // past it read as zeros, and so do the columns of threads without a place.
  typedef Granule<R> Gr;
  Gr pB[LB], pC[OUT ? LB : 1], pX[LX];
  const size_t rB = (size_t)a.G * N, rX = (size_t)a.H * P;
  const R *Bg = (const R *)a.Bm + (size_t)begin * rB + (size_t)g * N;
  const R *Cg = (const R *)a.Cm + (size_t)begin * rB + (size_t)g * N;
  const R *Xg = (const R *)a.x + (size_t)begin * rX + (size_t)h0 * P + c0;
  const float *dtg = a.dt + (size_t)begin * a.H + h;
  constexpr int kNowhere = 0x7fffff00;
  float dtv = 0.f;
  // Places in global memory and LDS are computed anew from the thread's number at each
  // use: a few operations, where 14 registers would otherwise push others into memory.
  auto fetch = [&](int t0, bool bc, bool x_) {
    const int id = again(tid);
    const int tB = id / NV, cB = id % NV * 8, tX = id / XV, cX = id % XV * 8;
    const int cC = 32 * (id % NV / 4) + 4 * (id % 4);  // C's granules go by operands
    const bool hasB = RB <= Q || tB < Q;               // narrow states leave threads without a piece of B and C
    const int oB = hasB && cB < N ? (int)((tB * rB + cB) * sizeof(R)) : kNowhere;
    const int oC = hasB && cC < N ? (int)((tB * rB + cC) * sizeof(R)) : kNowhere;
    const int oC1 = NK > 1 || cC + 16 < N ? oC + 16 * (int)sizeof(R) : kNowhere;
    const int oX = cX < ncols ? (int)((tX * rX + cX) * sizeof(R)) : kNowhere;
    const int odt = id % kWave < Q ? id % kWave * a.H * 4 : kNowhere;
    const int rem = min(Q, t_end - t0);  // none left: empty buffers, which read nothing
    auto size = [&](size_t row, int last) { return rem > 0 ? ((rem - 1) * row + last) * sizeof(R) : 0; };
    if (bc) {
      dtv = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          buffer_of(dtg + (size_t)t0 * a.H, rem > 0 ? ((rem - 1) * (size_t)a.H + 1) * 4 : 0), odt, 0, 0));
      const auto bB = buffer_of(Bg + t0 * rB, size(rB, N));
#pragma unroll
      for (int i = 0; i < LB; ++i) pB[i].load(bB, oB, (int)(i * RB * rB * sizeof(R)));
      if constexpr (OUT) {
        const auto bC = buffer_of(Cg + t0 * rB, size(rB, N));
#pragma unroll
        for (int i = 0; i < LB; ++i) pC[i].load2(bC, oC, oC1, (int)(i * RB * rB * sizeof(R)));
      }
    }
    if (x_) {
      const auto bX = buffer_of(Xg + t0 * rX, size(rX, ncols));
#pragma unroll
      for (int i = 0; i < LX; ++i) pX[i].load(bX, oX, (int)(i * RX * rX * sizeof(R)));
    }
  };
  auto spill = [&]() {
    const int id = again(tid);
    const int tB = id / NV, tX = id / XV;
    char *toB = lds + Z::B0 + tB * RS + in_row(tB, id % NV * 8), *toC = lds + Z::C0 + tB * RS + in_row_c(tB, id % NV / 4, id % 4);
    char *toX = lds + Z::X0 + tX * XS + in_row_x<XS>(tX, id % XV * 8);
    if (RB <= Q || tB < Q) {
#pragma unroll
      for (int i = 0; i < LB; ++i) {
        pB[i].put(toB + i * RB * RS, Q * RS);
        if constexpr (OUT) pC[i].put(toC + i * RB * RS, Q * RS);
      }
    }
#pragma unroll
    for (int i = 0; i < LX; ++i) pX[i].put(toX + i * RX * XS, Q * XS);
  };

  // Operand of 32 columns (step k) of rows 16 b + r, in the order of an accumulator
  // pair: columns 32 k + 4 q .. + 3, then 32 k + 16 + 4 q .. + 3.
  auto rows = [&](int tile, int b, int k, int oR) {
    Frag f;
    const char *p = lds + tile + 16 * b * RS;
    f.h[0] = *reinterpret_cast<const s16x4 *>(p + (oR ^ (k * 64)));
    f.h[1] = *reinterpret_cast<const s16x4 *>(p + (oR ^ (k * 64 + 32)));
    return f;
  };
  auto rows_c = [&](int tile, int b, int k, int oC) {
    Frag f;
    f.v = *reinterpret_cast<const s16x8 *>(lds + tile + 16 * b * RS + (oC ^ (k * 64)));
    return f;
  };
  // Operand of 32 tokens (step k) of column 16 c + r, tokens in the same order.
  auto cols = [&](int tile, int c, int k, int oT) {
    Frag f;
    const char *p = lds + tile + 32 * k * RS + (oT ^ (c * 32));
    f.h[0] = read_tr(p);
    f.h[1] = read_tr(p + 16 * RS);
    return f;
  };

  float decay = 1.f;
  fetch(t_first, true, true);
  for (int t0 = t_first; t0 < t_end; t0 += Q) {
    // Two workgroups share a SIMD, and the older one's instructions go first: it would end
    // early and leave the other alone for the last quarter, so they take turns of two
    // chunks.  The stretch of M is a chain of dependent steps and goes before both
    // (prompts of 16384 tokens: 415 us; turns alone 424, M alone 413, neither 442; of 8192:
    // 203, 205, 206, 209).
    if ((t0 / Q / 2 + (blockIdx.x >= gridDim.x / 2)) & 1)
      __builtin_amdgcn_s_setprio(1);
    else
      __builtin_amdgcn_s_setprio(0);
    // Decays: lane = token.
    const float dt = dtv;
    double sum = dt;
    float suf = dt;
    sum += row_shift<0x111>(sum), suf += row_shift<0x101>(suf);
    sum += row_shift<0x112>(sum), suf += row_shift<0x102>(suf);
    sum += row_shift<0x114>(sum), suf += row_shift<0x104>(suf);
    sum += row_shift<0x118>(sum), suf += row_shift<0x108>(suf);
    suf = row_shift<0x101>(suf);  // the tokens after this one
    sum *= Al;                    // as an exponent of 2
    const float pre = (float)sum, epre = __builtin_amdgcn_exp2f(pre), edt = __builtin_amdgcn_exp2f(Al * suf) * dt;
    float E[QB];  // the blocks' decays
#pragma unroll
    for (int b = 0; b < QB; ++b) E[b] = __uint_as_float(__builtin_amdgcn_readlane(bits(epre), 16 * b + 15));
    float all = 1.f, after = 1.f;  // the chunk's decay, and from the end of the lane's block to the chunk's
#pragma unroll
    for (int b = QB - 1; b >= 0; --b) {
      after = lane / 16 == b ? all : after;
      all *= E[b];
    }
    decay *= all;

    lds_barrier();  // every wave is done with the last chunk's tiles
    spill();
    if (first && lane < Q) {
      my[lane] = edt * after;
      if constexpr (OUT) {
        my[Q + lane] = epre;
        my[2 * Q + lane] = pre;
        my[3 * Q + lane] = (float)(sum - (double)pre);
        my[4 * Q + lane] = dt;
        my[5 * Q + lane] = edt;
      }
    }
    lds_barrier();

    // All of this is independent of the other waves: their tiles of G^T (rows j,
    // columns t), S0 C^T transposed (rows p, columns t), and the state after the chunk.
    floatx4 Yt[QB][CT];
    const int la = again(lane), lr = la % 16, lq = la / 16;
    const int tr = 4 * lq + lr / 4, oT = tr * RS + in_row(tr, lr % 4 * 4);
    Frag xf[KB][CT][IP], xw[KB][CT][3];
    float4 w4[KB][2];
    // The weighted inputs, in three pieces: step k, column tile pt.
    auto weigh = [&](int k, int pt) {
      const float w[8] = {w4[k][0].x, w4[k][0].y, w4[k][0].z, w4[k][0].w, w4[k][1].x, w4[k][1].y, w4[k][1].z, w4[k][1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Frag(&x)[IP] = xf[k][pt];
        float lo = lower(x[IP - 1].w[i]), up = upper(x[IP - 1].w[i]);
#pragma unroll
        for (int u = IP - 2; u >= 0; --u) lo += lower(x[u].w[i]), up += upper(x[u].w[i]);
        uint32_t pw[3];
        pieces<3>(lo * w[2 * i], up * w[2 * i + 1], pw);
#pragma unroll
        for (int u = 0; u < 3; ++u) xw[k][pt][u].w[i] = pw[u];
      }
    };
    auto load_x = [&]() {
#pragma unroll
      for (int pt = 0; pt < CT; ++pt) {
        const char *p = lds + Z::X0 + tr * XS + in_row_x<XS>(tr, xcol + (pt < np ? 16 * pt : 0) + lr % 4 * 4);
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
          for (int u = 0; u < IP; ++u) {
            xf[k][pt][u].h[0] = read_tr(p + (u * Q + 32 * k) * XS);
            xf[k][pt][u].h[1] = read_tr(p + (u * Q + 32 * k + 16) * XS);
          }
      }
#pragma unroll
      for (int k = 0; k < KB; ++k) w4[k][0] = ld4(my + 32 * k + 4 * lq), w4[k][1] = ld4(my + 32 * k + 16 + 4 * lq);
    };

    if constexpr (OUT) {
      const int oR = lr * RS + in_row(lr, 4 * lq), oC = lr * RS + in_row_c(lr, 0, lq);
      constexpr int GT = (TILES + kWaves - 1) / kWaves;  // a wave's tiles; the last ones are computed twice over
      Frag gb[GT][NK], gc[GT][NK];                       // the pieces v of both, one at a time
      floatx4 acc[GT];
      auto tile_of = [&](int g) { return min(g * kWaves + wave, TILES - 1); };
#pragma unroll
      for (int g = 0; g < GT; ++g) acc[g] = floatx4{0.f, 0.f, 0.f, 0.f};
      auto load_g = [&](int g, int u, int v) {
        const int i = tile_of(g), tb = tile_row(i), jb = tile_col(i);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          gb[g][k] = rows(Z::B0 + u * Q * RS, jb, k, oR);
          gc[g][k] = rows_c(Z::C0 + v * Q * RS, tb, k, oC);
        }
      };
#pragma unroll
      for (int u = IP - 1; u >= 0; --u)
#pragma unroll
        for (int v = IP - 1 - u; v >= 0; --v) {
#pragma unroll
          for (int g = 0; g < GT; ++g) load_g(g, u, v);
          if (u == 0 && v == 0) load_x();
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int g = 0; g < GT; ++g) acc[g] = mfma32(gb[g][k], gc[g][k], acc[g]);
        }
      Frag sp[NK][CT][MP];
      auto cut_state = [&](int k) {
#pragma unroll
        for (int pt = 0; pt < CT; ++pt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const floatx4 &s = S[2 * k + i / 2][pt];
            uint32_t w[MP];
            pieces<MP>(s[i % 2 * 2], s[i % 2 * 2 + 1], w);
#pragma unroll
            for (int u = 0; u < MP; ++u) sp[k][pt][u].w[i] = w[u];
          }
      };
      Frag cf[2][QB];
      auto load_c = [&](int at) {  // at: step k and piece v as k IP + v
#pragma unroll
        for (int tb = 0; tb < QB; ++tb) cf[at % 2][tb] = rows_c(Z::C0 + at % IP * Q * RS, tb, at / IP, oC);
      };
      load_c(0);
      cut_state(0);
#pragma unroll
      for (int g = 0; g < GT; ++g) sG[tile_of(g) * kWave] = make_float4(acc[g][0], acc[g][1], acc[g][2], acc[g][3]);
#pragma unroll
      for (int tb = 0; tb < QB; ++tb)
#pragma unroll
        for (int pt = 0; pt < CT; ++pt) Yt[tb][pt] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int at = 0; at < NK * IP; ++at) {
        __builtin_amdgcn_sched_barrier(0);
        const int k = at / IP, v = at % IP;
        if (at + 1 < NK * IP) load_c(at + 1);
        if (v == IP - 1 && k + 1 < NK) cut_state(k + 1);
        if (at < KB * CT) weigh(at / CT, at % CT);
#pragma unroll
        for (int u = MP - 1; u >= 0; --u)
          if (u + v < 3) {
#pragma unroll
            for (int tb = 0; tb < QB; ++tb)
#pragma unroll
              for (int pt = 0; pt < CT; ++pt) Yt[tb][pt] = mfma32(sp[k][pt][u], cf[at % 2][tb], Yt[tb][pt]);
          }
        interleave<QB * CT * (IP == 1 ? MP : 2), 4>();
      }
#pragma unroll
      for (int i = NK * IP; i < KB * CT; ++i) weigh(i / CT, i % CT);
    } else {
      load_x();
#pragma unroll
      for (int i = 0; i < KB * CT; ++i) weigh(i / CT, i % CT);
    }
    {
      // Steps of two state tiles and one piece of B, their operands read one step ahead.
      constexpr int STEPS = KB * NK * IP;
      Frag bf[2][2];
      auto load_b = [&](int at) {
        const int k = at / (NK * IP), n0 = at / IP % NK * 2, v = at % IP;
        bf[at % 2][0] = cols(Z::B0 + v * Q * RS, n0, k, oT);
        bf[at % 2][1] = cols(Z::B0 + v * Q * RS, n0 + 1, k, oT);
      };
      load_b(0);
#pragma unroll
      for (int at = 0; at < STEPS; ++at) {
        __builtin_amdgcn_sched_barrier(0);
        const int k = at / (NK * IP), n0 = at / IP % NK * 2, v = at % IP;
        if (at + 1 < STEPS) load_b(at + 1);
        if (k == 0 && v == 0) {
#pragma unroll
          for (int pt = 0; pt < CT; ++pt) S[n0][pt] *= all, S[n0 + 1][pt] *= all;
        }
#pragma unroll
        for (int u = 2; u >= 0; --u)
          if (u + v < 3) {
#pragma unroll
            for (int pt = 0; pt < CT; ++pt) {
              S[n0][pt] = mfma32(bf[at % 2][0], xw[k][pt][u], S[n0][pt]);
              S[n0 + 1][pt] = mfma32(bf[at % 2][1], xw[k][pt][u], S[n0 + 1][pt]);
            }
          }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (OUT) __builtin_amdgcn_s_setprio(2);
    fetch(t0 + Q, true, !OUT);

    if constexpr (OUT) {
      // What M needs of block tb: the values of this lane's token in it, and of its own four tokens.
      float et[2], p1[2], l1[2];
      float4 g4[2][QB];
      auto load_t = [&](int tb) {
        et[tb % 2] = my[Q + 16 * tb + lr];
        p1[tb % 2] = my[2 * Q + 16 * tb + lr], l1[tb % 2] = my[3 * Q + 16 * tb + lr];
      };
      auto load_gt = [&](int tb) {
#pragma unroll
        for (int jb = 0; jb <= tb; ++jb) g4[tb % 2][jb] = sG[(tb * (tb + 1) / 2 + jb) * kWave];
      };
      load_t(0);
      lds_barrier();  // G is complete
      load_gt(0);
      float f = 1.f;
#pragma unroll
      for (int tb = 0; tb < QB; ++tb) {
        __builtin_amdgcn_sched_barrier(0);
        if (tb == QB / 2) fetch(t0 + Q, false, true);
        if (tb + 1 < QB) load_t(tb + 1), load_gt(tb + 1);
        const int c = tb % 2;
        const float4 p4 = ld4(my + 2 * Q + 16 * tb + 4 * lq), l4 = ld4(my + 3 * Q + 16 * tb + 4 * lq);
        const float4 d4 = ld4(my + 4 * Q + 16 * tb + 4 * lq);
        const float e = f * et[c];
#pragma unroll
        for (int pt = 0; pt < CT; ++pt) Yt[tb][pt] *= e;
        f *= E[tb];
        // M^T from G^T, and x M^T.
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
            const float4 gt = g4[c][jb];
            float m[4];
            if (jb < tb) {
              float g = et[c];  // t's block up to t, and the whole blocks between
#pragma unroll
              for (int b = 0; b < QB; ++b)
                if (b > jb && b < tb) g *= E[b];
              const float4 wj = ld4(my + 5 * Q + 16 * jb + 4 * lq);
              m[0] = gt.x * (g * wj.x), m[1] = gt.y * (g * wj.y), m[2] = gt.z * (g * wj.z), m[3] = gt.w * (g * wj.w);
            } else {
              const float gj[4] = {gt.x, gt.y, gt.z, gt.w}, pj[4] = {p4.x, p4.y, p4.z, p4.w};
              const float lj[4] = {l4.x, l4.y, l4.z, l4.w}, dj[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int j = 4 * lq + i;
                const float v = gj[i] * (__builtin_amdgcn_exp2f((p1[c] - pj[i]) + (l1[c] - lj[i])) * dj[i]);
                m[i] = j < lr ? v : j == lr ? v + D : 0.f;  // D x_t rides along
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t w[MP];
              pieces<MP>(m[2 * i], m[2 * i + 1], w);
#pragma unroll
              for (int u = 0; u < MP; ++u) mf[u].w[2 * half + i] = w[u];
            }
          }
#pragma unroll
          for (int u = MP - 1; u >= 0; --u)
#pragma unroll
            for (int v = 0; v < IP; ++v)
              if (u + v < 3) {
#pragma unroll
                for (int pt = 0; pt < CT; ++pt) Yt[tb][pt] = mfma32(xf[k][pt][v], mf[u], Yt[tb][pt]);
              }
        }
      }
      // y: this lane holds four neighbouring channels of token 16 tb + r.
      if (active) {
        const int rem = min(Q, t_end - t0);
        const auto bY = buffer_of((Y *)a.y + (size_t)(begin + t0) * rX + (size_t)h * P + 16 * pt0,
                                  ((rem - 1) * rX + 16 * np) * sizeof(Y));  // rows past the end are not written
        const int oY = (int)((lr * rX + 4 * lq) * sizeof(Y));
#pragma unroll
        for (int tb = 0; tb < QB; ++tb)
#pragma unroll
          for (int pt = 0; pt < CT; ++pt) {
            if (pt >= np) continue;
            const floatx4 o = Yt[tb][pt];
            const int step = (int)(16 * tb * rX * sizeof(Y)), at = oY + 16 * pt * (int)sizeof(Y);
            if constexpr (sizeof(Y) == 2)
              __builtin_amdgcn_raw_buffer_store_b64(i32x2{(int)pack_bf16(o[0], o[1]), (int)pack_bf16(o[2], o[3])}, bY, at, step, 0);
            else  // step in the vector offset: a 16-byte store with a scalar offset may send the registers'
                  // next values if an instruction rewrites them right behind it (seen: the last lanes of a row)
              __builtin_amdgcn_raw_buffer_store_b128(
                  i32x4{__float_as_int(o[0]), __float_as_int(o[1]), __float_as_int(o[2]), __float_as_int(o[3])}, bY, at + step, 0, 0);
          }
      }
    }
  }

  float *to = MODE == kOwn ? plan.state + item * states : t_end == len ? a.state + row * states : nullptr;
  if (to && active) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < CT; ++pt)
        if (16 * nt < N && pt < np)
          st4(to + tile0 + (size_t)16 * pt * N + 16 * nt, make_float4(S[nt][pt][0], S[nt][pt][1], S[nt][pt][2], S[nt][pt][3]));
  }
  if (MODE == kOwn && first && part == 0 && lane == 0) plan.decay[(size_t)item * a.H + h] = decay;
}

// Where each segment of a split sequence starts: the segment before it decays
// that one's start and adds its own state.  One thread, four state elements.  HBM bound
// (8192 tokens of 128 heads, 59 MB: 10.6 us); with many segments the loads' latency
// counts, so four are under way together (4096 tokens of 16 heads: a pass of 56 us, one
// by one 59).
constexpr int kAhead = 4;
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
  float *const at = plan.state + item0 * states + e;
  const float *const decay = plan.decay + (size_t)item0 * a.H + h;
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    float4 own[kAhead];
    float d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = min(i0 + i, n - 2);  // the last segment has no own state
      own[i] = ld4(at + j * states);
      d[i] = decay[(size_t)j * a.H];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= n) break;
      st4(at + (i0 + i) * states, run);
      run = make_float4(fmaf(run.x, d[i], own[i].x), fmaf(run.y, d[i], own[i].y), fmaf(run.z, d[i], own[i].z),
                        fmaf(run.w, d[i], own[i].w));
    }
  }
}

// The workgroups of an item with ct tiles a wave.
void set_tiles(const ScanArgs &a, ScanPlan &p, int ct) {
  const int Hg = a.H / a.G, waves = (a.P / 16 + ct - 1) / ct;  // of a head
  p.parts = (waves + kWaves - 1) / kWaves;
  p.wph = (waves + p.parts - 1) / p.parts;
  p.hw = kWaves / p.wph < Hg ? kWaves / p.wph : Hg;
  p.nb = (Hg + p.hw - 1) / p.hw * p.parts;
  p.fnb = make_fastdiv((uint32_t)p.nb);
  p.fG = make_fastdiv((uint32_t)a.G);
  p.fparts = make_fastdiv((uint32_t)p.parts);
}

ScanPlan make_plan(const ScanArgs &a) {
  ScanPlan p{};
  set_tiles(a, p, 2);
  const int per = a.G * p.nb;
  // Split sequences along the length when there are too few to fill the card, which
  // holds 512 workgroups.  Lengths are on the device, so the rules go by the number of
  // sequences and all their tokens: a long prompt among enough short ones to fill the
  // card by their number stays whole (128 heads: 8000 tokens alone 236 us, with six
  // prompts of ten 269, with seven 672).  The thresholds in tokens were measured with 32
  // and 128 heads of 64 columns and stand for where a segment's start and the launches
  // cost what its length saves; they do not depend on the heads.  Each sequence ends with a part of a segment, half of one on
  // average; with those counted, few segments wait for a second round (2048 float32
  // tokens of five sequences: 99 us against 104, 4096 of nine: 93 against 99).
  const int want = (512 + per - 1) / per, whole = max(want - a.p.n / 2, 1);
  const int seg = ((a.p.tokens + whole - 1) / whole + 63) / 64 * 64;
  // Below 128 tokens a segment costs more than it saves, and up to 320 tokens so do two
  // launches (300 tokens of 128 heads: 25 us whole, 28 split; 400: 39 and 32).
  // Up to four segments add up the own states before them as they start, without
  // combine_k's launch, and up to 768 tokens four are enough (600 tokens of 128 heads: 37
  // us, five and combine_k 46); more would keep the last one waiting (8192 tokens, eight:
  // 212 us against 201), and fewer of more tokens take longer (800 tokens of 32 heads,
  // four: 33 us against 30).
  const int least = a.p.tokens > 512 && a.p.tokens <= 768 ? 192 : 128;
  p.seg = a.p.n >= want || seg >= a.p.tokens || a.p.tokens <= 320 ? 0 : max(seg, least);
  if (p.seg >= a.p.tokens) p.seg = 0;
  p.adds = p.seg && (a.p.tokens + p.seg - 1) / p.seg <= 4;
  p.items = p.seg ? items_of(a.p.tokens, a.p.n, p.seg) : a.p.n;
  p.units = (int64_t)p.items * a.G;
  return p;
}

// Column tiles of a wave with outputs.  At most one workgroup a CU: waves of half the
// columns, on twice as many, end sooner (200 tokens of 32 heads: 20 us against 25; 600:
// 28 against 34).
int tiles(const ScanPlan &p) { return p.units * p.nb <= 256 ? 1 : 2; }

size_t decay_bytes(const ScanArgs &a, const ScanPlan &p) { return ((size_t)p.items * a.H * 4 + 255) / 256 * 256; }

template <typename R, typename Y, int NK, int CT, int MODE>
int launch_part(const ScanArgs &a, ScanPlan p, hipStream_t st) {
  set_tiles(a, p, CT);
  const int64_t blocks = (p.units + kXcds - 1) / kXcds * kXcds * p.nb;
  if (blocks > kMostBlocks) return kTooLarge;
  hipLaunchKernelGGL((scan_k<R, Y, NK, CT, MODE>), dim3((uint32_t)blocks), dim3(kThreads), (Shape_<R, Y, NK, CT, MODE>::lds(p.hw)),
                     st, a, p);
  return (int)hipGetLastError();
}

template <typename R, typename Y, int NK>
int launch(const ScanArgs &a, const ScanPlan &p, hipStream_t st) {
  const int per_seq = (a.H * a.P * a.N / 4 + kThreads - 1) / kThreads;
  if (p.seg && !p.adds && (int64_t)a.p.n * per_seq > kMostBlocks) return kTooLarge;
  const bool few = tiles(p) == 1;
  if (!p.seg) return few ? launch_part<R, Y, NK, 1, kAll>(a, p, st) : launch_part<R, Y, NK, 2, kAll>(a, p, st);
  // Own states of float32 records: half the columns leave LDS for four workgroups a CU
  // (2048 tokens of 64 heads: 100 us a pass against 109).
  const int e = sizeof(R) == 4 || few ? launch_part<R, Y, NK, 1, kOwn>(a, p, st) : launch_part<R, Y, NK, 2, kOwn>(a, p, st);
  if (e) return e;
  if (!p.adds)
    hipLaunchKernelGGL(combine_k, dim3((uint32_t)(a.p.n * per_seq)), dim3(kThreads), 0, st, a, p, make_fastdiv((uint32_t)per_seq));
  return few ? launch_part<R, Y, NK, 1, kFrom>(a, p, st) : launch_part<R, Y, NK, 2, kFrom>(a, p, st);
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

void scan_plan(const ScanArgs &a, int32_t (&plan)[4]) {
  ScanPlan p = make_plan(a);
  plan[0] = p.seg, plan[1] = p.adds, plan[2] = 16 * tiles(p);
  set_tiles(a, p, tiles(p));
  plan[3] = (int32_t)(p.units * p.nb < INT32_MAX ? p.units * p.nb : INT32_MAX);
}

int launch_scan(const ScanArgs &a, hipStream_t st) {
  ScanPlan p = make_plan(a);
  p.decay = (float *)a.workspace;
  p.state = p.seg ? (float *)((char *)a.workspace + decay_bytes(a, p)) : nullptr;
  if (!a.bf16) return launch_n<float, float>(a, p, st);
  return a.y_bf16 ? launch_n<bf16_t, bf16_t>(a, p, st) : launch_n<bf16_t, float>(a, p, st);
}

}  // namespace rssm
