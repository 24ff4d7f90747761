// Gated delta rule over packed prompts: S <- a S (I - b k k^T) + b v k^T, o = S q.
//
// Chunks of 64 tokens turn it into matrix products.  With g_t the sum of log a over
// the chunk's tokens up to t and S0 the state before it:
//   T[t][j] = b_t e^{g_t - g_j} k_t.k_j  (j < t, else 0),   A = (I + T)^-1 diag(b),
//   P[t][j] = e^{g_t - g_j} q_t.k_j      (j <= t, else 0),
//   U = A (V - diag(e^g) K S0^T),   O = diag(e^g) Q S0^T + P U,
//   S1 = e^{g_C} S0 + sum_j e^{g_C - g_j} u_j k_j^T.
//
// The least that a call moves is q, k, v and y; what bounds it is the walk along a sequence,
// whose chunks need the state before them, and in a chunk the float32 accuracy of the state:
// its products take three bf16 pieces of S, V - K S0^T and U.  Two forms of it:
//
// cells_k and chain_k, a call's few heads and sequences.  cells_k makes A and P of every
// chunk and head (a cell), all at once: they do not depend on the state.  chain_k walks a
// sequence's chunks, a workgroup for 16 (or 32) rows of a head's state, which evolve independently
// of the others, so that even one sequence's 32 heads are a workgroup for every CU; its
// waves share the products and hand each other S, V - K S0^T and U through LDS.  A chunk
// takes 1.5 us: one sequence of 8192 tokens, 32 heads, 128 x 128 (bf16): 269 us, of which
// cells_k 68 (it writes 270 MB at 3.9 TB/s) and chain_k 200.
//
// walk_k, calls of many (bf16 records): both in one launch, 128 rows to a workgroup, no cell
// in memory.  A chunk takes 5.5 us, for eight times the rows.  24 sequences of 16384 tokens together, 32
// heads, 128 x 128, float32 outputs: 305 us, 669 by the other two; eight of 2048 tokens: 236
// (2.3 TB/s of q, k, v and y), 525; one of 8192 and 64 heads: 529, 511.
//
// The inverse is a forward substitution inside the diagonal blocks of 16 tokens, joined
// block by block below them in float32 matrix products; no power of T is formed, whose
// entries would grow where keys are alike.  Decays are exponentials of differences of g, taken
// in float64.
#include <algorithm>

#include "ops.h"
#include "pieces.h"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int Q = 64;                 // tokens of a chunk
constexpr int kCus = 256;             // compute units of the card
constexpr int kSteps = 6;             // 32-token steps of the lower triangle, by rows of 16 tokens: 1, 1, 2, 2
constexpr int kFrag = kWave * 16;     // bytes of an operand, a lane's 16 bytes each
constexpr int kNowhere = 0x7fffff00;  // past the end of every buffer

__device__ __forceinline__ int step_of(int w, int s) { return w < 2 ? w : 2 * w - 2 + s; }

// What cells_k leaves for chain_k of one chunk and head (walk_k keeps K and Q as rows): operands as the lanes hold
// them.  Operands with tokens along the sum take them in the order of an accumulator
// pair: slot 8 q + 4 h + i of step s is token 32 s + 16 h + 4 q + i.
template <typename R, typename Y, int NK>
struct Cell {
  static constexpr int IP = sizeof(R) == 4 ? 3 : 1;  // pieces of an input
  // Pieces of P, U and S in the output products: two are within 2^-16 of a term, where a bf16
  // output is then rounded by up to 2^-8 (8192 tokens 268 us, 299 with three; eight of 2048 229, 247).
  static constexpr int MP = sizeof(Y) == 4 ? 3 : 2;
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
  int sort, apart; // walk_k: whether sequences go by length; chunks from which a head's rows are split,
  int halves;      // of so many sequences at most
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

// Place of granule g of a row of K or Q in LDS, permuted so that neither 16 rows at one
// granule nor four rows at four neighbouring ones meet in a bank.
template <int NK>
__device__ __forceinline__ int place_of(int row, int g) {
  const int turn = NK == 4 ? (row & 3) << 2 | (row >> 2 & 3) : NK == 2 ? (row >> 1 & 1) << 2 | (row >> 2 & 3) : row >> 2 & 3;
  return row * 64 * NK + (g ^ turn) * 16;
}

// v where `keep`, else 0: a mask, since a condition would become a branch around v.
__device__ __forceinline__ float only(float v, bool keep) { return __uint_as_float(bits(v) & (keep ? ~0u : 0u)); }

// A chunk's decays by token.  Off the diagonal tiles of 16 x 16 tokens e^{g_t - g_j} is
// `row` times `col`, neither above 1, with the first token of t's tile between them.
struct Decays {
  double g[Q];       // sums of log2 a
  float b[Q], row[Q], col[3][Q];
};
// By a wave, lane = token: past the end a = 1 and b = 0.  A decay of zero forgets everything.
__device__ __forceinline__ void make_decays(Decays &to, float al, float be, int rem, int lane, float &eg, float &left) {
  double g = lane < rem ? (double)log2f(al) : 0.0;
  g = scan64(g < -4096.0 ? -4096.0 : g);
  const double g1 = lane_value(g, 16), g2 = lane_value(g, 32), g3 = lane_value(g, 48);
  eg = __builtin_amdgcn_exp2f((float)g);
  left = __builtin_amdgcn_exp2f((float)(lane_value(g, kWave - 1) - g));
  to.g[lane] = g;
  to.b[lane] = lane < rem ? be : 0.f;
  to.row[lane] = __builtin_amdgcn_exp2f((float)(g - (lane < 16 ? lane_value(g, 0) : lane < 32 ? g1 : lane < 48 ? g2 : g3)));
  to.col[0][lane] = __builtin_amdgcn_exp2f((float)(g1 - g));  // read where token < 16, < 32, < 48
  to.col[1][lane] = __builtin_amdgcn_exp2f((float)(g2 - g));
  to.col[2][lane] = __builtin_amdgcn_exp2f((float)(g3 - g));
}

// A and P of a chunk by four waves.  `rows` is K in LDS by place_of, Q behind it.  T's tiles
// may lie where K and Q do, with `over`; the inverses of the diagonal ones take their place.
// `image` takes K and Q as operands, where given.
typedef float Tile[16][20];
__device__ __forceinline__ constexpr int tri(int i, int j) { return i * (i + 1) / 2 + j; }
struct Square {
  Tile T[10], turn[kWaves];  // T's tiles of the lower triangle, a place to transpose one
};

template <int S, int T>
__device__ __forceinline__ void below_row(float v, float (&x)[16]) {
  if constexpr (T < 16) {
    x[T] = fmaf(__uint_as_float(__builtin_amdgcn_update_dpp(0, bits(v), 0x150 + T, 0xF, 0xF, true)), x[S], x[T]);
    below_row<S, T + 1>(v, x);
  }
}
// x[t] += T[t][s] x[s] for the rows t below s, from s on: T[s] of lane t of every 16.
template <int S>
__device__ __forceinline__ void below(const float (&T)[16], float (&x)[16]) {
  if constexpr (S < 15) {
    below_row<S, S + 1>(T[S], x);
    below<S + 1>(T, x);
  }
}

template <typename R, typename Y, int NK, typename Sync, typename Last>
__device__ __forceinline__ void make_cell(const char *rows, Square &sq, const Decays &de, char *toA, char *toP, char *image, bool over,
                                          int wave, int lane, Sync sync, Last last) {
  typedef Cell<R, Y, NK> C;
  constexpr int IP = C::IP, MP = C::MP;
  constexpr int PL = sizeof(R) / 2, ROWS = Q * 64 * NK;
  const int r = lane % 16, q = lane / 16;

  // P^T of this wave's rows of 16 tokens, G^T = (K K^T)^T of the rows 3 - wave; all four
  // tiles of a row, of which those right of the diagonal are not used.
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
      row.staged(rows + place_of<NK>(16 * j + r, 4 * s + q), ROWS);
      row.cut(k[j]);
    }
    row.staged(rows + PL * ROWS + place_of<NK>(16 * wave + r, 4 * s + q), ROWS);
    if (image) row.put(image + (4 * NK + wave * NK + s) * C::ROW, lane);
    row.cut(qf);
    row.staged(rows + place_of<NK>(16 * wg + r, 4 * s + q), ROWS);
    if (image) row.put(image + (wg * NK + s) * C::ROW, lane);
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
  if (over) sync();
  {
    // Row w's factors: e^{g_t - g_j} times `by`, this lane's t = row r and columns 4 q + i of
    // the tiles left of the diagonal, and of the diagonal one.
    struct Factors {
      float4 col[3];
      float row, own[4];
    };
    auto factors = [&](int w, float by) {
      Factors f;
#pragma unroll
      for (int j = 0; j < 3; ++j) f.col[j] = ld4(de.col[max(w, 1) - 1] + 16 * j + 4 * q);
      f.row = by * de.row[16 * w + r];
      const double gt = de.g[16 * w + r];
#pragma unroll
      for (int i = 0; i < 4; ++i) f.own[i] = by * __builtin_amdgcn_exp2f((float)(gt - de.g[16 * w + 4 * q + i]));
      return f;
    };
    // Tile j of the row; on the diagonal where the column is below `to`, none right of it.
    auto decayed = [&](const floatx4 &v, const Factors &f, int w, int j, int to, float (&x)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float left = j < 3 ? f4get(f.col[j < 3 ? j : 0], i) * f.row : 0.f;
        x[i] = only(v[i] * (j == w ? f.own[i] : left), j < w || (j == w && 4 * q + i < to));
      }
    };
    const Factors fT = factors(wg, de.b[16 * wg + r]), fP = factors(wave, 1.f);
    char *const to = toP + step_of(wave, 0) * kFrag;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Frag f[MP];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 2 * s + e;
        float t[4], p[4];
        decayed(aG[j], fT, wg, j, r, t);
        if (j <= wg) st4(&sq.T[tri(wg, j)][r][4 * q], make_float4(t[0], t[1], t[2], t[3]));
        decayed(aP[j], fP, wave, j, r + 1, p);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[MP];
          pieces<MP>(p[2 * i], p[2 * i + 1], w);
#pragma unroll
          for (int u = 0; u < MP; ++u) f[u].w[2 * e + i] = w[u];
        }
      }
      if (s <= wave / 2) {
#pragma unroll
        for (int u = 0; u < MP; ++u) put(to + (u * kSteps + s) * kFrag, lane, f[u]);
      }
    }
  }
  const float bj = de.b[16 * wave + r];

  // The inverse of the diagonal tile of T's row by substitution: column r in every 16 lanes,
  // which have a row of T each and give it to the others.
  {
    Tile &own = sq.T[tri(wg, wg)];
    float T[16], x[16];
#pragma unroll
    for (int s = 0; s < 16; s += 4) {
      const float4 v = ld4(&own[r][s]);
#pragma unroll
      for (int i = 0; i < 4; ++i) T[s + i] = -f4get(v, i);
    }
#pragma unroll
    for (int t = 0; t < 16; ++t) x[t] = t == r ? 1.f : 0.f;
    below<0>(T, x);
    // This lane's four of the column: rows 4 q + e.
#pragma unroll
    for (int e = 0; e < 4; ++e) own[4 * q + e][r] = q < 2 ? (q == 0 ? x[e] : x[4 + e]) : (q == 2 ? x[8 + e] : x[12 + e]);
  }
  sync();
  last();
  // Block column `wave` of the inverse, tile d below the diagonal: rows 16 (wave + d) + 4 q + e,
  // column r.  A's, transposed, are halves of operands; zeros right of the diagonal.
  floatx4 X[4], acc[4];
  float4 tv[4][4];
#pragma unroll
  for (int d = 0; d < 4; ++d)
    if (wave + d < 4) {
      const Tile *const row = &sq.T[tri(wave + d, wave)];
#pragma unroll
      for (int m = 0; m <= d; ++m) {
        if (d == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) X[0][e] = row[0][4 * q + e][r];
        } else {
          tv[d][m] = ld4(&row[m][r][4 * q]);
        }
      }
    }
  char *const half = toA + lane * 16 + 8 * (wave % 2);
  Tile &turn = sq.turn[wave];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if (wave + d >= 4) break;
    if (d > 0) {
      X[d] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) X[d] = mfma_16x16x4(-f4get(tv[d][d], e), acc[d][e], X[d]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) turn[4 * q + e][r] = X[d][e] * bj;
    const float4 v = ld4(&turn[r][4 * q]);
#pragma unroll
    for (int n = d + 1; n < 4; ++n)
      if (wave + n < 4) {
        if (d == 0) acc[n] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n] = mfma_16x16x4(f4get(tv[n][d], e), X[d][e], acc[n]);
      }
    uint32_t w0[3], w1[3];
    pieces<3>(v.x, v.y, w0);
    pieces<3>(v.z, v.w, w1);
#pragma unroll
    for (int u = 0; u < 3; ++u)
      *reinterpret_cast<uint2 *>(half + (u * kSteps + step_of(wave + d, wave / 2)) * kFrag) = make_uint2(w0[u], w1[u]);
  }
  if (wave % 2) {
#pragma unroll
    for (int u = 0; u < 3; ++u)
      *reinterpret_cast<uint2 *>(half + (u * kSteps + step_of(wave - 1, wave / 2)) * kFrag) = make_uint2(0, 0);
  }
}

template <typename R, typename Y, int NK>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(sizeof(R) == 4 ? 2 : 4)))
void cells_k(DeltaArgs a, DeltaPlan plan) {
  typedef Cell<R, Y, NK> C;
  constexpr int NV = 4 * NK, RB = kThreads / NV;           // granules of eight columns in a row, rows a load
  constexpr int PL = sizeof(R) / 2, ROWS = Q * 16 * NV;    // planes of 16 bytes a granule, bytes of one
  constexpr int KQ = 2 * PL * ROWS, ALL = KQ > (int)sizeof(Square) ? KQ : (int)sizeof(Square);  // K and Q, then T
  __shared__ __attribute__((aligned(16))) char pool[ALL];
  __shared__ __attribute__((aligned(16))) Decays de;
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int place = fdiv(blockIdx.x, plan.fH), h = blockIdx.x - place * a.H;
  const Item it = find_item(a.p, plan.lo + place, Q);
  const int t0 = it.index * Q;
  if (it.index < 0 || t0 >= it.len) return;
  const int rem = min(Q, it.len - t0), N = a.N;
  const int64_t row0 = (int64_t)it.begin + t0;
  char *const cell = plan.cells + ((int64_t)place * a.H + h) * C::BYTES;

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
    float eg, left;
    make_decays(de, al, be, rem, lane, eg, left);
    float *const e = reinterpret_cast<float *>(cell + C::G0);
    e[lane] = eg, e[Q + lane] = left;
  }
  __syncthreads();

  make_cell<R, Y, NK>(
      pool, *reinterpret_cast<Square *>(pool), de, cell + C::A0, cell + C::P0, cell + C::K0, true, wave, lane, [] { __syncthreads(); }, [] {});
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
        Frag rf[2][3];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int u = 0; u < 3; ++u) rf[s][u].v = *reinterpret_cast<const s16x8 *>(sR[u] + 16 * ct * TR + oF + 64 * s);
        if (most) {
#pragma unroll
          for (int u = 2; u >= 0; --u)
#pragma unroll
            for (int w = 2 - u; w >= 0; --w)
#pragma unroll
              for (int s = 0; s < 2; ++s) U = mfma32(af[s][u], rf[s][w], U);
        } else {
#pragma unroll
          for (int u = 2; u >= 0; --u)
#pragma unroll
            for (int w = 2 - u; w >= 0; --w) U = mfma32(af[0][u], rf[0][w], U);
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
            for (int w = MP - 1; w >= 0; --w)
#pragma unroll
              for (int u = MP - 1 - w; u >= 0; --u) O[ct] = mfma32(uf[u], pf[s][w], O[ct]);
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

// Both in one launch, for calls of enough sequences and heads to fill the card: nothing
// between them goes through memory.  Four waves make the next chunk's A and P in LDS, out of
// K and Q that they put there, while up to eight use this chunk's: each carries 16 rows of
// the head's state through the chunk by itself, all 64 tokens and all columns, so that S,
// V - K S^T and U never leave its registers.  bf16 records, 64 or 128 columns.
// Eight sequences of 2048 tokens, 32 heads, 128 x 128: the matrix cores are busy 53% of the
// time, the vector pipes 60% and LDS 45%.  A chunk by four waves of users, the other half of
// a head's rows elsewhere, takes 4.1 us and not 5.5: so the longest sequences go, which would
// outlast the rest (24 sequences of up to 3258 tokens: 344 us without, 305 with it and with
// the longest first).
constexpr int kUsers = 8, kWalkThreads = (kUsers + kWaves) * kWave;

template <typename Y, int NK>
__global__ __launch_bounds__(kWalkThreads) __attribute__((amdgpu_waves_per_eu(3, 3)))
void walk_k(DeltaArgs a, DeltaPlan plan) {
  typedef Cell<bf16_t, Y, NK> C;
  constexpr int MP = C::MP, NT = 2 * NK;  // tiles of the state's columns
  __shared__ __attribute__((aligned(16))) char cells[2][C::BYTES];  // K0 and Q0: rows, by place_of
  __shared__ __attribute__((aligned(16))) Square sq;
  __shared__ __attribute__((aligned(16))) Decays de;
  __shared__ int met[kWaves], chosen;
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane % 16, q = lane / 16;
  // Unit, a sequence's head, and part of its rows.  With plan.sort the longest sequences come
  // first; those of plan.apart chunks and more have a head's rows in two parts, on one XCD.
  const int P = a.P, N = a.N;
  auto length = [&](int s) { return max(0, clamp_start(a.p, s + 1) - clamp_start(a.p, s)); };
  int unit = blockIdx.x, split = 0, before = 0, halved = plan.apart ? 0 : a.p.n;
  if (plan.sort) {
    int *const lens = reinterpret_cast<int *>(cells[0]), t = threadIdx.x;
    const int mine = t < a.p.n ? length(t) : -1;  // -1: behind all others
    lens[t] = mine;
    __syncthreads();
    for (int s = 0; s < a.p.n; s += 16) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int4 l = *reinterpret_cast<const int4 *>(lens + s + i);
        const int four[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          before += four[j] > mine || (four[j] == mine && s + i + j < t);
          halved += four[j] > (plan.apart - 1) * Q;
        }
      }
    }
  }
  const int two = min(halved, plan.halves) * a.H, round = (two + kXcds - 1) / kXcds * kXcds;
  if (unit < 2 * round) {
    split = 1 + unit / kXcds % 2;
    unit = unit / (2 * kXcds) * kXcds + unit % kXcds;
    if (unit >= two) return;
  } else {
    unit += two - 2 * round;
  }
  if (unit >= plan.units) return;
  int seq = fdiv(unit, plan.fH);
  const int h = unit - seq * a.H, slice = split == 2;
  if (plan.sort) {
    if (before == seq && (int)threadIdx.x < a.p.n) chosen = threadIdx.x;
    __syncthreads();
    seq = __builtin_amdgcn_readfirstlane(chosen);
  }
  const int begin = clamp_start(a.p, seq), len = length(seq);
  const int chunks = (len + Q - 1) / Q;
  const int first = 4 * slice, users = split == 1 ? 4 : P / 16 - first;
  const int row = batch_row(a.p, seq, h == 0 && slice == 0 && threadIdx.x == 0);
  if (row < 0) return;

  if (wave >= kUsers) {
    __builtin_amdgcn_s_setprio(2);  // what the others wait for
    const int tid = threadIdx.x - kUsers * kWave, w4 = wave - kUsers;
    const int64_t rK = (int64_t)a.H * N;
    constexpr int NV = 4 * NK, RB = kThreads / NV, NL = Q / RB;  // granules of a row, rows a load, loads
    const int trow = tid / NV, g = tid % NV;
    const int at = (int)((trow * rK + 8 * g) * 2);
    const uint16_t *pK = (const uint16_t *)a.k + begin * rK + (int64_t)h * N, *pQ = (const uint16_t *)a.q + begin * rK + (int64_t)h * N;
    const float *pa = a.alpha + (int64_t)begin * a.H + h, *pb = a.beta + (int64_t)begin * a.H + h;
    Rows<bf16_t> k[NL], x[NL];
    float al = 1.f, be = 0.f;
    int rem = len, loaded = 0;  // tokens from the chunk to be loaded next, of the one loaded last
    auto load = [&]() {
      const int m = loaded = min(rem, Q);
      rem -= Q;
      const size_t n = m > 0 ? (size_t)((m - 1) * rK + N) * 2 : 0;
      const auto bK = buffer_of(pK, n), bQ = buffer_of(pQ, n);
#pragma unroll
      for (int i = 0; i < NL; ++i) k[i].load(bK, at, (int)(i * RB * rK * 2));
#pragma unroll
      for (int i = 0; i < NL; ++i) x[i].load(bQ, at, (int)(i * RB * rK * 2));
      const size_t ng = m > 0 ? (size_t)((m - 1) * (int64_t)a.H + 1) * 4 : 0;
      al = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buffer_of(pa, ng), lane * a.H * 4, 0, 0));
      be = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buffer_of(pb, ng), lane * a.H * 4, 0, 0));
      pK += Q * rK, pQ += Q * rK, pa += (int64_t)Q * a.H, pb += (int64_t)Q * a.H;
    };
    if (tid < kWaves) met[tid] = 0;
    if (chunks) load();
    lds_barrier();
    // The four waves meet without the others: everyone says how often and waits for all four.
    // A wave's LDS accesses are done in their order.
    int often = 0;
    auto meet = [&]() {
      ++often;
      asm volatile("" ::: "memory");
      __hip_atomic_store(&met[w4], often, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      while (__any(__hip_atomic_load(&met[lane % kWaves], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) < often)) {
      }
      asm volatile("" ::: "memory");
    };
    // The next chunk's, by the wave that has the fewest tiles of the inverse.
    float eg, left;
    auto decays = [&]() {
      if (w4 == 3) make_decays(de, al, be, loaded, lane, eg, left);
    };
    decays();
    for (int c = 0; c < chunks; ++c) {
      char *const cell = cells[c & 1];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        k[i].stage(cell + C::K0 + place_of<NK>(trow + i * RB, g), 0);
        x[i].stage(cell + C::Q0 + place_of<NK>(trow + i * RB, g), 0);
      }
      if (w4 == 3) {
        float *const e = reinterpret_cast<float *>(cell + C::G0);
        e[lane] = eg, e[Q + lane] = left;
      }
      load();
      meet();
      make_cell<bf16_t, Y, NK>(cell + C::K0, sq, de, cell + C::A0, cell + C::P0, nullptr, false, w4, lane, meet, decays);
      lds_barrier();
    }
    return;
  }

  if (wave >= users) {
    for (int c = 0; c <= chunks; ++c) lds_barrier();
    return;
  }
  // The state, transposed: tile 2 s + m, row 4 q + i is column 32 s + 8 q + 4 m + i.
  floatx4 S[NT];
  const int col = (first + wave) * 16;  // the wave's first row of the state
  const size_t tile0 = ((size_t)row * a.H + h) * P * N + (size_t)(col + r) * N + 8 * q;
  const bool known = a.initial && (!a.p.resume || a.p.resume[seq]);
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    S[m] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (known) {
      const float4 v = ld4(a.initial + tile0 + 32 * (m / 2) + 4 * (m % 2));
      S[m] = floatx4{v.x, v.y, v.z, v.w};
    }
  }
  const int64_t rV = (int64_t)a.H * P;
  const char *pV = (const char *)((const uint16_t *)a.v + begin * rV + (int64_t)h * P + col);
  char *pY = (char *)((Y *)a.y + begin * rV + (int64_t)h * P + col);
  const int oV = (int)((4 * q * rV + r) * 2), oY = (int)((r * rV + 4 * q) * sizeof(Y));
  int rem = len;  // of the chunk to be loaded next
  auto rows_v = [&](const void *p, int esize) {
    const int m = min(rem, Q);
    return buffer_of(p, m > 0 ? (size_t)((m - 1) * rV + 16) * esize : 0);
  };
  uint16_t v[4][4];
  auto load_v = [&]() {
    const auto b = rows_v(pV, 2);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[t][i] = __builtin_amdgcn_raw_buffer_load_b16(b, oV, (int)((16 * t + i) * rV * 2), 0);
  };
  if (chunks) load_v();
  lds_barrier();  // the makers' counter is there
  // Rows r of a tile of tokens and granule q; for the transposing reads, four rows 4 q .. + 3
  // and granules 0 to 3.
  int atK[NK], atT[NK];
#pragma unroll
  for (int s = 0; s < NK; ++s)
    atK[s] = place_of<NK>(r, 4 * s + q), atT[s] = C::K0 + place_of<NK>(4 * q + r / 4, 4 * s + r % 4);
  for (int c = 0; c < chunks; ++c) {
    lds_barrier();  // the cell is there, and every wave is done with the one before
    const char *const now = cells[c & 1];
    auto frag = [&](int at) {
      Frag f;
      f.v = *reinterpret_cast<const s16x8 *>(now + at + lane * 16);
      return f;
    };
    const float *const G = reinterpret_cast<const float *>(now + C::G0);
    const auto bY = rows_v(pY, sizeof(Y));  // rows past the end are not written
    rem -= Q;
    pV += Q * rV * 2, pY += Q * rV * sizeof(Y);
    floatx4 X[4], O[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) X[t] = O[t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      Frag sf[3], kf[4], qf[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        kf[t].v = *reinterpret_cast<const s16x8 *>(now + C::K0 + atK[s] + 16 * t * 64 * NK);
        qf[t].v = *reinterpret_cast<const s16x8 *>(now + C::Q0 + atK[s] + 16 * t * 64 * NK);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t w0[3], w1[3];
        pieces<3>(S[2 * s + m][0], S[2 * s + m][1], w0);
        pieces<3>(S[2 * s + m][2], S[2 * s + m][3], w1);
#pragma unroll
        for (int u = 0; u < 3; ++u) sf[u].w[2 * m] = w0[u], sf[u].w[2 * m + 1] = w1[u];
      }
#pragma unroll
      for (int u = 2; u >= 0; --u)
#pragma unroll
        for (int t = 0; t < 4; ++t) X[t] = mfma32(kf[t], sf[u], X[t]);
#pragma unroll
      for (int u = MP - 1; u >= 0; --u)
#pragma unroll
        for (int t = 0; t < 4; ++t) O[t] = mfma32(sf[u], qf[t], O[t]);
    }
    Frag rf[2][3];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float4 eg = ld4(G + 16 * t + 4 * q);
      const float e4[4] = {eg.x, eg.y, eg.z, eg.w};
      float d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = fmaf(-e4[i], X[t][i], lower((uint32_t)v[t][i]));
      uint32_t w0[3], w1[3];
      pieces<3>(d[0], d[1], w0);
      pieces<3>(d[2], d[3], w1);
#pragma unroll
      for (int u = 0; u < 3; ++u) rf[t / 2][u].w[t % 2 * 2] = w0[u], rf[t / 2][u].w[t % 2 * 2 + 1] = w1[u];
    }
    load_v();
    floatx4 U[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) U[t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 2; u >= 0; --u) {
      Frag af[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) af[i] = frag(C::A0 + (u * kSteps + i) * kFrag);
#pragma unroll
      for (int w = 2 - u; w >= 0; --w)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int t = 2 * s; t < 4; ++t) U[t] = mfma32(af[t < 2 ? t : 2 * t - 2 + s], rf[s][w], U[t]);
    }
    Frag uf[2][MP], wf[2][3];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float4 left = ld4(G + Q + 16 * t + 4 * q);
      const floatx4 x = U[t];
      uint32_t p0[MP], p1[MP];
      pieces<MP>(x[0], x[1], p0);
      pieces<MP>(x[2], x[3], p1);
#pragma unroll
      for (int u = 0; u < MP; ++u) uf[t / 2][u].w[t % 2 * 2] = p0[u], uf[t / 2][u].w[t % 2 * 2 + 1] = p1[u];
      uint32_t w0[3], w1[3];
      pieces<3>(x[0] * left.x, x[1] * left.y, w0);
      pieces<3>(x[2] * left.z, x[3] * left.w, w1);
#pragma unroll
      for (int u = 0; u < 3; ++u) wf[t / 2][u].w[t % 2 * 2] = w0[u], wf[t / 2][u].w[t % 2 * 2 + 1] = w1[u];
    }
    const float whole = G[Q - 1];
#pragma unroll
    for (int ts = 0; ts < 2; ++ts)
#pragma unroll
      for (int m = 0; m < NT; m += 4) {
        Frag kt[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) kt[j].h[e] = read_tr(now + atT[(m + j) / 2] + (2 * ts + e) * 16 * 64 * NK + 8 * (j % 2));
        if (ts == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) S[m + j] *= whole;
        }
#pragma unroll
        for (int u = 2; u >= 0; --u)
#pragma unroll
          for (int j = 0; j < 4; ++j) S[m + j] = mfma32(kt[j], wf[ts][u], S[m + j]);
      }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float eg = G[16 * t + r];
      O[t] *= eg;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int w = MP - 1; w >= 0; --w) {
        Frag pf[4];
#pragma unroll
        for (int t = 2 * s; t < 4; ++t) pf[t] = frag(C::P0 + (w * kSteps + (t < 2 ? t : 2 * t - 2 + s)) * kFrag);
#pragma unroll
        for (int u = MP - 1 - w; u >= 0; --u)
#pragma unroll
          for (int t = 2 * s; t < 4; ++t) O[t] = mfma32(uf[s][u], pf[t], O[t]);
      }
    // This lane holds rows 4 q .. + 3 of the wave's, for token 16 t + r.
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const floatx4 o = O[t];
      // All of it in the vector offset: a 16-byte store with a scalar one may send the registers'
      // next values if an instruction rewrites them right behind it.
      const int to = oY + (int)(16 * t * rV * sizeof(Y));
      if constexpr (sizeof(Y) == 2)
        __builtin_amdgcn_raw_buffer_store_b64(i32x2{(int)pack_bf16(o[0], o[1]), (int)pack_bf16(o[2], o[3])}, bY, to, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b128(
            i32x4{__float_as_int(o[0]), __float_as_int(o[1]), __float_as_int(o[2]), __float_as_int(o[3])}, bY, to, 0, 0);
    }
  }
#pragma unroll
  for (int m = 0; m < NT; ++m)
    st4(a.state + tile0 + 32 * (m / 2) + 4 * (m % 2), make_float4(S[m][0], S[m][1], S[m][2], S[m][3]));
}

// Cells of one pass: 256 MB of them at most, so that long prompts need no more than that (24
// prompts of 16384 tokens by cells_k and chain_k: 128 MB 683 us, 256 MB 660, 768 MB 616), but eight
// chunks of all heads at least, whose states each pass reads and writes (float32 records, 128 x 128:
// 2048 tokens of 400 heads 1399 us, 1469 in 256 MB; 1024 of 1000 heads 1667, 2038).
constexpr size_t kCells = 256u << 20;

// Whether a call walks: heads of all sequences, and their rows, that give at least half of
// the CUs something to do.  Sequences of 640 tokens, 32 heads (the other form in brackets):
// 128 rows, four of them 54 us (77), two 48 (43); 64 rows, four 49 (58); 32 rows, four of 1024
// tokens 67 (65), 24 of 683 162 (338).  And a chunk or so a sequence, where one launch and no
// workspace count: 37 tokens 12.5 (16.1), three of 64 13.5 (17.2), but one of 128 16.4 (16.8)
// and 16.8 (13.7) in a graph.  The lengths are on the device, so a prompt that outlasts the others walks
// with them: one of 8192 with three of ten tokens 527 (287), with 15 528 (312), alone 270; four
// of 4000 288 (503).
// Heads past what a launch of workgroups so large holds go by the other form, in passes.
constexpr int64_t kWalk = 128, kWalkRows = 64;

// How a call would walk, and its workgroups.
int64_t walk_plan(const DeltaArgs &a, DeltaPlan &p) {
  p.fH = make_fastdiv((uint32_t)a.H);
  const int64_t units = (int64_t)a.p.n * a.H, all = items_of(a.p.tokens, a.p.n, Q);
  // By length where it can matter: 24 sequences of 64 tokens take 46 us without it, 62 with it.
  p.sort = units >= kCus && a.p.n > 1 && a.p.n <= kWalkThreads && all >= 4 * (int64_t)a.p.n;
  p.apart = units < kCus ? 0 : p.sort ? (int)std::max<int64_t>(all * a.H / kCus, 1) : 0x1000000;
  p.halves = a.P <= 64 ? 0 : p.apart ? (int)std::min<int64_t>(a.p.n, all / p.apart) : a.p.n;  // more only with offsets that fall
  p.units = (int)units;
  return units + (int64_t)p.halves * a.H + 2 * kXcds;
}

template <typename R>
bool walks(const DeltaArgs &a) {
  const int64_t units = (int64_t)a.p.n * a.H;
  const bool brief = a.p.tokens <= Q * std::min(a.p.n, 3) && a.P >= kWalkRows;
  if (!(sizeof(R) == 2 && a.N >= 64 && (brief || (units >= kWalk && units * a.P >= kWalk * kWalkRows)))) return false;
  DeltaPlan p{};
  return walk_plan(a, p) * kWalkThreads < (int64_t)1 << 32;
}

template <typename Y, int NK>
int launch_walk(const DeltaArgs &a, hipStream_t st) {
  DeltaPlan p{};
  const int64_t blocks = walk_plan(a, p);
  hipLaunchKernelGGL((walk_k<Y, NK>), dim3((uint32_t)blocks), dim3(kWalkThreads), 0, st, a, p);
  return (int)hipGetLastError();
}

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
  if (walks<R>(a)) return 0;
  if (a.N <= 32) return (size_t)places_of<R, Y, 1>(a) * a.H * Cell<R, Y, 1>::BYTES;
  if (a.N == 64) return (size_t)places_of<R, Y, 2>(a) * a.H * Cell<R, Y, 2>::BYTES;
  return (size_t)places_of<R, Y, 4>(a) * a.H * Cell<R, Y, 4>::BYTES;
}

template <typename R, typename Y>
int launch_n(const DeltaArgs &a, hipStream_t st) {
  if constexpr (sizeof(R) == 2)
    if (walks<R>(a)) return a.N == 64 ? launch_walk<Y, 2>(a, st) : launch_walk<Y, 4>(a, st);
  // 32 rows of float32 records, which leave one workgroup to a CU, once every CU has one:
  // four sequences of 512 tokens, 32 heads, 128 x 128, 105 us, 131 with 16; one of 2048, 161 and 141.
  if constexpr (sizeof(R) == 4)
    if (a.P % 32 == 0 && (int64_t)a.p.n * a.H * (a.P / 16) >= 2 * kCus) {
      if (a.N <= 32) return launch<R, Y, 1, 2>(a, st);
      return a.N == 64 ? launch<R, Y, 2, 2>(a, st) : launch<R, Y, 4, 2>(a, st);
    }
  if (a.N <= 32) return launch<R, Y, 1, 1>(a, st);
  return a.N == 64 ? launch<R, Y, 2, 1>(a, st) : launch<R, Y, 4, 1>(a, st);
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
