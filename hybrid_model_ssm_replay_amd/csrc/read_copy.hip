// The read copy of some sequences, from their float32 checkpoint: what a caller that
// has written checkpoint rows itself (a prompt's scan) leaves to do.
//
// A workgroup a head, as in the kernels that read the copy; those of the other
// sequences return at once.  HBM bound: read S, write the 4-bit copy.
#include "ops.h"
#include "state_io.h"

namespace rssm {
namespace {

constexpr int kCols = 128;  // state_dim of layers with a separate read copy
constexpr int kNch = kCols / 16;

template <int RF, int RBW>
__global__ __launch_bounds__(256) void renew_read_copy_k(Shape sh, StateBufs sb, const uint8_t *mask) {
  constexpr int CM = col_map(REPLAY_FMT_F32, RF);
  typedef SIO<RF, kNch, RBW, CM> Copy;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = xcd_remap(blockIdx.x, gridDim.x);
  const int b = fdiv(tile, sh.fH), h = tile - b * sh.H;
  if (mask && !mask[b]) return;  // the whole workgroup
  const int rb0 = wave * RBW;
  const size_t head = ((size_t)b * sh.H + h) * sh.P * kCols;
  float4 s[RBW][kNch];
  load_rows_g<kNch, RBW, CM>(s, (const float *)sb.ck.data + head, rb0, lane);
  typename Copy::Raw raw;
  if constexpr (RF == REPLAY_FMT_F4E2M1_CS) Copy::prepare(raw, s, lane, wave);
  Copy::encode(raw, s, rb0, lane, SRKey{});  // rounds to nearest: the key is not read
  Copy::write(raw, sb.rd, head, rb0, lane);
}

template <int RF>
int launch(const Shape &s, const StateBufs &sb, const uint8_t *mask, hipStream_t st) {
  const dim3 grid((unsigned)((size_t)s.B * s.H)), block(256);
  if (s.P == 64)
    hipLaunchKernelGGL((renew_read_copy_k<RF, 1>), grid, block, 0, st, s, sb, mask);
  else if (s.P == 128)
    hipLaunchKernelGGL((renew_read_copy_k<RF, 2>), grid, block, 0, st, s, sb, mask);
  else
    return (int)hipErrorInvalidValue;
  return (int)hipGetLastError();
}

}  // namespace

int launch_renew_read_copy(const Shape &s, const FormatBufs &f, const uint8_t *mask, hipStream_t st) {
  if (s.N != kCols) return (int)hipErrorInvalidValue;
  if (f.read_fmt == REPLAY_FMT_F4E2M1_CS) return launch<REPLAY_FMT_F4E2M1_CS>(s, state_bufs(f), mask, st);
  return launch<REPLAY_FMT_F4E2M1_B16>(s, state_bufs(f), mask, st);
}

}  // namespace rssm
