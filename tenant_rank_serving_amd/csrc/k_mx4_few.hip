// Products of an MXFP4 matrix with bf16 activations for more than 16 tokens,
// y_t[o] = sum_k w_ok x_tk.
//
// A block takes (16 RT WR) rows x (16 TT) tokens, WR x WK waves: wave (r, c) rows
// 16 RT r .. and every WK-th 128 columns, whose sums are added through LDS at the
// end.  Matrix and activations go straight to LDS (global_load_lds), NS - 1 steps
// ahead: a KiB of x is 4 tokens x 128 columns side by side there, which are 16 cache
// lines; as operands straight from memory (16 tokens x 4 pieces of 16 bytes) each
// KiB touches 64, and a CU's L1 takes about one a cycle (32000 x 4096 with 64 tokens
// 36 us that way).  The codes become bf16 with their block's scale on the way to
// the matrix core (v_cvt_scalef32_pk_bf16_fp4, exact).  Operands as for k_mx4: lane
// l holds row (token) l%16 and columns 32(l/16) + 8j .. +8 of the 128 for product j.
//
// Measured, 32000 x 4096 with 64 tokens: 23.4 us, weights from memory at 3.0 TB/s.
// A block is alone on its CU there, and its waves meet at a barrier every 256
// columns, so what a step takes adds up: products alone 9.2 us, reading and filling
// LDS 5 to 8, launch, first loads and last sums 4.4.  Not faster: loads through
// registers (24.0), operands fetched a half step ahead and spread among the products
// (26), other first columns for every block (21.5, and 3 more for few rows), two
// waves a SIMD that take turns at reading and multiplying (26).
#include <hip/hip_runtime.h>

#include "step.h"

namespace dc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

#include "mx4_common.h"

// What a token's number in a tile is XOR-ed into the numbers of its 16-byte pieces
// as: a read serves 8 tokens' pieces of one number and 8 others' of the number 4
// above at a time (tokens 0-3, 12-15 and 4-11), which this sends to different banks.
__device__ __forceinline__ int turned(int t) { return (t & 3) | (0xD2 >> ((t >> 1) & 6) & 3) << 2; }

template <int RT, int TT, int WR, int WK, int NS>
struct FewLds {
  alignas(256) uint8_t x[NS][WK][TT * 4096];
  alignas(256) uint8_t w[NS][WK][WR][RT * 1024];
  alignas(256) uint8_t s[NS][WK][WR][RT * 256];
};

template <int RT, int TT, int WR, int WK, int NS>
__global__ void __launch_bounds__(64 * WR * WK) k_mx4_few(Mx4Args g) {
  typedef FewLds<RT, TT, WR, WK, NS> Lds;
  constexpr int kRows = 16 * RT * WR, kRed = (WK - 1) * kRows * (TT * 16 + 1) * 4;
  __shared__ union {
    Lds l;
    float red[WK > 1 ? kRed / 4 : 1];
  } sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave % WR, wk = wave / WR;
  const int r0 = blockIdx.x * RT * WR, t0 = blockIdx.y * TT * 16;   // first row tile, first token
  const int gc = g.in / 128, hc = (gc + 3) / 4, rts = g.out / 16;
  const int steps = (gc + WK - 1) / WK;

  constexpr int LX = TT * 4 / WR, L = LX + 2 * RT;   // loads of a wave and step
  static_assert(LX * WR == TT * 4, "the waves share the loads of x");
  const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)&sh.l;
  uint32_t xo[LX];   // offsets of the lane's pieces in x
#pragma unroll
  for (int i = 0; i < LX; ++i) {
    const int t = 4 * (wr * LX + i) + (lane >> 4), p = (lane & 15) ^ turned(t & 15);
    xo[i] = (uint32_t)min(t, g.T - 1 - t0) * (uint32_t)g.in * 2 + 16 * p;
  }
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(g.x) + (size_t)t0 * g.in * 2;
  const uint8_t* wsc = g.w + (size_t)rts * gc * 1024;
  const int wrow = r0 + wr * RT;
  auto load = [&](int s, int b) {
    const int c = min(s * WK + wk, gc - 1);
#pragma unroll
    for (int i = 0; i < LX; ++i)
      to_lds16(xb + (size_t)c * 256, xo[i], at + (uint32_t)offsetof(Lds, x) + (b * WK + wk) * (TT * 4096) + (wr * LX + i) * 1024);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const size_t T = min(wrow + r, rts - 1);
      to_lds16(g.w + (T * gc + c) * 1024, lane * 16,
               at + (uint32_t)offsetof(Lds, w) + ((b * WK + wk) * WR + wr) * (RT * 1024) + r * 1024);
      to_lds4(wsc + (T * hc + (c >> 2)) * 256, lane * 4,
              at + (uint32_t)offsetof(Lds, s) + ((b * WK + wk) * WR + wr) * (RT * 256) + r * 256);
    }
  };

  f32x4 acc[RT][TT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) load(s, s);
  int b = 0;
  uint64_t large = 0;
  for (int s = 0; s < steps; ++s) {
    wait_barrier<(NS - 2) * L>();   // this step's tiles are here, the last one's have been read
    load(s + NS - 1, b == 0 ? NS - 1 : b - 1);
    const int c = s * WK + wk;
    if (c < gc) {
      const uint8_t* x = sh.l.x[b][wk];
      bf16x8 xv[TT][4];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xv[t][j] = *reinterpret_cast<const bf16x8*>(x + t * 4096 + (lane & 15) * 256 + (((lane >> 4) * 4 + j) ^ turned(lane & 15)) * 16);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const uint4 w = *reinterpret_cast<const uint4*>(sh.l.w[b][wk][wr] + r * 1024 + lane * 16);
        const uint32_t sc = *reinterpret_cast<const uint32_t*>(sh.l.s[b][wk][wr] + r * 256 + lane * 4);
        const float f = scale_unless_large(sc >> (8 * (c & 3)) & 255u, &large);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 cv = codes8(u[j], f);
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cv, xv[t][j], acc[r][t], 0, 0, 0);
        }
      }
    }
    b = b + 1 == NS ? 0 : b + 1;
  }
  if (large) add_large<RT, TT>(g, acc, wrow, t0, wk, WK);
  wait_barrier<0>();   // nothing is on its way to LDS, and everyone has left it

  if constexpr (WK > 1) {
    if (wk > 0) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sh.red[((wk - 1) * kRows + (wr * RT + r) * 16 + 4 * (lane >> 4) + i) * (TT * 16 + 1) + 16 * t + (lane & 15)] = acc[r][t][i];
    }
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < WK - 1; ++n)
            acc[r][t][i] += sh.red[(n * kRows + (wr * RT + r) * 16 + 4 * (lane >> 4) + i) * (TT * 16 + 1) + 16 * t + (lane & 15)];
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = 16 * (wrow + r) + 4 * (lane >> 4);
    if (row >= g.out) continue;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int tok = t0 + 16 * t + (lane & 15);
      if (tok < g.T)
        *reinterpret_cast<uint2*>(g.y + (size_t)tok * g.out + row) =
            uint2{pack2(acc[r][t][0], acc[r][t][1]), pack2(acc[r][t][2], acc[r][t][3])};
    }
  }
}

template <int RT, int TT, int WR, int WK, int NS>
void go(const Mx4Args& a) {
  const dim3 b((unsigned)((a.out + 16 * RT * WR - 1) / (16 * RT * WR)), (unsigned)((a.T + TT * 16 - 1) / (TT * 16)));
  hipLaunchKernelGGL((k_mx4_few<RT, TT, WR, WK, NS>), b, dim3(64 * WR * WK), 0, reinterpret_cast<hipStream_t>(a.stream), a);
}

}  // namespace

// The block's tile by what the fullest CU takes: n blocks at `step` ns for 128
// columns each, and `first` for the call; a block of 64 x 32 alone takes as long as
// 1.55 of several.  us, where two part: 4096 x 4096: 32 tokens 32x16 5.7, 32x32 7.3;
// 64 tokens 32x32 7.5, 32x16 8.1, 64x32 of 8 waves 8.6; 128 tokens 8.9 of 8 waves,
// 11.0 of 4; 256 tokens 16.5 and 13.4, 128x64 18.6; 512 tokens 64x32 24.9, 128x64
// 19.6; 11008 x 4096, 32 tokens 64x32 of 8 waves 9.4, of 4 11.0, 32x16 11.3
int mx4_few_tile(int32_t out, int32_t in, int32_t T) {
  constexpr struct {
    int rows, toks, first, step, least;   // least: hundredths of a block
  } kTiles[] = {{32, 16, 2200, 88, 100}, {32, 32, 1500, 183, 100}, {64, 32, 1500, 235, 100}, {64, 32, 1500, 186, 155}, {128, 64, 1000, 540, 100}};
  int best = 0;
  int64_t least = INT64_MAX;
  for (int c = 0; c < 5; ++c) {
    const int64_t blocks = (int64_t)((out + kTiles[c].rows - 1) / kTiles[c].rows) * ((T + kTiles[c].toks - 1) / kTiles[c].toks);
    int64_t n = (blocks + 255) / 256 * 100;
    if (n < kTiles[c].least) n = kTiles[c].least;
    const int64_t cost = kTiles[c].first + n * kTiles[c].step * (in / 128) / 100;
    if (cost < least) least = cost, best = c;
  }
  return best;
}

int launch_mx4_few(const Mx4Args& a) {
  switch (mx4_few_tile(a.out, a.in, a.T)) {
    case 0: go<1, 1, 2, 4, 3>(a); break;
    case 1: go<1, 2, 2, 4, 3>(a); break;
    case 2: go<2, 2, 2, 4, 2>(a); break;
    case 3: go<2, 2, 2, 2, 3>(a); break;
    default: go<2, 4, 4, 2, 3>(a); break;
  }
  return (int)hipGetLastError();
}

}  // namespace dc
