// Microscaled 4-bit floating point (MXFP4): the packer, its inverse, and
// products with bf16 or MXFP4 activations.
//
// y_t[o] = sum over blocks B of 32 columns of 2^(s_oB - 127) sum_{k in B} c_ok x_tk.
// A lane's piece is one block of one row, so the conversions take the block's
// scale as their operand (bf16 activations: v_cvt_scalef32_pk_bf16_fp4, exact),
// and so does the matrix core (MXFP4 activations: v_mfma_scale, products exact,
// sums fp32).
#include <hip/hip_runtime.h>

#include "step.h"

namespace dc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

#include "mx4_common.h"

constexpr int kFp4 = 4;   // the matrix core's format number

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ v8i piece(uint4 w) { return v8i{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0}; }

// ------------------------------------------------------------------ packer
// A wave takes 16 rows x 512 columns, lane l row l%16 and block l/16 of each
// 128 columns: loads are 256 bytes of a row, stores whole KiB of codes.
// Bound by HBM: 4096 x 14336 (0.15 GB) 29 us, 5.1 TB/s.
__global__ void __launch_bounds__(256) k_mx4_pack(const uint16_t* __restrict__ X, int64_t stride, uint8_t* __restrict__ dst,
                                                  uint32_t* __restrict__ flag, int rows, int cols) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int gc = cols / 128, hc = (gc + 3) / 4;
  const int T = blockIdx.x / hc * 4 + wave, H = blockIdx.x % hc;
  if (T * 16 >= rows) return;
  const int row = T * 16 + (lane & 15);
  const bool have = row < rows;
  const uint16_t* src = X + (int64_t)(have ? row : rows - 1) * stride + 512 * H + 32 * (lane >> 4);
  uint4 x[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = min(4 * H + j, gc - 1) - 4 * H;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[j][i] = *reinterpret_cast<const uint4*>(src + 128 * g + 8 * i);
  }
  uint32_t scales = 0;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (4 * H + j >= gc) break;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u[4] = {x[j][i].x, x[j][i].y, x[j][i].z, x[j][i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max2(m, u[e] & 0x7FFF7FFFu);
    }
    m = max(m & 0xFFFFu, m >> 16);
    const uint32_t ex = m >> 7;   // the exponent field of the largest
    uint32_t s = ex > 2 ? ex - 2 : 0;
    if (ex == 255) s = 255, bad |= have;
    uint32_t w[4];
    const float f = __uint_as_float(s << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t r = 0;
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x[j][i].x), f, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x[j][i].y), f, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x[j][i].z), f, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x[j][i].w), f, 3);
      w[i] = have && ex < 255 ? r : 0u;
    }
    scales |= (have ? s : 0u) << (8 * j);
    *reinterpret_cast<uint4*>(dst + ((size_t)T * gc + 4 * H + j) * 1024 + lane * 16) = uint4{w[0], w[1], w[2], w[3]};
  }
  const size_t codes = (size_t)((rows + 15) / 16) * gc * 1024;
  *reinterpret_cast<uint32_t*>(dst + codes + ((size_t)T * hc + H) * 256 + lane * 4) = scales;
  if (bad && flag) atomicOr(flag, 1u);
}

__global__ void k_mx4_flag(uint32_t* flag) { *flag = 0; }

// The same tiles the other way.  Lane l takes 8 codes of row l/4 at a time, so
// that 4 lanes write a block's 64 bytes side by side (a lane's whole block is 64
// bytes in 4 stores, each of 16 bytes of as many cache lines: 40 us for 4096 x 14336
// where this takes 24).
__global__ void __launch_bounds__(256) k_mx4_dequant(const uint8_t* __restrict__ w, uint16_t* __restrict__ X, int64_t stride,
                                                     int rows, int cols) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int gc = cols / 128, hc = (gc + 3) / 4;
  const int T = blockIdx.x / hc * 4 + wave, H = blockIdx.x % hc;
  if (T * 16 >= rows) return;
  const int i = lane >> 2, e = lane & 3, row = T * 16 + i;
  const uint8_t* code = w + ((size_t)T * gc + 4 * H) * 1024 + i * 16 + e * 4;
  const uint8_t* scale = w + (size_t)((rows + 15) / 16) * gc * 1024 + ((size_t)T * hc + H) * 256 + i * 4;
  const int n = min(4, gc - 4 * H);
  uint32_t s[4], c[4][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    s[q] = *reinterpret_cast<const uint32_t*>(scale + q * 64);
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j][q] = *reinterpret_cast<const uint32_t*>(code + min(j, n - 1) * 1024 + q * 256);
  }
  if (row >= rows) return;
  uint16_t* dst = X + (int64_t)row * stride + 512 * H + 8 * e;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (j < n) *reinterpret_cast<uint4*>(dst + 128 * j + 32 * q) = __builtin_bit_cast(uint4, codes8(c[j][q], scale_of(s[q] >> (8 * j) & 255u)));
}

// ---------------------------------------------------------------- products
// Block: RT 16-row tiles of the matrix x TT 16-token tiles, all columns; NW
// waves take the 128-column groups in turn and add their sums through LDS: one
// launch, no workspace.  Lane l holds row (token) l%16 and block l/16 of 128
// columns; result: token l%16, rows 4(l/16) .. +4.
// Bound by latency (4096 x 4096, 1 token: 3.4 us, of which the weights at HBM's rate
// take 1.7) and for more tokens by accesses of the L1 (the rule's times, below).
template <int RT, int TT, int NW, bool XQ>
__global__ void __launch_bounds__(64 * NW, NW / 4) k_mx4(Mx4Args a) {
  __shared__ float red[NW][RT * 16][TT * 16 + 1];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int r0 = blockIdx.x * RT, t0 = blockIdx.y * TT;   // first tiles
  const int gc = a.in / 128, hc = (gc + 3) / 4, rts = a.out / 16, tts = (a.T + 15) / 16;
  const uint8_t* ws = a.w + (size_t)rts * gc * 1024;
  const uint8_t* xs = a.xq + (size_t)tts * gc * 1024;
  f32x4 acc[RT][TT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint64_t large = 0;
  for (int g = wave; g < gc; g += NW) {
    const int H = g >> 2, j8 = 8 * (g & 3);
    uint4 w[RT];
    uint32_t s[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const size_t T = min(r0 + r, rts - 1);
      w[r] = *reinterpret_cast<const uint4*>(a.w + (T * gc + g) * 1024 + lane * 16);
      s[r] = *reinterpret_cast<const uint32_t*>(ws + (T * hc + H) * 256 + lane * 4) >> j8 & 255u;
    }
    if constexpr (XQ) {
      uint4 x[TT];
      uint32_t xsc[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const size_t T = min(t0 + t, tts - 1);
        x[t] = *reinterpret_cast<const uint4*>(a.xq + (T * gc + g) * 1024 + lane * 16);
        xsc[t] = *reinterpret_cast<const uint32_t*>(xs + (T * hc + H) * 256 + lane * 4) >> j8 & 255u;
      }
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          acc[r][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(piece(w[r]), piece(x[t]), acc[r][t], kFp4, kFp4, 0,
                                                                      (int)s[r], 0, (int)xsc[t]);
    } else {
      bf16x8 b[TT][4];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint16_t* xp = a.x + (size_t)min(16 * (t0 + t) + (lane & 15), a.T - 1) * a.in + 128 * g + 32 * (lane >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[t][j] = *reinterpret_cast<const bf16x8*>(xp + 8 * j);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float f = scale_unless_large(s[r], &large);
        const uint32_t u[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 c = codes8(u[j], f);
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[r][t] = mfma(c, b[t][j], acc[r][t]);
        }
      }
    }
  }
  if constexpr (!XQ) {
    if (large) add_large<RT, TT>(a, acc, r0, 16 * t0, wave, NW);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][16 * r + 4 * (lane >> 4) + i][16 * t + (lane & 15)] = acc[r][t][i];
  __syncthreads();
  for (int e = tid; e < RT * 16 * TT * 16; e += 64 * NW) {   // consecutive threads: consecutive rows of a token
    const int row = e % (RT * 16), tok = e / (RT * 16);
    float v = 0.f;
#pragma unroll
    for (int n = 0; n < NW; ++n) v += red[n][row][tok];
    if (16 * t0 + tok < a.T && 16 * r0 + row < a.out)
      a.y[(size_t)(16 * t0 + tok) * a.out + 16 * r0 + row] = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
}

template <int RT, int TT, bool XQ>
void go(const Mx4Args& a) {
  const dim3 g((unsigned)((a.out / 16 + RT - 1) / RT), (unsigned)((a.T + TT * 16 - 1) / (TT * 16)));
  hipLaunchKernelGGL((k_mx4<RT, TT, 8, XQ>), g, dim3(512), 0, reinterpret_cast<hipStream_t>(a.stream), a);
}

}  // namespace

// Up to 16 tokens: row tiles a block, by the accesses of the fullest CU's L1 (17 for
// a row tile, 4 for a token's x) and the rounds of 256 blocks.  us, 1 / 7 / 16
// tokens: 4096 x 4096 16 rows 3.4 / 4.4 / 5.9, 48 rows 4.7 / 5.3 / 6.8; 11008 x 4096
// 16 rows 5.7 / 8.9 / 13.4, 48 rows 4.8 / 5.5 / 7.2; 32000 x 4096 32 rows 11.9 / 12.7
// / 18.6, 64 rows 13.1 / 13.3 / 15.5.
int mx4_row_tiles(int32_t out, int32_t T) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int rt = 1; rt <= 4; ++rt) {
    const int64_t cost = ((out / 16 + rt - 1) / rt + 255) / 256 * (17 * rt + 4 * T);
    if (cost < least) least = cost, best = rt;
  }
  return best;
}

int launch_mx4(const Mx4Args& a) {
  if (a.T > 16) return launch_mx4_few(a);
  switch (mx4_row_tiles(a.out, a.T)) {
    case 1: go<1, 1, false>(a); break;
    case 2: go<2, 1, false>(a); break;
    case 3: go<3, 1, false>(a); break;
    default: go<4, 1, false>(a); break;
  }
  return (int)hipGetLastError();
}

// The block's tile, rows x tokens, by what the fullest CU takes: `first` for the
// call, and for each of its tiles `end` and `step` for 128 columns, in ns.
// Measured, us, where two tiles part (weights in the caches):
//   4096 x 4096: 32 tokens 16x32 3.4, 32x32 3.7; 64 tokens 16x32 4.3, 32x32 3.9;
//   128 tokens 32x64 5.1, 32x32 5.3, 64x64 6.3; 256 tokens 64x64 6.6, 32x64 7.1;
//   512 tokens 64x64 9.0, 64x128 9.0, 128x128 11.7; 1024 tokens 64x128 12.8,
//   128x128 12.5; 4096 x 11008: 128 tokens 32x64 9.1, 64x64 11.4; 11008 x 4096: 64
//   tokens 64x64 6.5, 32x64 7.5 (codes drawn evenly); with normal numbers, 128x128
//   and 256x256: 4096 x 4096 2048 tokens 21.6 and 30.5, 4096 42.3 and 40.2, 8192
//   84.9 and 78.7; 11008 x 4096 2048 tokens 57 and 62, 4096 118 and 108, 8192 219
//   and 212; 32000 x 4096, 8192 tokens 588 and 516
int mx4q_tile(int32_t out, int32_t in, int32_t T) {
  constexpr struct {
    int rows, toks, first, end, step;
  } kTiles[] = {{16, 16, 2200, 0, 32}, {16, 32, 2300, 0, 35},    {32, 32, 2100, 0, 48},      {32, 64, 2600, 0, 70},
                {64, 64, 3200, 0, 92}, {64, 128, 3400, 0, 148}, {128, 128, 2000, 1600, 200}, {256, 256, 2000, 5000, 730}};
  int best = 0;
  int64_t least = INT64_MAX;
  for (int c = 0; c < 8; ++c) {
    const int64_t tiles = (int64_t)((out + kTiles[c].rows - 1) / kTiles[c].rows) * ((T + kTiles[c].toks - 1) / kTiles[c].toks);
    const int64_t cost = kTiles[c].first + (tiles + 255) / 256 * (kTiles[c].end + (int64_t)kTiles[c].step * (in / 128));
    if (cost < least) least = cost, best = c;
  }
  return best;
}

int launch_mx4q(const Mx4Args& a) {
  const int best = mx4q_tile(a.out, a.in, a.T);
  switch (best) {
    case 0: go<1, 1, true>(a); break;
    case 1: go<1, 2, true>(a); break;
    case 2: go<2, 2, true>(a); break;
    case 3: go<2, 4, true>(a); break;
    default: return launch_mx4_tiles(a, best - 4);
  }
  return (int)hipGetLastError();
}

// Pieces of 64 rows and 512 columns (columns: up to 2^31 less 128).
static unsigned pieces_of(int32_t rows, int32_t cols) { return ((unsigned)rows + 63) / 64 * (((unsigned)cols + 511) / 512); }

int launch_mx4_pack(int32_t rows, int32_t cols, const uint16_t* X, int64_t stride, uint8_t* dst, uint32_t* flag,
                    void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (flag) hipLaunchKernelGGL(k_mx4_flag, dim3(1), dim3(1), 0, st, flag);
  hipLaunchKernelGGL(k_mx4_pack, dim3(pieces_of(rows, cols)), dim3(256), 0, st, X, stride, dst, flag, rows, cols);
  return (int)hipGetLastError();
}

int launch_mx4_dequant(int32_t rows, int32_t cols, const uint8_t* w, uint16_t* X, int64_t stride, void* stream) {
  hipLaunchKernelGGL(k_mx4_dequant, dim3(pieces_of(rows, cols)), dim3(256), 0, reinterpret_cast<hipStream_t>(stream), w, X, stride, rows, cols);
  return (int)hipGetLastError();
}

}  // namespace dc
