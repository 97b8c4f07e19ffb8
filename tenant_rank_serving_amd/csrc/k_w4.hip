// Products with a 4-bit backbone: y_t[o] = sum_g s_og sum_{k in g} (q_ok - z_og) x_tk
// over groups of 128 inputs, and the packer of that format from a bf16 matrix.
//
// A nibble or-ed into the low mantissa bits of the bf16 number 128 is the
// value 128 + q exactly, so unpacking two codes is one shift and one and-or,
// and the matrix core multiplies them with the bf16 activations as they are:
//   sum_k (q_k - z) x_k = sum_k (128 + q_k) x_k - (128 + z) sum_k x_k.
// The sums of x come from the matrix core too, against a tile of ones (the
// same for every row).  What the 128 adds cancels to 2^-24 * 128 of the sum of
// |x|: 2^-17 of it, below the output's rounding of 2^-8.
#include <hip/hip_runtime.h>

#include "layer.h"

namespace dc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float h2f(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }

__device__ __forceinline__ bf16x8 codes8(uint32_t w) {
  uint4 r;
  r.x = (w & 0x000F000Fu) | 0x43004300u;
  r.y = ((w >> 4) & 0x000F000Fu) | 0x43004300u;
  r.z = ((w >> 8) & 0x000F000Fu) | 0x43004300u;
  r.w = ((w >> 12) & 0x000F000Fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8, r);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Block: RT 16-row tiles of the matrix x TT 16-token tiles, all inputs; NW
// waves take the 128-groups in turn (wave w: groups w, w + NW, ..), U of its
// groups at a time with all their loads issued first, and add their sums
// through LDS, so a call is one launch without a workspace.
// Operands: lane l holds row (token) l%16 and columns 32(l/16) + 8j .. +8 of
// the group for op j; result: token l%16, rows 4(l/16) .. +4.
template <int RT, int TT, int NW, int U>
__global__ void __launch_bounds__(64 * NW, NW / 4) k_w4(const uint8_t* __restrict__ wq, const uint16_t* __restrict__ x,
                                                        uint16_t* __restrict__ y, int out, int in, int T) {
  __shared__ float red[NW][RT * 16][TT * 16 + 1];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int r0 = blockIdx.x * RT * 16, t0 = blockIdx.y * TT * 16;
  const int gi = in / kGroup;
  const uint32_t* sz = reinterpret_cast<const uint32_t*>(wq + (size_t)out * in / 2);
  bf16x8 ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.f;
  const uint16_t* xp[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
    xp[t] = x + (size_t)min(t0 + 16 * t + (lane & 15), T - 1) * in + 32 * (lane >> 4);
  const int rt = min(RT, (out - r0) / 16);   // out is a multiple of 128 rows: whole tiles
  f32x4 tot[RT][TT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) tot[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int g0 = wave; g0 < gi; g0 += NW * U) {
    uint4 w[U][RT], s4[U][RT];
    bf16x8 b[U][TT][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = min(g0 + u * NW, gi - 1);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int row = r0 + 16 * min(r, rt - 1);
        w[u][r] = *reinterpret_cast<const uint4*>(wq + ((size_t)(row / 16) * gi + g) * 1024 + lane * 16);
        s4[u][r] = *reinterpret_cast<const uint4*>(sz + (size_t)g * out + row + 4 * (lane >> 4));
      }
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) b[u][t][j] = *reinterpret_cast<const bf16x8*>(xp[t] + (size_t)g * kGroup + 8 * j);
    }
    __builtin_amdgcn_sched_barrier(0);   // the loads stay ahead of the products
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (U > 1 && g0 + u * NW >= gi) break;
      f32x4 xs[TT];   // the group's sums of x, the same for every row
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        xs[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) xs[t] = mfma(ones, b[u][t][j], xs[t]);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const uint32_t ww[4] = {w[u][r].x, w[u][r].y, w[u][r].z, w[u][r].w};
        const uint32_t zz[4] = {s4[u][r].x, s4[u][r].y, s4[u][r].z, s4[u][r].w};
        f32x4 acc[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 c = codes8(ww[j]);
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[t] = mfma(c, b[u][t][j], acc[t]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = h2f(zz[i] & 0xFFFFu), z = 128.f + h2f(zz[i] >> 16);
#pragma unroll
          for (int t = 0; t < TT; ++t) tot[r][t][i] += s * (acc[t][i] - z * xs[t][i]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][16 * r + 4 * (lane >> 4) + i][16 * t + (lane & 15)] = tot[r][t][i];
  __syncthreads();
  for (int e = tid; e < RT * 16 * TT * 16; e += 64 * NW) {   // consecutive threads: consecutive rows of a token
    const int row = e % (RT * 16), tok = e / (RT * 16);
    float v = 0.f;
#pragma unroll
    for (int n = 0; n < NW; ++n) v += red[n][row][tok];
    if (t0 + tok < T && row < 16 * rt) y[(size_t)(t0 + tok) * out + r0 + row] = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
}

// ------------------------------------------------------------------ packer
// One wave per (row, 128-group), two columns a lane: the quantizer of dc_pack
// at 4 bits (range with 0, fp16 scale, integer zero, round half to even), in
// fp64 from the bf16 values.  The words are or-ed together across the 4 lanes
// that share one.
__global__ void __launch_bounds__(256) k_w4_pack(const uint16_t* __restrict__ W, uint8_t* __restrict__ dst,
                                                 uint32_t* __restrict__ flag, int out, int in) {
  const int gi = in / kGroup, lane = threadIdx.x & 63;
  const size_t item = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= (size_t)out * gi) return;
  const int row = (int)(item / gi), g = (int)(item % gi);
  const uint32_t two = *reinterpret_cast<const uint32_t*>(W + (size_t)row * in + (size_t)g * kGroup + 2 * lane);
  const float a = __uint_as_float(two << 16), b = __uint_as_float(two & 0xFFFF0000u);
  const bool bad = !(__builtin_isfinite(a) && __builtin_isfinite(b));
  float mn = fminf(fminf(a, b), 0.f), mx = fmaxf(fmaxf(a, b), 0.f);
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    mn = fminf(mn, __shfl_xor(mn, m));
    mx = fmaxf(mx, __shfl_xor(mx, m));
  }
  uint16_t sh = f64_to_f16(((double)mx - (double)mn) / 15.0);
  if ((sh & 0x7FFF) == 0) sh = 0x3C00;   // 1.0
  const double s = f16_to_f64(sh);
  double z = rint(-(double)mn / s);
  z = z > 0.0 ? (z > 15.0 ? 15.0 : z) : 0.0;   // -0.0 counts as 0
  double qa = rint((double)a / s) + z, qb = rint((double)b / s) + z;
  qa = qa < 0.0 ? 0.0 : (qa > 15.0 ? 15.0 : qa);
  qb = qb < 0.0 ? 0.0 : (qb > 15.0 ? 15.0 : qb);
  const bool fail = bad || (sh & 0x7C00) == 0x7C00;
  const uint64_t any = __ballot(fail);
  // lane: columns 2 lane, 2 lane + 1 = elements 2 (lane % 4), +1 of word lane / 4
  uint32_t w = 0;
  if (!any) w = ((uint32_t)qa | ((uint32_t)qb << 16)) << (4 * (lane & 3));
  w |= __shfl_xor(w, 1);
  w |= __shfl_xor(w, 2);
  if ((lane & 3) == 0) {
    const int wi = lane >> 2;   // 0..15: chunk wi / 4, word wi % 4
    uint32_t* p = reinterpret_cast<uint32_t*>(dst + ((size_t)(row / 16) * gi + g) * 1024);
    p[((wi >> 2) * 16 + row % 16) * 4 + (wi & 3)] = w;
  }
  if (lane == 0) {
    reinterpret_cast<uint32_t*>(dst + (size_t)out * in / 2)[(size_t)g * out + row] =
        (uint32_t)sh | ((uint32_t)f64_to_f16(z) << 16);
    if (any) atomicOr(flag, 1u);
  }
}

__global__ void k_w4_flag(uint32_t* flag) { *flag = 0; }

template <int RT, int TT, int U = 1>
void go(const W4Args& a) {
  const dim3 g((unsigned)((a.out / 16 + RT - 1) / RT), (unsigned)((a.T + TT * 16 - 1) / (TT * 16)));
  hipLaunchKernelGGL((k_w4<RT, TT, 8, U>), g, dim3(512), 0, reinterpret_cast<hipStream_t>(a.stream), a.w, a.x, a.y,
                     a.out, a.in, a.T);
}

}  // namespace

// The tile of a block.  With more than a token or two the time is that of a
// CU's L1, about an access a cycle.  A wave's load makes 16 accesses where its
// bytes lie together (codes; x of one token, whose row all lanes read), and
// more where they are 16 rows of x: counted 16 a load with 1 token, 29 with 7,
// 36 in the tile (6,2) with 64, whose 23000 accesses a CU take two thirds of the
// time.  Each block loads x again for its rows, so the rule weighs, for the
// fullest CU, RT row tiles (17 each) against the tokens' x (4 each), for each
// round of 256 blocks; of 4096 inputs 14 to 17 such units take a us.  Measured,
// us, all 10 tiles timed: 4096 x 4096 with 64 tokens (1,1) 18.6, (1,4) 17.1,
// (4,1) 8.8; 11008 x 4096 with 16 (1,1) 14.7, (2,1) 11.6, (3,1) 8.2, (4,1) 9.0,
// with 64 (4,4) 21.5, (3,4) 20.3, (6,2) 15.1; 4096 x 14336 with 1 (1,1) 10.3 (3.0
// TB/s: few bytes on their way), (2,1) 12.6.  4096 x 14336 with 7 tokens takes
// 10.6 however many groups are loaded ahead (2 to 8), with 8 waves or 16, and
// wherever a block begins in x.  4096 x 4096 with 128, 512 and 2048 tokens 13, 36
// and 128: every 32 tokens unpack the codes again.
int launch_w4(const W4Args& a) {
  constexpr int kTiles[][2] = {{1, 1}, {2, 1}, {3, 1}, {4, 1}, {6, 1}, {8, 1}, {2, 2}, {4, 2}, {6, 2}, {8, 2}};
  int best = 0;
  int64_t least = INT64_MAX;
  for (int c = 0; c < 10; ++c) {
    const int64_t rt = kTiles[c][0], tok = 16 * kTiles[c][1];
    const int64_t blocks = (a.out / 16 + rt - 1) / rt * ((a.T + tok - 1) / tok);
    const int64_t cost = (blocks + 255) / 256 * (17 * rt + 4 * (a.T < tok ? a.T : tok));
    if (cost < least) least = cost, best = c;
  }
  switch (best) {
    case 0: go<1, 1, 4>(a); break;
    case 1: go<2, 1>(a); break;
    case 2: go<3, 1>(a); break;
    case 3: go<4, 1>(a); break;
    case 4: go<6, 1>(a); break;
    case 5: go<8, 1>(a); break;
    case 6: go<2, 2>(a); break;
    case 7: go<4, 2>(a); break;
    case 8: go<6, 2>(a); break;
    default: go<8, 2>(a); break;
  }
  return (int)hipGetLastError();
}

int launch_w4_pack(int32_t out, int32_t in, const uint16_t* W, uint8_t* dst, uint32_t* flag, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(k_w4_flag, dim3(1), dim3(1), 0, st, flag);
  const size_t items = (size_t)out * (in / kGroup);
  hipLaunchKernelGGL(k_w4_pack, dim3((unsigned)((items + 3) / 4)), dim3(256), 0, st, W, dst, flag, out, in);
  return (int)hipGetLastError();
}

}  // namespace dc
