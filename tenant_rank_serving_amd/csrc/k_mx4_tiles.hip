// Products of two MXFP4 matrices for many tokens: y[t][o] = sum_k w_ok x_tk.
//
// A block takes (16 MA WM) rows of the matrix x (16 NB WN) tokens, WM x WN waves, and
// 128 columns a step.  Operands come as whole KiB pieces of the format, which are
// the lanes of v_mfma_scale_f32_16x16x128 as they lie: straight to LDS
// (global_load_lds, four tiles in flight, one barrier a step), then to registers
// one step ahead of the products.
//
// Rows are dealt to a wave's MA products so that a lane ends with 8 rows side by
// side in each two of them, and the 4 lanes of a token with 32: operand row i of
// product a is row 32 (a / 2) + 8 (i / 4) + 4 (a % 2) + i % 4 of the wave's, and lane
// l gets rows 32 (a / 2) + 8 (l / 16) + 4 (a % 2) + r of token l % 16.  Reading
// operands in that order takes pieces of two tiles at once; the tiles are padded
// in LDS such that they lie in different banks.
//
// Blocks stay for several tiles and load the next one's first steps under the last
// one's products.  The largest tile has two waves a SIMD, which take turns: while
// one multiplies, the other reads the operands of its next step and sends for
// tiles.  (All waves reading, then all multiplying: 398 us where this takes 360,
// 32000 x 4096 with 8192 tokens 548 and 516; and operands of two steps in registers
// at once, 7 more than there are.)
//
// Measured, 16384 tokens x 11008 x 4096 (1.48 TFLOP), normal numbers: 335 to 375 us,
// 4.0 to 4.4 PFLOP/s.  Two things bound it.  A turn takes twice its products' cycles:
// of 640000 cycles the matrix pipes are busy 352000; LDS serves reads for 149000
// (no bank conflicts), and waves wait for it 11 % of their time, so it is not the
// port that fills the rest but what a turn waits for in a row, loads, reads and two
// barriers.  And the power that the card may take: with all codes zero the same
// cycles run at 2.45 GHz and take 264 us, with normal numbers at 1.97.  Parts taken
// away in a copy: results 315, loads 327, operands that stay 290; products alone, from
// registers, 206 (zero codes 156).  Not faster: results written over the next tile's
// steps instead of at once (361), products of 32 x 32 x 64 (365), wave tiles of 128 x
// 128 (the compiler moves their sums about).  Results go out as 64 bytes a token, past
// the caches: 16-byte pieces cost 10 % more, 32-byte pieces 70 %, cached stores 3 %.
#include <hip/hip_runtime.h>

#include "step.h"

namespace dc {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#include "mx4_common.h"

constexpr int kFp4 = 4;
constexpr int NS = 4;   // tiles in LDS: as many as steps that share a scale word

__device__ __forceinline__ v8i piece(u32x4 w) { return v8i{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0}; }

template <int TA, int TB>
struct TilesLds {
  static constexpr int kA = 1024 + 64, kB = 1024;   // bytes of a tile's codes of a step
  static constexpr int kAs = 256 + 16, kBs = 256;   // of its scales of four steps
  alignas(256) uint8_t a[NS][TA * kA];
  alignas(256) uint8_t b[NS][TB * kB];
  alignas(256) uint8_t as[TA * kAs];
  alignas(256) uint8_t bs[TB * kBs];
};

// wait_barrier, and with no wait for loads where `fresh`.  (The branch is hidden from
// the compiler, which makes copies of the steps for either side.)
template <int N>
__device__ __forceinline__ void wait_barrier_unless(int fresh) {
  asm volatile(
      "s_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 .Lfresh%=\n\ts_waitcnt vmcnt(%1)\n.Lfresh%=:\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"s"(__builtin_amdgcn_readfirstlane(fresh)),
      "n"(N)
      : "memory", "scc");
}

// wait_barrier, with M more on their way where `fresh`.
template <int N, int M>
__device__ __forceinline__ void wait_barrier_more(int fresh) {
  asm volatile(
      "s_waitcnt vmcnt(%2)\n\ts_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 .Lmore%=\n\ts_waitcnt vmcnt(%1)\n.Lmore%=:\n\ts_waitcnt "
      "lgkmcnt(0)\n\ts_barrier" ::"s"(__builtin_amdgcn_readfirstlane(fresh)),
      "n"(N), "n"(N + M)
      : "memory", "scc");
}
__device__ __forceinline__ void only_barrier() { asm volatile("s_barrier" ::: "memory"); }

template <int MA, int NB>
struct Operands {
  u32x4 a[MA], b[NB];
};

// The compiler does not know that the barrier waited for these: without this it
// waits again, behind the next step's reads.
__device__ __forceinline__ void here(u32x4& w) { asm volatile("" : "+v"(w)); }
template <int MA, int NB>
__device__ __forceinline__ void arrived(Operands<MA, NB>& o) {
#pragma unroll
  for (int a = 0; a < MA; ++a) here(o.a[a]);
#pragma unroll
  for (int b = 0; b < NB; ++b) here(o.b[b]);
}

// Where a tile's operands are: offsets of the wave's pieces of the matrix and of
// x, and of their scales.
template <int LA, int LB>
struct Sources {
  uint32_t a[LA], b[LB], as[LA], bs[LB];
};

template <int MA, int NB, int WM, int WN, int WAVES>
__global__ void __launch_bounds__(64 * WM * WN, WAVES) k_mx4_tiles(Mx4Args g, int mt, int nt) {
  typedef TilesLds<MA * WM, NB * WN> Lds;
  __shared__ Lds sh;
  constexpr int TA = MA * WM, TB = NB * WN, LA = MA / WN, LB = NB / WM;   // tiles of the block; loads of a wave
  static_assert(LA * WN == MA && LB * WM == NB, "every wave loads as many tiles");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  constexpr bool TURNS = WM * WN == 8;   // waves w and w + 4 share a SIMD and take turns
  const int gc = g.in / 128, hc = (gc + 3) / 4, rts = g.out / 16, tts = (g.T + 15) / 16;
  // The 8 XCDs take consecutive blocks in turn; each gets a stretch of the tiles
  // in an order where blocks that run together share rows and tokens: bands of
  // 8 tiles of tokens.
  const int per = (mt * nt + 7) / 8, stride = gridDim.x >> 3;
  const int from = (blockIdx.x & 7) * per, until = min(per, mt * nt - from);   // of the XCD: from + j for j < until
  auto place = [&](int j, int* m, int* n) {
    const int id = from + j, band = id / (8 * mt), first = band * 8, wide = min(8, nt - first), rest = id - band * 8 * mt;
    *m = __builtin_amdgcn_readfirstlane(rest / wide);
    *n = __builtin_amdgcn_readfirstlane(first + rest % wide);
  };
  typedef Sources<LA, LB> Src;
  auto sources = [&](int m, int n) {
    Src r;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const uint32_t T = min(m * TA + wave * LA + i, rts - 1);
      r.a[i] = T * gc * 1024;
      r.as[i] = T * hc * 256;
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const uint32_t T = min(n * TB + wave * LB + i, tts - 1);
      r.b[i] = T * gc * 1024;
      r.bs[i] = T * hc * 256;
    }
    return r;
  };
  const uint8_t* ws = g.w + (size_t)rts * gc * 1024;
  const uint8_t* xs = g.xq + (size_t)tts * gc * 1024;
  const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)&sh.a[0][0];
  const uint32_t la = at + wave * LA * Lds::kA, lb = at + (uint32_t)offsetof(Lds, b) + wave * LB * Lds::kB;
  const uint32_t lsa = at + (uint32_t)offsetof(Lds, as) + wave * LA * Lds::kAs;
  const uint32_t lsb = at + (uint32_t)offsetof(Lds, bs) + wave * LB * Lds::kBs;
  auto load = [&](const Src& p, int k, int s) {
    const int voff = k * 1024 + lane * 16;
#pragma unroll
    for (int i = 0; i < LA; ++i) to_lds16(g.w + p.a[i], voff, la + i * Lds::kA + s * (uint32_t)sizeof(sh.a[0]));
#pragma unroll
    for (int i = 0; i < LB; ++i) to_lds16(g.xq + p.b[i], voff, lb + i * Lds::kB + s * (uint32_t)sizeof(sh.b[0]));
  };
  auto load_scales = [&](const Src& p, int h) {
    const int voff = h * 256 + lane * 4;
#pragma unroll
    for (int i = 0; i < LA; ++i) to_lds4(ws + p.as[i], voff, lsa + i * Lds::kAs);
#pragma unroll
    for (int i = 0; i < LB; ++i) to_lds4(xs + p.bs[i], voff, lsb + i * Lds::kBs);
  };
  // where the lane's pieces and scales lie
  int ao[MA], aso[MA];
#pragma unroll
  for (int a = 0; a < MA; ++a) {
    const int row = 32 * (a / 2) + 8 * ((lane & 15) >> 2) + 4 * (a % 2) + (lane & 3), q = lane >> 4;
    ao[a] = (wm * MA + row / 16) * Lds::kA + (q * 16 + row % 16) * 16;
    aso[a] = (wm * MA + row / 16) * Lds::kAs + (q * 16 + row % 16) * 4;
  }
  const int bo = wn * NB * Lds::kB + lane * 16, bso = wn * NB * Lds::kBs + lane * 4;
  auto fetch = [&](Operands<MA, NB>& o, int s) {
#pragma unroll
    for (int a = 0; a < MA; ++a) o.a[a] = *reinterpret_cast<const u32x4*>(sh.a[s] + ao[a]);
#pragma unroll
    for (int b = 0; b < NB; ++b) o.b[b] = *reinterpret_cast<const u32x4*>(sh.b[s] + bo + b * Lds::kB);
  };
  int sa[MA], sb[NB];
  auto fetch_scales = [&](int* x, int* y) {
#pragma unroll
    for (int a = 0; a < MA; ++a) x[a] = *reinterpret_cast<const int*>(sh.as + aso[a]);
#pragma unroll
    for (int b = 0; b < NB; ++b) y[b] = *reinterpret_cast<const int*>(sh.bs + bso + b * Lds::kBs);
  };

  int j = blockIdx.x >> 3, m, n;
  if (j >= until) return;
  place(j, &m, &n);
  Src now = sources(m, n);
  Operands<MA, NB> o[TURNS ? 1 : 2];
  auto begin = [&] {
    load_scales(now, 0);
#pragma unroll
    for (int s = 0; s < (TURNS ? NS - 1 : NS); ++s) load(now, min(s, gc - 1), s);
    wait_barrier<0>();
    if constexpr (!TURNS) {
      fetch(o[0], 0);
      fetch_scales(sa, sb);
    }
  };
  begin();
  // from here on the second four are a barrier behind
  if (TURNS && wave >= 4) only_barrier();
  const bool whole = gc % 4 == 0;   // else a tile's last steps send for nothing, and the next tile begins anew

  constexpr int L = LA + LB, STORES = MA / 2 * NB;
  // Step J of four (which scale byte, which operands and place in LDS), k + J of
  // the tile; it sends for the step 4 later, of the next tile at the end.  What
  // may be on its way as a step begins: the tiles sent for since those of the
  // next step, and the scales, sent for in step 0.  In a tile's first steps
  // everything older is here, and stores of the last tile's results may be younger.
#define DC_STEP(J)                                                                                                          \
  {                                                                                                                         \
    if (J < NS - 1) wait_barrier_unless<(NS - 2) * L + (J > 0 ? L : 0)>(fresh);                                             \
    else wait_barrier<(NS - 2) * L>();                                                                                      \
    arrived(o[J & 1]);                                                                                                      \
    fetch(o[(J + 1) & 1], (J + 1) % NS);                                                                                    \
    if (J == 0) load_scales(src, min(ahead >> 2, hc - 1));                                                                  \
    load(src, min(ahead + J, gc - 1), J);                                                                                   \
    _Pragma("unroll") for (int b = 0; b < NB; ++b)                                                                          \
      _Pragma("unroll") for (int a = 0; a < MA; ++a)                                                                        \
        acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(piece(o[J & 1].a[a]), piece(o[J & 1].b[b]), acc[a][b], \
                                                                    kFp4, kFp4, J, sa[a], J, sb[b]);                        \
  }
  // The same in turns, in two halves with a barrier behind each: reading, and
  // sending for the tile 3 steps later (the place of the step before, which the
  // other four have read by then), then multiplying.  The next step's tile has to
  // be here at the first barrier, and the scales, sent for in step 1, at step 3's.
  // In a tile's first two steps the tiles have to be that were sent for before the
  // last one's results: STORES more may be on their way.  (As many stores as that
  // there are, or none older than those loads: below.)
#define DC_TURN(J)                                                                                                          \
  {                                                                                                                         \
    fetch(o[0], J);                                                                                                         \
    if (J == 0) fetch_scales(sa, sb);                                                                                       \
    if (J == 1) load_scales(src, min(ahead >> 2, hc - 1));                                                                  \
    load(src, min(ahead + J - 1, gc - 1), (J + NS - 1) % NS);                                                               \
    __builtin_amdgcn_sched_barrier(0);                                                                                      \
    if (J < 2) wait_barrier_more<J == 0 ? 2 * L : 3 * L, STORES>(fresh);                                                    \
    else wait_barrier<J == 2 ? 3 * L : 2 * L>();                                                                            \
    __builtin_amdgcn_sched_barrier(0);                                                                                      \
    arrived(o[0]);                                                                                                          \
    __builtin_amdgcn_s_setprio(1);                                                                                          \
    _Pragma("unroll") for (int b = 0; b < NB; ++b)                                                                          \
      _Pragma("unroll") for (int a = 0; a < MA; ++a)                                                                        \
        acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(piece(o[0].a[a]), piece(o[0].b[b]), acc[a][b],         \
                                                                    kFp4, kFp4, J, sa[a], J, sb[b]);                        \
    __builtin_amdgcn_s_setprio(0);                                                                                          \
    __builtin_amdgcn_sched_barrier(0);                                                                                      \
    only_barrier();                                                                                                         \
    __builtin_amdgcn_sched_barrier(0);                                                                                      \
  }
  for (;;) {
    int nm = m, nn = n;
    const bool more = j + stride < until;
    if (more) place(j + stride, &nm, &nn);
    Src src = now;
    now = sources(nm, nn);   // (behind the last tile: itself, and never used)
    f32x4 acc[MA][NB];
#pragma unroll
    for (int a = 0; a < MA; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    int k = 0, fresh = 1;
#pragma clang loop unroll(disable)
    for (; k + 4 <= gc; k += 4) {   // no branch among the products: the sums stay where they are
      int ahead = k + 4;            // what is sent for
      if constexpr (TURNS) DC_TURN(0)   // (the last of this tile)
      uint32_t over = whole && ahead >= gc ? ~0u : 0u;
      over = __builtin_amdgcn_readfirstlane(over);   // (no copy of the steps for this either)
      ahead &= ~over;
#pragma unroll
      for (int i = 0; i < LA; ++i) src.a[i] += (now.a[i] - src.a[i]) & over, src.as[i] += (now.as[i] - src.as[i]) & over;
#pragma unroll
      for (int i = 0; i < LB; ++i) src.b[i] += (now.b[i] - src.b[i]) & over, src.bs[i] += (now.bs[i] - src.bs[i]) & over;
      if constexpr (TURNS) {
        DC_TURN(1)
        DC_TURN(2)
        DC_TURN(3)
        fresh = 0;
      } else {
        DC_STEP(0)
        DC_STEP(1)
        DC_STEP(2)
        DC_STEP(3)
        fresh = 0;
        fetch_scales(sa, sb);   // of the next four steps: here since step 3's barrier
      }
    }
    if (k < gc) {
      const int ahead = k + 4;
      if constexpr (TURNS) {
        DC_TURN(0)
        if (k + 1 < gc) {
          DC_TURN(1)
          if (k + 2 < gc) DC_TURN(2)
        }
      } else {
        DC_STEP(0)
        if (k + 1 < gc) {
          DC_STEP(1)
          if (k + 2 < gc) DC_STEP(2)
        }
      }
    }
    // Loads and stores are counted together: the next tile's first tiles are here
    // before the results leave, unless (in turns) all STORES of them will and more
    // tiles follow.
    const int r0 = m * TA * 16 + wm * MA * 16;
    if (!TURNS || !whole || !more || r0 >= g.out || (n * TB + (wn + 1) * NB - 1) * 16 >= g.T) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (r0 < g.out) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int t = n * TB * 16 + (wn * NB + b) * 16 + (lane & 15);
        if (t < g.T) {
          uint16_t* y = g.y + (size_t)t * g.out + r0 + 8 * (lane >> 4);
#pragma unroll
          for (int a = 0; a < MA; a += 2) {
            const f32x4 u = acc[a][b], v = acc[a + 1][b];
            __builtin_nontemporal_store(u32x4{pack2(u[0], u[1]), pack2(u[2], u[3]), pack2(v[0], v[1]), pack2(v[2], v[3])},
                                        reinterpret_cast<u32x4*>(y + 16 * a));
          }
        }
      }
    }
    if (!more) break;
    j += stride;
    m = nm, n = nn;
    if (!whole) {
      if constexpr (TURNS) {
        begin();          // everyone has read the last tile's operands: the other four before this half
        only_barrier();   // and their loads are here
      } else {
        wait_barrier<0>();   // everyone has left the last tile's operands
        begin();
      }
    }
  }
  if (TURNS && wave < 4) only_barrier();
#undef DC_TURN
#undef DC_STEP
}

template <int MA, int NB, int WM, int WN, int WAVES>
void go(const Mx4Args& a) {
  const int rows = 16 * MA * WM, toks = 16 * NB * WN, mt = (a.out + rows - 1) / rows, nt = (a.T + toks - 1) / toks;
  // blocks that stay, as many as run at once: WAVES waves a SIMD
  const int all = (mt * nt + 7) / 8 * 8, stay = 256 * 4 * WAVES / (WM * WN);
  const unsigned blocks = (unsigned)(all < stay ? all : stay);
  hipLaunchKernelGGL((k_mx4_tiles<MA, NB, WM, WN, WAVES>), dim3(blocks), dim3(64 * WM * WN), 0, reinterpret_cast<hipStream_t>(a.stream), a,
                     mt, nt);
}

}  // namespace

int launch_mx4_tiles(const Mx4Args& a, int32_t size) {
  switch (size) {
    case 0: go<2, 2, 2, 2, 4>(a); break;   // 64 x 64
    case 1: go<2, 4, 2, 2, 3>(a); break;   // 64 x 128
    case 2: go<4, 4, 2, 2, 2>(a); break;   // 128 x 128
    default: go<4, 8, 4, 2, 2>(a); break;  // 256 x 256
  }
  return (int)hipGetLastError();
}

}  // namespace dc
