// Attention over the paged cache: y = sum_k softmax_k(scale q.k) v_k for
// ragged sequences whose groups share prefixes.
//
// Two walks over keys: Keys (attn_keys.h) for at most 32 query rows of a kv
// head, where the time is that of reading the cache, and Tiles (attn_tiles.h)
// for more.  Two forms of a call, chosen from the host's bounds (attn_plan):
//   split   a block takes the rows of one (sequence, kv head) or, for a
//           prefix, of one (group, kv head), and a range of the keys; its sums
//           go to the workspace and k_attn_join adds a row's.  A prefix is
//           read once for all sequences of its group.
//   rows    long queries: a block takes 128 rows of one (sequence, kv head)
//           and walks its prefix and its own keys; no partial sums.
// Measured (own keys and prefix are read once, us): one token on 1000 keys of
// 32 heads 7.7 + 3.0 for the join, latency; 64 tokens in 16 groups on prefixes
// of 2048 51 + 5, 4.3 TB/s, in two rounds of blocks; 48 tokens on one e4m3 prefix
// of 30000 keys 48 + 7, 192 rows in blocks of 128, 864 blocks of which 512 run at
// once; 20 x 5 tokens of 40 heads on 3 prefixes of 1111 41 + 6, 1160 blocks of
// which 768 run at once.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "layer.h"

namespace dc {
namespace {

#include "attn_common.h"
#include "attn_keys.h"
#include "attn_tiles.h"

// Where a block's partial sums go.
struct Out {
  int64_t at;      // (row, split) number
  uint16_t* y;
};
template <int D>
__device__ __forceinline__ Out out_of(const AttnArgs& a, const Item& it, int row, int h, int slot) {
  const int tok = a.gq_d.of(row), hh = row - tok * a.gq;
  Out o;
  o.at = ((int64_t)(it.t0 + tok) * a.hq + h * a.gq + hh) * (a.plan.sp + a.plan.so) + slot;
  o.y = a.y + (int64_t)(it.t0 + tok) * a.ys + (int64_t)(h * a.gq + hh) * D;
  return o;
}

// A block's work; `again`: every step is treated as one with masks.  True: it
// has to be done again (see Factor).
template <int D, bool F8, int N>
__device__ __forceinline__ bool keys_block(const AttnArgs& a, const Item& it, const Stream& st, Pages& pages, int row0, int h,
                                           int c0, int c1, int slot, bool again, KeysLds<D>& sh) {
  const int wave = __builtin_amdgcn_readfirstlane(thread_anew() >> 6);
  const int last = min(row0 + 16 * N, it.rows) - 1;
  const int lo = it.sees(a.gq_d.of(row0)), up = it.sees(a.gq_d.of(last));
  const int w0 = c0 + 32 * wave, w1 = min(c1, up);
  typename Keys<D, F8, N>::Stage g;
  if (w0 < w1) {   // the first keys and values go first
    g.seek(st, pages, w0, w1);
    g.load_k(st);
    g.load_v(st);
  }
  uint32_t flip;
  const float c = score_factor<F8>(a, h, &flip), vs = value_scale<F8>(a, h);
  Keys<D, F8, N> R;
  R.start(a, it, row0, h, flip);
  R.walk(st, g, pages, w0, w1, again ? 0 : lo, up, c);
  constexpr int J = D / 16;
  return join<D, F8, N>(R, sh, !again, [&](int row, int e, float m, float l, const float* x) __attribute__((always_inline)) {
    if (row0 + row >= it.rows) return;
    const Out w = out_of<D>(a, it, row0 + row, h, slot);
    if (a.plan.direct) {
      store_y<J>(w.y + e, x, l == 0.f ? 0.f : vs / l);
      return;
    }
#pragma unroll
    for (int j = 0; j < J; j += 4)
      *reinterpret_cast<f32x4*>(a.po + w.at * D + e + j) = f32x4{x[j] * vs, x[j + 1] * vs, x[j + 2] * vs, x[j + 3] * vs};
    if (e == 0) a.pml[2 * w.at] = m, a.pml[2 * w.at + 1] = l;
  });
}

// A wave's tile of results, to the output or the workspace.  The output goes
// through the wave's part of LDS (the walk is over), so that 16 bytes a lane
// cover whole rows.
template <int D, bool F8>
__device__ __forceinline__ void put_tiles(const AttnArgs& a, const Item& it, const Tiles<D, F8>& R, int row0, int h,
                                          int slot, float vs, TilesLds<D, F8>& sh) {
  const int tid = thread_anew(), lane = tid & 63, g = lane >> 5, i32 = lane & 31;
  const float l = R.l + __shfl_xor(R.l, 32);
  if (a.plan.direct) {
    constexpr int kRow = D * 2 + 16;   // of LDS: neighbouring rows in other banks
    static_assert(kWaves * kTileRows * kRow <= (int)sizeof(sh.k) + (int)sizeof(sh.v), "the rows fit over the tiles");
    uint8_t* mine = &sh.k[0][0] + (tid >> 6) * (kTileRows * kRow);
    const float f = l == 0.f ? 0.f : vs / l;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x[4] = {R.o[d][4 * i], R.o[d][4 * i + 1], R.o[d][4 * i + 2], R.o[d][4 * i + 3]};
        store_y<4>(reinterpret_cast<uint16_t*>(mine + i32 * kRow) + 32 * d + 8 * i + 4 * g, x, f);
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (other lanes wrote what a lane reads)
    constexpr int P = D / 8;   // pieces of a row
#pragma unroll
    for (int i = 0; i < kTileRows * P / 64; ++i) {
      const int rr = (i * 64 + lane) / P, c = lane % P;
      if (row0 + rr >= it.rows) continue;
      const Out w = out_of<D>(a, it, row0 + rr, h, slot);
      *reinterpret_cast<uint4*>(w.y + c * 8) = *reinterpret_cast<const uint4*>(mine + rr * kRow + c * 16);
    }
    return;
  }
  const int row = row0 + i32;
  if (row >= it.rows) return;
  const Out w = out_of<D>(a, it, row, h, slot);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4*>(a.po + w.at * D + 32 * d + 8 * i + 4 * g) =
          f32x4{R.o[d][4 * i] * vs, R.o[d][4 * i + 1] * vs, R.o[d][4 * i + 2] * vs, R.o[d][4 * i + 3] * vs};
  if (g == 0) a.pml[2 * w.at] = R.m, a.pml[2 * w.at + 1] = l;
}

// One walk of a block's rows over keys [c0, c1) of an item.
template <int D, bool F8>
__device__ __forceinline__ void tiles_walk(const AttnArgs& a, const Item& it, const Stream& st, const Pages& pages,
                                           Tiles<D, F8>& R, int blk0, int c0, int c1, bool again, float c,
                                           TilesLds<D, F8>& sh) {
  const int wave = __builtin_amdgcn_readfirstlane(thread_anew() >> 6);
  const int row0 = blk0 + kTileRows * wave;
  const bool live = row0 < it.rows;
  const int blast = min(blk0 + kBlockRows, it.rows) - 1, wlast = min(row0 + kTileRows, it.rows) - 1;
  const int blo = it.sees(a.gq_d.of(blk0)), bup = it.sees(a.gq_d.of(blast));
  const int lo = it.sees(a.gq_d.of(row0)), up = it.sees(a.gq_d.of(max(wlast, 0)));
  R.hi = it.sees(a.gq_d.of(min(row0 + (thread_anew() & 31), it.rows - 1)));
  R.walk(st, pages, c0, c1, lo, up, again ? 0 : blo, bup, c, live, sh);
}

template <int D, bool F8>
__device__ __forceinline__ bool tiles_block(const AttnArgs& a, const Item& it, const Stream& st, const Pages& pages, int blk0,
                                            int h, int c0, int c1, int slot, bool again, TilesLds<D, F8>& sh) {
  uint32_t flip;
  const float c = score_factor<F8>(a, h, &flip), vs = value_scale<F8>(a, h);
  const int row0 = blk0 + kTileRows * __builtin_amdgcn_readfirstlane(thread_anew() >> 6);
  Tiles<D, F8> R;
  R.clear();
  R.load_q(a, it, row0, h, flip);
  tiles_walk<D, F8>(a, it, st, pages, R, blk0, c0, c1, again, c, sh);
  if (!F8 && !again && __builtin_expect(R.unfinite_results(sh), 0)) return true;
  put_tiles<D, F8>(a, it, R, row0, h, slot, vs, sh);
  return false;
}

// Split form.  WO, WP: how own keys and prefixes are walked, by Keys of 16 or
// 32 rows (1, 2) or by Tiles (3).
constexpr int kByTiles = 3;
template <int D, bool F8, int WO, int WP>
union SplitLds {
  KeysLds<D> keys;
  TilesLds<WO == kByTiles || WP == kByTiles ? D : 8, F8> tiles;
};
template <int D, bool F8, int WO, int WP>
__device__ __forceinline__ bool split_block(const AttnArgs& a, int npre, int block, bool again, SplitLds<D, F8, WO, WP>& sh) {
  const bool prefix = block < npre;
  const int blk = prefix ? block : block - npre;
  const int rb = prefix ? a.plan.rbp : a.plan.rbo, ns = prefix ? a.plan.sp : a.plan.so;
  const int chunk = prefix ? a.plan.cp : a.plan.co;
  int u = (prefix ? a.plan.rbp_d : a.plan.rbo_d).of(blk);
  const int r = blk - u * rb;
  const int u2 = a.hkv_d.of(u), h = u - u2 * a.kv.heads;
  const int b = (prefix ? a.plan.sp_d : a.plan.so_d).of(u2), s = u2 - b * ns;
  const int c0 = s * chunk;
  // the page numbers are on their way while the lengths are read
  const Stream st = prefix ? prefix_stream(a, h, b) : own_stream(a, h, b);
  Pages pages;
  pages.fill(st, c0 >> st.shift);
  const Item it = prefix ? prefix_item(a, b) : own_item(a, b);
  const int how = prefix ? WP : WO;
  const int row0 = r * (how == kByTiles ? kBlockRows : 16 * how);
  if (row0 >= it.rows) return false;
  const int c1 = min(it.len, c0 + chunk);
  if (c0 >= c1 && !a.plan.direct) return false;   // the join knows that it holds nothing
  const int slot = prefix ? s : a.plan.sp + s;
#define DC_WALK(W_)                                                                                 \
  if constexpr (W_ == kByTiles) return tiles_block<D, F8>(a, it, st, pages, row0, h, c0, c1, slot, again, sh.tiles); \
  else return keys_block<D, F8, W_>(a, it, st, pages, row0, h, c0, c1, slot, again, sh.keys);
  if constexpr (WO == WP) {
    DC_WALK(WO)
  } else if (prefix) {
    DC_WALK(WP)
  } else {
    DC_WALK(WO)
  }
#undef DC_WALK
}
// (three blocks a CU where the tiles of bf16 leave room for them)
template <int D, bool F8, int WO, int WP>
__global__ void __launch_bounds__(64 * kWaves, !F8 && WO != 2 && WP == kByTiles ? 3 : 2) k_attn_split(AttnArgs, int npre) {
  __shared__ SplitLds<D, F8, WO, WP> sh;
  for (int again = 0; split_block<D, F8, WO, WP>(args_anew(), npre, block_anew(), one_code(again), sh) && !F8;) again = 1;
}

// Joins the splits of a row: one wave a row.  Everything that does not depend
// on the token's sequence is loaded at once: the sequences' starts and
// lengths (64 at a time, one a lane), the splits' maxima and weights (one a
// lane) and the first of their sums.  A half wave takes every other split, 16
// bytes a lane (D = 64: a quarter, every fourth).
template <int D>
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs a) {
  constexpr int L = D / 4, P = 64 / L;   // lanes of a split's sums, splits at a time
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= (int64_t)a.n * a.hq) return;
  const int tok = a.hq_d.of((int)row), h = (int)row - tok * a.hq;
  const int sp = a.plan.sp, slots = sp + a.plan.so;
  const f32x2* ml = reinterpret_cast<const f32x2*>(a.pml) + row * slots;
  const float* po = a.po + row * slots * D + (lane % L) * 4;
  // slots lane and lane + 64 (a prefix and the own keys have at most 64 each)
  const f32x2 mla = ml[min(lane, slots - 1)], mlb = ml[min(lane + 64, slots - 1)];
  f32x4 first[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    first[i] = *reinterpret_cast<const f32x4*>(po + (int64_t)min(i * P + lane / L, slots - 1) * D);
  // the token's sequence: the last one that starts at or before it
  int b = -1, len = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int i = min(b0 + lane, a.B - 1);
    const int s = a.q_start[i], e = a.q_start[i + 1], n = a.kv_len[i];
    const bool in = b0 + lane < a.B && s <= tok && tok < e && tok - clampi(s, 0, a.n) < a.max_q;
    const uint64_t hit = __builtin_amdgcn_ballot_w64(in);
    if (hit) {
      const int at = 63 - __builtin_clzll(hit);
      b = b0 + at;
      len = __builtin_amdgcn_readlane(n, at);
    }
  }
  int plen = 0;
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    const int g = min(g0 + lane, a.G - 1);
    const int n = a.p_len[g];
    const bool in = g0 + lane < a.G && a.g_start[g] <= b && b < a.g_start[g + 1];
    const uint64_t hit = __builtin_amdgcn_ballot_w64(in);
    if (hit) plen = __builtin_amdgcn_readlane(n, 63 - __builtin_clzll(hit));
  }
  if (b < 0) return;   // behind the last sequence: left as it is
  const int no = (clampi(len, 0, a.max_kv) + a.plan.co - 1) / a.plan.co;
  const int np = (clampi(plen, 0, a.max_pre) + a.plan.cp - 1) / a.plan.cp;
  // splits that hold keys were written by their blocks
  auto held = [&](int s) __attribute__((always_inline)) { return s < np || (s >= sp && s - sp < no); };
  float ma = held(lane) ? mla[0] : kLow, mb = held(lane + 64) ? mlb[0] : kLow;
  float m = fmaxf(ma, mb);
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) m = fmaxf(m, __shfl_xor(m, i));
  const float wa = held(lane) ? __builtin_amdgcn_exp2f(ma - m) : 0.f;
  const float wb = held(lane + 64) ? __builtin_amdgcn_exp2f(mb - m) : 0.f;
  float l = (held(lane) ? mla[1] * wa : 0.f) + (held(lane + 64) ? mlb[1] * wb : 0.f);
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) l += __shfl_xor(l, i);
  f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < slots; s0 += P * kAhead) {
    f32x4 o[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = s0 + i * P + lane / L;
      o[i] = s0 == 0 ? first[i] : *reinterpret_cast<const f32x4*>(po + (int64_t)min(s, slots - 1) * D);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = s0 + i * P + lane / L;
      const Factor w(s < 64 ? __shfl(wa, s & 63) : __shfl(wb, s & 63));
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] += held(s) ? w.of(o[i][j]) : 0.f;
    }
  }
#pragma unroll
  for (int i = L; i < 64; i <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] += __shfl_xor(x[j], i);
  if (lane < L) {
    const float xs[4] = {x[0], x[1], x[2], x[3]};
    store_y<4>(a.y + (int64_t)tok * a.ys + (int64_t)h * D + lane * 4, xs, l == 0.f ? 0.f : 1.f / l);
  }
}

// Long queries.  Blocks of one (sequence, kv head) follow each other on one
// XCD, so that its L2 serves their keys, the longest rows first; the quarter
// with the shortest rows of every sequence comes last and fills the end (187
// us without that, 183 with; all sequences' longest rows first 219: their keys
// do not fit).  PRE: some sequences have a prefix.
template <int D, bool F8, bool PRE>
__device__ __forceinline__ bool rows_block(const AttnArgs& a, int block, bool again, TilesLds<D, F8>& sh) {
  const int xcd = block & 7, j8 = block >> 3;
  const int light = a.plan.rbo >> 2, heavy = a.plan.rbo - light, h8 = (a.B * a.kv.heads + 7) / 8 * heavy;
  int p8, rblk;
  if (j8 < h8) {
    p8 = a.plan.heavy_d.of(j8);
    rblk = a.plan.rbo - 1 - (j8 - p8 * heavy);
  } else {
    p8 = a.plan.light_d.of(j8 - h8);
    rblk = light - 1 - (j8 - h8 - p8 * light);
  }
  const int pair = p8 * 8 + xcd;
  if (pair >= a.B * a.kv.heads) return false;
  const int b = a.hkv_d.of(pair), h = pair - b * a.kv.heads;
  // the page numbers are on their way while the lengths are read
  const Stream st = own_stream(a, h, b);
  Pages pages;
  pages.fill(st, 0);
  const Item own = own_item(a, b);
  const int blk0 = rblk * kBlockRows;
  if (blk0 >= own.rows) return false;
  uint32_t flip;
  const float c = score_factor<F8>(a, h, &flip), vs = value_scale<F8>(a, h);
  const int row0 = blk0 + kTileRows * __builtin_amdgcn_readfirstlane(thread_anew() >> 6);
  Tiles<D, F8> R;
  R.clear();
  R.load_q(a, own, row0, h, flip);
  if constexpr (PRE) {   // the group's prefix, all of it
    const int gr = group_of(a, b);
    Item it = own;
    it.len = gr < 0 ? 0 : clampi(a.p_len[gr], 0, a.max_pre);
    it.causal = false;
    const Stream ps = prefix_stream(a, h, max(gr, 0));
    Pages pp;
    pp.fill(ps, 0);
    tiles_walk<D, F8>(a, it, ps, pp, R, blk0, 0, it.len, again, c, sh);
  }
  tiles_walk<D, F8>(a, own, st, pages, R, blk0, 0, own.len, again, c, sh);
  if (!F8 && !again && __builtin_expect(R.unfinite_results(sh), 0)) return true;
  put_tiles<D, F8>(a, own, R, row0, h, 0, vs, sh);
  return false;
}
template <int D, bool F8, bool PRE>
__global__ void __launch_bounds__(64 * kWaves, F8 ? 2 : 3) k_attn_rows(AttnArgs) {
  __shared__ TilesLds<D, F8> sh;
  for (int again = 0; rows_block<D, F8, PRE>(args_anew(), block_anew(), one_code(again), sh) && !F8;) again = 1;
}

template <int D, bool F8>
void go(const AttnArgs& a) {
  hipStream_t st = reinterpret_cast<hipStream_t>(a.stream);
  const AttnPlan& p = a.plan;
  const dim3 blk(64 * kWaves);
  if (p.rows) {
    const int pairs8 = (int)(((int64_t)a.B * a.kv.heads + 7) / 8);
    const dim3 g((unsigned)(8 * pairs8 * p.rbo));
    if (a.G > 0) hipLaunchKernelGGL((k_attn_rows<D, F8, true>), g, blk, 0, st, a);
    else hipLaunchKernelGGL((k_attn_rows<D, F8, false>), g, blk, 0, st, a);
    return;
  }
  const int npre = a.G * a.kv.heads * p.rbp * p.sp, nown = a.B * a.kv.heads * p.rbo * p.so;
  const dim3 g((unsigned)(npre + nown));
#define DC_SPLIT(WO_, WP_) hipLaunchKernelGGL((k_attn_split<D, F8, WO_, WP_>), g, blk, 0, st, a, npre)
  switch (p.wo * 4 + p.wp) {
    case 5: DC_SPLIT(1, 1); break;
    case 6: DC_SPLIT(1, 2); break;
    case 7: DC_SPLIT(1, 3); break;
    case 10: DC_SPLIT(2, 2); break;
    case 11: DC_SPLIT(2, 3); break;
    default: DC_SPLIT(3, 3); break;
  }
#undef DC_SPLIT
  if (!p.direct)
    hipLaunchKernelGGL((k_attn_join<D>), dim3((unsigned)(((int64_t)a.n * a.hq + 3) / 4)), dim3(256), 0, st, a);
}

}  // namespace

int launch_attention(const AttnArgs& a) {
  if (a.dim == 64) {
    if (a.e4m3) go<64, true>(a);
    else go<64, false>(a);
  } else {
    if (a.e4m3) go<128, true>(a);
    else go<128, false>(a);
  }
  return (int)hipGetLastError();
}

}  // namespace dc
