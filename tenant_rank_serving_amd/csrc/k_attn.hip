// Attention over the paged cache: y = sum_k softmax_k(scale q.k) v_k for
// ragged sequences whose groups share prefixes.
//
// The matrix core takes the products transposed, S^T = K Q^T and
// O^T = V^T P^T (16x16x32, bf16 in, fp32 sums), so that every operand is
// where it is needed without a trip through LDS:
//   K   operand A: lane l holds key l%16 of a 16-key half of the 32-key step
//       and 8 consecutive elements: one 16-byte load from the cache.
//   S^T result: lane l holds query row l%16 and keys 4(l/16) .. +4 of each
//       half; the softmax state of a row is therefore in the lane.
//   P^T operand B: row l%16 and 8 keys of lane group l/16; the order of the
//       keys inside a product is free, so the lane's own 2 x 4 values of S^T
//       are the operand.
//   V^T operand A: lane l loads 8 keys (those of its P) x d/16 consecutive
//       elements, d = (d/16)(l%16) + j, and product j takes element j of each
//       key: a register transposition of 16-bit halves.  Row m of product j
//       is element (d/16) m + j, so a lane's results are consecutive elements.
//
// The running maximum m of a row moves only when a value passes it by
// 2^kSlack (most steps leave the sums as they are; the weights then reach
// 2^kSlack instead of 1, which floats do not mind).  The row's sum comes from
// the matrix core as well, against ones, from the rounded weights: numerator
// and denominator hold the same weights.
#include <hip/hip_runtime.h>

#include "layer.h"

namespace dc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLow = -3.402823466e38f;   // a row that has seen no key
constexpr float kSlack = 6.f;
constexpr int kWaves = 4;

__device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // round to nearest even
  bf16x2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// 2 of the 4 e4m3 codes of a word as bf16 (exact)
__device__ __forceinline__ uint32_t cvt2(uint32_t w, bool hi) {
  return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true))
            : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false));
}

template <int N> struct Words { uint32_t w[N]; };
template <int N> __device__ __forceinline__ Words<N> load_words(const uint8_t* p) {
  Words<N> r;
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}

// A run of keys of one kv head: its page table and the cache.
struct Stream {
  const uint8_t *k, *v;     // of the head
  int64_t page_stride;
  int32_t slot_stride;      // fits: a page's slots lie within 2^31 bytes
  const int32_t* table;
  int32_t npages;           // entries of the table that hold keys
  int32_t num_pages;        // pages of the cache
  int32_t shift;
};

// The state of NRT 16-row tiles of queries in one wave.
template <int D, bool F8, int NRT>
struct Rows {
  static constexpr int C = D / 32;   // products of a 16-key tile
  static constexpr int J = D / 16;   // products of a 32-key step's values
  uint4 q[NRT][C];
  f32x4 o[NRT][J];
  f32x4 l[NRT];
  float m[NRT];
  int32_t hi[NRT];   // keys the lane's row sees: [0, hi)

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NRT; ++n) {
#pragma unroll
      for (int j = 0; j < J; ++j) o[n][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      l[n] = f32x4{0.f, 0.f, 0.f, 0.f};
      m[n] = kLow;
    }
  }

  // Keys [k0, k1) of the stream (k0 a multiple of 32; k0 < k1), weights
  // exp2(c q.k).  SPLITP: the weights as two bf16 pieces.
  template <bool SPLITP>
  __device__ __forceinline__ void walk(const Stream& st, int k0, int k1, float c) {
    const int lane = threadIdx.x & 63, g = lane >> 4, i16 = lane & 15;
    // rows that see every key of a step need no masks
    int lo = hi[0], up = hi[0];
#pragma unroll
    for (int n = 1; n < NRT; ++n) lo = min(lo, hi[n]), up = max(up, hi[n]);
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) lo = min(lo, __shfl_xor(lo, s)), up = max(up, __shfl_xor(up, s));
    lo = __builtin_amdgcn_readfirstlane(lo);
    up = __builtin_amdgcn_readfirstlane(up);
    k1 = min(k1, up);
    if (k0 >= k1) return;
    constexpr int KB = F8 ? 1 : 2;                 // bytes of an element
    constexpr int KL = D * KB / 64;                // 16-byte loads of a key's lane group
    constexpr int VW = D * KB / 64;                // words of a lane's piece of a value row
    const int koff = i16 * st.slot_stride + g * 16;
    const int voff = 4 * g * st.slot_stride + i16 * (VW * 4);
    // page numbers of the next 64 pages, one a lane
    int pbase = k0 >> st.shift, pg = 0;
    auto pages = [&]() __attribute__((always_inline)) {
      pg = st.table[min(pbase + lane, st.npages - 1)];
      pg = (unsigned)pg < (unsigned)st.num_pages ? pg : 0;   // never outside the cache
    };
    pages();
    Words<4> kr[2][KL];
    Words<VW> vr[8];
    const uint8_t *kb[2], *vb[2];
    // the two 16-key halves of the step at k (the last one that holds keys
    // again past the end: masked by their numbers)
    auto seek = [&](int k) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int at = min(k + 16 * t, (k1 - 1) & ~15);
        int p = at >> st.shift;
        if (p - pbase >= 64) {
          pbase = p;
          pages();
        }
        const int64_t page = __builtin_amdgcn_readlane(pg, p - pbase);
        const int64_t off = page * st.page_stride + (int64_t)(at & ((1 << st.shift) - 1)) * st.slot_stride;
        kb[t] = st.k + off;
        vb[t] = st.v + off;
      }
    };
    auto load_k = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < KL; ++i) kr[t][i] = load_words<4>(kb[t] + koff + 64 * i);
    };
    auto load_v = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) vr[e] = load_words<VW>(vb[e >> 2] + voff + (e & 3) * st.slot_stride);
    };
    seek(k0);
    load_k();
    load_v();
    for (int k = k0; k < k1; k += 32) {
      f32x4 s[NRT][2];
#pragma unroll
      for (int n = 0; n < NRT; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          s[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < C; ++i) {
            uint4 a;
            if constexpr (F8) {
              const uint32_t w0 = kr[t][i >> 1].w[2 * (i & 1)], w1 = kr[t][i >> 1].w[2 * (i & 1) + 1];
              a = uint4{cvt2(w0, false), cvt2(w0, true), cvt2(w1, false), cvt2(w1, true)};
            } else {
              a = uint4{kr[t][i].w[0], kr[t][i].w[1], kr[t][i].w[2], kr[t][i].w[3]};
            }
            s[n][t] = mfma(a, q[n][i], s[n][t]);
          }
        }
      const bool more = k + 32 < k1;
      const bool masked = k + 32 > lo;
      // the values as 8-key operands
      if (more) {
        seek(k + 32);
        load_k();
      }
      uint4 va[J];
      auto operands = [&]() __attribute__((always_inline)) {
        uint32_t x[8][J / 2];   // bf16 pairs of elements
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int w = 0; w < J / 2; ++w)
            x[e][w] = F8 ? cvt2(vr[e].w[w >> 1], w & 1) : vr[e].w[w];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
          va[j] = uint4{__builtin_amdgcn_perm(x[1][j >> 1], x[0][j >> 1], sel),
                        __builtin_amdgcn_perm(x[3][j >> 1], x[2][j >> 1], sel),
                        __builtin_amdgcn_perm(x[5][j >> 1], x[4][j >> 1], sel),
                        __builtin_amdgcn_perm(x[7][j >> 1], x[6][j >> 1], sel)};
        }
      };
      bool careful = false;
      if (masked) {
        // values that no row sees count as zero: the slots may hold anything
        uint32_t odd = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool dead = k + 16 * (e >> 2) + 4 * g + (e & 3) >= up;
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            vr[e].w[w] = dead ? 0u : vr[e].w[w];
            const uint32_t u = vr[e].w[w];
            if constexpr (F8) {   // NaN is 0x7F
              const uint32_t b = u & 0x7F7F7F7Fu;
              odd |= (b + 0x01010101u) & 0x80808080u;
            } else {              // infinity or NaN: all exponent bits
              odd |= (((u & 0x7F807F80u) + 0x00800080u) & 0x80008000u);
            }
          }
        }
        careful = __builtin_amdgcn_ballot_w64(odd != 0) != 0;
      }
      operands();
      if (more) load_v();
#pragma unroll
      for (int n = 0; n < NRT; ++n) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = s[n][e >> 2][e & 3] * c;
        if (masked) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[e] = k + 16 * (e >> 2) + 4 * g + (e & 3) < hi[n] ? x[e] : -__builtin_inff();
        }
        float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        if (__builtin_amdgcn_ballot_w64(top > m[n] + kSlack)) {
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          const float mn = fmaxf(m[n], top);
          const float f = __builtin_amdgcn_exp2f(m[n] - mn);
          m[n] = mn;
#pragma unroll
          for (int r = 0; r < 4; ++r) l[n][r] *= f;
#pragma unroll
          for (int j = 0; j < J; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) o[n][j][r] *= f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_exp2f(x[e] - m[n]);
        const uint4 ph = uint4{pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
        uint4 pl = uint4{0, 0, 0, 0};
        if constexpr (SPLITP)
          pl = uint4{pack2(x[0] - lo_f(ph.x), x[1] - hi_f(ph.x)), pack2(x[2] - lo_f(ph.y), x[3] - hi_f(ph.y)),
                     pack2(x[4] - lo_f(ph.z), x[5] - hi_f(ph.z)), pack2(x[6] - lo_f(ph.w), x[7] - hi_f(ph.w))};
        const uint4 ones = uint4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        l[n] = mfma(ones, ph, l[n]);
        if constexpr (SPLITP) l[n] = mfma(ones, pl, l[n]);
        if (!careful) {
#pragma unroll
          for (int j = 0; j < J; ++j) {
            o[n][j] = mfma(va[j], ph, o[n][j]);
            if constexpr (SPLITP) o[n][j] = mfma(va[j], pl, o[n][j]);
          }
        } else {
          // a value that some row must not see is not finite, and zero times
          // it would be NaN: one key at a time, added where it is seen
          for (int kk = 0; kk < 32; ++kk) {
            const int e = (kk >> 4) * 4 + (kk & 3);         // its place in lane group (kk >> 2) & 3
            const bool mine = g == ((kk >> 2) & 3);
            const bool seen = k + kk < hi[n];
#pragma unroll
            for (int j = 0; j < J; ++j) {
              uint4 one = va[j];
              const uint32_t half = (e & 1) ? 0xFFFF0000u : 0x0000FFFFu;
              one.x = mine && (e >> 1) == 0 ? one.x & half : 0u;
              one.y = mine && (e >> 1) == 1 ? one.y & half : 0u;
              one.z = mine && (e >> 1) == 2 ? one.z & half : 0u;
              one.w = mine && (e >> 1) == 3 ? one.w & half : 0u;
              f32x4 t = mfma(one, ph, f32x4{0.f, 0.f, 0.f, 0.f});
              if constexpr (SPLITP) t = mfma(one, pl, t);
#pragma unroll
              for (int r = 0; r < 4; ++r) o[n][j][r] += seen ? t[r] : 0.f;
            }
          }
        }
      }
    }
  }
};

// The sequence (group) of an item and its rows.
struct Item {
  int32_t t0, rows;   // first token; rows = tokens * (query heads of a kv head)
  int32_t len;        // keys
  const int32_t* table;
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// Tokens [*t0, *t0 + *n) of sequence b (what the bounds allow of them).
__device__ __forceinline__ void tokens_of(const AttnArgs& a, int b, int* t0, int* n) {
  const int s = clampi(a.q_start[b], 0, a.n), e = clampi(a.q_start[b + 1], 0, a.n);
  *t0 = s;
  *n = clampi(e - s, 0, a.max_q);
}
// The group that holds sequence b, -1: none.
__device__ __forceinline__ int group_of(const AttnArgs& a, int b) {
  const int lane = threadIdx.x & 63;
  int r = -1;
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    const int g = g0 + lane;
    const bool in = g < a.G && a.g_start[g] <= b && b < a.g_start[min(g + 1, a.G)];
    const uint64_t hit = __builtin_amdgcn_ballot_w64(in);
    if (hit) r = g0 + 63 - __builtin_clzll(hit);
  }
  return r;
}

template <int D, bool F8, int NRT>
__device__ __forceinline__ void load_q(Rows<D, F8, NRT>& R, const AttnArgs& a, const Item& it, int row0, int h,
                                       int nq, int first) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
#pragma unroll
  for (int n = 0; n < NRT; ++n) {
    const int row = min(row0 + 16 * n + (lane & 15), it.rows - 1);   // past the last row: the last one again
    const int tok = row / a.gq, hh = row - tok * a.gq;
    const uint16_t* p = a.q + (int64_t)(it.t0 + tok) * a.qs + (int64_t)(h * a.gq + hh) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int d = F8 ? 64 * (i >> 1) + 16 * g + 8 * (i & 1) : 32 * i + 8 * g;   // as the keys' lanes hold them
      R.q[n][i] = *reinterpret_cast<const uint4*>(p + d);
    }
    R.hi[n] = nq < 0 ? it.len : clampi(first + tok + 1, 0, it.len);
  }
}

// The four waves' sums of one block (they walked different keys for the same
// rows) joined in LDS, 16 rows at a time, and handed to `put` as D/16
// consecutive elements a thread.
template <int D, int NRT>
struct Shared {
  float ml[kWaves][16 * NRT][2];
  float o[kWaves][16][D + 4];
};
template <int D, bool F8, int NRT, class Put>
__device__ __forceinline__ void join(const Rows<D, F8, NRT>& R, Shared<D, NRT>& sh, Put put) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4, i16 = lane & 15;
  constexpr int J = D / 16;
  if (g == 0) {
#pragma unroll
    for (int n = 0; n < NRT; ++n) {
      sh.ml[wave][16 * n + i16][0] = R.m[n];
      sh.ml[wave][16 * n + i16][1] = R.l[n][0];
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NRT; ++n) {
    float m = kLow;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sh.ml[w][16 * n + i16][0]);
    const float f = __builtin_amdgcn_exp2f(R.m[n] - m);
    // element (D/16)(4 g + r) + j of row i16 is o[j][r]
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < J; j += 4) {
        f32x4 t;
#pragma unroll
        for (int u = 0; u < 4; ++u) t[u] = R.o[n][j + u][r] * f;
        *reinterpret_cast<f32x4*>(&sh.o[wave][i16][J * (4 * g + r) + j]) = t;
      }
    __syncthreads();
    const int row = tid >> 4, e = (tid & 15) * J;
    float mm = kLow, ll = 0.f, x[J];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, sh.ml[w][16 * n + row][0]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      ll += sh.ml[w][16 * n + row][1] * __builtin_amdgcn_exp2f(sh.ml[w][16 * n + row][0] - mm);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      x[j] = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) x[j] += sh.o[w][row][e + j];
    }
    put(16 * n + row, e, mm, ll, x);
    if (n + 1 < NRT) __syncthreads();
  }
}

// J = D/16 consecutive results of a row, rounded once.
template <int J>
__device__ __forceinline__ void store_y(uint16_t* p, const float* x, float f) {
  if constexpr (J == 8)
    *reinterpret_cast<uint4*>(p) = uint4{pack2(x[0] * f, x[1] * f), pack2(x[2] * f, x[3] * f), pack2(x[4] * f, x[5] * f),
                                         pack2(x[6] * f, x[7] * f)};
  else
    *reinterpret_cast<uint2*>(p) = uint2{pack2(x[0] * f, x[1] * f), pack2(x[2] * f, x[3] * f)};
}

// Split form: a block takes up to 16 NRT rows of one (sequence or group, kv
// head) and one range of its keys; its four waves share the range by quarters.
template <int D, bool F8, int NRT, bool SPLITP>
__device__ __forceinline__ void split_block(const AttnArgs& a, bool prefix, int blk, void* lds) {
  const int rb = prefix ? a.plan.rbp : a.plan.rbo, ns = prefix ? a.plan.sp : a.plan.so;
  const int chunk = prefix ? a.plan.cp : a.plan.co;
  const int r = blk % rb;
  int u = blk / rb;
  const int h = u % a.kv.heads;
  u /= a.kv.heads;
  const int s = u % ns, b = u / ns;
  Item it;
  int nt;
  if (prefix) {
    const int b0 = clampi(a.g_start[b], 0, a.B), b1 = clampi(a.g_start[b + 1], 0, a.B);
    if (b0 >= b1) return;
    it.t0 = clampi(a.q_start[b0], 0, a.n);
    nt = clampi(clampi(a.q_start[b1], 0, a.n) - it.t0, 0, a.max_gq);
    it.len = clampi(a.p_len[b], 0, a.max_pre);
    it.table = a.p_pages + (int64_t)b * a.ppw;
  } else {
    tokens_of(a, b, &it.t0, &nt);
    it.len = clampi(a.kv_len[b], 0, a.max_kv);
    it.table = a.pages + (int64_t)b * a.pw;
  }
  it.rows = nt * a.gq;
  const int row0 = r * 16 * NRT;
  if (row0 >= it.rows) return;
  const int c0 = s * chunk, c1 = min(it.len, c0 + chunk);
  if (c0 >= c1 && !a.plan.direct) return;   // the join knows it holds nothing
  Rows<D, F8, NRT> R;
  load_q(R, a, it, row0, h, prefix ? -1 : nt, it.len - nt);
  R.clear();
  Stream st;
  st.k = a.kv.k + h * a.kv.head_stride;
  st.v = a.kv.v + h * a.kv.head_stride;
  st.page_stride = a.kv.page_stride;
  st.slot_stride = (int)a.kv.slot_stride;
  st.table = it.table;
  st.shift = a.kv.shift;
  st.npages = ((it.len - 1) >> st.shift) + 1;
  st.num_pages = a.kv.num_pages;
  float c = a.scale;
  float vs = 1.f;
  if constexpr (F8) {
    if (a.kv.ks) c *= a.kv.ks[h];
    if (a.kv.vs) vs = a.kv.vs[h];
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quarter = ((c1 - c0 + 32 * kWaves - 1) / (32 * kWaves)) * 32;
  const int w0 = c0 + wave * quarter, w1 = min(c1, w0 + quarter);
  if (w0 < w1) R.template walk<SPLITP>(st, w0, w1, c);
  constexpr int J = D / 16;
  const int slot = prefix ? s : a.plan.sp + s, slots = a.plan.sp + a.plan.so;
  join<D, F8, NRT>(R, *reinterpret_cast<Shared<D, NRT>*>(lds),
                   [&](int row, int e, float m, float l, const float* x) __attribute__((always_inline)) {
    if (row0 + row >= it.rows) return;
    const int tok = (row0 + row) / a.gq, hh = (row0 + row) - tok * a.gq;
    const int64_t at = (int64_t)(it.t0 + tok) * a.hq + h * a.gq + hh;
    if (a.plan.direct) {
      store_y<J>(a.y + (int64_t)(it.t0 + tok) * a.ys + (int64_t)(h * a.gq + hh) * D + e, x, l == 0.f ? 0.f : vs / l);
      return;
    }
    const int64_t p = at * slots + slot;
#pragma unroll
    for (int j = 0; j < J; j += 4)
      *reinterpret_cast<f32x4*>(a.po + p * D + e + j) = f32x4{x[j] * vs, x[j + 1] * vs, x[j + 2] * vs, x[j + 3] * vs};
    if (e == 0) a.pml[2 * p] = m, a.pml[2 * p + 1] = l;
  });
}

template <int D, bool F8, int NO, int NP>
__global__ void __launch_bounds__(64 * kWaves, NO > 2 || NP > 2 ? 1 : 2) k_attn_split(AttnArgs a, int npre) {
  constexpr int NM = NO > NP ? NO : NP;
  __shared__ Shared<D, NM> sh;
  const int blk = blockIdx.x;
  if (blk < npre)
    split_block<D, F8, NP, NP == 1>(a, true, blk, &sh);
  else
    split_block<D, F8, NO, NO == 1>(a, false, blk - npre, &sh);
}

// Joins the splits of a row: one wave a row, D/64 elements a lane.
template <int D>
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= (int64_t)a.n * a.hq) return;
  const int tok = (int)(row / a.hq), h = (int)(row - (int64_t)tok * a.hq);
  // the token's sequence: the last one that starts at or before it
  int b = -1;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int i = b0 + lane;
    const bool in = i < a.B && a.q_start[i] <= tok && tok < a.q_start[i + 1];
    const uint64_t hit = __builtin_amdgcn_ballot_w64(in);
    if (hit) b = b0 + 63 - __builtin_clzll(hit);
  }
  if (b < 0) return;   // behind the last sequence: left as it is
  int t0, nt;
  tokens_of(a, b, &t0, &nt);
  if (tok - t0 >= nt) return;
  const int len = clampi(a.kv_len[b], 0, a.max_kv);
  const int no = (len + a.plan.co - 1) / a.plan.co;
  int np = 0;
  const int gr = group_of(a, b);
  if (gr >= 0) np = (clampi(a.p_len[gr], 0, a.max_pre) + a.plan.cp - 1) / a.plan.cp;
  const int slots = a.plan.sp + a.plan.so;
  const float* ml = a.pml + 2 * row * slots;
  const float* o = a.po + row * slots * D + lane * (D / 64);
  float m = kLow, l = 0.f, x[D / 64];
#pragma unroll
  for (int j = 0; j < D / 64; ++j) x[j] = 0.f;
  for (int s = 0; s < slots; ++s)
    if (s < np || (s >= a.plan.sp && s - a.plan.sp < no)) m = fmaxf(m, ml[2 * s]);
  for (int s = 0; s < slots; ++s) {
    if (!(s < np || (s >= a.plan.sp && s - a.plan.sp < no))) continue;
    const float f = __builtin_amdgcn_exp2f(ml[2 * s] - m);
    l += ml[2 * s + 1] * f;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) x[j] += o[(int64_t)s * D + j] * f;
  }
  const float f = l == 0.f ? 0.f : 1.f / l;
  uint16_t* y = a.y + (int64_t)tok * a.ys + (int64_t)h * D + lane * (D / 64);
  if constexpr (D == 128)
    *reinterpret_cast<uint32_t*>(y) = pack2(x[0] * f, x[1] * f);
  else
    *y = (uint16_t)pack2(x[0] * f, 0.f);
}

// Long queries: a block takes 4 waves x 16 NRT rows of one (sequence, kv
// head); every wave walks all keys its rows see, the prefix first, so that
// the block's waves find the keys in the caches.  Blocks of one (sequence, kv
// head) follow each other on one XCD, the longest rows first.
template <int D, bool F8, int NRT>
__global__ void __launch_bounds__(64 * kWaves, NRT > 2 ? 1 : 2) k_attn_rows(AttnArgs a) {
  const int xcd = blockIdx.x & 7, j8 = blockIdx.x >> 3;
  const int rb = a.plan.rbo;
  const int pair = (j8 / rb) * 8 + xcd, rblk = rb - 1 - j8 % rb;
  if (pair >= a.B * a.kv.heads) return;
  const int b = pair / a.kv.heads, h = pair - b * a.kv.heads;
  Item it;
  int nt;
  tokens_of(a, b, &it.t0, &nt);
  it.rows = nt * a.gq;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int row0 = (rblk * kWaves + wave) * 16 * NRT;
  if (row0 >= it.rows) return;
  Rows<D, F8, NRT> R;
  R.clear();
  Stream st;
  st.k = a.kv.k + h * a.kv.head_stride;
  st.v = a.kv.v + h * a.kv.head_stride;
  st.page_stride = a.kv.page_stride;
  st.slot_stride = (int)a.kv.slot_stride;
  st.shift = a.kv.shift;
  st.num_pages = a.kv.num_pages;
  float c = a.scale, vs = 1.f;
  if constexpr (F8) {
    if (a.kv.ks) c *= a.kv.ks[h];
    if (a.kv.vs) vs = a.kv.vs[h];
  }
  const int gr = group_of(a, b);
  for (int part = gr < 0 ? 1 : 0; part < 2; ++part) {
    it.len = part == 0 ? clampi(a.p_len[gr], 0, a.max_pre) : clampi(a.kv_len[b], 0, a.max_kv);
    it.table = part == 0 ? a.p_pages + (int64_t)gr * a.ppw : a.pages + (int64_t)b * a.pw;
    load_q(R, a, it, row0, h, part == 0 ? -1 : nt, it.len - nt);
    st.table = it.table;
    st.npages = ((it.len - 1) >> st.shift) + 1;
    if (it.len > 0) R.template walk<false>(st, 0, it.len, c);
  }
  constexpr int J = D / 16;
#pragma unroll
  for (int n = 0; n < NRT; ++n) {
    const int row = row0 + 16 * n + (lane & 15);
    if (row >= it.rows) continue;
    const int tok = row / a.gq, hh = row - tok * a.gq;
    const float f = R.l[n][0] == 0.f ? 0.f : vs / R.l[n][0];
    uint16_t* y = a.y + (int64_t)(it.t0 + tok) * a.ys + (int64_t)(h * a.gq + hh) * D + J * 4 * (lane >> 4);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x[J];
#pragma unroll
      for (int j = 0; j < J; ++j) x[j] = R.o[n][j][r];
      store_y<J>(y + J * r, x, f);
    }
  }
}

template <int D, bool F8>
void go(const AttnArgs& a) {
  hipStream_t st = reinterpret_cast<hipStream_t>(a.stream);
  const AttnPlan& p = a.plan;
  if (p.rows) {
    const unsigned pairs = (unsigned)(((int64_t)a.B * a.kv.heads + 7) / 8 * 8);
    hipLaunchKernelGGL((k_attn_rows<D, F8, 4>), dim3(pairs * p.rbo), dim3(64 * kWaves), 0, st, a);
    return;
  }
  const int npre = a.G * a.kv.heads * p.rbp * p.sp, nown = a.B * a.kv.heads * p.rbo * p.so;
  const dim3 g((unsigned)(npre + nown)), blk(64 * kWaves);
  if (p.ro == 1) {
    if (p.rp == 1) hipLaunchKernelGGL((k_attn_split<D, F8, 1, 1>), g, blk, 0, st, a, npre);
    else if (p.rp == 2) hipLaunchKernelGGL((k_attn_split<D, F8, 1, 2>), g, blk, 0, st, a, npre);
    else hipLaunchKernelGGL((k_attn_split<D, F8, 1, 4>), g, blk, 0, st, a, npre);
  } else {
    hipLaunchKernelGGL((k_attn_split<D, F8, 2, 2>), g, blk, 0, st, a, npre);
  }
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
