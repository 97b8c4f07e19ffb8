// Device pieces that the attention kernels share.  Included inside namespace
// dc, anonymous namespace, of k_attn.hip.
#pragma once

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLow = -3.402823466e38f;   // the maximum of a row that has seen no key
// The running maximum of a row moves only when a score passes it by this
// (in powers of 2): most steps then leave the sums as they are, and a weight
// reaches 2^12 instead of 1, which floats do not mind.
constexpr float kSlack = 12.f;
constexpr int kWaves = 4;

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
// The top bits of those of a bf16 pair (e4m3 quadruple) that are not finite.
template <bool F8> __device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return F8 ? ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u : ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
// w with those replaced by zero.
template <bool F8> __device__ __forceinline__ uint32_t only_finite(uint32_t w, uint32_t odd) {
  if constexpr (F8) return w & ~((odd >> 7) * 0xFFu);
  return w & ~((odd >> 15) * 0xFFFFu);
}

// N words (or, N = 0, half a word) of a cache row.
template <int N> struct Words { uint32_t w[N ? N : 1]; };
template <int N> __device__ __forceinline__ Words<N> load_words(const uint8_t* p) {
  Words<N> r;
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else if constexpr (N == 1) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
  return r;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// The keys of one kv head of a sequence or a prefix, in pages.
struct Stream {
  const uint8_t *k, *v;     // of the head
  int64_t page_stride;
  int32_t slot_stride;      // a page's slots lie within 2^31 bytes
  const int32_t* table;
  int32_t width;            // entries of the table (those that hold no keys are read, not used)
  int32_t num_pages;        // pages of the cache
  int32_t shift;            // log2 of a page's slots
};

// Of a kv head; a sequence's own keys or a group's prefix.
__device__ __forceinline__ Stream stream_of(const AttnArgs& a, int h, const int32_t* table, int width) {
  Stream st;
  st.k = a.kv.k + h * a.kv.head_stride;
  st.v = a.kv.v + h * a.kv.head_stride;
  st.page_stride = a.kv.page_stride;
  st.slot_stride = (int)a.kv.slot_stride;
  st.table = table;
  st.width = width;
  st.shift = a.kv.shift;
  st.num_pages = a.kv.num_pages;
  return st;
}

__device__ __forceinline__ Stream own_stream(const AttnArgs& a, int h, int b) {
  return stream_of(a, h, a.pages + (int64_t)b * a.pw, a.pw);
}
__device__ __forceinline__ Stream prefix_stream(const AttnArgs& a, int h, int g) {
  return stream_of(a, h, a.p_pages + (int64_t)g * a.ppw, a.ppw);
}

// A stream's page numbers, 64 of them in a register, one a lane.
struct Pages {
  int base, pg;
  __device__ __forceinline__ void fill(const Stream& st, int p) {
    base = p;
    pg = st.table[min(p + (int)(threadIdx.x & 63), st.width - 1)];   // (used, and so waited for, by offset)
  }
  // Byte offset of key `at` (the first of 16 that share a page); ascending.
  __device__ __forceinline__ int64_t offset(const Stream& st, int at) {
    const int p = at >> st.shift;
    if (__builtin_expect(p - base >= 64, 0)) {
      fill(st, p);
      asm volatile("" : "+v"(pg));   // waited for here, not by the code that both ways share
    }
    const int n = __builtin_amdgcn_readlane(pg, p - base);
    const int64_t page = (unsigned)n < (unsigned)st.num_pages ? n : 0;   // never outside the cache
    return page * st.page_stride + (int64_t)(at & ((1 << st.shift) - 1)) * st.slot_stride;
  }
};

// What a step left out.  Zero times a value that is not finite would be NaN,
// so where some row must not see some key (its weight is zero), the products
// take such values as zero, and the rows that do see the key get them here,
// element by element.  (A weight is positive, so the value stands for weight
// times value.)
__device__ __forceinline__ const uint8_t* value_row(const Stream& st, int key) {
  int pg = st.table[min(key >> st.shift, st.width - 1)];
  pg = (unsigned)pg < (unsigned)st.num_pages ? pg : 0;
  return st.v + pg * st.page_stride + (int64_t)(key & ((1 << st.shift) - 1)) * st.slot_stride;
}
template <bool F8> __device__ __forceinline__ f32x2 unfinite_pair(const uint8_t* row, int e, bool seen) {
  const uint32_t w = F8 ? cvt2(*reinterpret_cast<const uint16_t*>(row + e), false)
                        : *reinterpret_cast<const uint32_t*>(row + 2 * e);
  const float a = lo_f(w), b = hi_f(w);
  return f32x2{seen && !__builtin_isfinite(a) ? a : 0.f, seen && !__builtin_isfinite(b) ? b : 0.f};
}
// Where every row sees every key of a step, values go into the products as they
// are.  An infinite one can then end as NaN: times a weight that is too small
// for its type, or times the second piece of a weight, which may be zero or
// negative.  So a block whose results are not all finite, though its rows'
// weights are, does its work once more and treats every step as one with masks
// (finite data pays for looking at the results only).  A row's sums of finite
// values are the same both times, bit for bit.

// The factor of sums of values whose maximum has moved.  Where it is zero (an
// exponential is, or 2^-126 or more), infinite sums stay and finite ones vanish
// all the same, as 2^-126 times 2^-126 of them.
struct Factor {
  float f, g;
  explicit __device__ __forceinline__ Factor(float x) : f(fmaxf(x, 0x1p-126f)), g(x < 0x1p-126f ? 0x1p-126f : 1.f) {}
  __device__ __forceinline__ float of(float x) const { return x * f * g; }
};

// The block's arguments, number and thread, taken anew each time it does its work:
// what is derived from them would else be kept for a second time and cost
// registers in the walk.
__device__ __forceinline__ const AttnArgs& args_anew() {
  auto p = (const __attribute__((address_space(4))) AttnArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnArgs*)p;
}
__device__ __forceinline__ int block_anew() {
  int b = blockIdx.x;
  asm volatile("" : "+s"(b));
  return b;
}
// (and both times by the same code)
__device__ __forceinline__ bool one_code(int again) {
  asm volatile("" : "+s"(again));
  return again != 0;
}
__device__ __forceinline__ int thread_anew() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// The query rows of a sequence (of a group) for one kv head: row r is token
// t0 + r / gq, query head r % gq of the kv head's.
struct Item {
  int32_t t0, nt, rows;
  int32_t len;            // keys
  int32_t first;          // own keys: token j sees first + j + 1 of them
  bool causal;
  // keys that token tok sees
  __device__ __forceinline__ int sees(int tok) const { return causal ? clampi(first + tok + 1, 0, len) : len; }
};

// Sequence b with its own keys; what the bounds do not cover is cut.
__device__ __forceinline__ Item own_item(const AttnArgs& a, int b) {
  Item it;
  const int s = clampi(a.q_start[b], 0, a.n), e = clampi(a.q_start[b + 1], 0, a.n);
  it.t0 = s;
  it.nt = clampi(e - s, 0, a.max_q);
  it.rows = it.nt * a.gq;
  it.len = clampi(a.kv_len[b], 0, a.max_kv);
  it.first = it.len - it.nt;
  it.causal = true;
  return it;
}
// The tokens of group g's sequences with its prefix.
__device__ __forceinline__ Item prefix_item(const AttnArgs& a, int g) {
  Item it;
  const int b0 = clampi(a.g_start[g], 0, a.B), b1 = clampi(a.g_start[g + 1], 0, a.B);
  const int s = clampi(a.q_start[b0], 0, a.n), e = clampi(a.q_start[b1], 0, a.n);
  it.t0 = s;
  it.nt = b0 < b1 ? clampi(e - s, 0, a.max_gq) : 0;
  it.rows = it.nt * a.gq;
  it.len = clampi(a.p_len[g], 0, a.max_pre);
  it.first = 0;
  it.causal = false;
  return it;
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

// The factor of the scores, positive: a negative scale of the keys (they are
// the caller's numbers) turns the queries' sign instead, and zero is the
// smallest number, so that a masked score stays minus infinity.
template <bool F8> __device__ __forceinline__ float score_factor(const AttnArgs& a, int h, uint32_t* flip) {
  float c = a.scale;
  *flip = 0;
  if constexpr (F8) {
    if (a.kv.ks) c *= a.kv.ks[h];
    if (c < 0.f) *flip = 0x80008000u;
    c = fabsf(c);
    if (c == 0.f) c = 1.1754944e-38f;
  }
  return c;
}
template <bool F8> __device__ __forceinline__ float value_scale(const AttnArgs& a, int h) {
  return F8 && a.kv.vs ? a.kv.vs[h] : 1.f;
}

// J consecutive results of a row, rounded once.
template <int J> __device__ __forceinline__ void store_y(uint16_t* p, const float* x, float f) {
  if constexpr (J == 8)
    *reinterpret_cast<uint4*>(p) = uint4{pack2(x[0] * f, x[1] * f), pack2(x[2] * f, x[3] * f), pack2(x[4] * f, x[5] * f),
                                         pack2(x[6] * f, x[7] * f)};
  else
    *reinterpret_cast<uint2*>(p) = uint2{pack2(x[0] * f, x[1] * f), pack2(x[2] * f, x[3] * f)};
}
