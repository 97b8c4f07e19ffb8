// Internal declarations of the decoder-layer operators: the paged key/value
// cache (append, attention) and the 4-bit backbone.  Not part of the public
// ABI (include/deltacome.h is).
#pragma once

#include "dc_internal.h"

namespace dc {

// The cache as the kernels see it: strides in bytes.
struct KvArgs {
  uint8_t* k;
  uint8_t* v;
  const float* ks;     // per kv head, null: 1
  const float* vs;
  int64_t page_stride, head_stride, slot_stride;
  int32_t heads, num_pages;
  int32_t shift;       // log2 of the tokens per page
};

struct AppendArgs {
  KvArgs kv;
  const uint16_t *q, *k, *v;
  int64_t qs, ks, vs, qos;   // row strides, elements
  const int32_t* pos;
  const int64_t* slots;
  const double* freq;
  uint16_t* qo;
  int32_t hq, dim, rot, interleaved, e4m3, n;
  void* stream;
};
int launch_append(const AppendArgs& a);

// n / d for 0 <= n < 2^31 with one multiplication: floor(n M / 2^(32+s)) with
// M = ceil(2^(32+s) / d) and 2^s < d <= 2^(s+1) (M < 2^32; exact for 31 bits).
struct Div {
  uint32_t m;
  int32_t s, d;
#if defined(__HIPCC__)
  __device__ __forceinline__ int32_t of(int32_t n) const { return d == 1 ? n : (int32_t)(__umulhi((uint32_t)n, m) >> s); }
#endif
};
inline Div div_by(int32_t d) {
  Div r{0, 0, d < 1 ? 1 : d};
  if (r.d == 1) return r;
  while ((INT64_C(2) << r.s) < r.d) ++r.s;
  r.m = (uint32_t)(((UINT64_C(1) << (32 + r.s)) + (uint64_t)r.d - 1) / (uint64_t)r.d);
  return r;
}

// How one attention call is split, from the host's bounds alone (the lengths
// stay on the device).
struct AttnPlan {
  bool rows;          // long queries: a block walks all keys of its 128 rows; else the keys are split
  int32_t wo, wp;     // split form, own keys / prefixes: by Keys of 16 or 32 rows (1, 2), by Tiles (3); wo <= wp
  int32_t rbo, rbp;   // row blocks of a sequence / of a group
  int32_t so, sp;     // key splits of a sequence's own keys / of a prefix
  int32_t co, cp;     // keys of a split (multiples of 128)
  bool direct;        // one split in all: the outputs are written at once
  Div rbo_d, rbp_d, so_d, sp_d;
  Div heavy_d, light_d;   // rows: row blocks of a sequence that come first, and last
  size_t o_off, ws;   // split form: partial sums at o_off of the workspace, its size
};

struct AttnArgs {
  KvArgs kv;
  AttnPlan plan;
  const uint16_t* q;
  uint16_t* y;
  int64_t qs, ys;     // row strides, elements
  float scale;        // times log2(e)
  int32_t hq, gq, n, dim, e4m3;
  Div hq_d, gq_d, hkv_d;
  int32_t B, max_q, max_kv, pw;
  const int32_t *q_start, *kv_len, *pages;
  int32_t G, max_gq, max_pre, ppw;
  const int32_t *g_start, *p_len, *p_pages;
  float* po;          // [n * hq][sp + so][dim] partial sums
  float* pml;         // [n * hq][sp + so][2] their maxima and weights
  void* stream;
};
AttnPlan attn_plan(int32_t hkv, int32_t gq, int32_t dim, int32_t n, int32_t B, int32_t max_q, int32_t max_kv, int32_t G,
                   int32_t max_gq, int32_t max_pre);
int launch_attention(const AttnArgs& a);

struct W4Args {
  const uint8_t* w;
  const uint16_t* x;
  uint16_t* y;
  int32_t out, in, T;
  void* stream;
};
int launch_w4(const W4Args& a);
int launch_w4_pack(int32_t out, int32_t in, const uint16_t* W, uint8_t* dst, uint32_t* flag, void* stream);

}  // namespace dc
