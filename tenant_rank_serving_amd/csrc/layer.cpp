// Entry points of the decoder-layer operators (paged key/value cache, 4-bit
// backbone): argument checks on the host, then one launcher.  No allocation,
// no synchronization.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "layer.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows of `w` bytes, `n` of them `stride` bytes apart: whether two such
// buffers share a byte.  Buffers of one stride may be interleaved (columns of
// one fused matrix); of other pairs whose ranges meet nothing is known, so
// they count as sharing.
bool rows_meet(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t n) {
  if (n <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const uintptr_t xe = x + (uintptr_t)((n - 1) * sa + wa), ye = y + (uintptr_t)((n - 1) * sb + wb);
  if (xe <= y || ye <= x) return false;
  if (n == 1 || sa != sb) return true;
  const int64_t d = (int64_t)((y >= x ? y - x : x - y) % (uintptr_t)sa);
  const int64_t u = y >= x ? wa : wb, v = y >= x ? wb : wa;   // the lower buffer's rows, the upper one's
  return d < u || d + v > sa;
}

// The bytes from the first row's first to the last row's last.
int64_t rows_span(int64_t stride, int64_t w, int64_t n) { return (n - 1) * stride + w; }

bool spans_meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// Whether n bytes at p reach into the cache's keys or values (into a page, not
// into room between pages).
bool in_cache(const dc::KvArgs& k, int64_t dim_bytes, const void* p, int64_t n) {
  const int64_t page =
      (k.heads - 1) * k.head_stride + ((INT64_C(1) << k.shift) - 1) * k.slot_stride + dim_bytes;
  const int64_t all = (k.num_pages - 1) * k.page_stride + page;
  for (const uint8_t* base : {k.k, k.v}) {
    if (!spans_meet(base, all, p, n)) continue;
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(base);
    if (x < b || k.num_pages == 1) return true;
    const int64_t at = (int64_t)((x - b) % (uintptr_t)k.page_stride);
    if (at < page || at + n > k.page_stride) return true;
  }
  return false;
}

bool mul_fits(int64_t a, int64_t b, int64_t lim) { return a == 0 || b <= lim / a; }

// A launch's threads along x are numbered with 32 bits; blocks of 256.
constexpr int64_t kMostBlocks = UINT32_MAX / 256;

// The cache's shape and strides; fills the kernels' view of it.
dc_status check_cache(const dc_kv_cache* c, dc::KvArgs* k) {
  if (!c) return DC_ERR_INVALID_ARG;
  if (c->dtype != DC_KV_BF16 && c->dtype != DC_KV_E4M3) return DC_ERR_INVALID_ARG;
  if (c->heads < 1 || (c->dim != 64 && c->dim != 128) || c->num_pages < 1) return DC_ERR_SHAPE;
  if (c->page < 16 || c->page > 1024 || (c->page & (c->page - 1))) return DC_ERR_SHAPE;
  if (!c->k || !c->v) return DC_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return DC_ERR_ALIGN;
  const int64_t e = c->dtype == DC_KV_BF16 ? 2 : 1;
  if (c->dtype == DC_KV_BF16 && (c->k_scale || c->v_scale)) return DC_ERR_INVALID_ARG;
  const int64_t lim = INT64_C(1) << 62;
  if (c->slot_stride < c->dim || c->head_stride < c->dim || c->page_stride < c->dim) return DC_ERR_SHAPE;
  if ((c->slot_stride * e) % 16 || (c->head_stride * e) % 16 || (c->page_stride * e) % 16) return DC_ERR_ALIGN;
  // no two rows share an element: heads behind slots or slots behind heads, pages behind both
  if (!mul_fits(c->page, c->slot_stride, lim / 4) || !mul_fits(c->heads, c->head_stride, lim / 4) ||
      !mul_fits(c->num_pages, c->page_stride, lim / 4))
    return DC_ERR_UNSUPPORTED;
  const int64_t slots = (c->page - 1) * c->slot_stride + c->dim, heads = (c->heads - 1) * c->head_stride + c->dim;
  if (!(c->heads == 1 || c->head_stride >= slots || c->slot_stride >= heads)) return DC_ERR_SHAPE;
  if (c->num_pages > 1 && c->page_stride < (c->page - 1) * c->slot_stride + (c->heads - 1) * c->head_stride + c->dim)
    return DC_ERR_SHAPE;
  if (slots * e > INT32_MAX / 2) return DC_ERR_UNSUPPORTED;   // 32-bit offsets inside a page
  k->k = static_cast<uint8_t*>(c->k);
  k->v = static_cast<uint8_t*>(c->v);
  k->ks = c->k_scale;
  k->vs = c->v_scale;
  k->page_stride = c->page_stride * e;
  k->head_stride = c->head_stride * e;
  k->slot_stride = c->slot_stride * e;
  k->heads = c->heads;
  k->num_pages = c->num_pages;
  k->shift = 0;
  while ((1 << k->shift) < c->page) ++k->shift;
  return DC_OK;
}

// A row-strided bf16 matrix [n][cols], within 2^47 bytes.
dc_status check_rows(const void* p, int64_t stride, int64_t cols, int64_t n) {
  if (!p) return DC_ERR_INVALID_ARG;
  if (stride < cols || !mul_fits(n > 1 ? n : 1, stride, INT64_C(1) << 46)) return DC_ERR_SHAPE;
  if (!aligned(p, 16) || stride % 8) return DC_ERR_ALIGN;
  return DC_OK;
}

dc_status check_batch(const dc_kv_cache* kv, const dc_attn_batch* b, int32_t q_heads, int32_t N) {
  if (!b || N < 0 || q_heads < 1) return DC_ERR_INVALID_ARG;
  if (q_heads % kv->heads) return DC_ERR_SHAPE;
  if (b->seqs < 0 || b->max_q < 0 || b->max_kv < 0 || b->groups < 0 || b->max_group_q < 0 || b->max_prefix < 0)
    return DC_ERR_INVALID_ARG;
  if (b->seq_pages < 0 || b->prefix_pages_per_group < 0) return DC_ERR_INVALID_ARG;
  if ((int64_t)b->seq_pages * kv->page < b->max_kv) return DC_ERR_SHAPE;
  if (b->groups > 0 && (int64_t)b->prefix_pages_per_group * kv->page < b->max_prefix) return DC_ERR_SHAPE;
  // the kernels number query rows and keys with 32 bits
  if ((int64_t)N * q_heads > INT32_MAX || (int64_t)b->max_q * q_heads > INT32_MAX / 2 ||
      (int64_t)b->max_group_q * q_heads > INT32_MAX / 2 || b->max_kv > INT32_MAX / 2 || b->max_prefix > INT32_MAX / 2)
    return DC_ERR_UNSUPPORTED;
  return DC_OK;
}

// Blocks of either form.
int64_t blocks_of(const dc::AttnPlan& p, int64_t B, int64_t G, int64_t heads) {
  if (p.rows) return (B * heads + 7) / 8 * 8 * p.rbo;
  return B * heads * p.rbo * p.so + G * heads * p.rbp * p.sp;
}

}  // namespace

namespace dc {

constexpr int64_t kOwnBlocks = 256, kPrefixBlocks = 512;

AttnPlan attn_plan(int32_t hkv, int32_t gq, int32_t dim, int32_t n, int32_t B, int32_t max_q, int32_t max_kv, int32_t G,
                   int32_t max_gq, int32_t max_pre) {
  AttnPlan p{};
  const int64_t ro = (int64_t)max_q * gq, rg = (int64_t)max_gq * gq;   // query rows of a sequence, of a group
  if (max_pre == 0 || max_gq == 0) G = 0;
  // long queries: enough blocks of 128 rows to fill the card, or to get through
  // few keys before split ones are joined (us, in rows / split: 256 blocks x
  // 4096 keys 108 / 110; 512 x 8192 263 / 274; 128 x 512 18.7 / 26.6, x 1024
  // 31.6 / 33.5, x 2048 56 / 47; 64 x 512 18.3 / 21.1, x 1024 31 / 25)
  const int64_t rb = (ro + 127) / 128, all = (int64_t)B * hkv * rb;
  // Each of those blocks walks its sequence's prefix too; split, the blocks of a
  // prefix are filled from all rows of its group, at the price of partial sums.
  // Keys walked by blocks, in rows / split (us, in rows / split; 36 rows of a
  // sequence and kv head, 8 kv heads, 300 own keys): 64 sequences on one prefix
  // of 16384 3.4 (433 / 208), of 2048 2.7 (78 / 60), of 512 1.8 (38 / 47); on 8
  // of 16384 2.6 (436 / 287), of 2048 2.2 (75 / 70), of 512 1.7 (36 / 48); 64
  // rows, one prefix of 16384 2.0 (434 / 310), of 2048 1.8 (76 / 76); 128 rows
  // (filled blocks) of 16384 1.0 (526 / 567).
  const int64_t keys = (int64_t)max_kv + (G > 0 ? max_pre : 0);
  const double in_rows = (double)B * rb * keys, in_split = (double)G * ((rg + 127) / 128) * max_pre + (double)B * rb * max_kv;
  const bool shared = G > 0 && in_rows >= 1.9 * in_split && ((int64_t)n * hkv * gq + 3) / 4 <= kMostBlocks;   // (a join of theirs)
  if (ro > 32 && !shared && (all >= 256 || (all >= 64 && keys <= 8 * all))) {
    p.rows = true;
    p.rbo = (int32_t)rb;
    p.co = p.cp = 128;
    p.direct = true;
    return p;
  }
  // us, 16 rows / 32 / 128 at a time: 8 x 4000 e4m3 keys with 16 rows 16.6 / 18.3
  // / -, with 32 rows 19.8 by 32, 31.5 by 128; with 48 rows 36.6 by 32 twice, 37.8
  auto walk = [](int64_t rows) { return rows <= 16 ? 1 : (rows <= 32 ? 2 : 3); };
  p.wo = walk(ro);
  p.wp = walk(rg) > p.wo ? walk(rg) : p.wo;
  auto blocks = [](int64_t rows, int32_t how) { return (int32_t)(how == 3 ? (rows + 127) / 128 : (rows + 16 * how - 1) / (16 * how)); };
  p.rbo = blocks(ro, p.wo);
  p.rbp = blocks(rg, p.wp);
  // n ranges of keys for each item, of 128 (a step a wave) or more
  auto split = [](int64_t n, int64_t keys, int64_t least, int32_t* s, int32_t* c) {
    const int64_t most = (keys + least - 1) / least;
    if (n > most) n = most;
    if (n > 64) n = 64;
    if (n < 1) n = 1;
    int64_t ch = ((keys + n - 1) / n + 127) / 128 * 128;
    if (ch < 128) ch = 128;
    *c = (int32_t)ch;
    *s = (int32_t)((keys + ch - 1) / ch);
  };
  // few keys and few rows: one range, which needs no join (256 keys 8.5 -> 6.1
  // us, 512: 8.4 -> 8.3, 640: 9.9 -> 10.6; 64 rows on 384 keys 11.8 -> 15.1)
  const bool one = G == 0 && p.wo < 3 && max_kv <= 512;
  const int64_t own = std::max<int64_t>((int64_t)B * hkv * p.rbo, 1), pre = std::max<int64_t>((int64_t)G * hkv * p.rbp, 1);
  // a block a CU (4 x 131072 keys 260 us, with two 265; own keys behind a long
  // prefix fill its end anyway)
  split(one ? 1 : (kOwnBlocks + own - 1) / own, max_kv, 128, &p.so, &p.co);
  p.cp = 128;
  // two a CU and no more, each of 256 keys or more when there are that many:
  // every range costs its rows' partial sums (20 rows of 4 on 4000 keys, ranges
  // of 128: 23.0 us, of 256: 19.2; on 400 keys 14.4 and 16.5)
  if (G > 0) split(kPrefixBlocks / pre, max_pre, max_pre > 512 ? 256 : 128, &p.sp, &p.cp);
  if (p.sp == 0 && p.so <= 1) {
    p.so = 1;
    p.direct = true;
    return p;
  }
  const size_t rows = (size_t)n * hkv * gq, slots = (size_t)p.sp + p.so;
  p.o_off = round_up(8 * rows * slots, kAlign);
  p.ws = round_up(p.o_off + 4 * rows * slots * dim, kAlign);
  return p;
}

}  // namespace dc

extern "C" {

dc_status dc_kv_append(const dc_kv_cache* kv, const dc_rope* rope, const uint16_t* q, int64_t q_stride,
                       const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* pos,
                       const int64_t* slots, uint16_t* q_out, int64_t q_out_stride, int32_t q_heads, int32_t N,
                       void* stream) {
  dc::AppendArgs a{};
  dc_status st = check_cache(kv, &a.kv);
  if (st != DC_OK) return st;
  if (N < 0 || q_heads < 0) return DC_ERR_INVALID_ARG;
  const int64_t qc = (int64_t)q_heads * kv->dim, kc = (int64_t)kv->heads * kv->dim;
  if ((qc + 2 * kc) / 16 > 65535 * 256) return DC_ERR_UNSUPPORTED;   // a launch's blocks along y
  if (rope) {
    if (rope->rot < 16 || rope->rot > kv->dim || rope->rot % 16) return DC_ERR_SHAPE;
    if (!rope->inv_freq || !pos) return DC_ERR_INVALID_ARG;
    if (!aligned(rope->inv_freq, 8) || !aligned(pos, 4)) return DC_ERR_ALIGN;
  }
  if (q_heads > 0) {
    if ((st = check_rows(q, q_stride, qc, N)) != DC_OK) return st;
    if ((st = check_rows(q_out, q_out_stride, qc, N)) != DC_OK) return st;
    const bool in_place = q == q_out && q_stride == q_out_stride;
    if (!in_place && rows_meet(q, 2 * q_stride, 2 * qc, q_out, 2 * q_out_stride, 2 * qc, N)) return DC_ERR_INVALID_ARG;
  }
  if ((st = check_rows(k, k_stride, kc, N)) != DC_OK) return st;
  if ((st = check_rows(v, v_stride, kc, N)) != DC_OK) return st;
  if (q_heads > 0 && (rows_meet(k, 2 * k_stride, 2 * kc, q_out, 2 * q_out_stride, 2 * qc, N) ||
                      rows_meet(v, 2 * v_stride, 2 * kc, q_out, 2 * q_out_stride, 2 * qc, N)))
    return DC_ERR_INVALID_ARG;
  if (!slots) return DC_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return DC_ERR_ALIGN;
  if (N > kMostBlocks) return DC_ERR_UNSUPPORTED;   // a block a token
  if (N == 0) return DC_OK;
  const int64_t row = (int64_t)kv->dim * (kv->dtype == DC_KV_BF16 ? 2 : 1);
  if (q_heads > 0 && in_cache(a.kv, row, q_out, rows_span(2 * q_out_stride, 2 * qc, N))) return DC_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.qos = q_out_stride;
  a.pos = pos;
  a.slots = slots;
  a.freq = rope ? rope->inv_freq : nullptr;
  a.qo = q_out;
  a.hq = q_heads;
  a.dim = kv->dim;
  a.rot = rope ? rope->rot : 0;
  a.interleaved = rope ? rope->interleaved != 0 : 0;
  a.e4m3 = kv->dtype == DC_KV_E4M3;
  a.n = N;
  a.stream = stream;
  return dc::launch_append(a) == 0 ? DC_OK : DC_ERR_HIP;
}

size_t dc_attention_workspace_bytes(const dc_kv_cache* kv, const dc_attn_batch* b, int32_t q_heads, int32_t N) {
  dc::KvArgs k{};
  if (check_cache(kv, &k) != DC_OK || check_batch(kv, b, q_heads, N) != DC_OK) return 0;
  const dc::AttnPlan p = dc::attn_plan(kv->heads, q_heads / kv->heads, kv->dim, N, b->seqs, b->max_q, b->max_kv,
                                       b->groups, b->max_group_q, b->max_prefix);
  return p.ws > 0 ? p.ws : dc::kAlign;
}

dc_status dc_attention(const dc_kv_cache* kv, const dc_attn_batch* b, const uint16_t* q, int64_t q_stride,
                       int32_t q_heads, float scale, uint16_t* y, int64_t y_stride, int32_t N, void* ws,
                       size_t ws_bytes, void* stream) {
  dc::AttnArgs a{};
  dc_status st = check_cache(kv, &a.kv);
  if (st != DC_OK) return st;
  if ((st = check_batch(kv, b, q_heads, N)) != DC_OK) return st;
  // the kernels' exponentials are base 2; a factor of zero or infinity would
  // turn masked or zero scores into NaN
  const float base2 = (float)((double)scale * 1.4426950408889634074);
  if (!(scale >= FLT_MIN) || !std::isfinite(base2)) return DC_ERR_INVALID_ARG;
  const int64_t qc = (int64_t)q_heads * kv->dim;
  if ((st = check_rows(q, q_stride, qc, N)) != DC_OK) return st;
  if ((st = check_rows(y, y_stride, qc, N)) != DC_OK) return st;
  if (rows_meet(q, 2 * q_stride, 2 * qc, y, 2 * y_stride, 2 * qc, N)) return DC_ERR_INVALID_ARG;
  if (!ws) return DC_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return DC_ERR_ALIGN;
  if (b->seqs > 0) {
    if (!b->q_start || !b->kv_len || (b->max_kv > 0 && !b->pages)) return DC_ERR_INVALID_ARG;
    if (!aligned(b->q_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->pages, 4)) return DC_ERR_ALIGN;
  }
  if (b->groups > 0) {
    if (!b->group_start || !b->prefix_len || (b->max_prefix > 0 && !b->prefix_pages)) return DC_ERR_INVALID_ARG;
    if (!aligned(b->group_start, 4) || !aligned(b->prefix_len, 4) || !aligned(b->prefix_pages, 4)) return DC_ERR_ALIGN;
  }
  a.plan = dc::attn_plan(kv->heads, q_heads / kv->heads, kv->dim, N, b->seqs, b->max_q, b->max_kv, b->groups,
                         b->max_group_q, b->max_prefix);
  if (ws_bytes < a.plan.ws) return DC_ERR_BUFFER;
  if (blocks_of(a.plan, b->seqs, b->groups, kv->heads) > kMostBlocks) return DC_ERR_UNSUPPORTED;
  if (!a.plan.direct && ((int64_t)N * q_heads + 3) / 4 > kMostBlocks) return DC_ERR_UNSUPPORTED;   // the join
  if (N == 0 || b->seqs == 0 || b->max_q == 0) return DC_OK;   // no query: nothing to write
  const int64_t row = (int64_t)kv->dim * (kv->dtype == DC_KV_BF16 ? 2 : 1), need = (int64_t)a.plan.ws;
  const int64_t y_span = rows_span(2 * y_stride, 2 * qc, N), q_span = rows_span(2 * q_stride, 2 * qc, N);
  if (in_cache(a.kv, row, y, y_span) || spans_meet(ws, need, y, y_span) || spans_meet(ws, need, q, q_span) ||
      (need > 0 && in_cache(a.kv, row, ws, need)))
    return DC_ERR_INVALID_ARG;
  a.q = q;
  a.y = y;
  a.qs = q_stride;
  a.ys = y_stride;
  a.scale = base2;
  a.hq = q_heads;
  a.gq = q_heads / kv->heads;
  a.hq_d = dc::div_by(a.hq);
  a.gq_d = dc::div_by(a.gq);
  a.hkv_d = dc::div_by(kv->heads);
  a.plan.rbo_d = dc::div_by(a.plan.rbo);
  a.plan.rbp_d = dc::div_by(a.plan.rbp);
  a.plan.so_d = dc::div_by(a.plan.so);
  a.plan.heavy_d = dc::div_by(a.plan.rbo - (a.plan.rbo >> 2));
  a.plan.light_d = dc::div_by(a.plan.rbo >> 2);
  a.plan.sp_d = dc::div_by(a.plan.sp);
  a.n = N;
  a.dim = kv->dim;
  a.e4m3 = kv->dtype == DC_KV_E4M3;
  a.B = b->seqs;
  a.max_q = b->max_q;
  a.max_kv = b->max_kv;
  a.pw = b->max_kv > 0 ? b->seq_pages : 1;
  a.q_start = b->q_start;
  a.kv_len = b->kv_len;
  a.pages = b->max_kv > 0 ? b->pages : b->kv_len;   // (the kernels read an entry ahead; without keys none is used)
  const bool pre = b->groups > 0 && b->max_prefix > 0 && b->max_group_q > 0;
  a.G = pre ? b->groups : 0;
  a.max_gq = b->max_group_q;
  a.max_pre = b->max_prefix;
  a.ppw = b->prefix_pages_per_group;
  a.g_start = b->group_start;
  a.p_len = b->prefix_len;
  a.p_pages = b->prefix_pages;
  a.pml = static_cast<float*>(ws);
  a.po = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + a.plan.o_off);
  a.stream = stream;
  return dc::launch_attention(a) == 0 ? DC_OK : DC_ERR_HIP;
}

size_t dc_w4_bytes(int32_t out, int32_t in) {
  if (out <= 0 || in <= 0 || out % dc::kGroup || in % dc::kGroup) return 0;
  return (size_t)out * in / 2 + 4 * (size_t)out * (in / dc::kGroup);
}

dc_status dc_w4_pack_device(int32_t out, int32_t in, const uint16_t* W, void* dst, size_t dst_bytes, uint32_t* flag,
                            void* stream) {
  const size_t need = dc_w4_bytes(out, in);
  if (need == 0) return DC_ERR_SHAPE;
  if (!W || !dst || !flag) return DC_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(dst, 16) || !aligned(flag, 4)) return DC_ERR_ALIGN;
  if (dst_bytes < need) return DC_ERR_BUFFER;
  if ((size_t)out * in > (size_t)INT32_MAX) return DC_ERR_UNSUPPORTED;
  if (spans_meet(W, 2 * (int64_t)out * in, dst, (int64_t)need)) return DC_ERR_INVALID_ARG;
  return dc::launch_w4_pack(out, in, W, static_cast<uint8_t*>(dst), flag, stream) == 0 ? DC_OK : DC_ERR_HIP;
}

dc_status dc_apply_w4(const dc_w4_view* w, const uint16_t* x, uint16_t* y, int32_t T, void* stream) {
  if (!w || T < 0) return DC_ERR_INVALID_ARG;
  if (dc_w4_bytes(w->out, w->in) == 0) return DC_ERR_SHAPE;
  if (!w->base || !x || !y) return DC_ERR_INVALID_ARG;
  if (!aligned(w->base, 16) || !aligned(x, 16) || !aligned(y, 16)) return DC_ERR_ALIGN;
  if (rows_meet(x, 2 * (int64_t)w->in, 2 * (int64_t)w->in, y, 2 * (int64_t)w->out, 2 * (int64_t)w->out, T))
    return DC_ERR_INVALID_ARG;
  if ((size_t)w->out * w->in > (size_t)INT32_MAX || T > 65535 * 16) return DC_ERR_UNSUPPORTED;
  if (T == 0) return DC_OK;
  if (spans_meet(w->base, (int64_t)dc_w4_bytes(w->out, w->in), y, 2 * (int64_t)w->out * T)) return DC_ERR_INVALID_ARG;
  const dc::W4Args a{static_cast<const uint8_t*>(w->base), x, y, w->out, w->in, T, stream};
  return dc::launch_w4(a) == 0 ? DC_OK : DC_ERR_HIP;
}

}  // extern "C"
