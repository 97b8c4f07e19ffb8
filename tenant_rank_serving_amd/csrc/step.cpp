// Entry points of the operators that close a decode step (verification, page
// tables and pages, MXFP4): argument checks on the host, then one launcher.
// No allocation, no synchronization.
#include <algorithm>
#include <cstdint>

#include "checks.h"
#include "step.h"

using namespace dc;

namespace dc {

// Pieces of 2048 logits until the call has two blocks of 8192 for each CU, else of
// 8192 (fewer sums to join).  us by 2048 and by 8192: 64 rows of 32000 16.8 and 19.3,
// 16 rows of 128256 fp32 14.7 and 16.0, 16 x 5 rows of 32000 fp32 15.6 and 18.6; with
// draft logits, which the size of the workspace knows nothing of, 8 x 4 rows of
// 128256 26.5 and 22.3, 20 x 5 of 32000 22.1 and 21.8.
VerifyPlan verify_plan(int32_t vocab, int32_t N, int32_t seqs) {
  VerifyPlan p{};
  // a row that is not aligned has a part of a vector at either end
  const int64_t vecs = ((int64_t)vocab + 2 * kVerifyVec - 2) / kVerifyVec;
  auto chunks = [&](int32_t per) { return (vecs + kVerifyThreads * per - 1) / (kVerifyThreads * per); };
  p.vecs = chunks(4) * N >= 512 ? 4 : 1;
  p.chunks = (int32_t)chunks(p.vecs);
  p.pieces = (int32_t)chunks(pick_threads(p.vecs) / kVerifyThreads);
  p.rest_off = round_up(sizeof(VerifyPart) * 2 * (size_t)N * p.chunks, kAlign);
  p.arrived_off = p.rest_off + round_up(2 * sizeof(double) * (size_t)seqs * p.pieces, kAlign);
  // What a call needs falls where longer pieces begin.  A workspace serves smaller
  // calls too, so its size is a bound that grows with each argument: short pieces
  // are taken while chunks(4) * N is 511 or less, when there are at most 4 * 511.
  const int64_t shorts = std::min<int64_t>(chunks(1) * N, 4 * 511), longs = chunks(4) * N;
  p.ws = round_up(sizeof(VerifyPart) * 2 * (size_t)std::max(shorts, longs), kAlign) +
         round_up(2 * sizeof(double) * (size_t)(chunks(1) * seqs), kAlign) + round_up(4 * (size_t)seqs, kAlign);
  return p;
}

}  // namespace dc

namespace {

dc_status check_logits(const void* p, int64_t stride, int64_t vocab, int64_t e, int64_t n) {
  if (!p) return DC_ERR_INVALID_ARG;
  if (stride < vocab) return DC_ERR_SHAPE;
  if (!mul_fits(n > 1 ? n : 1, stride, (INT64_C(1) << 47) / e)) return DC_ERR_UNSUPPORTED;
  if (!aligned(p, (uintptr_t)e)) return DC_ERR_ALIGN;
  return DC_OK;
}

// Whether any of the buffers that a call writes shares a byte with another
// one, or with one that it reads.
struct Span {
  const void* p;
  int64_t n;
};
template <int W, int R>
bool overlap(const Span (&w)[W], const Span (&r)[R]) {
  for (int i = 0; i < W; ++i) {
    if (!w[i].p) continue;
    for (int j = i + 1; j < W; ++j)
      if (w[j].p && spans_meet(w[i].p, w[i].n, w[j].p, w[j].n)) return true;
    for (int j = 0; j < R; ++j)
      if (r[j].p && spans_meet(w[i].p, w[i].n, r[j].p, r[j].n)) return true;
  }
  return false;
}

bool verify_size(int32_t vocab, int32_t N, int32_t seqs) {
  if (vocab < 1 || N < 0 || seqs < 0) return false;
  const int64_t most = ((int64_t)vocab + 14) / 8 / (4 * kVerifyThreads) + 1;
  // (a sequence has a block of 512 threads for 4096 logits, or one of up to 1024 threads)
  return mul_fits(most, 2 * (int64_t)N, kMostBlocks - 1) && mul_fits(most, seqs, (kMostBlocks - 1) / 4) && vocab <= (1 << 30);
}

dc_status check_table(const dc_kv_table* t, uint32_t* status, void* stream, TableArgs* a) {
  if (!t || t->seqs < 0 || t->width < 0) return DC_ERR_INVALID_ARG;
  if (t->page < 16 || t->page > 1024 || (t->page & (t->page - 1)) || t->num_pages < 1) return DC_ERR_SHAPE;
  if (t->width > INT32_MAX / t->page) return DC_ERR_SHAPE;   // lengths have 31 bits
  if (!t->refs || !status || (t->seqs > 0 && (!t->kv_len || (t->width > 0 && !t->pages)))) return DC_ERR_INVALID_ARG;
  if (!aligned(t->refs, 16) || !aligned(t->pages, 4) || !aligned(t->kv_len, 4) || !aligned(status, 4)) return DC_ERR_ALIGN;
  *a = TableArgs{t->pages, t->kv_len, t->refs, t->seqs, t->width, t->page, t->num_pages, status, stream};
  return DC_OK;
}

dc_status check_layers(const dc_kv_cache* c, int32_t n, LayerArgs* a) {
  if (!c || n < 1) return DC_ERR_INVALID_ARG;
  if (n > DC_KV_MAX_LAYERS) return DC_ERR_UNSUPPORTED;
  KvArgs first{};
  for (int32_t i = 0; i < n; ++i) {
    KvArgs k{};
    const dc_status st = check_cache(c + i, &k);
    if (st != DC_OK) return st;
    if (i == 0) first = k;
    if (c[i].dtype != c[0].dtype || c[i].dim != c[0].dim || k.heads != first.heads || k.shift != first.shift ||
        k.num_pages != first.num_pages || k.page_stride != first.page_stride || k.head_stride != first.head_stride ||
        k.slot_stride != first.slot_stride)
      return DC_ERR_SHAPE;
    a->k[i] = k.k;
    a->v[i] = k.v;
  }
  a->page_stride = first.page_stride;
  a->head_stride = first.head_stride;
  a->slot_stride = first.slot_stride;
  a->heads = first.heads;
  a->num_pages = first.num_pages;
  a->shift = first.shift;
  a->layers = n;
  const int32_t row = c[0].dim * (c[0].dtype == DC_KV_BF16 ? 2 : 1);
  for (a->pieces = 0; (16 << a->pieces) < row;) ++a->pieces;
  return DC_OK;
}

// Whether n bytes at p reach into a page of some layer.
bool in_layers(const LayerArgs& a, const void* p, int64_t n) {
  KvArgs k{};
  k.page_stride = a.page_stride;
  k.head_stride = a.head_stride;
  k.slot_stride = a.slot_stride;
  k.heads = a.heads;
  k.num_pages = a.num_pages;
  k.shift = a.shift;
  for (int32_t i = 0; i < a.layers; ++i) {
    k.k = a.k[i];
    k.v = a.v[i];
    if (in_cache(k, INT64_C(16) << a.pieces, p, n)) return true;
  }
  return false;
}

dc_status check_mx4(const dc_mx4_view* w) {
  if (!w) return DC_ERR_INVALID_ARG;
  if (dc_mx4_bytes(w->rows, w->cols) == 0) return DC_ERR_SHAPE;
  if (!w->base) return DC_ERR_INVALID_ARG;
  if (!aligned(w->base, 16)) return DC_ERR_ALIGN;
  if (((int64_t)w->rows + 15) / 16 * 16 * w->cols > INT32_MAX) return DC_ERR_UNSUPPORTED;
  return DC_OK;
}

}  // namespace

extern "C" {

size_t dc_verify_workspace_bytes(int32_t vocab, int32_t N, int32_t seqs) {
  if (!verify_size(vocab, N, seqs)) return 0;
  return std::max<size_t>(verify_plan(vocab, N, seqs).ws, kAlign);
}

dc_status dc_verify_drafts(const dc_verify_batch* b, int32_t dtype, int32_t vocab, const void* target,
                           int64_t target_stride, const void* draft, int64_t draft_stride, int32_t N, int32_t* out,
                           int32_t* count, float* prob, void* ws, size_t ws_bytes, void* stream) {
  if (!b || N < 0 || b->seqs < 0) return DC_ERR_INVALID_ARG;
  if (dtype != DC_LOGITS_BF16 && dtype != DC_LOGITS_F32) return DC_ERR_INVALID_ARG;
  if (vocab < 1) return DC_ERR_SHAPE;
  if (!verify_size(vocab, N, b->seqs)) return DC_ERR_UNSUPPORTED;
  const int64_t e = dtype == DC_LOGITS_BF16 ? 2 : 4;
  dc_status st = check_logits(target, target_stride, vocab, e, N);
  if (st != DC_OK) return st;
  if (draft && (st = check_logits(draft, draft_stride, vocab, e, N)) != DC_OK) return st;
  if (!ws || !out) return DC_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return DC_ERR_ALIGN;
  if (b->seqs > 0 && (!b->q_start || !b->tokens || !b->accept || !b->pick || !count)) return DC_ERR_INVALID_ARG;
  for (const void* p : {(const void*)b->q_start, (const void*)b->tokens, (const void*)b->accept, (const void*)b->pick,
                        (const void*)b->temperature, (const void*)out, (const void*)count, (const void*)prob})
    if (!aligned(p, 4)) return DC_ERR_ALIGN;
  const VerifyPlan plan = verify_plan(vocab, N, b->seqs);
  if (ws_bytes < plan.ws) return DC_ERR_BUFFER;
  if (b->seqs == 0) return DC_OK;
  const int64_t n4 = 4 * (int64_t)N, s4 = 4 * (int64_t)b->seqs;
  const Span w[] = {{out, n4}, {count, s4}, {prob, n4}, {ws, (int64_t)plan.ws}};
  const Span r[] = {{target, N > 0 ? e * rows_span(target_stride, vocab, N) : 0},
                    {draft, N > 0 ? e * rows_span(draft_stride, vocab, N) : 0},
                    {b->q_start, s4 + 4}, {b->tokens, n4}, {b->accept, n4}, {b->pick, s4}, {b->temperature, s4}};
  if (overlap(w, r)) return DC_ERR_INVALID_ARG;
  uint8_t* base = static_cast<uint8_t*>(ws);
  VerifyArgs a{};
  a.p = target;
  a.q = draft;
  a.ps = target_stride;
  a.qs = draft_stride;
  a.q_start = b->q_start;
  a.tokens = b->tokens;
  a.accept = b->accept;
  a.pick = b->pick;
  a.temperature = b->temperature;
  a.out = out;
  a.count = count;
  a.prob = prob;
  a.part = reinterpret_cast<VerifyPart*>(base);
  a.pieces = plan.pieces;
  a.rest = reinterpret_cast<double*>(base + plan.rest_off);
  a.arrived = reinterpret_cast<uint32_t*>(base + plan.arrived_off);
  a.vocab = vocab;
  a.n = N;
  a.seqs = b->seqs;
  a.chunks = plan.chunks;
  a.vecs = plan.vecs;
  a.f32 = dtype == DC_LOGITS_F32;
  a.stream = stream;
  return launch_verify(a) == 0 ? DC_OK : DC_ERR_HIP;
}

dc_status dc_kv_resize(const dc_kv_table* t, const int32_t* new_len, int32_t* copies, uint32_t* status, void* stream) {
  TableArgs a{};
  const dc_status st = check_table(t, status, stream, &a);
  if (st != DC_OK) return st;
  if (t->seqs > DC_KV_MAX_SEQS || (int64_t)t->seqs * (t->width + INT64_C(1)) > 1 << 30) return DC_ERR_UNSUPPORTED;
  if (t->seqs == 0) return DC_OK;
  if (!new_len || !copies) return DC_ERR_INVALID_ARG;
  if (!aligned(new_len, 4) || !aligned(copies, 4)) return DC_ERR_ALIGN;
  const int64_t s4 = 4 * (int64_t)t->seqs;
  const Span w[] = {{t->pages, s4 * t->width}, {t->kv_len, s4}, {t->refs, 4 * (int64_t)t->num_pages}, {copies, 2 * s4}, {status, 4}};
  const Span r[] = {{new_len == t->kv_len ? nullptr : new_len, s4}};
  if (overlap(w, r)) return DC_ERR_INVALID_ARG;
  return launch_resize(a, new_len, copies) == 0 ? DC_OK : DC_ERR_HIP;
}

dc_status dc_kv_fork(const dc_kv_table* t, const int32_t* src, const int32_t* dst, int32_t n, uint32_t* status,
                     void* stream) {
  TableArgs a{};
  const dc_status st = check_table(t, status, stream, &a);
  if (st != DC_OK) return st;
  if (n < 0) return DC_ERR_INVALID_ARG;
  if (n > DC_KV_MAX_SEQS) return DC_ERR_UNSUPPORTED;   // (every block looks through dst)
  if (n == 0) return DC_OK;
  if (!src || !dst) return DC_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4)) return DC_ERR_ALIGN;
  const int64_t s4 = 4 * (int64_t)t->seqs;
  const Span w[] = {{t->pages, s4 * t->width}, {t->kv_len, s4}, {t->refs, 4 * (int64_t)t->num_pages}, {status, 4}};
  const Span r[] = {{src, 4 * (int64_t)n}, {dst, 4 * (int64_t)n}};
  if (overlap(w, r)) return DC_ERR_INVALID_ARG;
  return launch_fork(a, src, dst, n) == 0 ? DC_OK : DC_ERR_HIP;
}

dc_status dc_kv_copy(const dc_kv_cache* layers, int32_t n_layers, const int32_t* copies, int32_t n, void* stream) {
  LayerArgs a{};
  const dc_status st = check_layers(layers, n_layers, &a);
  if (st != DC_OK) return st;
  if (n < 0) return DC_ERR_INVALID_ARG;
  if (n > 0 && !copies) return DC_ERR_INVALID_ARG;
  if (!aligned(copies, 4)) return DC_ERR_ALIGN;
  const int64_t pieces = ((int64_t)a.heads << a.shift) << a.pieces, parts = (pieces + kCopyBlock - 1) / kCopyBlock;
  if (pieces > INT32_MAX / 2 || parts > 65535 || !mul_fits(2 * (int64_t)n_layers * parts, n, kMostBlocks)) return DC_ERR_UNSUPPORTED;
  if (n == 0) return DC_OK;
  if (in_layers(a, copies, 8 * (int64_t)n)) return DC_ERR_INVALID_ARG;
  return launch_copy(a, copies, n, stream) == 0 ? DC_OK : DC_ERR_HIP;
}

dc_status dc_kv_compact(const dc_kv_cache* layers, int32_t n_layers, const int32_t* from, int32_t seqs, int32_t width,
                        const int32_t* keep_start, const int32_t* keep, int32_t n, const int32_t* to, void* stream) {
  LayerArgs a{};
  const dc_status st = check_layers(layers, n_layers, &a);
  if (st != DC_OK) return st;
  if (n < 0 || seqs < 0 || width < 0) return DC_ERR_INVALID_ARG;
  if (width > (INT32_MAX >> a.shift)) return DC_ERR_SHAPE;
  const int64_t groups = ((int64_t)a.heads + 3) / 4;   // (64 >> pieces heads a block, 4 at least)
  const int64_t tiles = std::max<int64_t>(((int64_t)n + kCompactTokens - 1) / kCompactTokens, seqs);
  if (groups > 65535 || !mul_fits(2 * (int64_t)n_layers * groups, tiles, kMostBlocks)) return DC_ERR_UNSUPPORTED;
  if (n == 0 || seqs == 0 || width == 0) return DC_OK;
  if (!from || !keep_start || !keep) return DC_ERR_INVALID_ARG;
  if (!aligned(from, 4) || !aligned(keep_start, 4) || !aligned(keep, 4) || !aligned(to, 4)) return DC_ERR_ALIGN;
  if (from == to) return DC_ERR_INVALID_ARG;   // in place is to = NULL
  const int64_t table = 4 * (int64_t)seqs * width;
  if (in_layers(a, from, table) || (to && in_layers(a, to, table)) || in_layers(a, keep_start, 4 * (int64_t)seqs + 4) ||
      in_layers(a, keep, 4 * (int64_t)n))
    return DC_ERR_INVALID_ARG;
  return launch_compact(a, from, to, keep_start, keep, seqs, width, n, stream) == 0 ? DC_OK : DC_ERR_HIP;
}

size_t dc_mx4_bytes(int32_t rows, int32_t cols) {
  if (rows < 1 || cols < 1 || cols % 128) return 0;
  return mx4_codes(rows, cols) + ((size_t)rows + 15) / 16 * (((size_t)cols + 511) / 512) * 256;
}

dc_status dc_mx4_pack_device(int32_t rows, int32_t cols, const uint16_t* X, int64_t stride, void* dst, size_t dst_bytes,
                             uint32_t* flag, void* stream) {
  if (rows < 0) return DC_ERR_INVALID_ARG;
  if (cols < 1 || cols % 128) return DC_ERR_SHAPE;
  dc_status st = check_rows(X, stride, cols, rows);
  if (st != DC_OK) return st;
  if (!dst) return DC_ERR_INVALID_ARG;
  if (!aligned(dst, 16) || !aligned(flag, 4)) return DC_ERR_ALIGN;
  const size_t need = rows > 0 ? dc_mx4_bytes(rows, cols) : 0;
  if (dst_bytes < need) return DC_ERR_BUFFER;
  if (!mul_fits(((int64_t)rows + 63) / 64, ((int64_t)cols + 511) / 512, kMostBlocks)) return DC_ERR_UNSUPPORTED;
  if (rows == 0) return DC_OK;
  const Span w[] = {{dst, (int64_t)need}, {flag, 4}};
  const Span r[] = {{X, 2 * rows_span(stride, cols, rows)}};
  if (overlap(w, r)) return DC_ERR_INVALID_ARG;
  return launch_mx4_pack(rows, cols, X, stride, static_cast<uint8_t*>(dst), flag, stream) == 0 ? DC_OK : DC_ERR_HIP;
}

dc_status dc_mx4_dequant(const dc_mx4_view* w, uint16_t* X, int64_t stride, void* stream) {
  dc_status st = check_mx4(w);
  if (st != DC_OK) return st;
  if ((st = check_rows(X, stride, w->cols, w->rows)) != DC_OK) return st;
  if (spans_meet(w->base, (int64_t)dc_mx4_bytes(w->rows, w->cols), X, 2 * rows_span(stride, w->cols, w->rows)))
    return DC_ERR_INVALID_ARG;
  return launch_mx4_dequant(w->rows, w->cols, static_cast<const uint8_t*>(w->base), X, stride, stream) == 0 ? DC_OK
                                                                                                          : DC_ERR_HIP;
}

dc_status dc_apply_mx4(const dc_mx4_view* w, const uint16_t* x, uint16_t* y, int32_t T, void* stream) {
  const dc_status st = check_mx4(w);
  if (st != DC_OK) return st;
  if (T < 0 || !x || !y) return DC_ERR_INVALID_ARG;
  if (w->rows % 128) return DC_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16)) return DC_ERR_ALIGN;
  if (T > 65535 * 16) return DC_ERR_UNSUPPORTED;
  if (T == 0) return DC_OK;
  const Span o[] = {{y, 2 * (int64_t)w->rows * T}};
  const Span r[] = {{x, 2 * (int64_t)w->cols * T}, {w->base, (int64_t)dc_mx4_bytes(w->rows, w->cols)}};
  if (overlap(o, r)) return DC_ERR_INVALID_ARG;
  const Mx4Args a{static_cast<const uint8_t*>(w->base), x, nullptr, y, w->rows, w->cols, T, stream};
  return launch_mx4(a) == 0 ? DC_OK : DC_ERR_HIP;
}

dc_status dc_apply_mx4q(const dc_mx4_view* w, const dc_mx4_view* x, uint16_t* y, void* stream) {
  dc_status st = check_mx4(w);
  if (st != DC_OK) return st;
  if ((st = check_mx4(x)) != DC_OK) return st;
  if (!y) return DC_ERR_INVALID_ARG;
  if (w->rows % 128 || w->cols != x->cols) return DC_ERR_SHAPE;
  if (!aligned(y, 16)) return DC_ERR_ALIGN;
  if (x->rows > 65535 * 16) return DC_ERR_UNSUPPORTED;
  const Span o[] = {{y, 2 * (int64_t)w->rows * x->rows}};
  const Span r[] = {{x->base, (int64_t)dc_mx4_bytes(x->rows, x->cols)}, {w->base, (int64_t)dc_mx4_bytes(w->rows, w->cols)}};
  if (overlap(o, r)) return DC_ERR_INVALID_ARG;
  const Mx4Args a{static_cast<const uint8_t*>(w->base), nullptr, static_cast<const uint8_t*>(x->base), y, w->rows, w->cols,
                  x->rows, stream};
  return launch_mx4q(a) == 0 ? DC_OK : DC_ERR_HIP;
}

}  // extern "C"
