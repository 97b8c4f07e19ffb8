// Argument checks shared by the entry points of the decoder-layer and step
// operators: alignment, overlaps of strided buffers, a cache's shape.
#pragma once

#include <cstdint>

#include "layer.h"

namespace dc {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows of `w` bytes, `n` of them `stride` bytes apart: whether two such
// buffers share a byte.  Buffers of one stride may be interleaved (columns of
// one fused matrix); of other pairs whose ranges meet nothing is known, so
// they count as sharing.
inline bool rows_meet(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t n) {
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
inline int64_t rows_span(int64_t stride, int64_t w, int64_t n) { return (n - 1) * stride + w; }

inline bool spans_meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// Whether n bytes at p reach into the cache's keys or values (into a page, not
// into room between pages).
inline bool in_cache(const KvArgs& k, int64_t dim_bytes, const void* p, int64_t n) {
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

inline bool mul_fits(int64_t a, int64_t b, int64_t lim) { return a == 0 || b <= lim / a; }

// A launch's threads along x are numbered with 32 bits; blocks of 256.
constexpr int64_t kMostBlocks = UINT32_MAX / 256;

// The cache's shape and strides; fills the kernels' view of it.
inline dc_status check_cache(const dc_kv_cache* c, KvArgs* k) {
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
inline dc_status check_rows(const void* p, int64_t stride, int64_t cols, int64_t n) {
  if (!p) return DC_ERR_INVALID_ARG;
  if (stride < cols || !mul_fits(n > 1 ? n : 1, stride, INT64_C(1) << 46)) return DC_ERR_SHAPE;
  if (!aligned(p, 16) || stride % 8) return DC_ERR_ALIGN;
  return DC_OK;
}

}  // namespace dc
