// Internal declarations of the operators that close a decode step: verifying
// drafted tokens, page tables and pages, the MXFP4 backbone.  Not part of the
// public ABI (include/deltacome.h is).
#pragma once

#include "layer.h"

namespace dc {

// ------------------------------------------------------------ verification
// What one block found in its piece of one row's logits: the largest, the
// first index that has it, and the sum of 2^((l - largest) k), k = log2(e) / T
// (NaN if the piece holds one).
struct alignas(16) VerifyPart {
  float m;
  int32_t at;
  double z;
};

constexpr int kVerifyVec = 8;       // logits of a vector
constexpr int kVerifyThreads = 256;
constexpr int pick_threads(int vecs) { return vecs == 4 ? 2 * kVerifyThreads : kVerifyThreads; }

struct VerifyArgs {
  const void *p, *q;                // target, draft (null: none)
  int64_t ps, qs;                   // row strides, elements
  const int32_t *q_start, *tokens;
  const float *accept, *pick, *temperature;
  int32_t *out, *count;
  float* prob;
  VerifyPart* part;                 // [N][2][chunks]
  double* rest;                     // [seqs][pieces][2]: sums of max(p - q, 0) and of p
  uint32_t* arrived;                // [seqs]
  int32_t vocab, n, seqs, chunks, vecs, pieces, f32;   // vecs: vectors of a thread in a chunk; pieces: of one vector of pick_threads
  void* stream;
};
struct VerifyPlan {
  int32_t vecs, chunks, pieces;
  size_t rest_off, arrived_off, ws;
};
VerifyPlan verify_plan(int32_t vocab, int32_t N, int32_t seqs);
int launch_verify(const VerifyArgs& a);

// ------------------------------------------------------------ pages
struct TableArgs {
  int32_t *pages, *kv_len, *refs;
  int32_t seqs, width, page, num_pages;
  uint32_t* status;
  void* stream;
};
int launch_resize(const TableArgs& t, const int32_t* new_len, int32_t* copies);
int launch_fork(const TableArgs& t, const int32_t* src, const int32_t* dst, int32_t n);

struct LayerArgs {
  uint8_t* k[DC_KV_MAX_LAYERS];
  uint8_t* v[DC_KV_MAX_LAYERS];
  int64_t page_stride, head_stride, slot_stride;   // bytes
  int32_t heads, num_pages, shift, layers;
  int32_t pieces;                                  // log2 of the 16-byte pieces of a head's row
};
int launch_copy(const LayerArgs& a, const int32_t* copies, int32_t n, void* stream);
constexpr int kCopyBlock = 1024;                    // 16-byte pieces that a block of the copy moves
constexpr int kCompactTokens = 64;                  // tokens of a block of compaction; 64 >> pieces heads
int launch_compact(const LayerArgs& a, const int32_t* from, const int32_t* to, const int32_t* start,
                   const int32_t* keep, int32_t seqs, int32_t width, int32_t n, void* stream);

// ------------------------------------------------------------ MXFP4
struct Mx4Args {
  const uint8_t* w;
  const uint16_t* x;    // bf16, or
  const uint8_t* xq;    // MXFP4
  uint16_t* y;
  int32_t out, in, T;
  void* stream;
};
// Bytes of the codes of a matrix.
inline size_t mx4_codes(int32_t rows, int32_t cols) { return ((size_t)rows + 15) / 16 * 16 * (size_t)cols / 2; }
int launch_mx4(const Mx4Args& a);
int launch_mx4_few(const Mx4Args& a);   // of it, more than 16 tokens
int launch_mx4q(const Mx4Args& a);
// Which form a call takes: row tiles of 16 rows of a block (up to 16 tokens), and
// numbers in the lists of tiles of the other two.  Tests look at them.
int mx4_row_tiles(int32_t out, int32_t T);
int mx4_few_tile(int32_t out, int32_t in, int32_t T);
int mx4q_tile(int32_t out, int32_t in, int32_t T);
int launch_mx4_tiles(const Mx4Args& a, int32_t size);   // of it, by tiles in LDS: 64 x 64, 64 x 128, 128 x 128, 256 x 256
int launch_mx4_pack(int32_t rows, int32_t cols, const uint16_t* X, int64_t stride, uint8_t* dst, uint32_t* flag,
                    void* stream);
int launch_mx4_dequant(int32_t rows, int32_t cols, const uint8_t* w, uint16_t* X, int64_t stride, void* stream);

}  // namespace dc
