// Page tables of a cache's sequences, and pages: forking, growing and giving
// back, copying, compacting.
//
// The tables are a few thousand numbers, whose order matters (free pages go out
// lowest first, to the sequences in order): one block keeps them, so that a
// captured step needs no host.  Copies move bytes: every piece of 16 bytes is
// read and written once, blocks over pages (or tokens), layers, keys and values.
#include <hip/hip_runtime.h>

#include "step.h"

namespace dc {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ tables
constexpr int kResizeThreads = 1024, kWaves = kResizeThreads / 64;

// The counts of k_resize are one block's alone while it runs, so its atomics need
// not leave the XCD's L2.
__device__ __forceinline__ int32_t ld_block(const int32_t* p) {
  return __hip_atomic_load(const_cast<int32_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void add_block(int32_t* p, int32_t v) {
  __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void add_agent(int32_t* p, int32_t v) {
  __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What a block's 16 waves hold, added up for the waves before this one and in
// all; `box` [16].
__device__ __forceinline__ int before_wave(int mine, int* box, int* all) {
  const int wave = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) box[wave] = mine;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int v = box[w];
    before += w < wave ? v : 0;
    sum += v;
  }
  *all = sum;
  return before;
}

__device__ __forceinline__ int upto_lane(int v) {
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const int o = __shfl_up(v, x);
    if ((int)(threadIdx.x & 63) >= x) v += o;
  }
  return v;
}

// One block.  Pages behind the new lengths are given back; then each sequence's
// need is known, and the free pages, in the order of their numbers, are dealt
// to the sequences, in theirs: the k-th one to the sequence among whose running
// needs k falls.
//
// Bound by latency: lengths, entries, counts and free pages are read one after
// the other, about a microsecond each.  48 of 64 sequences giving back 5000 pages
// 7 us, growing by 255 pages out of 6100 7 us.
__global__ void __launch_bounds__(kResizeThreads) k_resize(TableArgs t, const int32_t* new_len, int32_t* copies) {
  // per sequence: pages needed up to and with it, and whether the first of its own is for an exchange;
  // its old length.  Before that, per page: how often it is given back
  constexpr int kCounted = 2 * DC_KV_MAX_SEQS;
  __shared__ union {
    struct {
      uint32_t upto[DC_KV_MAX_SEQS];
      int32_t old_of[DC_KV_MAX_SEQS];
    };
    alignas(16) int32_t freed[kCounted];
  } sh;
  uint32_t* upto = sh.upto;
  int32_t* old_of = sh.old_of;
  __shared__ int32_t given[kResizeThreads];   // what the first sequences get for their shared pages
  __shared__ int32_t list[4 * kResizeThreads];   // free pages, in order
  __shared__ int box[kWaves];
  __shared__ uint32_t status;
  __shared__ int giving;   // sequences that give pages back, 64 for one with 64
  __shared__ int part;     // the sequence that was dealt a part of what it needs
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int most = t.width * t.page, shift = 31 - __builtin_clz(t.page);
  auto pages_of = [&](int n) { return (int)(((int64_t)n + t.page - 1) >> shift); };
  if (tid == 0) status = 0, giving = 0, part = -1;
  __syncthreads();

  // the first kResizeThreads sequences' lengths, in the order in which the waves
  // take them now and in the one of later
  int old1 = 0, want1 = 0, old0 = 0, want0 = 0;
  if (wave + lane * kWaves < t.seqs) old1 = t.kv_len[wave + lane * kWaves], want1 = new_len[wave + lane * kWaves];
  if (tid < t.seqs) old0 = t.kv_len[tid], want0 = new_len[tid];
  const int give = old1 <= most && want1 >= 0 ? pages_of(old1) - pages_of(want1) : 0;
  // Many pages are counted in LDS and their counts fall once: one CU's atomics on
  // the L2 take 1.7 ns each (5000: 8.7 us, this way 3).  A few would not pay for it.
  const uint64_t some = __ballot(give >= 2), lots = __ballot(give >= 64);
  if (lane == 0 && some) atomicAdd(&giving, lots ? 64 : __builtin_popcountll(some));
  __syncthreads();
  const bool many = t.num_pages <= kCounted && giving >= 64;
  if (many) {
    for (int i = tid; i < (t.num_pages + 3) / 4; i += kResizeThreads) reinterpret_cast<int4*>(sh.freed)[i] = int4{0, 0, 0, 0};
    __syncthreads();
  }
  int32_t shared0 = -1;
  if (tid < t.seqs && old0 >= 0 && old0 < want0 && want0 <= most && (old0 & (t.page - 1)))
    shared0 = t.pages[(int64_t)tid * t.width + (old0 >> shift)];
  // 64 sequences of a wave at a time, a length in each lane; then those that give
  // pages back, 256 entries of one at a time, with the next ones' on their way
  for (int s0 = wave; s0 < t.seqs; s0 += 64 * kWaves) {
    const int b = s0 + lane * kWaves;
    int from = 0, to = 0;
    if (b < t.seqs) {
      const int old = s0 == wave ? old1 : t.kv_len[b], want = s0 == wave ? want1 : new_len[b];
      if (old < 0 || old > most || want < 0 || want > most) atomicOr(&status, (uint32_t)DC_KV_BAD);
      else from = pages_of(want), to = pages_of(old);
    }
    uint64_t todo = __ballot(from < to);
    if (!todo) continue;
    int l = __builtin_ctzll(todo), at = __builtin_amdgcn_readlane(from, l), end = __builtin_amdgcn_readlane(to, l);
    int32_t e[4], after[4];
    auto load = [&](int32_t* x) {
      const int32_t* row = t.pages + (int64_t)(s0 + l * kWaves) * t.width;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = at + 64 * j + lane < end ? row[at + 64 * j + lane] : 0;
    };
    load(e);
    for (;;) {
      const int l_ = l, at_ = at, end_ = end;
      at += 256;
      if (at >= end) {
        todo &= todo - 1;
        if (todo) l = __builtin_ctzll(todo), at = __builtin_amdgcn_readlane(from, l), end = __builtin_amdgcn_readlane(to, l);
      }
      if (todo) load(after);
      int32_t* row = t.pages + (int64_t)(s0 + l_ * kWaves) * t.width;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = at_ + 64 * j + lane;
        if (i >= end_) continue;
        if (e[j] < 0 || e[j] >= t.num_pages) atomicOr(&status, (uint32_t)DC_KV_BAD);
        else if (many) atomicAdd(&sh.freed[e[j]], 1);
        else add_block(t.refs + e[j], -1);
        row[i] = -1;
      }
      if (!todo) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = after[j];
    }
  }
  __builtin_amdgcn_s_waitcnt(0);   // the counts have fallen
  __syncthreads();
  const int vecs = (int)(((int64_t)t.num_pages + 3) / 4);
  if (many) {
    for (int v = tid; v < vecs; v += kResizeThreads) {
      const int4 n = reinterpret_cast<const int4*>(sh.freed)[v];
      if (!(n.x | n.y | n.z | n.w)) continue;
      if (4 * v + 3 < t.num_pages) {
        int4 r = reinterpret_cast<const int4*>(t.refs)[v];
        r.x -= n.x, r.y -= n.y, r.z -= n.z, r.w -= n.w;
        reinterpret_cast<int4*>(t.refs)[v] = r;
      } else {
        for (int i = 4 * v; i < t.num_pages; ++i) t.refs[i] -= sh.freed[i];
      }
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
  }

  // the free pages: 4 a thread, the next ones on their way while these are dealt
  auto load = [&](int v) {
    int4 r = int4{1, 1, 1, 1};
    if (v >= vecs) return r;   // (4 v may have 32 bits from here on)
    const unsigned p = 4u * (unsigned)v, pages = (unsigned)t.num_pages;
    if (p + 3 < pages) return reinterpret_cast<const int4*>(t.refs)[v];
    r.x = t.refs[p];
    if (p + 1 < pages) r.y = t.refs[p + 1];
    if (p + 2 < pages) r.z = t.refs[p + 2];
    return r;
  };
  // (counts that fell by atomics are in the L2; nothing of them is in this CU's L1 yet)
  int4 now = load(tid), next = load(kResizeThreads + tid);

  int total = 0;
  for (int b0 = 0; b0 < t.seqs; b0 += kResizeThreads) {
    const int b = b0 + tid;
    int need = 0;
    bool swap = false;
    if (b < t.seqs) {
      const int old = b0 ? t.kv_len[b] : old0, want = b0 ? new_len[b] : want0;
      old_of[b] = old;
      if (old >= 0 && old <= most && want > old && want <= most) {
        need = pages_of(want) - pages_of(old);
        if (old & (t.page - 1)) {
          const int32_t p = b0 ? t.pages[(int64_t)b * t.width + (old >> shift)] : shared0;
          if (p >= 0 && p < t.num_pages) swap = ld_block(t.refs + p) > 1;
          else atomicOr(&status, (uint32_t)DC_KV_BAD);
          need += swap;
        }
      }
      copies[2 * b] = copies[2 * b + 1] = -1;
    }
    const int sum = upto_lane(need);
    int all;
    const int before = before_wave(__shfl(sum, 63), box, &all);
    if (b < t.seqs) upto[b] = (uint32_t)(total + before + sum) << 1 | (uint32_t)swap;
    total += all;
  }
  __syncthreads();

  int dealt = 0;
  for (int v0 = 0; v0 < vecs && dealt < total; v0 += kResizeThreads) {
    const int4 later = load(v0 + 2 * kResizeThreads + tid);
    const int r[4] = {now.x, now.y, now.z, now.w};
    int mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) mine += r[j] <= 0;
    const int sum = upto_lane(mine);
    int all;
    int at = before_wave(__shfl(sum, 63), box, &all) + sum - mine;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (r[j] <= 0) list[at++] = 4 * (v0 + tid) + j;
    __syncthreads();
    const int deal = min(all, total - dealt);
    for (int i = tid; i < deal; i += kResizeThreads) {
      const int32_t p = list[i];
      const int k = dealt + i;
      int lo = 0, hi = t.seqs - 1;   // the first sequence with upto > k
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int)(upto[mid] >> 1) > k) hi = mid; else lo = mid + 1;
      }
      const int slot = k - (lo ? (int)(upto[lo - 1] >> 1) : 0);
      const bool swap = upto[lo] & 1;
      const int old = old_of[lo];
      int32_t* row = t.pages + (int64_t)lo * t.width;
      if (swap && slot == 0) {
        if (lo < kResizeThreads) {
          given[lo] = p;
        } else {
          copies[2 * lo] = row[old >> shift];
          copies[2 * lo + 1] = p;
          row[old >> shift] = p;
        }
      } else {
        row[pages_of(old) + slot - swap] = p;
      }
      t.refs[p] = 1;
    }
    dealt += all;
    now = next;
    next = later;
  }
  const int have = dealt < total ? dealt : total;
  __syncthreads();

  for (int b0 = 0; b0 < t.seqs; b0 += kResizeThreads) {
    const int b = b0 + tid;
    if (b >= t.seqs) continue;
    const int old = old_of[b], want = b0 ? new_len[b] : want0;
    if (old < 0 || old > most || want < 0 || want > most) continue;
    const int end = (int)(upto[b] >> 1), first = b ? (int)(upto[b - 1] >> 1) : 0;
    const bool swap = upto[b] & 1;
    if (end > first && end > have) {   // too few
      atomicOr(&status, (uint32_t)DC_KV_FULL);
      if (first < have) part = b;
      continue;
    }
    if (swap) {
      if (b0 == 0) {
        copies[2 * b] = shared0;
        copies[2 * b + 1] = given[tid];
        t.pages[(int64_t)b * t.width + (old >> shift)] = given[tid];
      }
      add_block(t.refs + (b0 ? copies[2 * b] : shared0), -1);
    }
    t.kv_len[b] = want;
  }
  __syncthreads();
  // What the one sequence was dealt that got some and not all goes back, by all
  // threads (8000 pages 4 us; by one, which waits for each entry, 1150).
  if (part >= 0) {
    const int b = part, first = b ? (int)(upto[b - 1] >> 1) : 0, old = old_of[b];
    const bool swap = upto[b] & 1;
    int32_t* row = t.pages + (int64_t)b * t.width;
    for (int slot = tid; slot < have - first; slot += kResizeThreads) {
      if (swap && slot == 0) {
        if (b < kResizeThreads) {
          t.refs[given[b]] = 0;
        } else {
          t.refs[copies[2 * b + 1]] = 0;
          row[old >> shift] = copies[2 * b];
          copies[2 * b] = copies[2 * b + 1] = -1;
        }
      } else {
        int32_t* e = row + pages_of(old) + slot - swap;
        t.refs[*e] = 0;
        *e = -1;
      }
    }
  }
  if (tid == 0 && status) atomicOr(t.status, status);
}

// Block: one branch.  Bound by latency, 4 us.  Every block looks through all of dst for rows that the call
// writes twice, or reads and writes.
__global__ void __launch_bounds__(256) k_fork(TableArgs t, const int32_t* src, const int32_t* dst, int count) {
  const int s = src[blockIdx.x], d = dst[blockIdx.x], tid = threadIdx.x;
  bool meets = false;
  for (int j = tid; j < count; j += 256) {
    const int other = dst[j];
    meets |= other == s || (other == d && j < (int)blockIdx.x);
  }
  bool ok = s >= 0 && s < t.seqs && d >= 0 && d < t.seqs && s != d;
  int n = 0;
  if (ok) {
    n = t.kv_len[s];
    ok = n >= 0 && n <= t.width * t.page && t.kv_len[d] == 0;
  }
  ok = !__syncthreads_or(meets) && ok;   // (everyone has read the lengths)
  if (!ok) {
    if (tid == 0) atomicOr(t.status, (uint32_t)DC_KV_BAD);
    return;
  }
  const int32_t* from = t.pages + (int64_t)s * t.width;
  int32_t* to = t.pages + (int64_t)d * t.width;
  const int pages = (int)(((int64_t)n + t.page - 1) / t.page);
  bool bad = false;
  for (int i = tid; i < pages; i += 256) {
    const int32_t p = from[i];
    to[i] = p;
    if (p >= 0 && p < t.num_pages) add_agent(t.refs + p, 1);
    else bad = true;
  }
  if (bad) atomicOr(t.status, (uint32_t)DC_KV_BAD);
  if (tid == 0) t.kv_len[d] = n;
}

// -------------------------------------------------------------------- copy
__device__ __forceinline__ uint8_t* pool_of(const LayerArgs& a, int lv) {
  return lv & 1 ? a.v[lv >> 1] : a.k[lv >> 1];
}

// Piece u of a page, in the order of memory: rows of a head, or heads of a row
// (Whole: a page without gaps).
template <bool Whole>
__device__ __forceinline__ int64_t piece_at(const LayerArgs& a, int u) {
  if constexpr (Whole) return 16 * (int64_t)u;
  const int c = u & ((1 << a.pieces) - 1), r = u >> a.pieces;
  int h, s;
  if (a.slot_stride <= a.head_stride) h = r >> a.shift, s = r & ((1 << a.shift) - 1);
  else s = r / a.heads, h = r - s * a.heads;
  return h * a.head_stride + s * a.slot_stride + 16 * c;
}

// Block: 16 KiB of a page of one layer's keys or values, 4 pieces a thread on their
// way at once.  Bound by HBM: 96 pages of 64 tokens of 32 layers x 8 heads (e4m3,
// 0.4 GB moved twice) 159 us, 5.1 TB/s, the rate of a large copy; 4 pages of 32 x 32
// heads of 128 bf16 numbers 15 us of which 13 are its bytes.  Addressing a page
// without gaps as one piece saves the division and the shifts (23 -> 15 us there).
template <bool Whole>
__global__ void __launch_bounds__(256) k_copy(LayerArgs a, const int32_t* copies) {
  const int64_t from = copies[2 * blockIdx.x], to = copies[2 * blockIdx.x + 1];
  if (from < 0 || from >= a.num_pages || to < 0 || to >= a.num_pages || from == to) return;
  uint8_t* pool = pool_of(a, blockIdx.y);
  const uint8_t* src = pool + from * a.page_stride;
  uint8_t* dst = pool + to * a.page_stride;
  const int pieces = a.heads << (a.shift + a.pieces), u0 = blockIdx.z * kCopyBlock + threadIdx.x;
  u32x4 x[kCopyBlock / 256];
#pragma unroll
  for (int i = 0; i < kCopyBlock / 256; ++i) {
    const int u = u0 + 256 * i;
    if (u < pieces) x[i] = *reinterpret_cast<const u32x4*>(src + piece_at<Whole>(a, u));
  }
#pragma unroll
  for (int i = 0; i < kCopyBlock / 256; ++i) {
    const int u = u0 + 256 * i;
    if (u < pieces) *reinterpret_cast<u32x4*>(dst + piece_at<Whole>(a, u)) = x[i];
  }
}

// ----------------------------------------------------------------- compact
// Byte offset of a token of a sequence, -1 if there is none.
__device__ __forceinline__ int64_t token_at(const LayerArgs& a, const int32_t* table, int width, int seq, int pos) {
  if (pos < 0 || (pos >> a.shift) >= width) return -1;
  const int32_t p = table[(int64_t)seq * width + (pos >> a.shift)];
  if (p < 0 || p >= a.num_pages) return -1;
  return p * a.page_stride + (pos & ((1 << a.shift) - 1)) * a.slot_stride;
}

// Block: 64 kept tokens of 64 >> a.pieces heads of one layer's keys or values, 16
// pieces of 16 bytes a thread.  Bound by HBM: 500 of 1000 tokens of 32 layers x 8
// heads 30 us (25 at a large copy's rate), 8 chats of 4000 395 us (373); with 4
// pieces a thread and a look-up for each 60 and 594.  To other pages the blocks are independent.  In
// place one block moves a sequence's tokens, a tile after the other: sources
// ascend and lie at or behind their places, so a tile's places hold nothing that
// is still to be read once the tile itself has been.  The next tile's places are
// looked up while this one's pieces are on their way.
template <bool InPlace>
__global__ void __launch_bounds__(256) k_compact(LayerArgs a, const int32_t* from, const int32_t* to,
                                                 const int32_t* start, const int32_t* keep, int seqs, int width, int n) {
  constexpr int kHalves = InPlace ? 2 : 1, kUnits = 16;
  __shared__ int64_t src[kHalves][kCompactTokens], dst[kHalves][kCompactTokens];
  const int tid = threadIdx.x;
  uint8_t* pool = pool_of(a, blockIdx.y);
  const int log_heads = 6 - a.pieces, h0 = blockIdx.z << log_heads, heads = min(1 << log_heads, a.heads - h0);
  int t0, t1, seq0 = 0;
  if constexpr (InPlace) {
    seq0 = blockIdx.x;
    t0 = min(max(start[seq0], 0), n);
    t1 = min(start[seq0 + 1], n);
  } else {
    t0 = blockIdx.x * kCompactTokens;
    t1 = min(t0 + kCompactTokens, n);
  }
  if (t0 >= t1) return;
  auto look_up = [&](int tile, int half) {
    if (tid >= kCompactTokens) return;
    const int j = tile + tid;
    int64_t s = -1, d = -1;
    if (j < t1) {
      const int at = keep[j];
      int seq = seq0;
      if constexpr (!InPlace) {   // the last sequence that starts at or before j
        int lo = 0, hi = seqs;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (start[mid] <= j) lo = mid + 1; else hi = mid;
        }
        seq = lo - 1;
      }
      if (seq >= 0 && j < start[seq + 1]) {
        s = token_at(a, from, width, seq, at);
        d = token_at(a, InPlace ? from : to, width, seq, j - max(start[seq], 0));
      }
    }
    src[half][tid] = s != d && d >= 0 ? s : -1;   // (in place: where it is already)
    dst[half][tid] = d;
  };
  // the thread's pieces: consecutive threads take a row's, then the next token's
  const int c = tid & ((1 << a.pieces) - 1), tok0 = tid >> a.pieces, log_step = 8 - a.pieces;
  auto piece_of = [&](int i, int* tok, int* h) {
    const int u = tok0 + (i << log_step);
    *tok = u & (kCompactTokens - 1);
    *h = u >> 6;
  };
  look_up(t0, 0);
  __syncthreads();
  int half = 0;
  for (int tile = t0; tile < t1; tile += kCompactTokens) {
    u32x4 x[kUnits];
    int64_t d[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      int tok, h;
      piece_of(i, &tok, &h);
      const int64_t s = src[half][tok], more = (h0 + h) * a.head_stride + 16 * c;
      d[i] = h < heads && s >= 0 ? dst[half][tok] + more : -1;
      if (d[i] >= 0) x[i] = *reinterpret_cast<const u32x4*>(pool + s + more);
    }
    if constexpr (InPlace) {
      if (tile + kCompactTokens < t1) look_up(tile + kCompactTokens, half ^ 1);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();   // every piece of the tile has been read
      half ^= 1;
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (d[i] >= 0) *reinterpret_cast<u32x4*>(pool + d[i]) = x[i];
  }
}

}  // namespace

int launch_resize(const TableArgs& t, const int32_t* new_len, int32_t* copies) {
  hipLaunchKernelGGL(k_resize, dim3(1), dim3(kResizeThreads), 0, reinterpret_cast<hipStream_t>(t.stream), t, new_len, copies);
  return (int)hipGetLastError();
}

int launch_fork(const TableArgs& t, const int32_t* src, const int32_t* dst, int32_t n) {
  hipLaunchKernelGGL(k_fork, dim3((unsigned)n), dim3(256), 0, reinterpret_cast<hipStream_t>(t.stream), t, src, dst, n);
  return (int)hipGetLastError();
}

int launch_copy(const LayerArgs& a, const int32_t* copies, int32_t n, void* stream) {
  const unsigned parts = (unsigned)(((a.heads << (a.shift + a.pieces)) + kCopyBlock - 1) / kCopyBlock);
  const int64_t row = INT64_C(16) << a.pieces, inner = a.slot_stride <= a.head_stride ? a.slot_stride : a.head_stride;
  const int64_t outer = a.slot_stride <= a.head_stride ? a.head_stride : a.slot_stride;
  const int64_t count = a.slot_stride <= a.head_stride ? INT64_C(1) << a.shift : a.heads;
  const dim3 g((unsigned)n, 2u * (unsigned)a.layers, parts);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (inner == row && outer == count * row) hipLaunchKernelGGL(k_copy<true>, g, dim3(256), 0, st, a, copies);
  else hipLaunchKernelGGL(k_copy<false>, g, dim3(256), 0, st, a, copies);
  return (int)hipGetLastError();
}

int launch_compact(const LayerArgs& a, const int32_t* from, const int32_t* to, const int32_t* start,
                   const int32_t* keep, int32_t seqs, int32_t width, int32_t n, void* stream) {
  const unsigned per = 64u >> a.pieces, groups = ((unsigned)a.heads + per - 1) / per;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (to)
    hipLaunchKernelGGL(k_compact<false>, dim3((unsigned)((n + kCompactTokens - 1) / kCompactTokens), 2u * (unsigned)a.layers, groups),
                       dim3(256), 0, st, a, from, to, start, keep, seqs, width, n);
  else
    hipLaunchKernelGGL(k_compact<true>, dim3((unsigned)seqs, 2u * (unsigned)a.layers, groups), dim3(256), 0, st, a, from,
                       from, start, keep, seqs, width, n);
  return (int)hipGetLastError();
}

}  // namespace dc
