// Verifying drafted tokens: with p = softmax(l / T) and q likewise of the draft
// model's logits, a draft t stands if u q(t) < p(t); at the first that does not
// the new token is drawn from max(p - q, 0), behind the last one from p.
//
// Two launches.  k_verify_stats: for every row its largest logit and the sum of
// the exponentials, a block for each piece of a row.  k_verify_pick: joins the
// rows' sums, decides, and looks for the piece, the vector and the token that
// r sum_k w_k falls on.
//
// The answers are whole numbers: a token changes when rounding moves one of V
// borders past r, which with sums good to d happens 2 V d times of all (V = 10^5
// and fp32's 1e-7: once in 50 calls).  So weights, sums and comparisons are fp64,
// exponentials to 2e-14 (2^f by a polynomial of degree 9).
#include <hip/hip_runtime.h>

#include "step.h"

namespace dc {
namespace {

#include "combine.h"

constexpr int kThreads = kVerifyThreads, kVec = kVerifyVec;
constexpr float kMinusInf = -__builtin_inff();
// What sums over max(p - q, 0) may be from rounding alone where p = q: p and q are
// good to 5e-14 each; ten times that counts as nothing.
constexpr double kNothing = 0x1p-40;

// s f + c with the constant in scalar registers: left to itself the compiler takes
// the accumulating form and moves each constant to vector registers first, two
// moves a step.
__device__ __forceinline__ double fma_c(double s, double f, double c) {
  double r;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(s), "v"(f), "s"(c));
  return r;
}

// 2^y for y <= 0 (a little above, too); 0 for -infinity and for NaN.  (The whole
// part by additions of 1.5 2^52 and an integer addition to the exponent instead of
// rint and ldexp: no faster.)
__device__ __forceinline__ double exp2_neg(double y) {
  y = __builtin_fmax(y, -1100.0);
  const double n = __builtin_rint(y), f = y - n;   // |f| <= 1/2
  // interpolates 2^f at the zeros of the Chebyshev polynomial of degree 10
  double s = fma_c(f, 1.0205905320493103e-07, 1.3259645243929057e-06);
  s = fma_c(s, f, 1.5252672925346873e-05);
  s = fma_c(s, f, 0.00015403433751254997);
  s = fma_c(s, f, 0.0013333558200793719);
  s = fma_c(s, f, 0.009618129193934304);
  s = fma_c(s, f, 0.05550410866465168);
  s = fma_c(s, f, 0.2402265069564034);
  s = fma_c(s, f, 0.6931471805599462);
  s = fma_c(s, f, 1.0000000000000135);
  return __builtin_ldexp(s, (int)n);
}

// Weight of a logit against the largest one.
__device__ __forceinline__ double weight(float l, float m, double k) { return exp2_neg(((double)l - (double)m) * k); }

template <bool F32>
__device__ __forceinline__ float logit(const void* row, int i) {
  if constexpr (F32) return static_cast<const float*>(row)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(row)[i] << 16);
}

template <bool F32>
__device__ __forceinline__ const void* row_of(const void* base, int64_t stride, int row) {
  return static_cast<const uint8_t*>(base) + (int64_t)row * stride * (F32 ? 4 : 2);
}

// Elements between the 16-byte border before a row (32 for fp32) and the row.
template <bool F32>
__device__ __forceinline__ int lead_of(const void* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) / (F32 ? 4 : 2)) % kVec);
}

// Logits i .. i+7 of a row of V; what lies outside it counts as -infinity.
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int i, int V, float* l) {
  const uint8_t* at = static_cast<const uint8_t*>(row) + (int64_t)i * (F32 ? 4 : 2);
  if (i >= 0 && i + kVec <= V && reinterpret_cast<uintptr_t>(at) % 16 == 0) {
    if constexpr (F32) {
      const float4 a = reinterpret_cast<const float4*>(at)[0], b = reinterpret_cast<const float4*>(at)[1];
      l[0] = a.x, l[1] = a.y, l[2] = a.z, l[3] = a.w, l[4] = b.x, l[5] = b.y, l[6] = b.z, l[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(at);
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) l[2 * j] = __uint_as_float(u[j] << 16), l[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) l[j] = i + j >= 0 && i + j < V ? logit<F32>(row, i + j) : kMinusInf;
}

// log2(e) / T of a sequence; 0: greedy.
__device__ __forceinline__ double factor(const float* temperature, int seq) {
  if (!temperature) return 1.4426950408889634074;
  const float t = temperature[seq];
  if (!(t > 0.f)) return 0.0;
  return 1.4426950408889634074 / (double)fminf(t, 3.402823466e38f);
}

__device__ __forceinline__ double shfl_xor(double v, int m) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl_xor((uint32_t)b, m), hi = __shfl_xor((uint32_t)(b >> 32), m);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ void st_dev64(double* p, double v) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double ld_dev64(const double* p) {
  return __builtin_bit_cast(double, __hip_atomic_load(reinterpret_cast<uint64_t*>(const_cast<double*>(p)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// The larger of two (value, index) pairs, the lower index of equal ones; a NaN
// is never the larger.
__device__ __forceinline__ void keep_larger(float& m, int& at, float m2, int at2) {
  if (m2 > m || (m2 == m && at2 < at)) m = m2, at = at2;
}

// ------------------------------------------------------------------ stats
// Block (piece, row, side).  Bound by the vector unit, whose 22 instructions for a
// logit are 18 fp64 ones of the exponential, the maximum, the test for NaN and the
// reductions' share, and for fp32 logits by HBM almost as much: 455 rows of 100003
// fp32 logits 43 us (4.2 TB/s), 829 rows of bf16 67 us (2.5 TB/s).
template <bool F32, int U>
__global__ void __launch_bounds__(kThreads) k_verify_stats(VerifyArgs a) {
  __shared__ float sm[4];
  __shared__ int sat[4], scount[8];
  __shared__ double sz[4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int sides = a.q ? 2 : 1, c = blockIdx.x % a.chunks, rs = blockIdx.x / a.chunks, side = rs % sides, row = rs / sides;
  // the counters of the next launch (the grid's threads are numbered with 32 bits: a step further needs more)
  for (size_t i = (size_t)blockIdx.x * kThreads + tid; i < (size_t)a.seqs; i += (size_t)gridDim.x * kThreads) a.arrived[i] = 0;
  const int V = a.vocab;
  const void* l = side ? row_of<F32>(a.q, a.qs, row) : row_of<F32>(a.p, a.ps, row);
  const int lead = lead_of<F32>(l);
  // The row's sequence: how many sequences end at or before it, by 256 of the starts
  // at a time, evenly spaced among those in question.  (All of them in every block are
  // the square of a batch: the statistics of 2^18 sequences of a row of 64 logits took
  // 18.6 ms that way, 1.6 this way.)
  const int first = a.q_start[0];
  int seq = 0;   // so many do, and perhaps some of the next `open`
  for (int open = a.seqs, turn = 0; open > 0; turn ^= 4) {
    const int step = (open + kThreads - 1) / kThreads, at = (tid + 1) * step;
    const uint64_t ends = __ballot(at <= open && a.q_start[seq + at] <= row);
    if (lane == 0) scount[turn + wave] = __builtin_popcountll(ends);
    __syncthreads();
    const int n = (scount[turn] + scount[turn + 1] + scount[turn + 2] + scount[turn + 3]) * step;
    seq += n;
    open = min(open - n, step - 1);
  }
  if (seq >= a.seqs || row < first) return;   // a row of no sequence
  if (side && row + 1 >= a.q_start[seq + 1]) return;   // behind the last draft
  const double k = factor(a.temperature, seq);
  if (side && k == 0.0) return;

  float v[U][kVec];
  const int v0 = c * U * kThreads + tid;
#pragma unroll
  for (int u = 0; u < U; ++u) load8<F32>(l, (v0 + u * kThreads) * kVec - lead, V, v[u]);
  // the largest logit; where it first is, for greedy rows alone
  float m = kMinusInf;
  int at = 0x7FFFFFFF;
  bool nan = false;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < kVec; j += 2) {
      nan |= __builtin_isunordered(v[u][j], v[u][j + 1]);
      m = fmaxf(fmaxf(m, v[u][j]), v[u][j + 1]);
    }
  if (k == 0.0) {
#pragma unroll
    for (int u = U - 1; u >= 0; --u)
#pragma unroll
      for (int j = kVec - 1; j >= 0; --j)
        if (v[u][j] == m) at = (v0 + u * kThreads) * kVec - lead + j;
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const float m2 = __shfl_xor(m, x);
    const int at2 = __shfl_xor(at, x);
    keep_larger(m, at, m2, at2);
  }
  if (lane == 0) sm[wave] = m, sat[wave] = at;
  __syncthreads();
  m = sm[0], at = sat[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) keep_larger(m, at, sm[w], sat[w]);
  double z = 0.0;
  if (k != 0.0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < kVec; ++j) z += weight(v[u][j], m, k);
  }
  if (nan) z = __builtin_nan("");
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) z += shfl_xor(z, x);
  if (lane == 0) sz[wave] = z;
  __syncthreads();
  if (tid == 0) {
    VerifyPart p;
    p.m = m;
    p.at = at;
    p.z = (sz[0] + sz[1]) + (sz[2] + sz[3]);
    a.part[((size_t)row * 2 + side) * a.chunks + c] = p;
  }
}

// ------------------------------------------------------------------- pick
struct RowStat {
  float m;
  int at;
  double z;     // > 0 unless the row has no distribution
};

// A row's sums from those of its pieces, by 16 lanes that all get the result
// (greedy, k = 0: z is 1, or NaN or 0 as for any row).
__device__ __forceinline__ RowStat join16(const VerifyPart* part, int chunks, double k) {
  const int i = threadIdx.x & 15;
  RowStat r{kMinusInf, 0x7FFFFFFF, 0.0};
  for (int c = i; c < chunks; c += 16) keep_larger(r.m, r.at, part[c].m, part[c].at);
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) {
    const float m2 = __shfl_xor(r.m, x);
    const int at2 = __shfl_xor(r.at, x);
    keep_larger(r.m, r.at, m2, at2);
  }
  for (int c = i; c < chunks; c += 16) r.z += part[c].z * (k == 0.0 ? 1.0 : weight(part[c].m, r.m, k));
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) r.z += shfl_xor(r.z, x);
  if (k == 0.0 && r.z == 0.0) r.z = __builtin_isfinite(r.m) ? 1.0 : 0.0;
  if (!__builtin_isfinite(r.m)) r.z = 0.0;
  return r;
}

// One row of a sequence as the decision needs it.
struct Judged {
  RowStat p, q;
  int token;
  int stands;        // its draft does
  float share;       // p(token)
};

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ double scan64(double v, int lane) {
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t o = (uint64_t)__shfl_up((uint32_t)(b >> 32), x) << 32 | __shfl_up((uint32_t)b, x);
    if (lane >= x) v += __builtin_bit_cast(double, o);
  }
  return v;
}
__device__ __forceinline__ double lane64(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)__shfl((uint32_t)(b >> 32), l) << 32 | __shfl((uint32_t)b, l));
}

// A thread for each vector of a piece.  With a draft model's logits (Q) every
// piece has its block and the last one to finish chooses.  Without them the
// pieces' sums are those of the statistics, but for the piece that holds the
// token taken off, and one block does it all (64 sequences of 100003 fp32 logits
// 42 -> 16.5 us).
//
// Bound by latency (decision, sums, search and the piece's own exponentials wait
// for each other) and with many blocks by the vector unit, half of it for the
// decision that each block repeats: 63 sequences of 9 rows of 100003 bf16 logits
// take 35 us by pieces of 2048 logits, 29 by 4096, 44 by 8192 (blocks of 16 waves
// leave CUs waiting for their slowest).  Blocks of 16 waves are started 0.2 us apart
// on an XCD, whatever they do: 2^20 sequences without rows take 25 ms.
template <bool F32, bool Q, int THREADS>
__global__ void __launch_bounds__(THREADS) k_verify_pick(VerifyArgs a) {
  constexpr int WAVES = THREADS / 64;
  __shared__ Judged judged[16];
  __shared__ double sr[WAVES], sp[WAVES];
  __shared__ int last_flag, found[2], first_of[WAVES], last_of[WAVES];
  __shared__ double left_of[1];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int pieces = Q ? a.pieces : a.chunks, blocks = Q ? pieces : 1;   // blocks of a sequence
  const int c = blockIdx.x % blocks, seq = blockIdx.x / blocks, V = a.vocab;
  const int lo = min(max(a.q_start[seq], 0), a.n), hi = min(max(a.q_start[seq + 1], lo), a.n);
  if (lo == hi) {
    if (c == 0 && tid == 0) a.count[seq] = 0;
    return;
  }
  const double k = factor(a.temperature, seq);
  const bool greedy = k == 0.0;

  // rows lo, lo + 1, .. 16 at a time, 16 lanes each, until a draft falls
  int stop = -1, base = lo;
  Judged end{};
  for (int r0 = lo; stop < 0; r0 += 16) {
    const int row = min(r0 + (tid >> 4), hi - 1);
    Judged g{};
    if (tid < 256 && r0 + wave * 4 < hi) {
      const bool drafted = row + 1 < hi;
      g.token = drafted ? a.tokens[row + 1] : -1;
      const bool inside = g.token >= 0 && g.token < V;
      float lp = kMinusInf, lq = kMinusInf;
      if (inside) lp = logit<F32>(row_of<F32>(a.p, a.ps, row), g.token);
      if (Q && inside) lq = logit<F32>(row_of<F32>(a.q, a.qs, row), g.token);
      g.p = join16(a.part + (size_t)row * 2 * a.chunks, a.chunks, k);
      if (Q && drafted && !greedy) g.q = join16(a.part + ((size_t)row * 2 + 1) * a.chunks, a.chunks, k);
      if (inside && g.p.z > 0.0) {
        if (greedy) {
          g.stands = g.token == g.p.at;
          g.share = 1.f;
        } else {
          const double pt = weight(lp, g.p.m, k) / g.p.z;
          g.share = (float)pt;
          // NaN sums (no distribution) compare false
          const double qt = Q ? (g.q.z > 0.0 ? weight(lq, g.q.m, k) / g.q.z : __builtin_nan("")) : 1.0;
          g.stands = (double)a.accept[row] * qt < pt;
        }
      }
    }
    __syncthreads();
    if (tid < 256 && (tid & 15) == 0) judged[tid >> 4] = g;
    __syncthreads();
    // the first that does not stand; the sequence's last row does not
    const int i = __builtin_ctzll(~__ballot(lane < 16 && judged[lane & 15].stands));
    base = r0;
    if (i < 16) {
      stop = r0 + i, end = judged[i];
    } else if (c == 0 && tid < 16) {
      a.out[r0 + tid] = judged[tid].token;
      if (a.prob) a.prob[r0 + tid] = judged[tid].share;
    }
  }
  // The other rows' results: drafts that stand, and -1 behind the new token at
  // row `stop`.  Written late: loads behind a store wait for it, too.
  auto settle = [&] {
    if (c > 0) return;
    if (tid < stop - base) {
      a.out[base + tid] = judged[tid].token;
      if (a.prob) a.prob[base + tid] = judged[tid].share;
    }
    for (int r = stop + 1 + tid; r < hi; r += THREADS) {
      a.out[r] = -1;
      if (a.prob) a.prob[r] = 0.f;
    }
  };
  const bool none = !(end.p.z > 0.0);
  if (none || greedy) {
    if (c == 0 && tid == 0) {
      a.out[stop] = none ? -1 : end.p.at;
      if (a.prob) a.prob[stop] = none ? 0.f : 1.f;
      a.count[seq] = stop - lo + (none ? 0 : 1);
    }
    settle();
    return;
  }
  const bool fell = stop + 1 < hi;
  const bool minus = Q && fell && end.q.z > 0.0;
  const int less = !Q && fell && end.token >= 0 && end.token < V ? end.token : -1;
  const void* rp = row_of<F32>(a.p, a.ps, stop);
  const void* rq = minus ? row_of<F32>(a.q, a.qs, stop) : rp;
  const int lead = lead_of<F32>(rp);
  const double ip = 1.0 / end.p.z, iq = minus ? 1.0 / end.q.z : 0.0;

  double w[kVec], pp[kVec];
  // weights of this thread's vector of a piece
  auto weigh = [&](int piece) {
    const int i0 = (piece * THREADS + tid) * kVec - lead;
    float lp[kVec], lq[kVec];
    load8<F32>(rp, i0, V, lp);
    if (minus) load8<F32>(rq, i0, V, lq);
#pragma unroll
    for (int j = 0; j < kVec; ++j) pp[j] = w[j] = weight(lp[j], end.p.m, k) * ip;
    if (minus) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) w[j] = fmax(pp[j] - weight(lq[j], end.q.m, k) * iq, 0.0);
    } else if (less - i0 >= 0 && less - i0 < kVec) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) w[j] = i0 + j == less ? 0.0 : w[j];
    }
    return i0;
  };
  auto sum8 = [&](const double* x) { return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7])); };

  double* rest = a.rest + (size_t)seq * pieces * 2;
  const int own = Q ? c : (less >= 0 ? (less + lead) / (THREADS * kVec) : -1);
  double own_sum = 0.0;
  if (own >= 0) {
    weigh(own);
    double tr = sum8(w), tp = Q ? sum8(pp) : 0.0;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
      tr += shfl_xor(tr, x);
      if (Q) tp += shfl_xor(tp, x);
    }
    if (lane == 0) sr[wave] = tr, sp[wave] = tp;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) own_sum += sr[i];
    if (Q) {
      if (tid == 0) {
        st_dev64(rest + 2 * c, own_sum);
        double p = 0.0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) p += sp[i];
        st_dev64(rest + 2 * c + 1, p);
      }
      const bool last = arrive_last(a.arrived + seq, pieces, &last_flag);
      settle();
      if (!last) return;
    }
  }

  // The piece that pick * total falls on, by wave 0: in order, lanes of 64
  // pieces at a time.
  if (wave == 0) {
    const VerifyPart* part = a.part + (size_t)stop * 2 * a.chunks;
    auto sum_of = [&](int b, bool all_p) {
      if (b >= pieces) return 0.0;
      if (Q) return ld_dev64(rest + 2 * b + all_p);
      // 0 exactly where the largest weight of the piece is, as it comes out below
      return !all_p && b == own ? own_sum : part[b].z * (weight(part[b].m, end.p.m, k) * ip);
    };
    const float r = a.pick[seq];
    const double mine0 = sum_of(lane, false);
    double all = mine0;
    for (int b = lane + 64; b < pieces; b += 64) all += sum_of(b, false);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) all += shfl_xor(all, x);
    // nothing left of p - q: p itself, whose sum is 1
    const bool all_p = !(all > (minus ? kNothing : 0.0));
    const double aim = (double)r * (all_p ? 1.0 : all);
    double run = 0.0, before = 0.0;
    int piece = -1, spare = 0;
    double spare_run = 0.0;
    for (int b0 = 0; b0 < pieces && piece < 0; b0 += 64) {
      const double mine = b0 == 0 && !all_p ? mine0 : sum_of(b0 + lane, all_p), upto = scan64(mine, lane);
      const uint64_t over = __ballot(mine > 0.0 && run + upto > aim), some = __ballot(mine > 0.0);
      const int l = over ? __builtin_ctzll(over) : (some ? 63 - __builtin_clzll(some) : 0);
      before = run + lane64(upto - mine, l);
      if (over) piece = b0 + l;
      else if (some) spare = b0 + l, spare_run = before;
      run += lane64(upto, 63);
    }
    if (piece < 0) piece = spare, before = spare_run;   // rounding: the last piece that has any
    if (lane == 0) found[0] = piece, found[1] = all_p, left_of[0] = aim - before;
  }
  __syncthreads();
  const bool all_p = found[1];
  const double aim = left_of[0];

  // Within it: sums of the vectors, in order.  The first one that passes the
  // aim, or the last one that has any weight.
  const int i0 = weigh(found[0]);
  if (all_p) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j] = pp[j];
  }
  const double mine = sum8(w);
  double upto = scan64(mine, lane);
  if (lane == 63) sr[wave] = upto;
  __syncthreads();
  double below = 0.0;
#pragma unroll
  for (int i = 0; i < WAVES - 1; ++i) below += i < wave ? sr[i] : 0.0;
  upto += below;
  const uint64_t over = __ballot(mine > 0.0 && upto > aim), some = __ballot(mine > 0.0);
  if (lane == 0) {
    first_of[wave] = over ? wave * 64 + __builtin_ctzll(over) : THREADS;
    last_of[wave] = some ? wave * 64 + 63 - __builtin_clzll(some) : -1;
  }
  __syncthreads();
  int hit = THREADS, last = -1;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) hit = min(hit, first_of[i]), last = max(last, last_of[i]);
  if (hit == THREADS) hit = last;
  if (!Q) settle();
  if (tid != hit) return;
  double run = upto - mine, share = 0.0;
  int token = -1;
  bool done = false;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    run += w[j];
    if (!done && w[j] > 0.0) token = i0 + j, share = pp[j], done = run > aim;
  }
  a.out[stop] = token;
  if (a.prob) a.prob[stop] = (float)share;
  a.count[seq] = stop - lo + 1;
}

}  // namespace

int launch_verify(const VerifyArgs& a) {
  hipStream_t st = reinterpret_cast<hipStream_t>(a.stream);
  const unsigned rows = (unsigned)a.n * (a.q ? 2u : 1u);
  const dim3 g1(rows * (unsigned)a.chunks);
#define DC_VERIFY(F32_, U_)                                                                                          \
  do {                                                                                                               \
    if (a.n > 0) hipLaunchKernelGGL((k_verify_stats<F32_, U_>), g1, dim3(kThreads), 0, st, a);                       \
    if (a.q)                                                                                                         \
      hipLaunchKernelGGL((k_verify_pick<F32_, true, pick_threads(U_)>), dim3((unsigned)a.seqs * a.pieces), dim3(pick_threads(U_)), 0, st, a); \
    else                                                                                                             \
      hipLaunchKernelGGL((k_verify_pick<F32_, false, U_ * kThreads>), dim3(a.seqs), dim3(U_ * kThreads), 0, st, a);   \
  } while (0)
  if (a.f32) {
    if (a.vecs == 4) DC_VERIFY(true, 4); else DC_VERIFY(true, 1);
  } else {
    if (a.vecs == 4) DC_VERIFY(false, 4); else DC_VERIFY(false, 1);
  }
#undef DC_VERIFY
  return (int)hipGetLastError();
}

}  // namespace dc
