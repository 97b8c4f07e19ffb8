// Verifying drafted tokens: with p = softmax(l / T) and q likewise of the draft
// model's logits, a draft t stands if u q(t) < p(t); at the first that does not
// the new token is drawn from max(p - q, 0), behind the last one from p.
//
// Two launches.  k_verify_stats: for every row its largest logit and the sum of
// the exponentials, a block for each piece of a row.  k_verify_pick: a block for
// each piece of a sequence's last row; every block joins the rows' sums and
// comes to the same decision, then sums its piece's weights max(p - q, 0), and
// the block that arrives last looks for the piece, the vector and the token
// that r sum_k w_k falls on.
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

// s f + c with the constant in scalar registers: left to itself the compiler takes
// the accumulating form and moves each constant to vector registers first, two
// moves a step.
__device__ __forceinline__ double fma_c(double s, double f, double c) {
  double r;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(s), "v"(f), "s"(c));
  return r;
}

// 2^y for y <= 0 (a little above, too); 0 for -infinity and for NaN.
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
// Block (piece, row, side).  Reads are bound by HBM where there are many; the 17
// fp64 operations of an exponential keep the vector unit busy for about as long.
template <bool F32, int U>
__global__ void __launch_bounds__(kThreads) k_verify_stats(VerifyArgs a) {
  __shared__ float sm[4];
  __shared__ int sat[4], scount[4];
  __shared__ double sz[4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int sides = a.q ? 2 : 1, c = blockIdx.x % a.chunks, rs = blockIdx.x / a.chunks, side = rs % sides, row = rs / sides;
  // the counters of the next launch
  for (int i = blockIdx.x * kThreads + tid; i < a.seqs; i += gridDim.x * kThreads) a.arrived[i] = 0;
  const int V = a.vocab;
  const void* l = side ? row_of<F32>(a.q, a.qs, row) : row_of<F32>(a.p, a.ps, row);
  const int lead = lead_of<F32>(l);
  // the row's sequence: how many sequences end at or before it
  int before = 0, first = 0;
  for (int i = tid; i <= a.seqs; i += kThreads) {
    const int s = a.q_start[i];
    before += i > 0 && s <= row;
    if (i == 0) first = s;
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) before += __shfl_xor(before, m);
  if (lane == 0) scount[wave] = before;
  if (tid == 0) sat[0] = first;
  __syncthreads();
  const int seq = scount[0] + scount[1] + scount[2] + scount[3];
  if (seq >= a.seqs || row < sat[0]) return;   // a row of no sequence
  if (side && row + 1 >= a.q_start[seq + 1]) return;   // behind the last draft
  const double k = factor(a.temperature, seq);
  if (side && k == 0.0) return;
  __syncthreads();

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

// The weights of a vector's logits: p - q where that is positive, and p.
template <bool F32>
__device__ __forceinline__ void weights8(const float* lp, const float* lq, const RowStat& p, const RowStat& q, double k,
                                         int i0, int less, bool minus, double* w, double* sp) {
  const double ip = 1.0 / p.z, iq = minus ? 1.0 / q.z : 0.0;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const double pj = weight(lp[j], p.m, k) * ip;
    double qj = 0.0;
    if (minus) qj = weight(lq[j], q.m, k) * iq;
    if (i0 + j == less) qj = 1.0;
    sp[j] = pj;
    w[j] = fmax(pj - qj, 0.0);
  }
}

template <bool F32, int U>
__global__ void __launch_bounds__(kThreads) k_verify_pick(VerifyArgs a) {
  __shared__ Judged judged[16];
  __shared__ double sr[U * 4], sp[U * 4];
  __shared__ int last_flag, found[2];
  __shared__ double left_of[1];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int c = blockIdx.x % a.chunks, seq = blockIdx.x / a.chunks, V = a.vocab;
  const int lo = min(max(a.q_start[seq], 0), a.n), hi = min(max(a.q_start[seq + 1], lo), a.n);
  if (lo == hi) {
    if (c == 0 && tid == 0) a.count[seq] = 0;
    return;
  }
  const double k = factor(a.temperature, seq);
  const bool greedy = k == 0.0;

  // rows lo, lo + 1, .. 16 at a time, 16 lanes each, until a draft falls
  int stop = -1;
  Judged end{};
  for (int r0 = lo; stop < 0; r0 += 16) {
    const int row = min(r0 + (tid >> 4), hi - 1);
    const bool drafted = row + 1 < hi;
    Judged g{};
    g.token = drafted ? a.tokens[row + 1] : -1;
    const bool inside = g.token >= 0 && g.token < V;
    float lp = kMinusInf, lq = kMinusInf;
    if (inside) lp = logit<F32>(row_of<F32>(a.p, a.ps, row), g.token);
    if (inside && a.q) lq = logit<F32>(row_of<F32>(a.q, a.qs, row), g.token);
    g.p = join16(a.part + (size_t)row * 2 * a.chunks, a.chunks, k);
    if (a.q && drafted && !greedy) g.q = join16(a.part + ((size_t)row * 2 + 1) * a.chunks, a.chunks, k);
    if (inside && g.p.z > 0.0) {
      if (greedy) {
        g.stands = g.token == g.p.at;
        g.share = 1.f;
      } else {
        const double pt = weight(lp, g.p.m, k) / g.p.z;
        g.share = (float)pt;
        // NaN sums (no distribution) compare false
        const double qt = a.q ? (g.q.z > 0.0 ? weight(lq, g.q.m, k) / g.q.z : __builtin_nan("")) : 1.0;
        g.stands = (double)a.accept[row] * qt < pt;
      }
    }
    __syncthreads();
    if ((tid & 15) == 0) judged[tid >> 4] = g;
    __syncthreads();
    const int n = min(16, hi - r0);
    int i = 0;
    while (i < n && judged[i].stands) {   // the last row's does not
      if (c == 0 && tid == 0) {
        a.out[r0 + i] = judged[i].token;
        if (a.prob) a.prob[r0 + i] = judged[i].share;
      }
      ++i;
    }
    if (i < n) stop = r0 + i, end = judged[i];
  }
  // the new token goes to row `stop`, -1 behind it
  if (c == 0)
    for (int r = stop + 1 + tid; r < hi; r += kThreads) {
      a.out[r] = -1;
      if (a.prob) a.prob[r] = 0.f;
    }
  const bool none = !(end.p.z > 0.0);
  if (none || greedy) {
    if (c == 0 && tid == 0) {
      a.out[stop] = none ? -1 : end.p.at;
      if (a.prob) a.prob[stop] = none ? 0.f : 1.f;
      a.count[seq] = stop - lo + (none ? 0 : 1);
    }
    return;
  }
  const bool fell = stop + 1 < hi;
  const bool minus = fell && a.q && end.q.z > 0.0;
  const int less = fell && !a.q && end.token >= 0 && end.token < V ? end.token : -1;
  const void* rp = row_of<F32>(a.p, a.ps, stop);
  const void* rq = minus ? row_of<F32>(a.q, a.qs, stop) : rp;
  const int lead = lead_of<F32>(rp);

  double w[kVec], pp[kVec];
  double tr = 0.0, tp = 0.0;
#pragma unroll 1
  for (int u = 0; u < U; ++u) {
    const int i0 = ((c * U + u) * kThreads + tid) * kVec - lead;
    if (i0 >= V) continue;
    float lp[kVec], lq[kVec];
    load8<F32>(rp, i0, V, lp);
    if (minus) load8<F32>(rq, i0, V, lq);
    weights8<F32>(lp, lq, end.p, end.q, k, i0, less, minus, w, pp);
#pragma unroll
    for (int j = 0; j < kVec; ++j) tr += w[j], tp += pp[j];
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) tr += shfl_xor(tr, x), tp += shfl_xor(tp, x);
  if (lane == 0) sr[wave] = tr, sp[wave] = tp;
  __syncthreads();
  double* rest = a.rest + (size_t)seq * a.chunks * 2;
  if (tid == 0) {
    st_dev64(rest + 2 * c, (sr[0] + sr[1]) + (sr[2] + sr[3]));
    st_dev64(rest + 2 * c + 1, (sp[0] + sp[1]) + (sp[2] + sp[3]));
  }
  if (!arrive_last(a.arrived + seq, a.chunks, &last_flag)) return;

  // The piece that pick * total falls on, by wave 0: in order, lanes of 64
  // pieces at a time.
  if (wave == 0) {
    double all = 0.0, allp = 0.0;
    for (int b = lane; b < a.chunks; b += 64) all += ld_dev64(rest + 2 * b), allp += ld_dev64(rest + 2 * b + 1);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) all += shfl_xor(all, x), allp += shfl_xor(allp, x);
    const int which = all > 0.0 ? 0 : 1;   // nothing left of p - q: p itself
    const double aim = (double)a.pick[seq] * (which ? allp : all);
    double run = 0.0, before = 0.0;
    int piece = -1, spare = -1;
    double spare_run = 0.0;
    for (int b0 = 0; b0 < a.chunks && piece < 0; b0 += 64) {
      const double mine = b0 + lane < a.chunks ? ld_dev64(rest + 2 * (b0 + lane) + which) : 0.0;
      double upto = mine;
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) {
        const uint64_t b = __builtin_bit_cast(uint64_t, upto);
        const uint64_t o = (uint64_t)__shfl_up((uint32_t)(b >> 32), x) << 32 | __shfl_up((uint32_t)b, x);
        if (lane >= x) upto += __builtin_bit_cast(double, o);
      }
      const uint64_t over = __ballot(mine > 0.0 && run + upto > aim), some = __ballot(mine > 0.0);
      const int l = over ? __builtin_ctzll(over) : (some ? 63 - __builtin_clzll(some) : 0);
      const double excl = upto - mine;
      const uint64_t eb = __builtin_bit_cast(uint64_t, excl), ub = __builtin_bit_cast(uint64_t, upto);
      before = run + __builtin_bit_cast(double, (uint64_t)__shfl((uint32_t)(eb >> 32), l) << 32 | __shfl((uint32_t)eb, l));
      if (over) piece = b0 + l;
      else if (some) spare = b0 + l, spare_run = before;
      run += __builtin_bit_cast(double, (uint64_t)__shfl((uint32_t)(ub >> 32), 63) << 32 | __shfl((uint32_t)ub, 63));
    }
    if (piece < 0) piece = spare, before = spare_run;   // rounding: the last piece that has any
    if (lane == 0) found[0] = piece, found[1] = which, left_of[0] = aim - before;
  }
  __syncthreads();
  const int piece = found[0], which = found[1];
  const double aim = left_of[0];

  // Within it: sums of the vectors, in order.
  double mine[U], upto[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i0 = ((piece * U + u) * kThreads + tid) * kVec - lead;
    float lp[kVec], lq[kVec];
    load8<F32>(rp, i0, V, lp);
    if (minus) load8<F32>(rq, i0, V, lq);
    weights8<F32>(lp, lq, end.p, end.q, k, i0, less, minus, w, pp);
    mine[u] = 0.0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) mine[u] += which ? pp[j] : w[j];
    upto[u] = mine[u];
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
      const uint64_t b = __builtin_bit_cast(uint64_t, upto[u]);
      const uint64_t o = (uint64_t)__shfl_up((uint32_t)(b >> 32), x) << 32 | __shfl_up((uint32_t)b, x);
      if (lane >= x) upto[u] += __builtin_bit_cast(double, o);
    }
    if (lane == 63) sr[u * 4 + wave] = upto[u];
  }
  if (tid == 0) found[0] = 0x7FFFFFFF, found[1] = -1;
  __syncthreads();
  // vectors in order: number (u, tid).  The first one that passes the aim, or
  // the last one that has any weight.
#pragma unroll
  for (int u = 0; u < U; ++u) {
    double base = 0.0;
    for (int i = 0; i < u * 4 + wave; ++i) base += sr[i];
    upto[u] += base;
    if (mine[u] > 0.0) {
      if (upto[u] > aim) atomicMin(&found[0], u * kThreads + tid);
      atomicMax(&found[1], u * kThreads + tid);
    }
  }
  __syncthreads();
  const int hit = found[0] != 0x7FFFFFFF ? found[0] : found[1];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (hit != u * kThreads + tid) continue;
    const int i0 = ((piece * U + u) * kThreads + tid) * kVec - lead;
    float lp[kVec], lq[kVec];
    load8<F32>(rp, i0, V, lp);
    if (minus) load8<F32>(rq, i0, V, lq);
    weights8<F32>(lp, lq, end.p, end.q, k, i0, less, minus, w, pp);
    double run = upto[u] - mine[u];
    int token = -1;
    double share = 0.0;
    bool done = false;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const double x = which ? pp[j] : w[j];
      run += x;
      if (!done && x > 0.0) token = i0 + j, share = pp[j], done = run > aim;
    }
    a.out[stop] = token;
    if (a.prob) a.prob[stop] = (float)share;
    a.count[seq] = stop - lo + 1;
  }
}

}  // namespace

int launch_verify(const VerifyArgs& a) {
  hipStream_t st = reinterpret_cast<hipStream_t>(a.stream);
  const unsigned rows = (unsigned)a.n * (a.q ? 2u : 1u);
  const dim3 g1(rows * (unsigned)a.chunks), g2((unsigned)a.seqs * (unsigned)a.chunks), b(kThreads);
#define DC_VERIFY(F32_, U_)                                                            \
  do {                                                                                 \
    if (a.n > 0) hipLaunchKernelGGL((k_verify_stats<F32_, U_>), g1, b, 0, st, a);      \
    hipLaunchKernelGGL((k_verify_pick<F32_, U_>), g2, b, 0, st, a);                    \
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
