// The walk for at most 32 query rows: each wave takes keys of its own (of
// every 128 keys 32) and holds all of the rows, in one or two tiles of 16.
// Included inside namespace dc, anonymous namespace, of k_attn.hip, behind
// attn_common.h.
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
// With so few rows the time is that of reading the cache: 4 sequences x 131072
// keys x 8 kv heads 260 us, 6.0 TB/s.  So the weights of a single tile enter as
// two bf16 pieces (16 bits) at no cost; their sum comes from the matrix core
// against ones, of the pieces as they entered.  A step's keys are loaded while
// the step before is worked on, its values behind them; the waves take turns
// in steps of 32 keys, so that a block's loads are neighbours.
#pragma once

__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int D, bool F8, int N>
struct Keys {
  static constexpr int C = D / 32;   // products of a 16-key half
  static constexpr int J = D / 16;   // products of a step's values
  static constexpr int kRows = 16 * N;
  static constexpr bool kTwo = N == 1;   // weights in two pieces
  uint4 q[N][C];
  f32x4 o[N][J];
  f32x4 l[N];
  float m[N];
  int32_t hi[N];   // keys the lane's row of a tile sees: [0, hi)

  __device__ __forceinline__ void start(const AttnArgs& a, const Item& it, int row0, int h, uint32_t flip) {
    const int lane = thread_anew() & 63, g = lane >> 4;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int row = min(row0 + 16 * n + (lane & 15), it.rows - 1);   // past the last row: the last one again
      const int tok = a.gq_d.of(row), hh = row - tok * a.gq;
      const uint16_t* p = a.q + (int64_t)(it.t0 + tok) * a.qs + (int64_t)(h * a.gq + hh) * D;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int d = F8 ? 64 * (i >> 1) + 16 * g + 8 * (i & 1) : 32 * i + 8 * g;   // as the keys' lanes hold them
        uint4 w = *reinterpret_cast<const uint4*>(p + d);
        if constexpr (F8) w.x ^= flip, w.y ^= flip, w.z ^= flip, w.w ^= flip;
        q[n][i] = w;
      }
      hi[n] = it.sees(tok);
#pragma unroll
      for (int j = 0; j < J; ++j) o[n][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      l[n] = f32x4{0.f, 0.f, 0.f, 0.f};
      m[n] = kLow;
    }
  }

  // Whether some result of the wave is not finite though its row's weights are.
  __device__ __forceinline__ bool unfinite_results() const {
    bool bad = false;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};   // NaN as soon as one is not finite
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) z[r] = __builtin_fmaf(o[n][j][r], 0.f, z[r]);
      bad |= (z[0] + z[1]) + (z[2] + z[3]) != 0.f && __builtin_isfinite(l[n][0]);
    }
    return __builtin_amdgcn_ballot_w64(bad) != 0;
  }

  static constexpr int KB = F8 ? 1 : 2;                // bytes of an element
  static constexpr int KL = D * KB / 64;               // 16-byte loads of a key's lane group
  static constexpr int VW = D * KB / 64;               // words of a lane's piece of a value row
  static constexpr int kStep = 32 * kWaves;            // from a wave's step to its next

  // A wave's keys and values on their way.
  struct Stage {
    Words<4> kr[2][KL];
    Words<VW> vr[8];
    const uint8_t *kb[2], *vb[2];
    // the two 16-key halves of the step at k (the last one that holds keys
    // again past the end, k1: masked by their numbers)
    __device__ __forceinline__ void seek(const Stream& st, Pages& pages, int k, int k1) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int64_t off = pages.offset(st, min(k + 16 * t, (k1 - 1) & ~15));
        kb[t] = st.k + off;
        vb[t] = st.v + off;
      }
    }
    __device__ __forceinline__ void load_k(const Stream& st) {
      const int lane = threadIdx.x & 63, koff = (lane & 15) * st.slot_stride + (lane >> 4) * 16;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < KL; ++i) kr[t][i] = load_words<4>(kb[t] + koff + 64 * i);
    }
    __device__ __forceinline__ void load_v(const Stream& st) {
      const int lane = threadIdx.x & 63, voff = 4 * (lane >> 4) * st.slot_stride + (lane & 15) * (VW * 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) vr[e] = load_words<VW>(vb[e >> 2] + voff + (e & 3) * st.slot_stride);
    }
  };

  // The wave's steps of keys [k0, k1) of the stream (its first at k0; k0 a
  // multiple of 32), the first of them loaded into g; scores c q.k in base 2.
  // Every row sees the keys below `lo`, none those from `up` on (k1 <= up).
  __device__ __forceinline__ void walk(const Stream& st, Stage& g_, Pages& pages, int k0, int k1, int lo, int up, float c) {
    // Q is here before the loop: loads return in order, so that a wait for it
    // inside would also be one for the values that are on their way.
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < C; ++i) asm volatile("" : "+v"(q[n][i].x), "+v"(q[n][i].y), "+v"(q[n][i].z), "+v"(q[n][i].w));
    int k = k0;
    for (; k + kStep < k1; k += kStep) step<true>(st, g_, pages, k, k1, lo, up, c);
    if (k < k1) step<false>(st, g_, pages, k, k1, lo, up, c);
  }

 private:
  // One step; MORE: another one follows, whose keys and values are sent for as
  // soon as their registers are free.  (Without branches on it, so that the
  // waits count what is really on its way.)
  template <bool MORE>
  __device__ __forceinline__ void step(const Stream& st, Stage& g_, Pages& pages, int k, int k1, int lo, int up, float c) {
    const int g = (threadIdx.x & 63) >> 4;
    f32x4 s[N][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int n = 0; n < N; ++n) s[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < C; ++i) {
        uint4 a;
        if constexpr (F8) {
          const uint32_t w0 = g_.kr[t][i >> 1].w[2 * (i & 1)], w1 = g_.kr[t][i >> 1].w[2 * (i & 1) + 1];
          a = uint4{cvt2(w0, false), cvt2(w0, true), cvt2(w1, false), cvt2(w1, true)};
        } else {
          a = uint4{g_.kr[t][i].w[0], g_.kr[t][i].w[1], g_.kr[t][i].w[2], g_.kr[t][i].w[3]};
        }
#pragma unroll
        for (int n = 0; n < N; ++n) s[n][t] = mfma16(a, q[n][i], s[n][t]);
      }
    }
    const bool masked = k + 32 > lo;
    if constexpr (MORE) {
      g_.seek(st, pages, k + kStep, k1);
      g_.load_k(st);
    }
    bool unfinite = false;
    if (__builtin_expect(masked, 0)) {
      // values that no row sees count as zero (the slots may hold
      // anything), and so do, for now, those that are not finite
      uint32_t any = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int key = k + 16 * (e >> 2) + 4 * g + (e & 3);
#pragma unroll
        for (int n = 0; n < N; ++n) s[n][e >> 2][e & 3] = key < hi[n] ? s[n][e >> 2][e & 3] : -__builtin_inff();
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t v = key >= up ? 0u : g_.vr[e].w[w], odd = not_finite<F8>(v);
          g_.vr[e].w[w] = only_finite<F8>(v, odd);
          any |= odd;
        }
      }
      unfinite = __builtin_amdgcn_ballot_w64(any != 0) != 0;
    }
    uint4 ph[N], pl[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = s[n][e >> 2][e & 3];
      float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      top *= c;
      if (__builtin_expect(__builtin_amdgcn_ballot_w64(top > m[n] + kSlack) != 0, 0)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m[n], top);
        const float f = __builtin_amdgcn_exp2f(m[n] - mn);
        m[n] = mn;
#pragma unroll
        for (int r = 0; r < 4; ++r) l[n][r] *= f;
        const Factor k(f);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[n][j][r] = k.of(o[n][j][r]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_exp2f(x[e] * c - m[n]);
      ph[n] = uint4{pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
      const uint4 ones = uint4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
      l[n] = mfma16(ones, ph[n], l[n]);
      if constexpr (kTwo) {
        pl[n] = uint4{pack2(x[0] - lo_f(ph[n].x), x[1] - hi_f(ph[n].x)), pack2(x[2] - lo_f(ph[n].y), x[3] - hi_f(ph[n].y)),
                      pack2(x[4] - lo_f(ph[n].z), x[5] - hi_f(ph[n].z)), pack2(x[6] - lo_f(ph[n].w), x[7] - hi_f(ph[n].w))};
        l[n] = mfma16(ones, pl[n], l[n]);
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {   // element j of the 8 keys
      const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
      uint32_t y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = F8 ? cvt2(g_.vr[e].w[j >> 2], (j >> 1) & 1) : g_.vr[e].w[j >> 1];
      const uint4 v = uint4{__builtin_amdgcn_perm(y[1], y[0], sel), __builtin_amdgcn_perm(y[3], y[2], sel),
                            __builtin_amdgcn_perm(y[5], y[4], sel), __builtin_amdgcn_perm(y[7], y[6], sel)};
#pragma unroll
      for (int n = 0; n < N; ++n) {
        o[n][j] = mfma16(v, ph[n], o[n][j]);
        if constexpr (kTwo) o[n][j] = mfma16(v, pl[n], o[n][j]);
      }
    }
    if constexpr (MORE) g_.load_v(st);
    if (__builtin_expect(unfinite, 0)) {
#pragma unroll 1
      for (int key = k; key < min(k + 32, up); ++key) {
        const uint8_t* row = value_row(st, key) + (F8 ? 1 : 2) * J * 4 * g;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < J; j += 2)
#pragma unroll
            for (int n = 0; n < N; ++n) {
              const f32x2 v = unfinite_pair<F8>(row, J * r + j, key < hi[n]);
              o[n][j][r] += v[0];
              o[n][j + 1][r] += v[1];
            }
      }
    }
  }
};

// The four waves' sums of one block (they walked different keys for the same
// rows) joined in LDS, 16 rows at a time, and handed to `put`, D/16
// consecutive elements a thread.  With `look`, results that are not finite (see
// Factor) are not joined: true.
template <int D>
struct KeysLds {
  uint32_t odd[kWaves];
  float ml[kWaves][32][2];
  alignas(16) float o[kWaves][16][D + 4];
};
template <int D, bool F8, int N, class Put>
__device__ __forceinline__ bool join(const Keys<D, F8, N>& R, KeysLds<D>& sh, bool look, Put put) {
  const int tid = thread_anew(), wave = tid >> 6, lane = tid & 63, g = lane >> 4, i16 = lane & 15;
  constexpr int J = D / 16;
  if constexpr (!F8) {
    const bool odd = R.unfinite_results();
    if (lane == 0) sh.odd[wave] = odd;
  }
  if (g == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      sh.ml[wave][16 * n + i16][0] = R.m[n];
      sh.ml[wave][16 * n + i16][1] = R.l[n][0];
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (n > 0) __syncthreads();
    // element (D/16)(4 g + r) + j of row i16 is o[j][r]
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < J; j += 4)
        *reinterpret_cast<f32x4*>(&sh.o[wave][i16][J * (4 * g + r) + j]) =
            f32x4{R.o[n][j][r], R.o[n][j + 1][r], R.o[n][j + 2][r], R.o[n][j + 3][r]};
    __syncthreads();
    if (!F8 && n == 0 && look &&
        __builtin_expect(__builtin_amdgcn_readfirstlane(sh.odd[0] | sh.odd[1] | sh.odd[2] | sh.odd[3]) != 0, 0)) {
      __syncthreads();   // read before the next time writes there
      return true;
    }
    const int row = tid >> 4, e = (tid & 15) * J;
    float m = kLow, l = 0.f, x[J];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sh.ml[w][16 * n + row][0]);
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(sh.ml[w][16 * n + row][0] - m);
      l += sh.ml[w][16 * n + row][1] * f;
      const Factor k(f);
#pragma unroll
      for (int j = 0; j < J; ++j) x[j] += k.of(sh.o[w][row][e + j]);
    }
    put(16 * n + row, e, m, l, x);
  }
  return false;
}
