// The walk for more than 32 query rows: a block takes 128 rows, wave w rows
// 32w .. 32w+31, and its keys come through LDS in tiles that all waves share.
// Included inside namespace dc, anonymous namespace, of k_attn.hip, behind
// attn_common.h.
//
// Products transposed as for few rows, S^T = K Q^T and O^T = V^T P^T, here
// 32x32x16: a wave reads a tile's keys and values once for 32 rows.
//   S^T result: lane l holds row l%32 and keys 8(i/4) + 4(l/32) + i%4, i < 16.
//   P^T operand B: row l%32, 8 keys of half l/32: results 8a .. 8a+7 as they
//       are, so product a of a 32-key half takes keys 16a + 4(l/32) + {0..3}
//       and those + 8.
//   V^T operand A: element 32 d + l%32, the same 8 keys: two transposing reads
//       of LDS (ds_read_b64_tr_b16: of 16 lanes, lane 4r + c supplies elements
//       4c .. 4c+3 of row r, lane j receives element j of the 4 rows).
//   LDS holds K and V as the cache does, [keys][D] in bf16, the 16-byte
//       pieces of a key permuted by an XOR with its number such that the lanes
//       that are served together reach different banks (key_swizzle,
//       value_swizzle).  bf16 keys go straight to LDS (global_load_lds, no
//       registers; the lanes choose the permuted pieces); e4m3 codes pass
//       through registers and are converted, once a block.
// Weights enter as one bf16 piece, rounded like the output (2^-8), and their sum
// is taken as they entered; a second piece would cost half of the products again
// (8 prompts 185 -> 242 us, 48 chats on an e4m3 prefix 52.7 -> 61.8).
// Measured, 8 prompts of up to 2048 tokens, 32 heads on 8, bf16: 181 to 191 us
// from one card to another, 840 to 800 TFLOP/s; with e4m3 keys 212 where bf16
// takes 191.  The matrix cores are busy 41 % of the call, at 1.84 GHz: 68 % inside
// the loop, less a block's first loads and its output (14000 of its 60000 cycles)
// and the last blocks (25 us).  Without any exponentials it would take 9 us
// less, without reading LDS 12.
#pragma once

__device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

constexpr int kStepKeys = 32;        // keys of a step
constexpr int kTileRows = 32;    // rows of a wave
constexpr int kBlockRows = kWaves * kTileRows;

// What a key's number is XOR-ed into the numbers of its pieces.  A read of K
// serves 16 keys' pieces of one number at a time, a transposing read of V 64
// bytes of 4 keys; the banks are 256 bytes wide (a key, or two of D = 64).
template <int D> __device__ __forceinline__ int key_swizzle(int key) { return D == 128 ? key & 15 : (key >> 1) & 7; }
template <int D> __device__ __forceinline__ int value_swizzle(int key) {
  return D == 128 ? (key & 3) << 2 : ((key >> 1) & 1) << 2;
}

// bf16: three tiles of one step; e4m3: two of two steps.
template <int D, bool F8>
struct TilesLds {
  static constexpr int kTiles = F8 ? 2 : 3, kKeys = F8 ? 2 * kStepKeys : kStepKeys;
  alignas(256) uint8_t k[kTiles][kKeys * D * 2];
  alignas(256) uint8_t v[kTiles][kKeys * D * 2];
  uint32_t odd[kTiles][kWaves];       // of a tile with masks: some of the values that a wave carried are not finite
};

template <int D, bool F8>
struct Tiles {
  typedef TilesLds<D, F8> Lds;
  static constexpr int KS = D / 16;   // products of 32 keys' scores
  static constexpr int DT = D / 32;   // 32-element tiles of the result
  uint4 q[KS];
  f32x16 o[DT];
  float l, m;
  int32_t hi;        // keys the lane's row sees

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    l = 0.f;
    m = kLow;
  }
  // row0: the wave's first row
  __device__ __forceinline__ void load_q(const AttnArgs& a, const Item& it, int row0, int h, uint32_t flip) {
    const int lane = thread_anew() & 63;
    const int row = min(row0 + (lane & 31), it.rows - 1);   // past the last row: the last one again
    const int tok = a.gq_d.of(row), hh = row - tok * a.gq;
    const uint16_t* p = a.q + (int64_t)(it.t0 + tok) * a.qs + (int64_t)(h * a.gq + hh) * D + 8 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      q[i] = *reinterpret_cast<const uint4*>(p + 16 * i);
      if constexpr (F8) q[i].x ^= flip, q[i].y ^= flip, q[i].z ^= flip, q[i].w ^= flip;
    }
  }

  // Whether some result of the block is not finite though its row's weights
  // are; every wave has left the walk.
  __device__ __forceinline__ bool unfinite_results(Lds& sh) const {
    f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};   // NaN as soon as one is not finite
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i & 3] = __builtin_fmaf(o[d][i], 0.f, z[i & 3]);
    const bool found = __builtin_amdgcn_ballot_w64((z[0] + z[1]) + (z[2] + z[3]) != 0.f && __builtin_isfinite(l + __shfl_xor(l, 32))) != 0;
    if ((threadIdx.x & 63) == 0) sh.odd[0][threadIdx.x >> 6] = found;
    wait_lds_barrier();
    const bool any = __builtin_amdgcn_readfirstlane(sh.odd[0][0] | sh.odd[0][1] | sh.odd[0][2] | sh.odd[0][3]) != 0;
    if (__builtin_expect(any, 0)) wait_lds_barrier();   // read before the next time writes there
    return any;
  }

  // Keys [k0, k1) of the stream (k0 a multiple of 64, its page in `pages`) for
  // the block; a wave without rows (live = false) only carries tiles.  The
  // wave's rows all see the keys below lo and none see those from up on; blo,
  // bup: the block's.
  //
  // Step h multiplies the keys of step h + 1, takes the exponentials of step h
  // and multiplies its values, in one stretch of code without branches, so
  // that the matrix core and the vector unit work at the same time within a
  // wave.  What a maximum moves is decided between steps.
  __device__ __forceinline__ void walk(const Stream& st, const Pages& pages, int k0, int k1, int lo, int up, int blo,
                                       int bup, float c, bool live, Lds& sh) {
    k1 = min(k1, bup);
    if (k0 >= k1) return;
    const int lane = thread_anew() & 63, half = lane >> 5, i32 = lane & 31;
    int ko[KS], vo[DT];
#pragma unroll
    for (int i = 0; i < KS; ++i) ko[i] = i32 * (D * 2) + (((2 * i + half) ^ key_swizzle<D>(i32)) * 16);
    const int r = (lane & 15) >> 2;   // a transposing read: the lane's key of 4, its 8 bytes of 32
#pragma unroll
    for (int d = 0; d < DT; ++d)
      vo[d] = (4 * half + r) * (D * 2) +
              (((4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ value_swizzle<D>(r)) * 16) + (lane & 1) * 8;
    if (!live) up = k0;   // no key is of interest
    Stage g(st, pages, sh);
    if constexpr (F8) {
      g.load_k(st, k0, k1);
      g.load_v(st);
      g.store_k(sh.k[0]);
      g.store_v(sh.v[0]);
      arrived();
      mend_v(sh.v[0], sh.odd[0], k0, blo, bup);
      g.load_k(st, k0 + kTile, k1);
    } else {
      g.load_k(st, k0, k1, 0);
      g.load_v(st, 0);
      if (k0 + kTile < k1) g.load_k(st, k0 + kTile, k1, 1);
      wait_loads<0>();
      arrived();
      if (k0 + kTile < k1) g.load_v(st, 1);
      if (k0 + 2 * kTile < k1) g.load_k(st, k0 + 2 * kTile, k1, 2);
      mend_v(sh.v[0], sh.odd[0], k0, blo, bup);
    }
    wait_lds_barrier();
    f32x16 s;
    if (k0 < up) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) s = mfma32(*reinterpret_cast<const uint4*>(sh.k[0] + ko[i]), q[i], s);
      prepare(s, largest(s), k0, lo, c);
    }
    if constexpr (F8) {
      for (int k = k0; k < k1; k += 2 * kTile) {
        two_steps<0>(g, st, s, k, k1, lo, up, blo, bup, c, ko, vo, sh);
        if (k + kTile < k1) two_steps<1>(g, st, s, k + kTile, k1, lo, up, blo, bup, c, ko, vo, sh);
      }
    } else {
      wait_lds_barrier();   // the first keys' place is free
      for (int k = k0; k < k1; k += 3 * kTile) {
        one_step<0>(g, st, s, k, k1, lo, up, blo, bup, c, ko, vo, sh);
        if (k + kTile < k1) one_step<1>(g, st, s, k + kTile, k1, lo, up, blo, bup, c, ko, vo, sh);
        if (k + 2 * kTile < k1) one_step<2>(g, st, s, k + 2 * kTile, k1, lo, up, blo, bup, c, ko, vo, sh);
      }
    }
    wait_lds_barrier();   // the buffers are free
  }

 private:
  static constexpr int kTile = Lds::kKeys;
  static constexpr int KW = kTile / kWaves;                       // keys of a tile that a wave carries (one page)
  static constexpr int KL = KW * D * (F8 ? 1 : 2) / 1024;         // 16-byte loads of theirs, a lane
  static constexpr int KP = D * (F8 ? 1 : 2) / 16;                // 16-byte pieces of a key
  static constexpr int KI = 64 / KP;                              // keys of a wave's load

  // At most N loads of the wave still on their way.
  template <int N> static __device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
  }
  // The wave's own LDS accesses are done, and so are every other wave's.
  static __device__ __forceinline__ void wait_lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
  // Q is here: a wait for it inside the loop would be one for younger loads
  // (they return in order; 8x2048 prompt: 187 us, 210 with it).
  __device__ __forceinline__ void arrived() {
#pragma unroll
    for (int i = 0; i < KS; ++i) asm volatile("" : "+v"(q[i].x), "+v"(q[i].y), "+v"(q[i].z), "+v"(q[i].w));
  }

  // A wave's part of the tiles on their way from the cache to LDS: wave w
  // carries keys KW w .. of each.  bf16: straight to LDS.
  struct Direct {
    Pages pages;
    int64_t off;
    int wave, ko[KL], vo;   // the lane's offsets in the keys' rows
    uint32_t at;            // LDS address of the wave's part of the first tile of keys
    __device__ __forceinline__ Direct(const Stream& st, const Pages& p, const Lds& sh) : pages(p) {
      const int lane = thread_anew() & 63;
      wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)&sh.k[0][0] + wave * (KW * D * 2);
      const int key = lane / KP, pos = lane % KP;   // LDS takes 16 bytes a lane, in the order of the lanes
#pragma unroll
      for (int i = 0; i < KL; ++i)
        ko[i] = key * st.slot_stride + (pos ^ key_swizzle<D>(KW * wave + key + KI * i)) * 16;
      vo = key * st.slot_stride + (pos ^ value_swizzle<D>(key)) * 16;
    }
    // 16 bytes a lane from base + voff to lds + 16 lane
    static __device__ __forceinline__ void to_lds(const uint8_t* base, int voff, uint32_t lds) {
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(base) : "memory", "m0");
    }
    // the keys of the tile at k into buffer b, and where its values are
    __device__ __forceinline__ void load_k(const Stream& st, int k, int k1, int b) {
      off = pages.offset(st, min(k + KW * wave, (k1 - 1) & -KW));
#pragma unroll
      for (int i = 0; i < KL; ++i)
        to_lds(st.k + off + (int64_t)(KI * i) * st.slot_stride, ko[i], at + b * (kTile * D * 2) + i * 1024);
    }
    // the values of the tile whose keys were loaded last
    __device__ __forceinline__ void load_v(const Stream& st, int b) {
#pragma unroll
      for (int i = 0; i < KL; ++i)
        to_lds(st.v + off + (int64_t)(KI * i) * st.slot_stride, vo,
               at + (uint32_t)sizeof(Lds::k) + b * (kTile * D * 2) + i * 1024);
    }
  };

  // e4m3: codes to registers, to be converted on their way to LDS.
  struct Codes {
    Words<4> kr[KL], vr[KL];
    Pages pages;
    int64_t off;
    int wave, ko;   // the lane's offset in the keys' rows
    __device__ __forceinline__ Codes(const Stream& st, const Pages& p, const Lds&) : pages(p) {
      const int lane = threadIdx.x & 63;
      wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      ko = lane / KP * st.slot_stride + lane % KP * 16;
    }
    __device__ __forceinline__ void load_k(const Stream& st, int k, int k1) {
      off = pages.offset(st, min(k + KW * wave, (k1 - 1) & -KW));
#pragma unroll
      for (int i = 0; i < KL; ++i) kr[i] = load_words<4>(st.k + off + (int64_t)(KI * i) * st.slot_stride + ko);
    }
    __device__ __forceinline__ void load_v(const Stream& st) {
#pragma unroll
      for (int i = 0; i < KL; ++i) vr[i] = load_words<4>(st.v + off + (int64_t)(KI * i) * st.slot_stride + ko);
    }
    static __device__ __forceinline__ void store(const Words<4>& w, uint8_t* row, int cc, int swizzle) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        *reinterpret_cast<uint4*>(row + (((2 * cc + u) ^ swizzle) * 16)) =
            uint4{cvt2(w.w[2 * u], false), cvt2(w.w[2 * u], true), cvt2(w.w[2 * u + 1], false), cvt2(w.w[2 * u + 1], true)};
    }
    __device__ __forceinline__ void store_k(uint8_t* lds) {
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int lane = threadIdx.x & 63, key = KW * wave + lane / KP + KI * i;
        store(kr[i], lds + key * (D * 2), lane % KP, key_swizzle<D>(key));
      }
    }
    __device__ __forceinline__ void store_v(uint8_t* lds) {
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int lane = threadIdx.x & 63, key = KW * wave + lane / KP + KI * i;
        store(vr[i], lds + key * (D * 2), lane % KP, value_swizzle<D>(key));
      }
    }
  };
  typedef std::conditional_t<F8, Codes, Direct> Stage;

  // The values of the tile at k, if it has masks: those that no row of the
  // block sees count as zero (the slots may hold anything), and so do, for
  // now, those that are not finite.  The wave's own keys, once they are in LDS.
  static __device__ __forceinline__ void mend_v(uint8_t* lds, uint32_t* odd, int k, int blo, int bup) {
    if (__builtin_expect(k + kTile <= blo, 1)) return;
    const int tid = thread_anew(), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if constexpr (F8) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (one wave wrote, other lanes read)
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < KW * D * 2 / 1024; ++i) {
      uint4* p = reinterpret_cast<uint4*>(lds + wave * (KW * D * 2) + i * 1024 + lane * 16);
      const bool dead = k + KW * wave + (i * 64 + lane) / (D / 8) >= bup;
      const uint4 u = *p;
      uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = dead ? 0u : w[j];
        const uint32_t bad = not_finite<false>(w[j]);
        w[j] = only_finite<false>(w[j], bad);
        any |= bad;
      }
      *p = uint4{w[0], w[1], w[2], w[3]};
    }
    const bool found = __builtin_amdgcn_ballot_w64(any != 0) != 0;
    if (lane == 0) odd[wave] = found;
  }

  // bf16: the step at k, its values in buffer B and the next step's keys in
  // B + 1; `s` holds its scores.  The values of the step after the next and
  // the keys of the one behind that set out, into the places that the step
  // before freed: each is on its way for two steps, with one barrier a step.
  // Three tiles of 32 keys take 48 KB (D = 128), so three blocks share a CU
  // (three waves a SIMD at 168 registers).
  template <int B>
  __device__ __forceinline__ void one_step(Stage& g, const Stream& st, f32x16& s, int k, int k1, int lo, int up, int blo,
                                           int bup, float c, const int* ko, const int* vo, Lds& sh) {
    constexpr int N = (B + 1) % 3, P = (B + 2) % 3;
    const bool more = k + kTile < k1;
    if (k + 2 * kTile < k1) g.load_v(st, P);
    if (k + 3 * kTile < k1) g.load_k(st, k + 3 * kTile, k1, B);
    float t;
    if (__builtin_expect(k < up, 1)) {
      step(s, t, sh.k[N], sh.v[B], c, ko, vo);   // (the scores of a step that is not there are not used)
      unfinite(st, k, k + kTile, up, blo, sh.odd[B]);
      if (__builtin_expect(more && k + kTile < up, 1)) prepare(s, t, k + kTile, lo, c);
    }
    if (__builtin_expect(more, 1)) {
      if (k + 3 * kTile < k1) wait_loads<2 * KL>();   // the next step's values and the keys behind; younger: this step's
      else wait_loads<0>();
      mend_v(sh.v[N], sh.odd[N], k + kTile, blo, bup);
      wait_lds_barrier();
    }
  }

  // e4m3: the two steps of the tile at k, in buffer B; `s` holds the scores of
  // the first.  K of the next tile is needed in the second step and V in the
  // next tile's first; each is on its way for two steps.  The loads (to
  // registers) do not depend on whether a tile follows, the last one is loaded
  // again: else the compiler would count only the loads that leave on every
  // path, and wait for younger ones too.
  template <int B>
  __device__ __forceinline__ void two_steps(Stage& g, const Stream& st, f32x16& s, int k, int k1, int lo, int up, int blo,
                                            int bup, float c, const int* ko, const int* vo, Lds& sh) {
    const bool more = k + kTile < k1;
    const int mid = k + kStepKeys;
    constexpr int kHalf = kStepKeys * D * 2;   // bytes of a step's keys
    float t;
    g.load_v(st);
    if (__builtin_expect(k < up, 1)) {
      step(s, t, sh.k[B] + kHalf, sh.v[B], c, ko, vo);
      unfinite(st, k, k + kTile, up, blo, sh.odd[B]);
      if (__builtin_expect(mid < up, 1)) prepare(s, t, mid, lo, c);
    }
    if (__builtin_expect(more, 1)) {
      g.store_k(sh.k[B ^ 1]);
      wait_lds_barrier();
    }
    g.load_k(st, k + 2 * kTile, k1);
    if (__builtin_expect(mid < up, 1)) {
      step(s, t, sh.k[B ^ 1], sh.v[B] + kHalf, c, ko, vo);   // (the scores of a tile that is not there are not used)
      unfinite(st, mid, k + kTile, up, blo, sh.odd[B]);
      if (__builtin_expect(more && k + kTile < up, 1)) prepare(s, t, k + kTile, lo, c);
    }
    if (__builtin_expect(more, 1)) {
      g.store_v(sh.v[B ^ 1]);
      mend_v(sh.v[B ^ 1], sh.odd[B ^ 1], k + kTile, blo, bup);
      wait_lds_barrier();
    }
  }

  // The largest of 16 scores of the lane's row.
  static __device__ __forceinline__ float largest(const f32x16& s) {
    float t = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) t = fmaxf(t, s[i]);
    return t;
  }

  // Scores of the 32 keys at k, the largest of them in t: masks, and the
  // running maximum.
  __device__ __forceinline__ void prepare(f32x16& s, float t, int k, int lo, float c) {
    if (__builtin_expect(k + kStepKeys > lo, 0)) {
      const int g = (threadIdx.x & 63) >> 5;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = k + 8 * (i >> 2) + 4 * g + (i & 3) < hi ? s[i] : -__builtin_inff();
      t = largest(s);
    }
    float top = t * c;
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(top > m + kSlack) != 0, 0)) {
      top = fmaxf(top, __shfl_xor(top, 32));
      const float mn = fmaxf(m, top);
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
      const Factor k(f);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = k.of(o[d][i]);
    }
  }

  // 8 keys of element 32 d + l%32 (16-key group a of the half at v)
  static __device__ __forceinline__ uint4 values(const uint8_t* v, int off, int a) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_t;
    union {
      s16x4 h[2];
      uint4 u;
    } r;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      r.h[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(v + off + (16 * a + 8 * e) * (D * 2)));
    return r.u;
  }

  // The weights of scores s and their values (32 keys at v); s becomes the
  // scores of the 32 keys at kn, t their largest.
  __device__ __forceinline__ void step(f32x16& s, float& t, const uint8_t* kn, const uint8_t* v, float c, const int* ko,
                                       const int* vo) {
    const bf16x2 ones = __builtin_bit_cast(bf16x2, 0x3F803F80u);
    f32x16 sn;
#pragma unroll
    for (int i = 0; i < 16; ++i) sn[i] = 0.f;
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      sn = mfma32(*reinterpret_cast<const uint4*>(kn + ko[i]), q[i], sn);
#pragma unroll
      for (int j = 8 / KS * i; j < 8 / KS * (i + 1); ++j) {
        p[j] = pack2(__builtin_amdgcn_exp2f(s[2 * j] * c - m), __builtin_amdgcn_exp2f(s[2 * j + 1] * c - m));
        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, p[j]), ones, l, false);
      }
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const uint4 pa = uint4{p[4 * a], p[4 * a + 1], p[4 * a + 2], p[4 * a + 3]};
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = mfma32(values(v, vo[d], a), pa, o[d]);
    }
    t = largest(sn);
    s = sn;
  }

  // See unfinite_pair: keys [k, k + 32) of the tile that ends at `end`.
  __device__ __forceinline__ void unfinite(const Stream& st, int k, int end, int up, int blo, const uint32_t* odd) {
    if (__builtin_expect(end <= blo, 1)) return;
    if (__builtin_expect(!(odd[0] | odd[1] | odd[2] | odd[3]), 1)) return;
    const int g = (thread_anew() & 63) >> 5;
#pragma unroll 1
    for (int key = k; key < min(k + kStepKeys, up); ++key) {
      const uint8_t* row = value_row(st, key) + (F8 ? 1 : 2) * 4 * g;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const f32x2 v = unfinite_pair<F8>(row, 32 * d + 8 * (i >> 2) + (i & 3), key < hi);
          o[d][i] += v[0];
          o[d][i + 1] += v[1];
        }
    }
  }
};
