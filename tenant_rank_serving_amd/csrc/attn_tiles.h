// The walk for more than 16 query rows: a block takes 128 rows, wave w rows
// 32w .. 32w+31, and its keys come through LDS in tiles of 64 that all waves
// share.  Included inside namespace dc, anonymous namespace, of k_attn.hip,
// behind attn_common.h.
//
// Products transposed as for few rows, S^T = K Q^T and O^T = V^T P^T, here
// 32x32x16: a wave reads a tile's keys and values once for 32 rows.
//   S^T result: lane l holds row l%32 and keys 8(i/4) + 4(l/32) + i%4, i < 16.
//   P^T operand B: row l%32, 8 keys of half l/32: results 8a .. 8a+7 as they
//       are, so product a of a 32-key half takes keys 16a + 4(l/32) + {0..3}
//       and those + 8.
//   LDS holds K as [64 keys][D] and V^T as [D][64 keys in that order], both
//       bf16 (e4m3 codes are converted on the way in, once a block), in lines
//       of 256 bytes, the width of the banks; the 16 pieces of a line are
//       permuted by an XOR such that 16 neighbouring lanes reach 16 different
//       ones, in the reads and in the writes (key_at, value_at).
// V is transposed on the way in: a thread loads 8 keys x D/32 elements and
// writes D/32 pieces.
#pragma once

__device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

constexpr int kTile = 64;        // keys of a tile
constexpr int kTileRows = 32;    // rows of a wave
constexpr int kBlockRows = kWaves * kTileRows;

// A line holds one key of D = 128, or keys i and i + 16 of a half of D = 64.
template <int D> __device__ __forceinline__ int key_at(int key, int c) {
  if constexpr (D == 128) return key * 256 + ((c ^ (key & 15)) * 16);
  const int line = key & 15, f = ((line & 1) << 3) | (line >> 1);
  return (key >> 5) * 4096 + line * 256 + (((((key >> 4) & 1) * 8 + c) ^ f) * 16);
}
// Element d's values, 8 keys (piece kg): regions of 32 elements, a line holds
// elements i and i + 16 of it; the regions are 64 bytes apart in the banks.
constexpr int kRegion = 4096 + 64;
template <int D> __device__ __forceinline__ int value_at(int d, int kg) {
  const int line = d & 15, f = D == 128 ? (line >> 2) | ((line & 3) << 2) : ((line & 1) << 3) | (line >> 1);
  return (d >> 5) * kRegion + line * 256 + (((((d >> 4) & 1) * 8 + kg) ^ f) * 16);
}

template <int D>
struct TilesLds {
  alignas(256) uint8_t k[2][kTile * D * 2];
  alignas(256) uint8_t v[2][D / 32 * kRegion];
  uint32_t odd[2][kWaves];       // of a tile with masks: some of the values that a wave carried are not finite
};

template <int D, bool F8>
struct Tiles {
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
    const int lane = threadIdx.x & 63;
    const int row = min(row0 + (lane & 31), it.rows - 1);   // past the last row: the last one again
    const int tok = row / a.gq, hh = row - tok * a.gq;
    const uint16_t* p = a.q + (int64_t)(it.t0 + tok) * a.qs + (int64_t)(h * a.gq + hh) * D + 8 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      q[i] = *reinterpret_cast<const uint4*>(p + 16 * i);
      if constexpr (F8) q[i].x ^= flip, q[i].y ^= flip, q[i].z ^= flip, q[i].w ^= flip;
    }
  }

  // Keys [k0, k1) of the stream (k0 a multiple of 64) for the block; a wave
  // without rows (live = false) only carries tiles.  The wave's rows all see
  // the keys below lo and none see those from up on; blo, bup: the block's.
  //
  // Half tiles of 32 keys: step h multiplies the keys of half h + 1, takes the
  // exponentials of half h and multiplies its values, in one stretch of code
  // without branches, so that the matrix core and the vector unit work at the
  // same time within a wave.  What a maximum moves is decided between steps.
  // K of the next tile is stored to LDS in a tile's first step and needed in
  // its second, V is stored in the second and needed in the next tile's first:
  // with two buffers, one barrier a step.
  __device__ __forceinline__ void walk(const Stream& st, int k0, int k1, int lo, int up, int blo, int bup, float c,
                                       bool live, TilesLds<D>& sh) {
    k1 = min(k1, bup);
    if (k0 >= k1) return;
    Stage g(st);
    const int lane = threadIdx.x & 63, half = lane >> 5, i32 = lane & 31;
    int ko[KS], vo[4];
#pragma unroll
    for (int i = 0; i < KS; ++i) ko[i] = key_at<D>(i32, 2 * i + half);
#pragma unroll
    for (int a = 0; a < 4; ++a) vo[a] = value_at<D>(i32, 2 * a + half);
    if (!live) up = k0;   // no key is of interest
    g.load_k(st, k0, k1);
    g.load_v(st);
    g.store_k(sh.k[0]);
    g.store_v(sh.v[0], sh.odd[0], k0, blo, bup);
    if (k0 + kTile < k1) g.load_k(st, k0 + kTile, k1);
    __syncthreads();
    f32x16 s;
    if (k0 < up) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) s = mfma32(*reinterpret_cast<const uint4*>(sh.k[0] + ko[i]), q[i], s);
      prepare(s, k0, lo, c);
    }
    for (int k = k0; k < k1; k += 2 * kTile) {
      tile<0>(g, st, s, k, k1, lo, up, blo, bup, c, ko, vo, sh);
      if (k + kTile < k1) tile<1>(g, st, s, k + kTile, k1, lo, up, blo, bup, c, ko, vo, sh);
    }
    __syncthreads();   // the buffers are free
  }

 private:
  static constexpr int KB = F8 ? 1 : 2;              // bytes of an element of the cache
  static constexpr int KL = 16 * D * KB / 1024;      // 16-byte pieces of a wave's 16 keys, a lane
  static constexpr int KP = D * KB / 16;             // pieces of a key
  static constexpr int DW = D / 32;                  // elements of a lane's piece of a value
  static constexpr int VW = DW * KB / 4;             // its words (0: half a word)

  // A wave's part of a tile on its way from the cache to LDS: wave w carries
  // keys 16w .. 16w+15 (one page).
  struct Stage {
    Words<4> kr[KL];
    Words<VW> vr[8];
    Pages pages;
    const uint8_t* vp;
    int koff, voff, wave;
    __device__ __forceinline__ Stage(const Stream& st) {
      const int lane = threadIdx.x & 63;
      wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      koff = (lane / KP) * st.slot_stride + (lane % KP) * 16;
      voff = 4 * (lane >> 5) * st.slot_stride + (lane & 31) * (DW * KB);
      pages.base = -64;
    }
    // the keys of the tile at k, and where its values are
    __device__ __forceinline__ void load_k(const Stream& st, int k, int k1) {
      const int64_t off = pages.offset(st, min(k + 16 * wave, (k1 - 1) & ~15));
      vp = st.v + off;
#pragma unroll
      for (int i = 0; i < KL; ++i) kr[i] = load_words<4>(st.k + off + (int64_t)(64 / KP * i) * st.slot_stride + koff);
    }
    // the values of the tile whose keys were loaded last
    __device__ __forceinline__ void load_v(const Stream& st) {
#pragma unroll
      for (int e = 0; e < 8; ++e) vr[e] = load_words<VW>(vp + (int64_t)((e & 3) + 8 * (e >> 2)) * st.slot_stride + voff);
    }
    __device__ __forceinline__ void store_k(uint8_t* lds) {
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int key = 16 * wave + lane / KP + 64 / KP * i, cc = lane % KP;
        if constexpr (F8) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<uint4*>(lds + key_at<D>(key, 2 * cc + u)) =
                uint4{cvt2(kr[i].w[2 * u], false), cvt2(kr[i].w[2 * u], true), cvt2(kr[i].w[2 * u + 1], false),
                      cvt2(kr[i].w[2 * u + 1], true)};
        } else {
          *reinterpret_cast<uint4*>(lds + key_at<D>(key, cc)) = uint4{kr[i].w[0], kr[i].w[1], kr[i].w[2], kr[i].w[3]};
        }
      }
    }
    // transposed; k: the tile's first key
    __device__ __forceinline__ void store_v(uint8_t* lds, uint32_t* odd, int k, int blo, int bup) {
      const int lane = threadIdx.x & 63, g = lane >> 5;
      constexpr int NW = VW ? VW : 1;
      if (k + kTile > blo) {
        // values that no row of the block sees count as zero, and so do, for
        // now, those that are not finite
        uint32_t any = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const bool dead = k + 16 * wave + 4 * g + (e & 3) + 8 * (e >> 2) >= bup;
            const uint32_t v = dead ? 0u : vr[e].w[w], bad = not_finite<F8>(v);
            vr[e].w[w] = only_finite<F8>(v, bad);
            any |= bad;
          }
        const bool found = __builtin_amdgcn_ballot_w64(any != 0) != 0;
        if (lane == 0) odd[wave] = found;
      }
      uint32_t x[8][DW / 2];
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int w = 0; w < DW / 2; ++w) x[e][w] = F8 ? cvt2(vr[e].w[0], w & 1) : vr[e].w[w];
#pragma unroll
      for (int j = 0; j < DW; ++j) {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
        *reinterpret_cast<uint4*>(lds + value_at<D>(DW * (lane & 31) + j, 2 * wave + g)) =
            uint4{__builtin_amdgcn_perm(x[1][j >> 1], x[0][j >> 1], sel), __builtin_amdgcn_perm(x[3][j >> 1], x[2][j >> 1], sel),
                  __builtin_amdgcn_perm(x[5][j >> 1], x[4][j >> 1], sel), __builtin_amdgcn_perm(x[7][j >> 1], x[6][j >> 1], sel)};
      }
    }
  };

  // The tile at k, in buffer B; `s` holds the scores of its first half.
  template <int B>
  __device__ __forceinline__ void tile(Stage& g, const Stream& st, f32x16& s, int k, int k1, int lo, int up, int blo,
                                       int bup, float c, const int* ko, const int* vo, TilesLds<D>& sh) {
    const bool more = k + kTile < k1;
    const int mid = k + kTile / 2;
    if (more) g.load_v(st);
    if (k < up) {
      step(s, sh.k[B] + kTile / 2 * D * 2, sh.v[B], c, ko, vo);
      unfinite(st, k, k, up, blo, sh.odd[B]);
      if (mid < up) prepare(s, mid, lo, c);
    }
    if (more) {
      g.store_k(sh.k[B ^ 1]);
      __syncthreads();
      if (k + 2 * kTile < k1) g.load_k(st, k + 2 * kTile, k1);
    }
    if (mid < up) {
      step(s, sh.k[B ^ 1], sh.v[B], c, ko, vo + 2);   // (the scores of a tile that is not there are not used)
      unfinite(st, mid, k, up, blo, sh.odd[B]);
      if (more && k + kTile < up) prepare(s, k + kTile, lo, c);
    }
    if (more) {
      g.store_v(sh.v[B ^ 1], sh.odd[B ^ 1], k + kTile, blo, bup);
      __syncthreads();
    }
  }

  // Scores of the 32 keys at k: masks, and the running maximum.
  __device__ __forceinline__ void prepare(f32x16& s, int k, int lo, float c) {
    if (k + kTile / 2 > lo) {
      const int g = (threadIdx.x & 63) >> 5;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = k + 8 * (i >> 2) + 4 * g + (i & 3) < hi ? s[i] : -__builtin_inff();
    }
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    top *= c;
    if (__builtin_amdgcn_ballot_w64(top > m + kSlack)) {
      top = fmaxf(top, __shfl_xor(top, 32));
      const float mn = fmaxf(m, top);
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
  }

  // The weights of scores s and their values (pieces vo[0], vo[1] of v); s
  // becomes the scores of the 32 keys at kn.
  __device__ __forceinline__ void step(f32x16& s, const uint8_t* kn, const uint8_t* v, float c, const int* ko,
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
      for (int d = 0; d < DT; ++d) o[d] = mfma32(*reinterpret_cast<const uint4*>(v + vo[a] + d * kRegion), pa, o[d]);
    }
    s = sn;
  }

  // See unfinite_pair: keys [k, k + 32) of the tile at k0.
  __device__ __forceinline__ void unfinite(const Stream& st, int k, int k0, int up, int blo, const uint32_t* odd) {
    if (k0 + kTile <= blo || !(odd[0] | odd[1] | odd[2] | odd[3])) return;
    const int g = (threadIdx.x & 63) >> 5;
#pragma unroll 1
    for (int key = k; key < min(k + kTile / 2, up); ++key) {
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
