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
//       bf16 (e4m3 codes are converted on the way in, once a block), in
//       16-byte pieces whose number is XOR-ed with the row's: 8 neighbouring
//       lanes reach 8 different bank groups, in the reads and in the writes.
// V is transposed on the way in: a thread loads 8 keys x D/32 elements and
// writes D/32 pieces.  The next tile's loads are in flight while a tile is
// multiplied; one barrier a tile.
// Per tile a wave has 32 products of 32 cycles for 64 KB of LDS reads (with
// two blocks a CU the reads and the products take about the same time) and 32
// exponentials a lane.
#pragma once

__device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

constexpr int kTile = 64;        // keys of a tile
constexpr int kTileRows = 32;    // rows of a wave
constexpr int kBlockRows = kWaves * kTileRows;

template <int D>
struct TilesLds {
  uint8_t k[2][kTile * D * 2];
  uint8_t v[2][D * kTile * 2];
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
  __device__ __forceinline__ void walk(const Stream& st, int k0, int k1, int lo, int up, int blo, int bup, float c,
                                       bool live, TilesLds<D>& sh) {
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5, i32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    k1 = min(k1, bup);
    if (k0 >= k1) return;
    constexpr int KB = F8 ? 1 : 2;
    constexpr int KL = 16 * D * KB / 1024;      // 16-byte pieces of a wave's 16 keys, a lane
    constexpr int KP = D * KB / 16;             // pieces of a key
    constexpr int DW = D / 32;                  // elements of a lane's piece of a value
    constexpr int VW = DW * KB / 4;             // its words (0: half a word)
    Words<4> kr[KL];
    Words<VW> vr[8];
    const int koff = (lane / KP) * st.slot_stride + (lane % KP) * 16;
    const int voff = 4 * g * st.slot_stride + i32 * (DW * KB);
    Pages pages;
    pages.fill(st, k0 >> st.shift);
    // wave w carries keys 16w .. 16w+15 of a tile (one page)
    auto load = [&](int k) __attribute__((always_inline)) {
      const int64_t off = pages.offset(st, min(k + 16 * wave, (k1 - 1) & ~15));
      const uint8_t *kp = st.k + off, *vp = st.v + off;
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        kr[i] = load_words<4>(kp + (int64_t)(64 / KP * i) * st.slot_stride + koff);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        vr[e] = load_words<VW>(vp + (int64_t)((e & 3) + 8 * (e >> 2)) * st.slot_stride + voff);
    };
    auto store = [&](int b, int k) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int p = lane + 64 * i, key = 16 * wave + p / KP, cc = p % KP;
        uint8_t* row = sh.k[b] + key * (D * 2);
        if constexpr (F8) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<uint4*>(row + (((2 * cc + u) ^ (key & 7)) * 16)) =
                uint4{cvt2(kr[i].w[2 * u], false), cvt2(kr[i].w[2 * u], true), cvt2(kr[i].w[2 * u + 1], false),
                      cvt2(kr[i].w[2 * u + 1], true)};
        } else {
          *reinterpret_cast<uint4*>(row + ((cc ^ (key & 7)) * 16)) = uint4{kr[i].w[0], kr[i].w[1], kr[i].w[2], kr[i].w[3]};
        }
      }
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
            const uint32_t v = dead ? 0u : vr[e].w[w], odd = not_finite<F8>(v);
            vr[e].w[w] = only_finite<F8>(v, odd);
            any |= odd;
          }
        const bool found = __builtin_amdgcn_ballot_w64(any != 0) != 0;
        if (lane == 0) sh.odd[b][wave] = found;
      }
      uint32_t x[8][DW / 2];
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int w = 0; w < DW / 2; ++w) x[e][w] = F8 ? cvt2(vr[e].w[0], w & 1) : vr[e].w[w];
#pragma unroll
      for (int j = 0; j < DW; ++j) {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
        const int d = DW * i32 + j, kg = 2 * wave + g;
        const int f = (d & 7) ^ ((d >> 3) & 3);
        *reinterpret_cast<uint4*>(sh.v[b] + d * (kTile * 2) + ((kg ^ f) * 16)) =
            uint4{__builtin_amdgcn_perm(x[1][j >> 1], x[0][j >> 1], sel), __builtin_amdgcn_perm(x[3][j >> 1], x[2][j >> 1], sel),
                  __builtin_amdgcn_perm(x[5][j >> 1], x[4][j >> 1], sel), __builtin_amdgcn_perm(x[7][j >> 1], x[6][j >> 1], sel)};
      }
    };
    load(k0);
    store(0, k0);
    __syncthreads();
    int b = 0;
    for (int k = k0; k < k1; k += kTile) {
      const bool more = k + kTile < k1;
      if (more) load(k + kTile);
      if (live && k < up) {
        multiply(k, lo, c, sh, b, i32, g);
        // a tile without masks in this wave may have had some in the block
        if (k + kTile > blo && (sh.odd[b][0] | sh.odd[b][1] | sh.odd[b][2] | sh.odd[b][3])) {
#pragma unroll 1
          for (int key = k; key < min(k + kTile, up); ++key) {
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
      }
      if (more) store(b ^ 1, k + kTile);
      __syncthreads();
      b ^= 1;
    }
  }

  __device__ __forceinline__ void multiply(int k, int lo, float c, const TilesLds<D>& sh, int b, int i32, int g) {
    f32x16 s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[t][i] = 0.f;
      const uint8_t* row = sh.k[b] + (32 * t + i32) * (D * 2);
#pragma unroll
      for (int i = 0; i < KS; ++i)
        s[t] = mfma32(*reinterpret_cast<const uint4*>(row + (((2 * i + g) ^ (i32 & 7)) * 16)), q[i], s[t]);
    }
    const bool masked = k + kTile > lo;
    if (masked) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[t][i] = k + 32 * t + 8 * (i >> 2) + 4 * g + (i & 3) < hi ? s[t][i] : -__builtin_inff();
    }
    float top = s[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
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
    uint32_t p[2][8];
    const bf16x2 ones = __builtin_bit_cast(bf16x2, 0x3F803F80u);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[t][i] = pack2(__builtin_amdgcn_exp2f(s[t][2 * i] * c - m), __builtin_amdgcn_exp2f(s[t][2 * i + 1] * c - m));
        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, p[t][i]), ones, l, false);
      }
    const int f = (i32 & 7) ^ ((i32 >> 3) & 3);
    const uint8_t* vt = sh.v[b] + i32 * (kTile * 2);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const uint32_t* pp = &p[a >> 1][4 * (a & 1)];
      const uint4 pa = uint4{pp[0], pp[1], pp[2], pp[3]};
#pragma unroll
      for (int d = 0; d < DT; ++d)
        o[d] = mfma32(*reinterpret_cast<const uint4*>(vt + d * (32 * kTile * 2) + (((2 * a + g) ^ f) * 16)), pa, o[d]);
    }
  }
};
