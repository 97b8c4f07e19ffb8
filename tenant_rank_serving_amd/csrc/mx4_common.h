// Device helpers of the MXFP4 kernels.  Included inside namespace dc, anonymous
// namespace, of the .hip files that use them, behind bf16x8 and f32x4.
#pragma once

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// The scale byte as the fp32 number whose exponent field it is: the conversions
// read that field (0: 2^-127), and 255 has to be NaN, not infinity.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : byte << 23);
}

// Scales of 253 and 254: the block's numbers may pass bf16's largest (they reach
// 6 2^127).  In the products of all blocks such a block, or one of NaN, counts as
// 2^-127 times its codes, 2^-253 of it, and is added behind them.  (As a branch among
// the products: 32000 x 4096 with 64 tokens 23.9 us, without any of it
// 21.4, so 21.7.)
__device__ __forceinline__ bool is_large(uint32_t byte) { return byte >= 253; }
__device__ __forceinline__ float scale_unless_large(uint32_t byte, uint64_t* any) {
  *any |= __builtin_amdgcn_ballot_w64(is_large(byte));
  return __uint_as_float(is_large(byte) ? 0u : byte << 23);
}

// 8 codes as bf16.
__device__ __forceinline__ bf16x8 codes8(uint32_t w, float s) {
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  return __builtin_bit_cast(bf16x8, r);
}

// Adds the products of the large blocks (above) of row tiles r0 .. and tokens t0 ..,
// columns 128 c for c = c0, c0 + step, ..: at a quarter, four times.  A matrix that
// holds any is read once more; the packer makes none (its scales end with 252).
template <int RT, int TT>
__device__ __forceinline__ void add_large(const Mx4Args& g, f32x4 (&acc)[RT][TT], int r0, int t0, int c0, int step) {
  const int lane = threadIdx.x & 63, gc = g.in / 128, hc = (gc + 3) / 4, rts = g.out / 16;
  const uint8_t* scales = g.w + (size_t)rts * gc * 1024;
#pragma clang loop unroll(disable)
  for (int c = c0; c < gc; c += step)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const size_t T = min(r0 + r, rts - 1);
      const uint32_t byte = *reinterpret_cast<const uint32_t*>(scales + (T * hc + (c >> 2)) * 256 + lane * 4) >> (8 * (c & 3)) & 255u;
      const bool large = is_large(byte);
      if (!__builtin_amdgcn_ballot_w64(large)) continue;
      const uint4 w = *reinterpret_cast<const uint4*>(g.w + (T * gc + c) * 1024 + lane * 16);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      const float f = scale_of(byte == 255 ? byte : large ? byte - 2 : 0);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint16_t* x = g.x + (size_t)min(t0 + 16 * t + (lane & 15), g.T - 1) * g.in + 128 * c + 32 * (lane >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 v = codes8(large ? u[j] : 0, f), xv = *reinterpret_cast<const bf16x8*>(x + 8 * j);
#pragma unroll
          for (int n = 0; n < 4; ++n) acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, xv, acc[r][t], 0, 0, 0);
        }
      }
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  bf16x2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

// 16 (4) bytes a lane from base + voff to lds + 16 (4) lane.
__device__ __forceinline__ void to_lds16(const uint8_t* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void to_lds4(const uint8_t* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}

// At most N of the wave's loads still on their way; its LDS reads are done, and
// so are every other wave's.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
