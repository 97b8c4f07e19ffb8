// Appending to the paged cache with the position rotation on the way.
//
// For token t, pair i of a head's first `rot` elements and the angle
// a = pos_t f_i:  (x_i, x_j) -> (x_i cos a - x_j sin a, x_j cos a + x_i sin a).
// q goes to q_out, k to the token's cache slot, v to its slot as it is.
//
// The angle is formed and reduced in fp64 (a position of 10^5 radians has
// only 2^-7 left of fp32); its fraction of a turn is then an fp32 whose sine
// and cosine are taken once per (token, pair) and shared by all heads of the
// block through LDS.  Bound by memory: each element is read and written once.
// 16384 tokens of 40 + 80 heads of 128: 190 us, 5.3 TB/s (a large copy reaches
// 5.2); 64 tokens of 32 + 16 heads into an e4m3 cache 3.5 us, one token 2.2 us
// (an empty kernel in a graph: 1.6).
#include <hip/hip_runtime.h>

#include "layer.h"

namespace dc {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // round to nearest even
  bf16x2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}
// e4m3 holds up to 448 and no infinity: saturate, keep NaN.
__device__ __forceinline__ float sat(float x) { return x != x ? x : fminf(fmaxf(x, -448.f), 448.f); }
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), w, true);
}

__device__ __forceinline__ void unpack8(uint4 w, float* f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = lo_f(u[i]), f[2 * i + 1] = hi_f(u[i]);
}

// A unit is 16 elements of one head of one token as two 8-element pieces: in
// the half-split pairing pieces rot/2 apart (every pair inside the unit),
// else, and past rot, neighbouring ones.  A thread holds kUnits units at a
// time.  Block: one token, a slice of its units (blockIdx.y).
template <int D, bool F8, int kUnits>
__global__ void __launch_bounds__(kThreads) k_append(AppendArgs a, int per) {
  constexpr int U = D / 16;
  __shared__ float cs[D / 2], sn[D / 2];
  const int t = blockIdx.x, tid = threadIdx.x;
  const int hkv = a.kv.heads;
  const int units = (a.hq + 2 * hkv) * U;
  const int u0 = blockIdx.y * per, u1 = min(units, u0 + per);
  const int rh = a.rot >> 1;
  const int64_t slot = a.slots[t];
  const int64_t nslots = (int64_t)a.kv.num_pages << a.kv.shift;
  const bool stored = slot >= 0 && slot < nslots;
  if (tid < rh) {
    // turns = pos f / 2 pi; its distance to the nearest whole one is exact in
    // fp64 to pos f 2^-53, and sincospi takes twice that
    const double turn = (double)a.pos[t] * a.freq[tid] * 0.15915494309189533577;
    const float fr = (float)(2.0 * (turn - rint(turn)));
    float s, c;
    sincospif(fr, &s, &c);
    cs[tid] = c;
    sn[tid] = s;
  }
  for (int ub = u0; ub < u1; ub += kThreads * kUnits) {
    uint4 x0[kUnits], x1[kUnits];
    int head[kUnits], e0[kUnits], e1[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = min(ub + i * kThreads + tid, u1 - 1);
      const int h = u / U, c = u % U;
      head[i] = h;
      const bool half = !a.interleaved && h < a.hq + hkv && 16 * c < a.rot;
      e0[i] = half ? 8 * c : 16 * c;
      e1[i] = half ? 8 * c + rh : 16 * c + 8;
      const uint16_t* src = h < a.hq ? a.q + t * a.qs + h * D
                            : h < a.hq + hkv ? a.k + t * a.ks + (h - a.hq) * D
                                             : a.v + t * a.vs + (h - a.hq - hkv) * D;
      x0[i] = *reinterpret_cast<const uint4*>(src + e0[i]);
      x1[i] = *reinterpret_cast<const uint4*>(src + e1[i]);
    }
    if (ub == u0) __syncthreads();   // the angles
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (ub + i * kThreads + tid >= u1) continue;
      const int h = head[i];
      float f0[8], f1[8];
      unpack8(x0[i], f0);
      unpack8(x1[i], f1);
      if (h < a.hq + hkv && e0[i] < a.rot) {
        if (a.interleaved) {   // pairs inside a piece
          const int p = e0[i] >> 1;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float c0 = cs[p + j], s0 = sn[p + j], c1 = cs[p + 4 + j], s1 = sn[p + 4 + j];
            const float a0 = f0[2 * j], b0 = f0[2 * j + 1], a1 = f1[2 * j], b1 = f1[2 * j + 1];
            f0[2 * j] = a0 * c0 - b0 * s0;
            f0[2 * j + 1] = b0 * c0 + a0 * s0;
            f1[2 * j] = a1 * c1 - b1 * s1;
            f1[2 * j + 1] = b1 * c1 + a1 * s1;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float c0 = cs[e0[i] + j], s0 = sn[e0[i] + j], p = f0[j], r = f1[j];
            f0[j] = p * c0 - r * s0;
            f1[j] = r * c0 + p * s0;
          }
        }
      }
      if (h < a.hq) {
        uint16_t* d = a.qo + t * a.qos + h * D;
        *reinterpret_cast<uint4*>(d + e0[i]) =
            uint4{pack2(f0[0], f0[1]), pack2(f0[2], f0[3]), pack2(f0[4], f0[5]), pack2(f0[6], f0[7])};
        *reinterpret_cast<uint4*>(d + e1[i]) =
            uint4{pack2(f1[0], f1[1]), pack2(f1[2], f1[3]), pack2(f1[4], f1[5]), pack2(f1[6], f1[7])};
        continue;
      }
      if (!stored) continue;
      const bool isv = h >= a.hq + hkv;
      const int kh = h - a.hq - (isv ? hkv : 0);
      uint8_t* d = (isv ? a.kv.v : a.kv.k) + (slot >> a.kv.shift) * a.kv.page_stride + kh * a.kv.head_stride +
                   (slot & ((1 << a.kv.shift) - 1)) * a.kv.slot_stride;
      if constexpr (F8) {
        const float* sp = isv ? a.kv.vs : a.kv.ks;
        const float s = sp ? sp[kh] : 1.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f0[j] = f0[j] / s, f1[j] = f1[j] / s;
        *reinterpret_cast<uint2*>(d + e0[i]) =
            uint2{pack4(f0[0], f0[1], f0[2], f0[3]), pack4(f0[4], f0[5], f0[6], f0[7])};
        *reinterpret_cast<uint2*>(d + e1[i]) =
            uint2{pack4(f1[0], f1[1], f1[2], f1[3]), pack4(f1[4], f1[5], f1[6], f1[7])};
      } else {
        *reinterpret_cast<uint4*>(d + 2 * e0[i]) =
            uint4{pack2(f0[0], f0[1]), pack2(f0[2], f0[3]), pack2(f0[4], f0[5]), pack2(f0[6], f0[7])};
        *reinterpret_cast<uint4*>(d + 2 * e1[i]) =
            uint4{pack2(f1[0], f1[1]), pack2(f1[2], f1[3]), pack2(f1[4], f1[5]), pack2(f1[6], f1[7])};
      }
    }
  }
}

}  // namespace

int launch_append(const AppendArgs& a) {
  const int units = (a.hq + 2 * a.kv.heads) * (a.dim / 16);
  // few tokens: one unit a thread, so that the whole call is in flight at
  // once; many: four, so that a block shares its token's angles (us, one / four:
  // 64 tokens of 48 heads 3.5 / 4.0, 1024 7.0 / 7.4, 4096 19.8 / 19.3; 512 of 120
  // heads 7.6 / 8.7, 2048 29.6 / 28.7)
  const bool few = a.n <= 1024;
  const int per = few ? kThreads : kThreads * 4;
  const dim3 g((unsigned)a.n, (unsigned)((units + per - 1) / per));
  hipStream_t st = reinterpret_cast<hipStream_t>(a.stream);
#define DC_APPEND(D_, F8_)                                                                       \
  if (few) hipLaunchKernelGGL((k_append<D_, F8_, 1>), g, dim3(kThreads), 0, st, a, per);         \
  else hipLaunchKernelGGL((k_append<D_, F8_, 4>), g, dim3(kThreads), 0, st, a, per);
  if (a.dim == 64) {
    if (a.e4m3) { DC_APPEND(64, true) } else { DC_APPEND(64, false) }
  } else {
    if (a.e4m3) { DC_APPEND(128, true) } else { DC_APPEND(128, false) }
  }
#undef DC_APPEND
  return (int)hipGetLastError();
}

}  // namespace dc
