// The 4-bit quantization of one group of values, shared by the weight and the
// cache quantizers.  Files that include it are compiled with -ffp-contract=off:
// every fp32 operation below is one correctly rounded IEEE operation.
#pragma once
#include "wq_device.h"

namespace wq {

// Eight values from index idx on as fp32 (DT: 0 fp32, 1 bf16, 2 fp16; exact).
template <int DT>
__device__ __forceinline__ void load8(const void* W, int64_t idx, float* out) {
  if constexpr (DT == 0) {  // fp32
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(W) + idx);
    float4 a = p[0], b = p[1];
    out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
    out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
  } else {
    uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + idx);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == 1) {  // bf16: exact widening
        out[2 * i] = __builtin_bit_cast(float, w[i] << 16);
        out[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
      } else {  // fp16: exact widening
        out[2 * i] = f16_bits_to_f32((uint16_t)(w[i] & 0xffffu));
        out[2 * i + 1] = f16_bits_to_f32((uint16_t)(w[i] >> 16));
      }
    }
  }
}

// Scale (fp16 bits), its fp32 value, an approximate reciprocal of it and the
// zero-point of a group whose min and max are lo and hi.
struct GroupParams {
  uint16_t s_bits;
  float s;
  float r;  // v_rcp_f32(s): only steers the rounding shortcut below
  float z;
};

__device__ __forceinline__ GroupParams group_params(float lo, float hi) {
  lo = fminf(lo, 0.0f);  // range widened to contain 0: z is then a code
  hi = fmaxf(hi, 0.0f);
  float range = hi - lo;
  float s32 = range / 15.0f;
  GroupParams p;
  p.s_bits = f32_to_f16_bits(s32);
  p.s = f16_bits_to_f32(p.s_bits);
  p.r = __builtin_amdgcn_rcpf(p.s);
  if (p.s == 0.0f) {  // degenerate group: s = 0, z = 0, codes 0
    p.s_bits = 0;
    p.z = 0.0f;
    return p;
  }
  float z = rintf(-lo / p.s);
  p.z = fminf(fmaxf(z, 0.0f), 15.0f);
  return p;
}

// rne(fl32(fl32(w / s) + z)) -- the encoding's two correctly rounded fp32
// operations and the rounding to an integer -- without the division wherever
// it cannot matter.  t = fma(w, r, z) with r = v_rcp_f32(s) (1 ulp) lies within
// |w/s| * 2^-22 + ulp(t) of the real w/s + z, and the exact steps lie within
// 2^-24 * (|w/s| + |t|) of it; with |w/s| <= 2^(B-1) + 1 for B-bit codes both
// are below 2^(B-1) * 2^-21.  So when t is farther than `margin` (2^-14 for
// 4-bit codes, 2^-10 for 8-bit: room for an rcp error of 16 ulp) from every
// half-integer, t, the real value and the exact result all round to the same
// integer; otherwise the exact steps run.
__device__ __forceinline__ float round_quotient(float w, const GroupParams& p, float z, float margin) {
  const float t = fmaf(w, p.r, z);
  const float f = t - floorf(t);  // exact for |t| < 2^23
  if (fabsf(f - 0.5f) > margin) return rintf(t);
  const float u = w / p.s;  // correctly rounded
  return rintf(u + z);
}

__device__ __forceinline__ uint32_t encode(float w, const GroupParams& p) {
  if (p.s == 0.0f) return 0u;
  float r = round_quotient(w, p, p.z, 0x1p-14f);
  r = fminf(fmaxf(r, 0.0f), 15.0f);
  return (uint32_t)r;
}

// Nibble position of column e (0..7) inside a packed word.
__device__ __forceinline__ int nibble_pos(int e) { return 4 * (e & 1) + (e >> 1); }

}  // namespace wq
