// Pieces that the attention kernels share.
#pragma once
#include "wq_device.h"
#include "wq_kernels.h"

namespace wq {

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

constexpr float kNegInf = -__builtin_inff();
// A row's reference point may lag its largest weight by this many powers of two,
// so that it rarely moves.
constexpr float kLag = 8.0f;
// The reference point of fp16 weights lies this many powers of two below the largest
// one.  With kLag they stay below 2^15, and keep all of their bits down to 2^-21 of
// the largest and some down to 2^-32 (from 1 on, 2^-14 and 2^-25): many small
// weights count where one large weight meets a value near 0.
constexpr float kLift = 7.0f;

// Four 16-bit values of each lane of 16, transposed in blocks of 4 x 16: lane i
// gets value i % 4 of lanes i / 4, i / 4 + 4, i / 4 + 8, i / 4 + 12.
__device__ __forceinline__ u2 read_transposed(const u2* p) {
  return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)p));
}

__device__ __forceinline__ float max_over_halves(float v) {  // over the lanes l, l ^ 32
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
}
__device__ __forceinline__ float sum_over_halves(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
}

// Exchanges within a wave by DPP, a few cycles each where one through LDS takes 60 or
// more: lane l gets the value of lane l - n of its row of 16 (0x110 + n), the same
// rotated within the row (0x120 + n), of lane l ^ 1 (0xB1), l ^ 2 (0x4E) or of its mirror
// image in eight (0x141), of the row before's last lane (0x142), of lane 31 (0x143), or of
// lane l - 1 (0x138); `none` where there is no such lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int none, int v) {
  return __builtin_amdgcn_update_dpp(none, v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float none, float v) {
  return __builtin_bit_cast(float, dpp<CTRL, ROWS>(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double none, double v) {
  const uint64_t o = __builtin_bit_cast(uint64_t, none), u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = dpp<CTRL, ROWS>((int)o, (int)u), hi = dpp<CTRL, ROWS>((int)(o >> 32), (int)(u >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// A lane's v and that of lane l ^ 32 (halves) or l ^ 16.
__device__ __forceinline__ double add_swapped(double v, bool halves) {
  const u2 w = __builtin_bit_cast(u2, v);
  uint32_t x[2], y[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    auto a = halves ? __builtin_amdgcn_permlane32_swap(w[i], w[i], false, false)
                    : __builtin_amdgcn_permlane16_swap(w[i], w[i], false, false);
    x[i] = a[0], y[i] = a[1];
  }
  return __builtin_bit_cast(double, u2{x[0], x[1]}) + __builtin_bit_cast(double, u2{y[0], y[1]});
}

// The queries of sequence b: `all` of them from q0 on, the first n are computed.
struct Queries {
  int q0, n, all;
};
__device__ __forceinline__ Queries queries_of(const KvAttnArgs& a, int b) {
  if (!a.q_starts) return {b, 1, 1};
  const int q0 = max(a.q_starts[b], 0);
  const int64_t all = max((int64_t)0, min((int64_t)a.q_starts[b + 1], a.T) - q0);
  return {q0, (int)min(all, a.max_queries), (int)all};
}
__device__ __forceinline__ int length_of(const KvAttnArgs& a, int b) {
  return (int)max((int64_t)0, min((int64_t)a.lens[b], a.max_context));
}

// The sequence that holds token t, its first token, and how many it has; none: b < 0.
struct Place {
  int b, q0, n;
};
__device__ __forceinline__ Place place_of(const int32_t* starts, int B, int64_t T, int t, int lane) {
  if (!starts) return {t < B ? t : -1, t, 1};
  // the last of the starts 0..B that is not above t: 64 probes at a time
  int lo = 0, len = B + 1, c;
  while (true) {
    const int step = (len + 63) / 64;
    const int at = lo + min(lane * step, len - 1);
    c = __popcll(__ballot(lane * step < len && starts[at] <= t));
    if (c == 0) return {-1, 0, 0};
    lo += (c - 1) * step;
    len = min(step, len - (c - 1) * step);
    if (step == 1) break;
  }
  if (lo >= B) return {-1, 0, 0};
  const int q0 = max(starts[lo], 0);
  return {lo, q0, (int)(min((int64_t)starts[lo + 1], T) - q0)};
}

// Bit i: node `node` (a query of the call) sees the token `rel` + i places behind
// its sequence's first node: all before that one, then as its mask words say.
__device__ __forceinline__ uint64_t tree_window(const KvAttnArgs& a, int node, int rel) {
  if (rel <= -64) return ~0ull;
  const uint64_t* w = a.tree + (int64_t)node * a.tree_words;
  if (rel < 0) return w[0] << -rel | ~(~0ull << -rel);
  const int i = rel >> 6, s = rel & 63;
  uint64_t v = i < a.tree_words ? w[i] >> s : 0;
  if (s && i + 1 < a.tree_words) v |= w[i + 1] << (64 - s);
  return v;
}

// fp32 pair -> 16-bit pair, round to nearest even
template <bool BF>
__device__ __forceinline__ uint32_t pack_pair(float x, float y) {
  if constexpr (BF) {
    const b2 v = {(__bf16)x, (__bf16)y};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    const h2 v = {(_Float16)x, (_Float16)y};
    return as_u32(v);
  }
}
__device__ __forceinline__ uint32_t pack_out(int dtype, float x, float y) {
  return dtype == 1 ? pack_pair<true>(x, y) : pack_pair<false>(x, y);
}
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? kNegInf : (m + __builtin_log2f(l)) * 0.6931471805599453f;
}

// Eight 16-bit values of a query row as fp32.
__device__ __forceinline__ void widen8(const u4& raw, int dtype, float (&y)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    y[e] = dtype == 1 ? __builtin_bit_cast(float, e % 2 ? raw[e / 2] & 0xffff0000u : raw[e / 2] << 16)
                      : (float)__builtin_bit_cast(h8, raw)[e];
}
// The power of two that a row is divided by so that its largest value lies in
// [1, 2) (zeros, subnormals and infinities: the nearest power), and its inverse.
struct RowPower {
  float up, down;
};
__device__ __forceinline__ RowPower row_power(float top) {
  int ex = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
  ex = min(max(ex, -126), 126);
  return {__builtin_bit_cast(float, (uint32_t)(127 + ex) << 23), __builtin_bit_cast(float, (uint32_t)(127 - ex) << 23)};
}
// The factor from such a row's scores to units of log2; never 0, which times the
// -inf of a masked score is no number.
__device__ __forceinline__ float score_factor(float scale, float up) {
  return fmaxf(scale * 1.4426950408889634f * up, 1.17549435e-38f);
}

// The power of two above a V scale.  A scale of 0 counts as 2^kNoPower: its token adds
// to the sum of weights, which stays within fp32, and to nothing else.
constexpr float kNoPower = -64.0f;
__device__ __forceinline__ float scale_power(float s) {
  return (float)__builtin_amdgcn_frexp_expf(fmaxf(fabsf(s), 0x1p-65f));
}

// top: the largest of the powers seen so far, with those of the lanes now.
__device__ __forceinline__ void raise_top(float& top, float power) {
  if (__ballot(power > top)) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) power = fmaxf(power, __shfl_xor(power, d));
    top = fmaxf(top, __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, power))));
  }
}

// The eight codes of a word less their zero-point(s) as four fp16 pairs, of
// nibbles 0 and 4, 1 and 5, 2 and 6, 3 and 7: 1024 + c and 64 + c by OR-ing an
// exponent in (wq_device.h), less the same of z.  The exponents come in vector
// registers: v_and_or_b32 takes one scalar operand and no literal.
struct Magic {
  uint32_t e10 = 0x64006400u, e6 = 0x54005400u;
  __device__ __forceinline__ Magic() {
    asm("" : "+v"(e10));
    asm("" : "+v"(e6));
  }
};
__device__ __forceinline__ u4 code_pairs(uint32_t w, uint32_t z10, uint32_t z6, const Magic& g) {
  const uint32_t w8 = w >> 8;
  return u4{as_u32(as_h2((w & 0x000F000Fu) | g.e10) - as_h2(z10)), as_u32(as_h2((w & 0x00F000F0u) | g.e6) - as_h2(z6)),
            as_u32(as_h2((w8 & 0x000F000Fu) | g.e10) - as_h2(z10)), as_u32(as_h2((w8 & 0x00F000F0u) | g.e6) - as_h2(z6))};
}

}  // namespace wq
