// Norm of every query and key head and the rotation of its position, one pass
// (gfx950).
//
// For a head row x of D 16-bit values: n = x * rsqrt(mean(x^2) + eps) * w with
// the channel weights w, then the pairs (a, b) of the first `rot` channels turn
// by the token's angle: a' = a cos - b sin, b' = b cos + a sin, with cos and
// sin from row positions[t] of two fp32 tables (tables, so that the angles of
// far positions and any scaled frequencies are the caller's, made once in 64
// bits).  Everything between the load and the store is fp32, one rounding at
// the end.
//
// Bound by memory: a row is read once and written once.  A lane holds four
// pairs: in the half form values 4l..4l+3 and their partners rot/2 further on
// (two 8-byte loads), in the interleaved form eight neighbours (one 16-byte
// load), so the rotation needs no exchange between lanes and the sum of squares
// is one xor-shuffle tree over the D/8 lanes of the row.  A prompt of 32768 tokens
// (64 + 8 heads of 128) moves 1.2 GB in 240-250 us, the rate of a large copy
// (5.0 TB/s); with 64-bit row numbers and outputs rounded in integer arithmetic the
// vector instructions took all of the cycles (268 us).  A decode step of 64 tokens
// takes 2.7 us a call in a replayed graph (traced alone 3.4), the latency of one row.
#include "wq_attn.h"

namespace wq {
namespace {

template <int DT>
__device__ __forceinline__ void unpack4(u2 w, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (DT == 1) {
      v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
    } else {
      const h2 h = as_h2(w[i]);
      v[2 * i] = (float)h[0];
      v[2 * i + 1] = (float)h[1];
    }
  }
}

template <int DT>
__device__ __forceinline__ u2 pack4(const float (&v)[4]) {
  u2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = pack_pair<DT == 1>(v[2 * i], v[2 * i + 1]);
  return w;
}

// LPH: lanes of a row (D = 8 LPH).  U: rows a lane works through, whose loads
// are all issued before the first is used.
template <int DT, bool INTER, int LPH, int U>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(QkNormRopeArgs a) {
  constexpr int D = 8 * LPH, RPB = 256 / LPH;  // rows in flight per workgroup and u
  const int l = threadIdx.x % LPH;
  const int H = a.Hq + a.Hkv, half = a.rot / 2, p0 = 4 * l;
  const bool turned = p0 < half;
  // channels of the lane's two quads: the pairs of the rotated part, then (half
  // form) the two halves of the rest
  int ca, cb;
  if constexpr (INTER) {
    ca = 8 * l;
    cb = 8 * l + 4;
  } else if (turned) {
    ca = p0;
    cb = p0 + half;
  } else {
    ca = a.rot + (p0 - half);
    cb = ca + (D - a.rot) / 2;
  }
  const uint32_t rows = (uint32_t)(a.T * H);  // below 2^31
  const uint32_t r0 = blockIdx.x * (RPB * U) + threadIdx.x / LPH;
  u2 xa[U], xb[U];
  int pos[U];
  uint32_t tok[U];
  int head[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = min(r0 + u * RPB, rows - 1);  // past the end: a real row, not stored
    tok[u] = r / (uint32_t)H;
    head[u] = (int)(r - tok[u] * H);
    const bool isq = head[u] < a.Hq;
    const uint16_t* x = isq ? a.q + (int64_t)tok[u] * a.q_stride + (int64_t)head[u] * D
                            : a.k + (int64_t)tok[u] * a.k_stride + (int64_t)(head[u] - a.Hq) * D;
    xa[u] = *reinterpret_cast<const u2*>(x + ca);
    xb[u] = *reinterpret_cast<const u2*>(x + cb);
    pos[u] = a.positions[tok[u]];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool isq = head[u] < a.Hq;
    float v[8];
    {
      float t[4];
      unpack4<DT>(xa[u], t);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = t[i];
      unpack4<DT>(xb[u], t);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 + i] = t[i];
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += v[i] * v[i];
#pragma unroll
    for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor(ss, m);
    const float rn = rsqrtf(ss * (1.0f / D) + a.eps);
    const uint16_t* w = isq ? a.q_weight : a.k_weight;
    float wa[4] = {1, 1, 1, 1}, wb[4] = {1, 1, 1, 1};
    if (w) {
      unpack4<DT>(*reinterpret_cast<const u2*>(w + ca), wa);
      unpack4<DT>(*reinterpret_cast<const u2*>(w + cb), wb);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = v[i] * rn * wa[i];
      v[4 + i] = v[4 + i] * rn * wb[i];
    }
    const bool in_table = pos[u] >= 0 && pos[u] < a.P;
    if (turned) {
      const int64_t at = (int64_t)(in_table ? pos[u] : 0) * half + p0;
      const f4 c = *reinterpret_cast<const f4*>(a.cos + at), s = *reinterpret_cast<const f4*>(a.sin + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : 4 + i;
        const float x0 = v[ia], x1 = v[ib];
        v[ia] = x0 * c[i] - x1 * s[i];
        v[ib] = x1 * c[i] + x0 * s[i];
      }
    }
    if (r0 + u * RPB < rows && in_table) {
      uint16_t* o = isq ? a.q_out + (int64_t)tok[u] * a.qo_stride + (int64_t)head[u] * D
                        : a.k_out + (int64_t)tok[u] * a.ko_stride + (int64_t)(head[u] - a.Hq) * D;
      const float oa[4] = {v[0], v[1], v[2], v[3]}, ob[4] = {v[4], v[5], v[6], v[7]};
      *reinterpret_cast<u2*>(o + ca) = pack4<DT>(oa);
      *reinterpret_cast<u2*>(o + cb) = pack4<DT>(ob);
    }
  }
}

template <int DT, bool INTER, int LPH>
hipError_t launch_lph(const QkNormRopeArgs& a, hipStream_t stream) {
  const int64_t rows = a.T * (a.Hq + a.Hkv);
  constexpr int RPB = 256 / LPH;
  // four rows a lane once that still leaves two thousand workgroups (32768 tokens of
  // 72 heads: 247 us, 265 with one); one below, where the time is the latency of a
  // row (64 tokens: 2.7 us, 4.6 with four; all in replayed graphs)
  if (rows >= (int64_t)2048 * RPB * 4)
    qk_norm_rope_kernel<DT, INTER, LPH, 4><<<(unsigned)((rows + 4 * RPB - 1) / (4 * RPB)), 256, 0, stream>>>(a);
  else
    qk_norm_rope_kernel<DT, INTER, LPH, 1><<<(unsigned)((rows + RPB - 1) / RPB), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <int DT, bool INTER>
hipError_t launch_d(const QkNormRopeArgs& a, hipStream_t stream) {
  if (a.D == 64) return launch_lph<DT, INTER, 8>(a, stream);
  if (a.D == 128) return launch_lph<DT, INTER, 16>(a, stream);
  return launch_lph<DT, INTER, 32>(a, stream);
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormRopeArgs& a, hipStream_t stream) {
  if (a.dtype == 1) return a.interleaved ? launch_d<1, true>(a, stream) : launch_d<1, false>(a, stream);
  return a.interleaved ? launch_d<2, true>(a, stream) : launch_d<2, false>(a, stream);
}

}  // namespace wq
