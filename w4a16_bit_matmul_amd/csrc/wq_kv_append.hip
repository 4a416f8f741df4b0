// Rotation of queries and keys and the quantization of keys and values into the
// pages of the INT4 KV cache, one pass (gfx950); and cache rows moved together.
//
// For a head row x of a query or key: with a norm, n = x r w, where
// r = 1 / sqrt(mean(x^2) + eps), else n = x; the pairs (a, b) of the first `rot`
// channels turn by the token's angle, a' = a c - b s, b' = b c + a s; the result
// is rounded to the tensors' 16-bit type.  The rounded keys, and the values as
// they come, are cut into blocks of 128 and quantized like weight groups.
//
// The codes are whole numbers: whether a value lands on one side of a half or the
// other hangs on its last bit, and on every operation before it.  So every step is
// one correctly rounded fp32 operation (this file is compiled with
// -ffp-contract=off), and the sum of squares, whose order would matter, is taken in
// 64 bits: products of 16-bit values are exact there and 256 of them add up to
// within 2^-45, so that its fp32 rounding does not depend on the order.  Keys are
// rounded to 16 bits first so that the cache holds what wq_kv_quantize makes of the
// rotated keys that a prompt's own attention reads (2^-9 of a value beside a step
// of a fifteenth of the block's range).
//
// Bound by memory: q, k and v are read once, q (and k, if asked for) written once,
// and 0.52 bytes a value of the cache.  A wave takes 512 neighbouring values of one
// token's q, k or v, eight a lane: a block is 16 lanes, so its range is four
// exchanges, a lane's codes are one word, and two blocks' zero-points a byte.  In the
// half form a value's partner sits rot / 2 further on: the lane loads those eight
// values too, from the line that its neighbour brings in, instead of exchanging
// them.
#include "wq_attn.h"
#include "wq_group.h"

namespace wq {
namespace {

// Row of a sequence's token in a paged cache, or -1.
__device__ __forceinline__ int64_t cache_row(const int32_t* table, int64_t width, int lg, int64_t pages, int b,
                                             int64_t token) {
  if (token < 0 || token >> lg >= width) return -1;
  const int pg = table[(int64_t)b * width + (token >> lg)];
  return pg < 0 || pg >= pages ? -1 : ((int64_t)pg << lg) + (token & ((1 << lg) - 1));
}

template <int DT>
__device__ __forceinline__ u4 pack8(const float (&v)[8]) {
  u4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_pair<DT == 1>(v[2 * i], v[2 * i + 1]);
  return w;
}
template <int DT>
__device__ __forceinline__ void unpack8(const u4& w, float (&v)[8]) {
  widen8(w, DT, v);
}

// v[0..7] times the head's r and the weights from w on (null: ones)
template <int DT>
__device__ __forceinline__ void scale8(float (&v)[8], float r, const uint16_t* w) {
  float y[8] = {1, 1, 1, 1, 1, 1, 1, 1};
  if (w) load8<DT>(w, 0, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * r * y[i];
}

template <int DT, bool INTER>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, uint32_t q_units, uint32_t k_units,
                                                        uint32_t waves) {
  const int lane = threadIdx.x & 63;
  const uint32_t id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= waves) return;
  const uint32_t units = q_units + 2 * k_units, t = id / units;
  uint32_t u = id - t * units;
  const bool isq = u < q_units, isv = u >= q_units + k_units;
  u -= isq ? 0 : isv ? q_units + k_units : q_units;
  const int D = a.D;
  const int vals = (isq ? a.Hq : a.Hkv) * D;
  const int v0 = min((int)(512 * u) + 8 * lane, vals - 8);  // past the end: real values, not stored
  const bool active = (int)(512 * u) + 8 * lane < vals;
  const uint16_t* x = isq ? a.q + (int64_t)t * a.q_stride : isv ? a.v + (int64_t)t * a.v_stride : a.k + (int64_t)t * a.k_stride;
  const u4 raw = *reinterpret_cast<const u4*>(x + v0);
  float y[8];
  unpack8<DT>(raw, y);

  const Place pl = place_of(a.q_starts, a.B, a.T, (int)t, lane);
  if (pl.b < 0) return;
  const int64_t token = (int64_t)a.lens[pl.b] - pl.n + ((int)t - pl.q0);
  const int64_t pos = a.positions ? (int64_t)a.positions[t] : token;
  if (pos < 0 || pos >= a.P) return;  // padding

  u4 out = raw;
  if (!isv) {
    const int half = a.rot / 2, e = v0 & (D - 1);  // the lane's channels e..e+7 of its head
    const uint16_t* w = isq ? a.q_weight : a.k_weight;
    float r = 1.0f;
    if (a.norm) {
      double ss = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += (double)y[i] * (double)y[i];
      for (int m = 1; m < D / 8; m <<= 1) ss += __shfl_xor(ss, m);
      r = 1.0f / sqrtf((float)(ss / D) + a.eps);
      scale8<DT>(y, r, w ? w + e : nullptr);
    }
    if (e < a.rot) {
      const float *cr = a.cos + pos * half, *sr = a.sin + pos * half;
      if constexpr (INTER) {
        const f4 c = *reinterpret_cast<const f4*>(cr + e / 2), s = *reinterpret_cast<const f4*>(sr + e / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = y[2 * i], q = y[2 * i + 1];
          y[2 * i] = p * c[i] - q * s[i];
          y[2 * i + 1] = q * c[i] + p * s[i];
        }
      } else {
        const bool first = e < half;
        const int pe = first ? e + half : e - half, at = first ? e : e - half;
        float z[8];  // the partners
        unpack8<DT>(*reinterpret_cast<const u4*>(x + v0 + (pe - e)), z);
        if (a.norm) scale8<DT>(z, r, w ? w + pe : nullptr);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f4 c = *reinterpret_cast<const f4*>(cr + at + 4 * h), s = *reinterpret_cast<const f4*>(sr + at + 4 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 4 * h + i;
            const float own = y[j] * c[i], other = z[j] * s[i];
            y[j] = first ? own - other : own + other;
          }
        }
      }
    }
    out = pack8<DT>(y);
    uint16_t* to = isq ? a.q_out + (int64_t)t * a.qo_stride : a.k_out ? a.k_out + (int64_t)t * a.ko_stride : nullptr;
    if (to && active) *reinterpret_cast<u4*>(to + v0) = out;
    if (isq) return;
    unpack8<DT>(out, y);
  }

  // a block of 128 values: 16 lanes
  float lo = y[0], hi = y[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, y[i]);
    hi = fmaxf(hi, y[i]);
  }
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, m));
    hi = fmaxf(hi, __shfl_xor(hi, m));
  }
  const GroupParams p = group_params(lo, hi);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) word |= encode(y[i], p) << (4 * nibble_pos(i));
  uint32_t z = active ? (uint32_t)p.z : 0u;
  z |= (uint32_t)__shfl_down((int)z, 16) << 4;  // the next block's beside it

  const int64_t row = cache_row(a.table, a.table_width, a.lg, a.pages, pl.b, token);
  if (row < 0 || !active) return;
  const int nb = vals / 128, blk = v0 / 128;
  uint8_t* codes = (isv ? a.v_codes : a.k_codes) + row * (vals / 2);
  *reinterpret_cast<uint32_t*>(codes + v0 / 2) = word;
  if ((lane & 15) == 0) (isv ? a.v_s : a.k_s)[row * nb + blk] = p.s_bits;
  if ((lane & 31) == 0) (isv ? a.v_zp : a.k_zp)[row * ((nb + 1) / 2) + blk / 2] = (uint8_t)z;
}

// Row len - n + path[j] of a sequence to row len - n + j, for its accepted nodes j.
// A thread owns 16 bytes of codes, a scale or a zero-point byte of every row and
// takes the nodes in order; path[j] >= j, so a row is read before any thread could
// write it.  Latency bounds: eight rows are in flight at a time.
__global__ __launch_bounds__(64) void kv_keep_kernel(KvKeepArgs a, int blocks) {
  const int lane = threadIdx.x;
  const int cb = blockIdx.x % blocks, bc = blockIdx.x / blocks, b = bc / 2;
  const bool isv = bc & 1;
  int q0 = b, n = 1;
  if (a.q_starts) {
    q0 = max(a.q_starts[b], 0);
    n = (int)(min((int64_t)a.q_starts[b + 1], a.T) - q0);
  }
  const int m = min(min(a.counts[b], a.width), n);
  const int64_t first = (int64_t)a.lens[b] - n;
  const int nb = a.nb, c16 = 4 * nb, zb = (nb + 1) / 2;
  const int item = cb * 64 + lane;
  uint8_t* codes = isv ? a.v_codes : a.k_codes;
  uint16_t* scales = isv ? a.v_s : a.k_s;
  uint8_t* zeros = isv ? a.v_zp : a.k_zp;
  for (int j0 = 0; j0 < m; j0 += 64) {
    // lane: the rows of node j0 + lane
    int64_t to = -1, from = -1;
    const int j = j0 + lane;
    if (j < m) {
      const int node = a.path[(int64_t)b * a.width + j];
      if (node > j && node < n) {
        to = cache_row(a.table, a.table_width, a.lg, a.pages, b, first + j);
        from = cache_row(a.table, a.table_width, a.lg, a.pages, b, first + node);
      }
    }
    if (to < 0 || from < 0) to = from = -1;
    for (int i0 = 0; i0 < min(64, m - j0); i0 += 8) {
      u4 v[8];
      int64_t dst[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t src = __shfl(from, i0 + i);
        dst[i] = __shfl(to, i0 + i);
        if (src < 0) continue;
        if (item < c16) v[i] = *reinterpret_cast<const u4*>(codes + src * (16 * c16) + 16 * item);
        else if (item < c16 + nb) v[i][0] = scales[src * nb + (item - c16)];
        else if (item < c16 + nb + zb) v[i][0] = zeros[src * zb + (item - c16 - nb)];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (dst[i] < 0) continue;
        if (item < c16) *reinterpret_cast<u4*>(codes + dst[i] * (16 * c16) + 16 * item) = v[i];
        else if (item < c16 + nb) scales[dst[i] * nb + (item - c16)] = (uint16_t)v[i][0];
        else if (item < c16 + nb + zb) zeros[dst[i] * zb + (item - c16 - nb)] = (uint8_t)v[i][0];
      }
    }
  }
}

template <int DT>
hipError_t launch_dt(const KvAppendArgs& a, hipStream_t stream) {
  const uint32_t qu = a.q ? (uint32_t)(((int64_t)a.Hq * a.D + 511) / 512) : 0;
  const uint32_t ku = (uint32_t)(((int64_t)a.Hkv * a.D + 511) / 512);
  const uint32_t waves = (uint32_t)a.T * (qu + 2 * ku);  // below 2^26 (checked by the caller)
  const unsigned grid = (waves + 3) / 4;
  if (a.interleaved) kv_append_kernel<DT, true><<<grid, 256, 0, stream>>>(a, qu, ku, waves);
  else kv_append_kernel<DT, false><<<grid, 256, 0, stream>>>(a, qu, ku, waves);
  return hipGetLastError();
}

}  // namespace

int64_t kv_append_waves(int64_t T, int Hq, int Hkv, int D) {
  return T * (((int64_t)Hq * D + 511) / 512 + 2 * (((int64_t)Hkv * D + 511) / 512));
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream) {
  return a.dtype == 1 ? launch_dt<1>(a, stream) : launch_dt<2>(a, stream);
}

int kv_keep_blocks(int nb) { return (5 * nb + (nb + 1) / 2 + 63) / 64; }

hipError_t launch_kv_keep(const KvKeepArgs& a, hipStream_t stream) {
  const int blocks = kv_keep_blocks(a.nb);
  kv_keep_kernel<<<(unsigned)(2 * a.B * blocks), 64, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace wq
