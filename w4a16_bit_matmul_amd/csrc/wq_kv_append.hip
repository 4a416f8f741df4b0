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
// -ffp-contract=off).  The sum of squares is taken in 64 bits, where products of 16-bit
// values are exact and 256 of them add up to within 2^-45, and in one order, eight neighbouring
// values and then neighbours' sums, pair by pair: near an fp32 midpoint 2^-45 too decides
// how the mean rounds.  Keys are
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
// them.  What the lines' second reading and the tables (four bytes of cosine and sine for
// two of a value) cost is the way through the L1 cache, so a wave of a long prompt
// takes two such runs, whose lanes have the same channels, with one reading of the
// tables: 32517 tokens of 64 + 8 heads of 128 move 1.32 GB in 234 us, 5.6 TB/s (a copy
// reaches 5.1); one run a wave takes 333.  A decode step of 64 tokens takes 4.0 us in a
// replayed graph.
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

// U: runs of 512 values that a wave works through, whose loads are all issued before the
// first is used; the lane's channels, and so its cosines and sines, are the same in each.
template <int DT, bool INTER, int U>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, uint32_t q_units, uint32_t k_units,
                                                        uint32_t waves) {
  const int lane = threadIdx.x & 63;
  const uint32_t id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= waves) return;
  const uint32_t units = q_units + 2 * k_units, t = id / units;
  uint32_t unit = id - t * units;
  const bool isq = unit < q_units, isv = unit >= q_units + k_units;
  unit -= isq ? 0 : isv ? q_units + k_units : q_units;
  const int D = a.D;
  const int vals = (isq ? a.Hq : a.Hkv) * D, start = (int)(512 * U * unit) + 8 * lane;
  const int half = a.rot / 2, e = start & (D - 1);  // the lane's channels e..e+7 of its heads
  const bool turned = !isv && e < a.rot;
  const int to_partner = INTER || !turned ? 0 : e < half ? half : -half;
  const uint16_t* x = isq ? a.q + (int64_t)t * a.q_stride : isv ? a.v + (int64_t)t * a.v_stride : a.k + (int64_t)t * a.k_stride;
  u4 raw[U], partner[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // past the end: the token's last head, not stored
    const int v0 = start + 512 * u < vals ? start + 512 * u : vals - D + e;
    raw[u] = *reinterpret_cast<const u4*>(x + v0);
    if (!INTER) partner[u] = *reinterpret_cast<const u4*>(x + v0 + to_partner);
  }

  const Place pl = place_of(a.q_starts, a.B, a.T, (int)t, lane);
  if (pl.b < 0) return;
  const int64_t token = (int64_t)a.lens[pl.b] - pl.n + ((int)t - pl.q0);
  const int64_t pos = a.positions ? (int64_t)a.positions[t] : token;
  if (pos < 0 || pos >= a.P) return;  // padding

  const uint16_t* w = isq ? a.q_weight : a.k_weight;
  f4 c[2] = {}, s[2] = {};
  if (turned) {
    const int at = INTER ? e / 2 : e < half ? e : e - half;
    const float *cr = a.cos + pos * half + at, *sr = a.sin + pos * half + at;
    c[0] = *reinterpret_cast<const f4*>(cr), s[0] = *reinterpret_cast<const f4*>(sr);
    if (!INTER) c[1] = *reinterpret_cast<const f4*>(cr + 4), s[1] = *reinterpret_cast<const f4*>(sr + 4);
  }
  const int64_t row = isq ? -1 : cache_row(a.table, a.table_width, a.lg, a.pages, pl.b, token);
  uint16_t* to = isq ? a.q_out + (int64_t)t * a.qo_stride : !isv && a.k_out ? a.k_out + (int64_t)t * a.ko_stride : nullptr;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int v0 = start + 512 * u;
    const bool active = v0 < vals;
    float y[8];
    unpack8<DT>(raw[u], y);
    if (!isv) {
      float r = 1.0f;
      if (a.norm) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += (double)y[i] * (double)y[i];
        ss += dpp<0xB1, 0xf>(0.0, ss);  // over the head's D / 8 lanes
        ss += dpp<0x4E, 0xf>(0.0, ss);
        ss += dpp<0x141, 0xf>(0.0, ss);
        if (D > 64) ss += dpp<0x128, 0xf>(0.0, ss);
        if (D > 128) ss = add_swapped(ss, false);
        r = 1.0f / sqrtf((float)(ss / D) + a.eps);
        scale8<DT>(y, r, w ? w + e : nullptr);
      }
      if (turned) {
        if constexpr (INTER) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = y[2 * i], q = y[2 * i + 1];
            y[2 * i] = p * c[0][i] - q * s[0][i];
            y[2 * i + 1] = q * c[0][i] + p * s[0][i];
          }
        } else {
          float z[8];
          unpack8<DT>(partner[u], z);
          if (a.norm) scale8<DT>(z, r, w ? w + e + to_partner : nullptr);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float own = y[i] * c[i / 4][i % 4], other = z[i] * s[i / 4][i % 4];
            y[i] = e < half ? own - other : own + other;
          }
        }
      }
      const u4 out = pack8<DT>(y);
      if (to && active) *reinterpret_cast<u4*>(to + v0) = out;
      if (isq) continue;
      unpack8<DT>(out, y);
    }

    // a block of 128 values: 16 lanes
    float lo = y[0], hi = y[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      lo = fminf(lo, y[i]);
      hi = fmaxf(hi, y[i]);
    }
    lo = fminf(lo, dpp<0x128, 0xf>(lo, lo)), hi = fmaxf(hi, dpp<0x128, 0xf>(hi, hi));
    lo = fminf(lo, dpp<0x124, 0xf>(lo, lo)), hi = fmaxf(hi, dpp<0x124, 0xf>(hi, hi));
    lo = fminf(lo, dpp<0x122, 0xf>(lo, lo)), hi = fmaxf(hi, dpp<0x122, 0xf>(hi, hi));
    lo = fminf(lo, dpp<0x121, 0xf>(lo, lo)), hi = fmaxf(hi, dpp<0x121, 0xf>(hi, hi));
    const GroupParams p = group_params(lo, hi);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) word |= encode(y[i], p) << (4 * nibble_pos(i));
    uint32_t z = active ? (uint32_t)p.z : 0u;
    z |= (uint32_t)__shfl_down((int)z, 16) << 4;  // the next block's beside it
    if (row < 0 || !active) continue;
    const int nb = vals / 128, blk = v0 / 128;
    *reinterpret_cast<uint32_t*>((isv ? a.v_codes : a.k_codes) + row * (vals / 2) + v0 / 2) = word;
    if ((lane & 15) == 0) (isv ? a.v_s : a.k_s)[row * nb + blk] = p.s_bits;
    if ((lane & 31) == 0) (isv ? a.v_zp : a.k_zp)[row * ((nb + 1) / 2) + blk / 2] = (uint8_t)z;
  }
}

// Row len - n + path[j] of a sequence to row len - n + j, for its accepted nodes j.
// A workgroup has 64 parts of a row (16 bytes of codes, or a scale or zero-point byte) of
// one sequence and cache; its four waves take every fourth node, read what 64 nodes
// need, meet, and write it.  path[j] >= j, so no row is written that later nodes
// still have to read.  It is all latency: lengths and path, pages, rows, stores one
// after the other, and each of them once for up to 64 nodes (up to 64 nodes of 200
// sequences, 9 blocks a row: 9.8 us; eight nodes at a time in one wave 12.9).
template <class T>
__device__ __forceinline__ void move_rows(T* base, int64_t stride, int64_t to, int64_t from, int m, int wave, bool mine) {
  constexpr int K = 16;
  T v[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int j = wave + 4 * i;
    const int64_t src = __shfl(from, j);
    if (j < m && src >= 0 && mine) v[i] = base[src * stride];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int j = wave + 4 * i;
    const int64_t dst = __shfl(to, j);
    if (j < m && dst >= 0 && mine) base[dst * stride] = v[i];
  }
}

__global__ __launch_bounds__(256) void kv_keep_kernel(KvKeepArgs a, int code_blocks, int blocks) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cb = blockIdx.x % (uint32_t)blocks, bc = blockIdx.x / (uint32_t)blocks, b = bc / 2;
  const bool isv = bc & 1;
  int q0 = b, n = 1;
  if (a.q_starts) {
    q0 = max(a.q_starts[b], 0);
    n = (int)(min((int64_t)a.q_starts[b + 1], a.T) - q0);
  }
  const int m = min(min(a.counts[b], a.width), n);
  const int64_t first = (int64_t)a.lens[b] - n;
  const int nb = a.nb, zb = (nb + 1) / 2;
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
    const int most = min(64, m - j0);
    if (cb < code_blocks) {
      const int item = cb * 64 + lane;
      move_rows(reinterpret_cast<u4*>(isv ? a.v_codes : a.k_codes) + item, 4 * nb, to, from, most, wave, item < 4 * nb);
    } else if (cb < code_blocks + (nb + 63) / 64) {
      const int item = (cb - code_blocks) * 64 + lane;
      move_rows((isv ? a.v_s : a.k_s) + item, nb, to, from, most, wave, item < nb);
    } else {
      const int item = (cb - code_blocks - (nb + 63) / 64) * 64 + lane;
      move_rows((isv ? a.v_zp : a.k_zp) + item, zb, to, from, most, wave, item < zb);
    }
  }
}

template <int DT, int U>
hipError_t launch_u(const KvAppendArgs& a, hipStream_t stream) {
  const uint32_t qu = a.q ? (uint32_t)(((int64_t)a.Hq * a.D + 512 * U - 1) / (512 * U)) : 0;
  const uint32_t ku = (uint32_t)(((int64_t)a.Hkv * a.D + 512 * U - 1) / (512 * U));
  const uint32_t waves = (uint32_t)a.T * (qu + 2 * ku);  // up to 2^26 - 4 (checked by the caller)
  const unsigned grid = (waves + 3) / 4;
  if (a.interleaved) kv_append_kernel<DT, true, U><<<grid, 256, 0, stream>>>(a, qu, ku, waves);
  else kv_append_kernel<DT, false, U><<<grid, 256, 0, stream>>>(a, qu, ku, waves);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const KvAppendArgs& a, hipStream_t stream) {
  // two runs a wave once there are waves for the whole GPU, two rounds of them (64 + 8 heads of 128, one run and
  // two: 64 tokens 4.0 and 5.0 us, 512 7.9 and 7.5, 1024 19.7 and 18.0, 8192 75 and 60; a prompt of
  // 32517 333 and 234, 265 with four); with the norm, whose arithmetic bounds then, always one (32 + 4
  // heads, 8192 tokens: 42.2 and 43.1 us)
  return !a.norm && kv_append_waves(a.T, a.q ? a.Hq : 0, a.Hkv, a.D) >= 8192 ? launch_u<DT, 2>(a, stream)
                                                                            : launch_u<DT, 1>(a, stream);
}

}  // namespace

int64_t kv_append_waves(int64_t T, int Hq, int Hkv, int D) {
  return T * (((int64_t)Hq * D + 511) / 512 + 2 * (((int64_t)Hkv * D + 511) / 512));
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream) {
  return a.dtype == 1 ? launch_dt<1>(a, stream) : launch_dt<2>(a, stream);
}

int kv_keep_blocks(int nb) { return (4 * nb + 63) / 64 + (nb + 63) / 64 + ((nb + 1) / 2 + 63) / 64; }

hipError_t launch_kv_keep(const KvKeepArgs& a, hipStream_t stream) {
  const int blocks = kv_keep_blocks(a.nb);
  kv_keep_kernel<<<(unsigned)(2 * a.B * blocks), 256, 0, stream>>>(a, (4 * a.nb + 63) / 64, blocks);
  return hipGetLastError();
}

}  // namespace wq
