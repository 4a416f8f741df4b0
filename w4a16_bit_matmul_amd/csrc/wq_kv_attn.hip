// Attention over the INT4 KV cache (gfx950).
//
// For a query row q (one query token and head) and the tokens t it sees,
//   out = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale * q.k_t - max),
// with k_t = s_t (c_t - z_t) and v_t alike, read from the codes in one pass: a
// running maximum and sum per row, no scores in memory.
//
// The matrix cores take the exact integers c - z in fp16 (|c - z| <= 15), decoded
// with the GEMV's shift, four AND-ORs and four packed subtractions a word; the
// scale of a token multiplies its score in fp32 (K) and its softmax weight in
// fp32 before that weight is rounded (V).  So nothing is rounded but q (bf16 rows
// are moved into fp16's range by a power of two) and the weights w_t = p_t s_t (to
// fp16, half a step of 2^-11 at most: their reference point is the largest score
// plus the exponent of the largest V scale so far, so the large ones lie near 1
// for any scale).  Leaving 64 + z of half of the codes to the fp32 sums saves a
// seventh of the vector instructions but not a microsecond, and loses bits where
// most codes equal z; codes as fp16 subnormals need no subtraction at all, but the
// matrix cores sum their products with 2^-15 of the sum lost (measured).
//
// Both products are computed transposed, S^T = K q^T and O^T = V^T P^T, with
// v_mfma_f32_16x16x32_f16 and 16 query rows as its columns (the heads of one KV
// head's group and the query tokens).  Then every value of a row lies in the
// lanes of that row (lane r + 16 c holds row r): the maximum is over a lane's
// eight scores and two lane swaps, rescaling needs no exchange, and a lane's
// scores of tokens {4c..4c+3, 16+4c..16+4c+3} of a 32-token tile are, in order,
// its operand of the second product.  For V that product needs eight tokens of
// one channel in a lane while a cache word holds eight channels of one token:
// a lane reads the same word of its eight tokens, and since the even channels of
// a word lie in its low half and the odd ones in its high half, one v_perm per
// pair of tokens turns them into words of one channel's token pairs.
//
// Reading is the bound: 2 (D/2 + 2.5 D/128) bytes a token and KV head.  A wave
// walks 32-token tiles of one KV head, the next tile's codes in flight while it
// computes; a workgroup's waves take neighbouring KV heads of the same tokens or
// different tiles of one head and join in LDS.  Where sequences and heads are too
// few to fill the GPU their walks are cut into pieces, whose fp32 results the last
// workgroup of each to arrive joins.
#include <stdio.h>

#include "wq_device.h"
#include "wq_kernels.h"

namespace wq {
namespace {

typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr float kNegInf = -__builtin_inff();
// A row's reference point may lag its largest weight by this many powers of two
// (fp16 weights stay below 2^9, the fp32 sums far below their limits), so that it
// rarely moves.
constexpr float kLag = 8.0f;
constexpr int kMaxShared = 256;  // sequences that a wave scans for its piece
constexpr int kMeta = 160;       // words of a wave's scales and zero-points of a tile and block
constexpr int kMinSteps = 4;     // steps of a piece, so that joining stays cheap
constexpr int kCounters = 1024;  // pieces that a launch can have

struct KvPlan {
  int HW;        // KV heads of a workgroup (its W / HW waves per head take different tiles)
  int RT;        // 16-row tiles of a wave
  int W;         // waves of a workgroup
  int rtiles;    // units along the query rows of one KV head
  int urows;     // query rows of a unit that a call can use
  int share;     // workgroups that the steps of all units are shared out to (0: one unit a workgroup)
  int64_t grid;  // workgroups launched
};

// A unit is HW heads of one sequence and one tile of query rows; its steps are
// the runs of 32 W / HW tokens that its waves take together.  With fewer units
// than the GPU holds workgroups they are cut into pieces of equal length (on the
// device, where the lengths are).
KvPlan plan_kv(int64_t T, int B, int Hq, int Hkv, int D, int page, int64_t max_context, int64_t max_queries) {
  KvPlan p;
  const int64_t G = Hq / Hkv, rows = max_queries * G;
  p.RT = rows <= 16 ? 1 : 2;
  p.W = 8;
  p.rtiles = (int)((rows + 16 * p.RT - 1) / (16 * p.RT));
  p.urows = (int)(rows < 16 * p.RT ? rows : 16 * p.RT);
  p.HW = Hkv % 2 == 0 ? 2 : 1;
  const int64_t want = 512;
  if ((int64_t)B * (Hkv / p.HW) * p.rtiles < want / 4) p.HW = 1;
  const int64_t units = (int64_t)B * (Hkv / p.HW) * p.rtiles;
  const int64_t steps = (max_context + 32 * (p.W / p.HW) - 1) / (32 * (p.W / p.HW));
  const bool cut = units < want && steps >= 2 * kMinSteps && B <= kMaxShared;
  p.share = cut ? (int)want : 0;
  p.grid = cut ? units + want : units;
  return p;
}

__device__ __forceinline__ int queries_of(const KvAttnArgs& a, int b, int* q0) {
  if (!a.q_starts) {
    *q0 = b;
    return 1;
  }
  *q0 = max(a.q_starts[b], 0);
  return (int)max((int64_t)0, min(min((int64_t)a.q_starts[b + 1], a.T) - *q0, a.max_queries));
}
__device__ __forceinline__ int length_of(const KvAttnArgs& a, int b) {
  return (int)max((int64_t)0, min((int64_t)a.lens[b], a.max_context));
}

// Units of sequence b and steps of each (one at least: a row that sees nothing
// is written too).
__device__ __forceinline__ uint32_t units_of(int nq, int G, int HG, int row_tile) {
  return (uint32_t)HG * ((uint32_t)(nq * G + row_tile - 1) / (uint32_t)row_tile);
}
__device__ __forceinline__ uint32_t steps_of(int len, int step) {
  return max((uint32_t)(len + step - 1) / (uint32_t)step, 1u);
}

// The piece of workgroup `id` when the units are cut, found by every wave for
// itself from the lengths.
struct Piece {
  int b, rt, hg;   // its unit
  int k, n;        // piece k of the unit's n
  uint32_t first;  // piece 0 of the unit (pieces of a unit are HG apart)
};
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = (uint32_t)__shfl_up((int)v, d);
    v += lane >= d ? up : 0u;
  }
  return v;
}
__device__ __forceinline__ bool find_piece(const KvAttnArgs& a, uint32_t id, uint32_t share, int G, int HG, int row_tile,
                                           int step, int lane, Piece* p) {
  uint32_t units[kMaxShared / 64], steps[kMaxShared / 64], total = 0;
#pragma unroll
  for (int w = 0; w < kMaxShared / 64; ++w) {
    units[w] = steps[w] = 0;
    const int b = 64 * w + lane;
    if (b < a.B) {
      int q0;
      units[w] = units_of(queries_of(a, b, &q0), G, HG, row_tile);
      steps[w] = steps_of(length_of(a, b), step);
    }
    if (64 * w < a.B) total += (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(units[w] * steps[w], lane), 63);
  }
  const uint32_t size = max((total + share - 1) / share, (uint32_t)kMinSteps);  // steps of a piece
  uint32_t before = 0;
#pragma unroll
  for (int w = 0; w < kMaxShared / 64; ++w) {
    if (64 * w >= a.B) break;
    const uint32_t n = max((steps[w] + size - 1) / size, 1u);
    const uint32_t incl = wave_scan(units[w] * n, lane);
    const uint64_t past = __ballot(before + incl > id);
    if (past) {
      const int i = __builtin_ctzll(past);
      const uint32_t ni = (uint32_t)__builtin_amdgcn_readlane((int)n, i);
      const uint32_t start = before + (uint32_t)__builtin_amdgcn_readlane((int)(incl - units[w] * n), i);
      const uint32_t x = id - start, y = x / (uint32_t)HG, rt = y / ni;
      p->b = 64 * w + i;
      p->hg = (int)(x - y * HG);
      p->rt = (int)rt;
      p->k = (int)(y - rt * ni);
      p->n = (int)ni;
      p->first = start + rt * ni * HG + p->hg;
      return true;
    }
    before += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  }
  return false;
}

__device__ __forceinline__ float max_over_rows16(float v) {  // over the lanes l, l ^ 16, l ^ 32, l ^ 48
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
__device__ __forceinline__ float sum_over_rows16(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return __builtin_bit_cast(float, (uint32_t)b[0]) + __builtin_bit_cast(float, (uint32_t)b[1]);
}

// Two floats of a piece's result, coherent across the chiplets' caches.
__device__ __forceinline__ void store_agent(float* p, float x, float y) {
  const uint64_t v = __builtin_bit_cast(uint32_t, x) | (uint64_t)__builtin_bit_cast(uint32_t, y) << 32;
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_agent(const float* p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__builtin_bit_cast(float, (uint32_t)v), __builtin_bit_cast(float, (uint32_t)(v >> 32)));
}
__device__ __forceinline__ void store_pair(const KvAttnArgs& a, int64_t at, float x, float y) {
  const uint32_t lo = a.dtype == 1 ? f32_to_bf16_bits(x) : f32_to_f16_bits(x);
  const uint32_t hi = a.dtype == 1 ? f32_to_bf16_bits(y) : f32_to_f16_bits(y);
  *reinterpret_cast<uint32_t*>(a.out + at) = lo | (hi << 16);
}
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? kNegInf : (m + __builtin_log2f(l)) * 0.6931471805599453f;
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

// One 32-token tile of one KV head as loaded, untouched.
template <int D>
struct Tile {
  static constexpr int NB = D == 256 ? 2 : 1;   // cache blocks of a head
  static constexpr int KL = D / 64;             // 16-byte loads of a lane that cover the tile's K codes
  u4 k[KL];
  uint32_t v[8][NB];  // (D = 64: half words)
  uint32_t s[NB];     // lanes 0..31: K scale of token l, lanes 32..63: V scale of token l - 32
  uint32_t z;         // the zero-point byte beside it
  bool ok;            // the tile's page (small pages: the page of the lane's token) exists
};

// K codes of a tile pass through LDS: they are loaded as whole 64-byte rows (four
// lanes a token) and read as operands (16 tokens of one chunk).  Chunk j of token
// t sits at k_place, so that those 16 fall in different banks.
template <int D>
__device__ __forceinline__ int k_place(int t, int j) {
  return D == 64 ? j ^ (t >> 3 & 1) : D == 128 ? j ^ (t >> 2 & 3) : j ^ (t >> 1 & 7);
}
// Words of LDS a wave walks with: scales and zero-points, K codes.
template <int D>
constexpr int kWave = kMeta * Tile<D>::NB + 4 * D;

template <int D, int RT, int W, bool P32>
__global__ __launch_bounds__(64 * W, RT == 1 && D <= 128 ? W / 2 : W / 4) void kv_attn_kernel(KvAttnArgs a, int HW, int rtiles,
                                                                                             int urows, int share) {
  constexpr int NB = Tile<D>::NB;
  constexpr int NS = D / 32;  // MFMA steps of a score
  constexpr int SB = NS / NB;
  constexpr int NE = D / 16;  // MFMAs of an output tile: 16 channels each
  constexpr int KL = Tile<D>::KL, kChunks = D / 32, kTok = 64 / kChunks;  // 16-byte chunks of a token, tokens of a load
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4, ml = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int TW = W / HW, tg = wave / HW, hw = wave - tg * HW, step = 32 * TW;
  const int HG = a.Hkv / HW, G = a.Hq / a.Hkv;
  const uint32_t rowb = (uint32_t)a.Hkv * (D / 2);  // code bytes of a cache row
  const uint32_t nbt = (uint32_t)a.Hkv * D / 128, zb = (nbt + 1) / 2;
  const int lg = 31 - __builtin_clz(a.page);
  const int pages = (int)(a.S >> lg);
  float* meta = reinterpret_cast<float*>(lds) + wave * kWave<D>;
  u4* kd = reinterpret_cast<u4*>(meta + kMeta * NB);

  const Magic magic;

  Piece u;
  if (share) {
    if (!find_piece(a, blockIdx.x, share, G, HG, 16 * RT, step, lane, &u)) return;
  } else {
    const uint32_t x = blockIdx.x / (uint32_t)HG;
    u.hg = (int)(blockIdx.x - x * HG);
    u.b = (int)(x / (uint32_t)rtiles);
    u.rt = (int)(x - u.b * rtiles);
    u.k = 0;
    u.n = 1;
    u.first = blockIdx.x;
  }
  const int b = u.b, hg = u.hg;
  int q0;
  const int nq = queries_of(a, b, &q0);
  const int len = length_of(a, b);
  const int row0 = u.rt * (16 * RT), rows = nq * G;
  if (row0 >= rows) return;
  const uint32_t steps = steps_of(len, step);
  const int s0 = (int)((uint64_t)steps * u.k / (uint32_t)u.n), s1 = (int)((uint64_t)steps * (u.k + 1) / (uint32_t)u.n);
  const int h = hg * HW + hw;
  const int row1 = min(row0 + 16 * RT, rows) - 1;
  // of these rows' tokens: what the last row sees ends the walk, what the first
  // sees ends the tiles that need no mask
  const int t_begin = s0 * step;
  const int t_end = min((int)min((int64_t)s1 * step, (int64_t)len), len - nq + (int)((uint32_t)row1 / (uint32_t)G) + 1);
  const int low = min(t_end, len - nq + (int)((uint32_t)row0 / (uint32_t)G) + 1);

  // the wave's queries, as the B operand of the scores: lane (r, c) channels
  // 32 c + 8 j (D = 64: 16 c + 8 j) of each block, brought into fp16's range by
  // the power of two that takes the row's largest value into [1, 2)
  h8 qf[RT][NS];
  float f[RT];   // score of a row in units of log2: raw * f
  int lim[RT];   // tokens the row sees, of those of this walk
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const uint32_t row = min(row0 + 16 * t + r, rows - 1);  // rows past the end repeat the last, not stored
    const uint32_t qi = row / (uint32_t)G;
    lim[t] = min(t_end, len - nq + (int)qi + 1);
    const uint16_t* qp = a.q + (int64_t)(q0 + qi) * a.q_stride + (int64_t)(h * G + (int)(row - qi * G)) * D;
    u4 raw[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const int ch = D == 64 ? 16 * c + 8 * j : 128 * (j / 4) + 32 * c + 8 * (j % 4);
      raw[j] = *reinterpret_cast<const u4*>(qp + ch);
    }
    float x[NS][8], top_q = 0.0f;
    if (a.dtype == 1) {
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[j][e] = __builtin_bit_cast(float, e % 2 ? raw[j][e / 2] & 0xffff0000u : raw[j][e / 2] << 16);
    } else {
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] = (float)__builtin_bit_cast(h8, raw[j])[e];
    }
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) top_q = fmaxf(top_q, fabsf(x[j][e]));
    top_q = max_over_rows16(top_q);
    int ex = (int)(__builtin_bit_cast(uint32_t, top_q) >> 23) - 127;
    ex = min(max(ex, -126), 126);  // zeros, subnormals and infinities: the nearest power
    const float down = __builtin_bit_cast(float, (uint32_t)(127 - ex) << 23);
    const float up = __builtin_bit_cast(float, (uint32_t)(127 + ex) << 23);
    f[t] = a.scale * 1.4426950408889634f * up;
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[t][j][e] = (_Float16)(x[j][e] * down);
  }

  f4 acc[RT][NE];
  float m[RT], l[RT];  // weights are 2^(score - m); m follows the largest score + v_exp
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = kNegInf;
    l[t] = 0.0f;
#pragma unroll
    for (int e = 0; e < NE; ++e) acc[t][e] = f4{0, 0, 0, 0};
  }
  // V scales so far are at most v_top (fp16 bits) < 2^v_exp
  uint32_t v_top = 0;
  float v_exp = -25.0f;

  const uint32_t blk = (uint32_t)h * D / 128;  // first block of the head
  const int zshift = D == 256 ? 0 : (blk & 1) * 4;
  const int32_t* table = a.table + (int64_t)b * a.table_width;
  const uint8_t* kc = a.k_codes + (uint32_t)h * (D / 2);
  const uint8_t* vc = a.v_codes + (uint32_t)h * (D / 2);
  const uint16_t* sp = (lane < 32 ? a.k_s : a.v_s) + blk + (P32 ? ml * nbt : 0);
  const uint8_t* zp = (lane < 32 ? a.k_zp : a.v_zp) + blk / 2 + (P32 ? ml * zb : 0);
  const uint32_t k_at = 16 * (lane % kChunks) + (P32 ? lane / kChunks * rowb : 0);
  const uint32_t v_at = (D == 64 ? 2 : 4) * r + (P32 ? 4 * c * rowb : 0);

  // page entries of a tile: one of the whole tile (P32) or one of lane ml's token
  auto page_entry = [&](int tk) -> int {
    if constexpr (P32) return table[min(tk, t_end - 1) >> lg];
    return table[min(tk + ml, t_end - 1) >> lg];
  };
  // row of the tile's first token (P32) or of lane ml's token
  auto rows_of = [&](int tk, int pg, bool* ok) -> int {
    *ok = pg >= 0 && pg < pages;
    return *ok ? (pg << lg) + ((P32 ? tk : tk + ml) & (a.page - 1)) : 0;  // none: the first rows of the cache
  };
  auto load_k = [&](Tile<D>& T, int row) {
#pragma unroll
    for (int n = 0; n < NB; ++n) T.s[n] = (sp + (int64_t)row * nbt)[n];
    T.z = (zp + (int64_t)row * zb)[0];
    uint32_t at = k_at;  // a lane's offset from a scalar address (not folded into a 64-bit one outside the loop)
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      const uint8_t* p = kc + (int64_t)(P32 ? row + kTok * i : __shfl(row, kTok * i + lane / kChunks)) * rowb;
      if constexpr (P32) asm volatile("" : "+s"(p));
      T.k[i] = *reinterpret_cast<const u4*>(p + at);
    }
  };
  auto load_v = [&](Tile<D>& T, int row) {
    uint32_t at = v_at;
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = 16 * (i / 4) + i % 4;
      const uint8_t* p = vc + (int64_t)(P32 ? row + t : __shfl(row, t + 4 * c)) * rowb;
      if constexpr (P32) asm volatile("" : "+s"(p));  // the tile's rows: a scalar address
      p += at;
      if constexpr (D == 64) {
        T.v[i][0] = *reinterpret_cast<const uint16_t*>(p);
      } else {
#pragma unroll
        for (int n = 0; n < NB; ++n) T.v[i][n] = *reinterpret_cast<const uint32_t*>(p + 64 * n);
      }
    }
  };

  // Works on tile tk; K and V of the next tile (rows `row`) replace this one's as
  // soon as they are decoded.
  auto compute = [&](Tile<D>& T, int tk, int row, bool next_ok) {
    const bool ok = T.ok;
    // scales and zero-points through LDS to the lanes that need them, in the form
    // they need; a token that is not attended has 0 for all, whatever its cache
    // row holds
    const bool off = !ok || tk + ml >= t_end;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const uint32_t z = off ? 0u : (D == 256 ? T.z >> (4 * n) : T.z >> zshift) & 15u;
      const uint32_t sb = off ? 0u : T.s[n];
      const float sv = f16_bits_to_f32((uint16_t)sb);
      float* mn = meta + kMeta * n;
      mn[lane] = sv;  // K's, then V's
      const uint32_t z10 = z | 0x6400u, z6 = (z << 4) | 0x5400u;  // 1024 + z, 64 + z
      if (lane < 32) {
        *reinterpret_cast<u2*>(mn + 64 + 2 * ml) = u2{z10 * 0x00010001u, z6 * 0x00010001u};
      } else {
        reinterpret_cast<uint16_t*>(mn + 128)[ml] = (uint16_t)z10;
        reinterpret_cast<uint16_t*>(mn + 144)[ml] = (uint16_t)z6;
      }
      // a V scale above all so far (rare): the next power of two from the largest
      if (__ballot(lane >= 32 && sb > v_top)) {
        uint32_t top = lane >= 32 ? sb & 0x7fffu : 0u;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
        top = __builtin_amdgcn_readfirstlane(top);
        v_exp = (float)((int)(__builtin_bit_cast(uint32_t, f16_bits_to_f32((uint16_t)top)) >> 23) - 126);
        v_top = top >> 10 ? top | 0x3ffu : 0xffffffffu >> __builtin_clz(top);
      }
    }
    // tokens of small pages that do not exist, a bit each (P32: all or none)
    const uint32_t gone = P32 ? 0u : ~(uint32_t)__ballot(ok);
    const bool masked = tk + 32 > low || (P32 ? !ok : gone != 0);
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      const int t = kTok * i + lane / kChunks;
      kd[t * kChunks + k_place<D>(t, lane % kChunks)] = T.k[i];
    }
    f4 sc[RT][2][NB];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const int t16 = 16 * g + r;
        uint32_t kw[SB];
        if constexpr (D == 64) {
          const u2 w = reinterpret_cast<const u2*>(kd + t16 * kChunks + k_place<D>(t16, c / 2))[c % 2];
          kw[0] = w[0];
          kw[1] = w[1];
        } else {
          const u4 w = kd[t16 * kChunks + k_place<D>(t16, 4 * n + c)];
#pragma unroll
          for (int j = 0; j < 4; ++j) kw[j] = w[j];
        }
        const u2 z = *reinterpret_cast<const u2*>(meta + kMeta * n + 64 + 2 * (16 * g + r));
#pragma unroll
        for (int t = 0; t < RT; ++t) sc[t][g][n] = f4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < SB; ++j) {
          const u4 d = code_pairs(kw[j], z[0], z[1], magic);
#pragma unroll
          for (int t = 0; t < RT; ++t)
            sc[t][g][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, d), qf[t][SB * n + j],
                                                                 sc[t][g][n], 0, 0, 0);
        }
      }
    __builtin_amdgcn_sched_barrier(0);
    load_k(T, row);
    T.ok = next_ok;
    // scores times their token's scale
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      f4 ks[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) ks[n] = *reinterpret_cast<const f4*>(meta + kMeta * n + 16 * g + 4 * c);
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[t][g][0][i] *= ks[0][i];
          if constexpr (NB == 2) sc[t][g][0][i] = __builtin_fmaf(sc[t][g][1][i], ks[1][i], sc[t][g][0][i]);
        }
    }
    f4 vs[NB][2];
    u2 vz10[NB][2], vz6[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        vs[n][g] = *reinterpret_cast<const f4*>(meta + kMeta * n + 32 + 16 * g + 4 * c);
        vz10[n][g] = *reinterpret_cast<const u2*>(meta + kMeta * n + 128 + 8 * g + 2 * c);
        vz6[n][g] = *reinterpret_cast<const u2*>(meta + kMeta * n + 144 + 8 * g + 2 * c);
      }
    h8 pf[RT][NB];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float s8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) s8[i] = sc[t][i / 4][0][i % 4];
      if (masked) {
        const int seen = P32 && !ok ? 0 : lim[t] - tk;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = 16 * (i / 4) + 4 * c + i % 4;
          if (tok >= seen || (!P32 && (gone >> tok & 1))) s8[i] = kNegInf;
        }
      }
      float mx = s8[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s8[i]);
      mx = __builtin_fmaf(max_over_rows16(mx), f[t], v_exp);
      if (__ballot(mx > m[t] + kLag)) {
        const float mn = fmaxf(m[t], mx);
        const float al = m[t] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[t] - mn);
        m[t] = mn;
        l[t] *= al;
#pragma unroll
        for (int e = 0; e < NE; ++e) acc[t][e] *= al;
      }
      const float ms = m[t] == kNegInf ? 0.0f : m[t];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s8[i], f[t], -ms));
        l[t] += p;
#pragma unroll
        for (int n = 0; n < NB; ++n) pf[t][n][i] = (_Float16)(p * vs[n][i / 4][i % 4]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // O^T += V^T P^T, 16 channels an MFMA
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      // 1024 + z and 64 + z of the token pairs
      const u4 z10 = {vz10[n][0][0], vz10[n][0][1], vz10[n][1][0], vz10[n][1][1]};
      const u4 z6 = {vz6[n][0][0], vz6[n][0][1], vz6[n][1][0], vz6[n][1][1]};
#pragma unroll
      for (int half = 0; half < (D == 64 ? 1 : 2); ++half) {
        u4 d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // even (odd) channels of two tokens
          const u4 x = code_pairs(
              __builtin_amdgcn_perm(T.v[2 * i + 1][n], T.v[2 * i][n], half ? 0x07060302u : 0x05040100u), z10[i],
              z6[i], magic);
#pragma unroll
          for (int p = 0; p < 4; ++p) d[p][i] = x[p];
        }
        // MFMA e of a block: channel 8 m + e of row m (D = 64: channel
        // 8 (m / 2) + m % 2 + 2 e)
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const int e = D == 64 ? p : 8 * n + 2 * p + half;
            acc[t][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, d[p]), pf[t][n], acc[t][e], 0, 0, 0);
          }
      }
    }
  };

  Tile<D> tile;
  int tk = t_begin + 32 * tg;
  if (tk < t_end) {
    int row = rows_of(tk, page_entry(tk), &tile.ok);
    load_k(tile, row);
    load_v(tile, row);
    int pg = page_entry(tk + step);
    do {
      // past the end the next tile repeats real rows and is not used
      bool ok;
      row = rows_of(min(tk + step, (t_end - 1) & ~31), pg, &ok);
      pg = page_entry(tk + 2 * step);
      compute(tile, tk, row, ok);
      load_v(tile, row);
      tk += step;
    } while (tk < t_end);
  }

  // Waves of one head join through LDS: the largest reference point, every
  // wave's sums scaled to it, added in wave order.  Slab: the 16 rows of one row
  // tile and block, [row][channel] per wave.
  constexpr int DB = D < 128 ? D : 128, NEB = DB / 16;
  // indices made here, not kept in registers through the walk
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int re = tid & 15, ce = (tid & 63) >> 4;
  // pieces' results: [piece][head of the unit][row], (reference point, sum) and sums
  float* stats = static_cast<float*>(a.workspace) + kCounters;
  float* part = stats + (int64_t)2 * gridDim.x * HW * urows;
  float* slab = reinterpret_cast<float*>(lds);  // over what the waves walked with (they meet before it is written)
  float* stat = slab + W * (kWave<D> > 16 * DB ? kWave<D> : 16 * DB);  // [wave][2][16]
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (t) __syncthreads();
    const float lt = sum_over_rows16(l[t]);
    if (ce == 0) {
      stat[wave * 32 + re] = m[t];
      stat[wave * 32 + 16 + re] = lt;
    }
    __syncthreads();
    float M = kNegInf;
    for (int g = 0; g < TW; ++g) M = fmaxf(M, stat[(hw + HW * g) * 32 + re]);
    // a wave whose sum is 0 saw nothing (a NaN sum stays one)
    const float k = lt == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m[t] - M);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (n) __syncthreads();
#pragma unroll
      for (int e = 0; e < NEB; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int mrow = 4 * ce + i;
          const int ch = D == 64 ? 8 * (mrow / 2) + mrow % 2 + 2 * e : 8 * mrow + e;
          slab[wave * 16 * DB + re * DB + ch] = acc[t][NEB * n + e][i] * k;
        }
      __syncthreads();
      // a thread: two channels of one row and head
      constexpr uint32_t per_head = 16 * DB / 2;
      for (uint32_t x = tid; x < HW * per_head; x += 64 * W) {
        const int hx = x / per_head, rr = x % per_head / (DB / 2), ch = 2 * (x % (DB / 2));
        const uint32_t row = row0 + 16 * t + rr;
        if ((int)row > row1) continue;
        float o0 = 0.0f, o1 = 0.0f, Mr = kNegInf, L = 0.0f;
        for (int g = 0; g < TW; ++g) Mr = fmaxf(Mr, stat[(hx + HW * g) * 32 + rr]);
        for (int g = 0; g < TW; ++g) {
          const int wv = hx + HW * g;
          const float lw = stat[wv * 32 + 16 + rr];
          if (lw == 0.0f) continue;
          o0 += slab[wv * 16 * DB + rr * DB + ch];
          o1 += slab[wv * 16 * DB + rr * DB + ch + 1];
          L += lw * __builtin_amdgcn_exp2f(stat[wv * 32 + rr] - Mr);
        }
        const uint32_t qi = row / (uint32_t)G;
        const int64_t orow = (int64_t)(q0 + qi) * a.Hq + (hg * HW + hx) * G + (row - qi * G);
        if (u.n == 1) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          store_pair(a, orow * D + 128 * n + ch, o0 * inv, o1 * inv);
          if (a.lse && ch == 0 && n == 0) a.lse[orow] = lse_of(Mr, L);
        } else {
          const int64_t slot = ((int64_t)blockIdx.x * HW + hx) * urows + (row - row0);
          store_agent(part + slot * D + 128 * n + ch, o0, o1);
          if (ch == 0 && n == 0) store_agent(stats + 2 * slot, Mr, L);
        }
      }
    }
  }
  if (u.n == 1) return;

  // The last workgroup of a unit to arrive joins its pieces, in order: a wave a
  // row, D / 64 channels a lane, whose loads do not wait for one another.
  unsigned* counter = static_cast<unsigned*>(a.workspace) + u.first;
  if (!split_arrive(counter, u.n)) return;
  constexpr int C = D / 64;
  const int vrows = row1 - row0 + 1, ln = tid & 63;
  const int64_t hop = (int64_t)HG * HW * urows;  // from a piece's rows to the next one's
  for (int x = wave; x < HW * vrows; x += W) {
    const int hx = x / vrows, rr = x - hx * vrows;
    const int64_t slot = ((int64_t)u.first * HW + hx) * urows + rr;
    const float* st = stats + 2 * slot;
    float M = kNegInf;
    for (int k = ln; k < u.n; k += 64) M = fmaxf(M, load_agent(st + 2 * k * hop).x);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) M = fmaxf(M, __shfl_xor(M, d));
    float o[C], L = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = 0.0f;
    constexpr int U = D == 256 ? 8 : 16;  // pieces whose loads are in flight together
    for (int k0 = 0; k0 < u.n; k0 += U) {
      float2 ml[U], v[U][(C + 1) / 2];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int64_t at = slot + min(k0 + j, u.n - 1) * hop;  // past the end: the last again, not added
        ml[j] = load_agent(stats + 2 * at);
        const float* p = part + at * D + ln * C;
        if constexpr (C == 1) {
          v[j][0] = make_float2(split_load(p), 0.0f);
        } else {
#pragma unroll
          for (int i = 0; i < C / 2; ++i) v[j][i] = load_agent(p + 2 * i);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        // 0: the piece saw nothing, or is past the end
        const float w = ml[j].y == 0.0f || k0 + j >= u.n ? 0.0f : __builtin_amdgcn_exp2f(ml[j].x - M);
        L += ml[j].y * w;
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] += (i % 2 ? v[j][i / 2].y : v[j][i / 2].x) * w;
      }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const uint32_t row = row0 + rr, qi = row / (uint32_t)G;
    const int64_t orow = (int64_t)(q0 + qi) * a.Hq + (hg * HW + hx) * G + (row - qi * G);
    if constexpr (C == 1) {
      a.out[orow * D + ln] = a.dtype == 1 ? f32_to_bf16_bits(o[0] * inv) : f32_to_f16_bits(o[0] * inv);
    } else {
#pragma unroll
      for (int i = 0; i < C; i += 2) store_pair(a, orow * D + ln * C + i, o[i] * inv, o[i + 1] * inv);
    }
    if (a.lse && ln == 0) a.lse[orow] = lse_of(M, L);
  }
}

// Arrival counters of the units that are cut.
__global__ __launch_bounds__(256) void kv_attn_clear_kernel(unsigned* counters) {
  for (int i = threadIdx.x; i < kCounters; i += 256) counters[i] = 0;
}

template <int D>
size_t lds_bytes(int W) {
  constexpr int DB = D < 128 ? D : 128;
  return (size_t)W * ((kWave<D> > 16 * DB ? kWave<D> : 16 * DB) + 32) * 4;
}

template <int D, int RT, int W, bool P32>
hipError_t launch_main(const KvAttnArgs& a, const KvPlan& p, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  const size_t lds = lds_bytes<D>(W);
  hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&kv_attn_kernel<D, RT, W, P32>), lds, raised);
  if (e != hipSuccess) return e;
  if (p.share) kv_attn_clear_kernel<<<1, 256, 0, stream>>>(static_cast<unsigned*>(a.workspace));
  kv_attn_kernel<D, RT, W, P32><<<(unsigned)p.grid, 64 * W, lds, stream>>>(a, p.HW, p.rtiles, p.urows, p.share);
  return hipGetLastError();
}

template <int D, int RT, int W>
hipError_t launch_p(const KvAttnArgs& a, const KvPlan& p, hipStream_t stream) {
  return a.page % 32 == 0 ? launch_main<D, RT, W, true>(a, p, stream) : launch_main<D, RT, W, false>(a, p, stream);
}

template <int D>
hipError_t launch_rt(const KvAttnArgs& a, const KvPlan& p, hipStream_t stream) {
  return p.RT == 1 ? launch_p<D, 1, 8>(a, p, stream) : launch_p<D, 2, 8>(a, p, stream);
}

}  // namespace

size_t kv_attn_workspace_bytes(int64_t T, int B, int Hq, int Hkv, int D, int page, int64_t max_context,
                               int64_t max_queries) {
  const KvPlan p = plan_kv(T, B, Hq, Hkv, D, page, max_context, max_queries);
  return p.share ? (size_t)kCounters * 4 + (size_t)p.grid * p.HW * p.urows * (D + 2) * 4 : 0;
}

int describe_kv_attn(int64_t T, int B, int Hq, int Hkv, int D, int page, int64_t max_context, int64_t max_queries,
                     char* buf, size_t len) {
  const KvPlan p = plan_kv(T, B, Hq, Hkv, D, page, max_context, max_queries);
  return snprintf(buf, len, "kv_attn_kernel<D=%d, RT=%d, W=%d, P32=%d> grid=%lld block=%d heads=%d %s", D, p.RT, p.W,
                  page % 32 == 0 ? 1 : 0, (long long)p.grid, 64 * p.W, p.HW, p.share ? "pieces" : "whole units");
}

hipError_t launch_kv_attn(const KvAttnArgs& a, hipStream_t stream) {
  const KvPlan p = plan_kv(a.T, a.B, a.Hq, a.Hkv, a.D, a.page, a.max_context, a.max_queries);
  if (a.D == 64) return launch_rt<64>(a, p, stream);
  if (a.D == 128) return launch_rt<128>(a, p, stream);
  return launch_rt<256>(a, p, stream);
}

}  // namespace wq
