// Attention over the INT4 KV cache (gfx950).
//
// For a query row q (one query token and head) and the tokens t it sees,
//   out = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale * q.k_t - max),
// with k_t = s_t (c_t - z_t) and v_t alike, read from the codes in one pass: a
// running maximum and sum per row, no scores in memory.
//
// The matrix cores take the exact integers c - z in fp16 (four bits and a
// zero-point: |c - z| <= 15); the scale of a token multiplies its score in fp32
// (K) and its softmax weight in fp32 before that weight is rounded to fp16 (V).
// So the codes are decoded with the GEMV's four AND-ORs and four packed
// subtractions a word and nothing is rounded but q (bf16 rows are moved into
// fp16's range by a power of two) and the weights p_t s_t (to fp16, half a step
// of 2^-11 at most: their reference point is the largest score plus the exponent
// of the largest V scale so far, so the large ones lie near 1 for any scale).
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
// computes; a workgroup's waves take neighbouring KV heads of the same tokens
// (whole cache rows are read) or, for short contexts, different tiles of one
// head.  Contexts split across workgroups leave fp32 partial results that a
// second kernel joins.
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
constexpr int kMaxFlat = 256;  // sequences that a wave scans for its share

struct KvPlan {
  int HW;           // KV heads of a workgroup (its W / HW waves per head take different tiles)
  int RT;           // 16-row tiles of a wave
  int W;            // waves of a workgroup
  int rtiles;       // units along the query rows of one KV head
  int urows;        // query rows of a unit that a call can use
  int64_t grid;     // workgroups
  bool flat;        // shared out in equal runs of steps; else one unit a workgroup
};

// A unit is HW heads of one sequence and one tile of query rows; its steps are
// the runs of 32 W / HW tokens that its waves take together.
KvPlan plan_kv(int64_t T, int B, int Hq, int Hkv, int D, int page, int64_t max_context, int64_t max_queries) {
  KvPlan p;
  const int64_t G = Hq / Hkv, rows = max_queries * G;
  p.RT = rows <= 16 ? 1 : 2;
  p.W = 8;
  p.rtiles = (int)((rows + 16 * p.RT - 1) / (16 * p.RT));
  p.urows = (int)(rows < 16 * p.RT ? rows : 16 * p.RT);
  p.HW = Hkv % 4 == 0 ? 4 : Hkv % 2 == 0 ? 2 : 1;
  if (max_context <= 2048) p.HW = 1;
  const int64_t units = (int64_t)B * (Hkv / p.HW) * p.rtiles;
  const int64_t steps = (max_context + 32 * (p.W / p.HW) - 1) / (32 * (p.W / p.HW));
  const int64_t want = 512;
  // runs of at least four steps, so that joining them stays cheap
  const int64_t n = units * steps / 4 < want ? units * steps / 4 : want;
  p.flat = n > units && B <= kMaxFlat && units * steps < (int64_t(1) << 31);
  p.grid = p.flat ? n : units;
  return p;
}

// Equal shares of the steps of all units.  The shares follow from the lengths
// alone, which only the device knows: each wave scans them.
struct Shares {
  uint32_t total, n;  // steps of all units, workgroups that share them
  uint32_t* lds;      // [2][kMaxFlat]: steps before each sequence's units, steps of one of its units
};

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

// Every wave scans all of it and writes the same words, so none waits for
// another.  A share is at least four steps while there are that many.
__device__ __forceinline__ Shares scan_shares(const KvAttnArgs& a, uint32_t wgs, int HG, int row_tile, int step,
                                              int lane, uint32_t* lds) {
  Shares s;
  s.total = 0;
  s.lds = lds;
  const int G = a.Hq / a.Hkv;
  for (int w = 0; w < a.B; w += 64) {
    const int b = w + lane;
    uint32_t cost = 0, steps = 1;
    if (b < a.B) {
      int q0;
      const int nq = queries_of(a, b, &q0);
      steps = steps_of(length_of(a, b), step);
      cost = units_of(nq, G, HG, row_tile) * steps;
    }
    uint32_t run = cost;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t up = (uint32_t)__shfl_up((int)run, d);
      run += lane >= d ? up : 0u;
    }
    lds[w + lane] = s.total + run - cost;
    lds[kMaxFlat + w + lane] = steps;
    s.total += (uint32_t)__builtin_amdgcn_readlane((int)run, 63);
  }
  s.n = max(min(wgs, (s.total + 3) / 4), 1u);
  return s;
}
// First step of share i of n.
__device__ __forceinline__ uint32_t share_start(uint32_t total, uint32_t i, uint32_t n) {
  return (uint32_t)((uint64_t)total * i / n);
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

// Two fp16 pairs (c - z) of the nibbles 0, 4 and 1, 5 of a word: (1024 + c) and
// (64 + c) by OR-ing an exponent in (wq_device.h), less the same of z.  The
// exponents come in vector registers (`magic`): v_and_or_b32 takes one scalar
// operand and no literal.
struct Magic {
  uint32_t e10 = 0x64006400u, e6 = 0x54005400u;
  __device__ __forceinline__ Magic() {
    asm("" : "+v"(e10));
    asm("" : "+v"(e6));
  }
};
__device__ __forceinline__ uint32_t code_pair(uint32_t w, h2 z1024, const Magic& g) {
  return as_u32(as_h2((w & 0x000F000Fu) | g.e10) - z1024);
}
__device__ __forceinline__ uint32_t code_pair16(uint32_t w, h2 z64, const Magic& g) {
  return as_u32(as_h2((w & 0x00F000F0u) | g.e6) - z64);
}
__device__ __forceinline__ h2 zero1024(uint32_t zz) { return as_h2(zz | 0x64006400u); }
__device__ __forceinline__ h2 zero64(uint32_t zz) { return as_h2((zz << 4) | 0x54005400u); }

// One 32-token tile of one KV head as loaded, untouched.
template <int D>
struct Tile {
  static constexpr int NB = D == 256 ? 2 : 1;   // cache blocks of a head
  static constexpr int KW = D / 32;             // code words of a K lane and 16-token group
  uint32_t k[2][KW];
  uint32_t v[8][NB];  // (D = 64: half words)
  uint32_t s[NB];     // lanes 0..31: K scale of token l, lanes 32..63: V scale of token l - 32
  uint32_t z;         // the zero-point byte beside it
  bool ok;            // the tile's page (small pages: the page of the lane's token) exists
};

template <int D, int RT, int W, bool P32>
__global__ __launch_bounds__(64 * W, RT == 1 && D <= 128 ? W / 2 : W / 4) void kv_attn_kernel(KvAttnArgs a, int HW, int rtiles,
                                                                                             int urows, bool flat) {
  constexpr int NB = Tile<D>::NB;
  constexpr int NS = D / 32;  // MFMA steps of a score
  constexpr int SB = NS / NB;
  constexpr int NE = D / 16;  // MFMAs of an output tile: 16 channels each
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4, ml = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int TW = W / HW, tg = wave / HW, hw = wave - tg * HW, step = 32 * TW;
  const int HG = a.Hkv / HW, G = a.Hq / a.Hkv;
  const uint32_t rowb = (uint32_t)a.Hkv * (D / 2);  // code bytes of a cache row
  const uint32_t nbt = (uint32_t)a.Hkv * D / 128, zb = (nbt + 1) / 2;
  const int lg = 31 - __builtin_clz(a.page);
  const int pages = (int)(a.S >> lg);
  uint32_t* meta = lds + wave * (64 * NB);
  const Magic magic;

  // this workgroup's steps, counted over all units
  uint32_t at = 0, at_end = 1;
  uint32_t* share_lds = lds + W * 64 * NB;
  if (flat) {
    const Shares sh = scan_shares(a, gridDim.x, HG, 16 * RT, step, lane, share_lds);
    if (blockIdx.x >= sh.n) return;
    at = share_start(sh.total, blockIdx.x, sh.n);
    at_end = share_start(sh.total, blockIdx.x + 1, sh.n);
  }
  for (int seg = 0; at < at_end; ++seg) {
  int b, rt0, hg, s0 = 0, s1 = 0;
  bool whole = true;  // all of a unit's steps are here
  if (flat) {
    // the last sequence that starts at or before `at` and is not empty
    b = 0;
    for (int w = 0; w < a.B; w += 64) {
      const uint64_t le = __ballot(w + lane < a.B && share_lds[w + lane] <= at);
      if (le) b = w + 63 - __builtin_clzll(le);
    }
    const uint32_t before = __builtin_amdgcn_readfirstlane(share_lds[b]);
    const uint32_t steps = __builtin_amdgcn_readfirstlane(share_lds[kMaxFlat + b]);
    const uint32_t unit = (at - before) / steps;
    rt0 = (int)(unit / (uint32_t)HG);
    hg = (int)(unit % (uint32_t)HG);
    s0 = (int)(at - before - unit * steps);
    s1 = (int)min(steps, (uint32_t)s0 + (at_end - at));
    whole = s0 == 0 && s1 == (int)steps;
    at += s1 - s0;
  } else {
    uint32_t id = blockIdx.x;
    hg = (int)(id % (uint32_t)HG);
    id /= (uint32_t)HG;
    rt0 = (int)(id % (uint32_t)rtiles);
    b = (int)(id / (uint32_t)rtiles);
    at = 1;
  }
  int q0;
  const int nq = queries_of(a, b, &q0);
  const int len = length_of(a, b);
  if (!flat) s1 = (int)steps_of(len, step);
  const int row0 = rt0 * (16 * RT), rows = nq * G;
  if (row0 >= rows) return;
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
  const uint32_t k_at = (D == 64 ? 8 : 16) * c + (P32 ? r * rowb : 0);
  const uint32_t v_at = (D == 64 ? 2 : 4) * r + (P32 ? 4 * c * rowb : 0);

  // page entries of a tile: one of the whole tile (P32) or one of lane ml's token
  auto page_entry = [&](int tk) -> int {
    if constexpr (P32) return table[min(tk, t_end - 1) >> lg];
    return table[min(tk + ml, t_end - 1) >> lg];
  };
  auto load = [&](Tile<D>& T, int tk, int pg) {
    const uint8_t *kr[2], *vr[8];
    const bool page_ok = pg >= 0 && pg < pages;
    T.ok = page_ok;
    if constexpr (P32) {
      // the tile lies inside one page (none: it reads the first rows of the cache)
      const int64_t base = page_ok ? ((int64_t)pg << lg) + (tk & (a.page - 1)) : 0;
#pragma unroll
      for (int g = 0; g < 2; ++g) kr[g] = kc + (base + 16 * g) * rowb;
#pragma unroll
      for (int i = 0; i < 8; ++i) vr[i] = vc + (base + 16 * (i / 4) + i % 4) * rowb;
#pragma unroll
      for (int n = 0; n < NB; ++n) T.s[n] = (sp + base * nbt)[n];
      T.z = (zp + base * zb)[0];
    } else {
      const int own = !page_ok ? 0 : (pg << lg) + ((tk + ml) & (a.page - 1));
#pragma unroll
      for (int g = 0; g < 2; ++g) kr[g] = kc + (uint64_t)(uint32_t)__shfl(own, 16 * g + r) * rowb;
#pragma unroll
      for (int i = 0; i < 8; ++i) vr[i] = vc + (uint64_t)(uint32_t)__shfl(own, 16 * (i / 4) + 4 * c + i % 4) * rowb;
#pragma unroll
      for (int n = 0; n < NB; ++n) T.s[n] = (sp + (uint64_t)(uint32_t)own * nbt)[n];
      T.z = (zp + (uint64_t)(uint32_t)own * zb)[0];
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if constexpr (D == 64) {
        const u2 w = *reinterpret_cast<const u2*>(kr[g] + k_at);
        T.k[g][0] = w[0];
        T.k[g][1] = w[1];
      } else {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const u4 w = *reinterpret_cast<const u4*>(kr[g] + k_at + 64 * n);
#pragma unroll
          for (int j = 0; j < 4; ++j) T.k[g][4 * n + j] = w[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (D == 64) {
        T.v[i][0] = *reinterpret_cast<const uint16_t*>(vr[i] + v_at);
      } else {
#pragma unroll
        for (int n = 0; n < NB; ++n) T.v[i][n] = *reinterpret_cast<const uint32_t*>(vr[i] + v_at + 64 * n);
      }
    }
  };

  auto compute = [&](Tile<D>& T, int tk) {
    // scale (low half) and zero-point (bits 16..19) of every token and cache
    // through LDS to the lanes that need them; a token that is not attended has
    // scale and zero-point 0, whatever its cache row holds
    const bool off = !T.ok || tk + ml >= t_end;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const uint32_t z = (D == 256 ? T.z >> (4 * n) : T.z >> zshift) & 15u;
      const uint32_t w = off ? 0u : T.s[n] | (z << 16);
      meta[64 * n + lane] = w;
      // a V scale above all so far (rare): the next power of two from the largest
      if (__ballot(lane >= 32 && (w & 0xffffu) > v_top)) {
        uint32_t top = lane >= 32 ? w & 0x7fffu : 0u;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
        top = __builtin_amdgcn_readfirstlane(top);
        v_exp = (float)((int)(__builtin_bit_cast(uint32_t, f16_bits_to_f32((uint16_t)top)) >> 23) - 126);
        v_top = top >> 10 ? top | 0x3ffu : 0xffffffffu >> __builtin_clz(top);
      }
    }
    // tokens of small pages that do not exist, a bit each (P32: all or none)
    const uint32_t gone = P32 ? 0u : ~(uint32_t)__ballot(T.ok);
    const bool masked = tk + 32 > low || (P32 ? !T.ok : gone != 0);
    f4 sc[RT][2][NB];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const uint32_t zz = (meta[64 * n + 16 * g + r] >> 16) * 0x00010001u;
        const h2 z1 = zero1024(zz), z6 = zero64(zz);
#pragma unroll
        for (int t = 0; t < RT; ++t) sc[t][g][n] = f4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < SB; ++j) {
          const uint32_t w = T.k[g][SB * n + j], w8 = w >> 8;
          const u4 d = {code_pair(w, z1, magic), code_pair16(w, z6, magic), code_pair(w8, z1, magic), code_pair16(w8, z6, magic)};
#pragma unroll
          for (int t = 0; t < RT; ++t)
            sc[t][g][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, d), qf[t][SB * n + j],
                                                                 sc[t][g][n], 0, 0, 0);
        }
      }
    // scores times their token's K scale
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const u4 w = *reinterpret_cast<const u4*>(meta + 64 * n + 16 * g + 4 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = f16_bits_to_f32((uint16_t)w[i]);
#pragma unroll
          for (int t = 0; t < RT; ++t) sc[t][g][0][i] = n ? __builtin_fmaf(sc[t][g][n][i], s, sc[t][g][0][i]) : sc[t][g][0][i] * s;
        }
      }
    u4 vm[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int g = 0; g < 2; ++g) vm[n][g] = *reinterpret_cast<const u4*>(meta + 64 * n + 32 + 16 * g + 4 * c);
    h8 pf[RT][NB];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float s8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) s8[i] = sc[t][i / 4][0][i % 4];
      if (masked) {
        const int seen = P32 && !T.ok ? 0 : lim[t] - tk;
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
        for (int n = 0; n < NB; ++n) pf[t][n][i] = (_Float16)(p * f16_bits_to_f32((uint16_t)vm[n][i / 4][i % 4]));
      }
    }
    // O^T += V^T P^T, 16 channels an MFMA
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      h2 z1[4], z6[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t zz = __builtin_amdgcn_perm(vm[n][i / 2][2 * (i % 2) + 1], vm[n][i / 2][2 * (i % 2)], 0x07060302u);
        z1[i] = zero1024(zz);
        z6[i] = zero64(zz);
      }
#pragma unroll
      for (int half = 0; half < (D == 64 ? 1 : 2); ++half) {
        u4 d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // even (odd) channels of two tokens
          const uint32_t w = __builtin_amdgcn_perm(T.v[2 * i + 1][n], T.v[2 * i][n], half ? 0x07060302u : 0x05040100u);
          const uint32_t w8 = w >> 8;
          d[0][i] = code_pair(w, z1[i], magic);
          d[1][i] = code_pair16(w, z6[i], magic);
          d[2][i] = code_pair(w8, z1[i], magic);
          d[3][i] = code_pair16(w8, z6[i], magic);
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

  Tile<D> ta, tb;
  int tk = t_begin + 32 * tg;
  if (tk < t_end) {
    load(ta, tk, page_entry(tk));
    int pg = page_entry(tk + step);
    while (true) {
      // past the end the next tile repeats real rows and is not computed
      load(tb, min(tk + step, (t_end - 1) & ~31), pg);
      pg = page_entry(tk + 2 * step);
      compute(ta, tk);
      tk += step;
      if (tk >= t_end) break;
      load(ta, min(tk + step, (t_end - 1) & ~31), pg);
      pg = page_entry(tk + 2 * step);
      compute(tb, tk);
      tk += step;
      if (tk >= t_end) break;
    }
  }

  // Waves of one head join through LDS: the largest reference point, every
  // wave's sums scaled to it, added in wave order.  Slab: the 16 rows of one row
  // tile and block, [row][channel] per wave.
  constexpr int DB = D < 128 ? D : 128, NEB = DB / 16;
  float* slab = reinterpret_cast<float*>(lds) + W * 64 * NB + 2 * kMaxFlat;
  float* stat = slab + W * 16 * DB;  // [wave][2][16]
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (t || seg) __syncthreads();
    const float lt = sum_over_rows16(l[t]);
    if (c == 0) {
      stat[wave * 32 + r] = m[t];
      stat[wave * 32 + 16 + r] = lt;
    }
    __syncthreads();
    float M = kNegInf;
    for (int g = 0; g < TW; ++g) M = fmaxf(M, stat[(hw + HW * g) * 32 + r]);
    // a wave whose sum is 0 saw nothing (a NaN sum stays one)
    const float k = lt == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m[t] - M);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (n) __syncthreads();
#pragma unroll
      for (int e = 0; e < NEB; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int mrow = 4 * c + i;
          const int ch = D == 64 ? 8 * (mrow / 2) + mrow % 2 + 2 * e : 8 * mrow + e;
          slab[wave * 16 * DB + r * DB + ch] = acc[t][NEB * n + e][i] * k;
        }
      __syncthreads();
      // a thread: two channels of one row and head
      constexpr uint32_t per_head = 16 * DB / 2;
      for (uint32_t x = threadIdx.x; x < HW * per_head; x += 64 * W) {
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
        if (whole) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          const uint32_t lo = a.dtype == 1 ? f32_to_bf16_bits(o0 * inv) : f32_to_f16_bits(o0 * inv);
          const uint32_t hi = a.dtype == 1 ? f32_to_bf16_bits(o1 * inv) : f32_to_f16_bits(o1 * inv);
          *reinterpret_cast<uint32_t*>(a.out + orow * D + 128 * n + ch) = lo | (hi << 16);
          if (a.lse && ch == 0 && n == 0)
            a.lse[orow] = L == 0.0f ? kNegInf : (Mr + __builtin_log2f(L)) * 0.6931471805599453f;
        } else {
          // partial result: a workgroup has two at most, of its first and its last unit
          const int64_t slot = ((int64_t)(2 * blockIdx.x + (seg > 0)) * HW + hx) * urows + (row - row0);
          float* ws = static_cast<float*>(a.workspace);
          float2* stats = reinterpret_cast<float2*>(ws + (int64_t)2 * gridDim.x * HW * urows * D);
          *reinterpret_cast<float2*>(ws + slot * D + 128 * n + ch) = make_float2(o0, o1);
          if (ch == 0 && n == 0) stats[slot] = make_float2(Mr, L);
        }
      }
    }
  }
  }
}

// Joins the partial results of the units that several workgroups shared: a
// workgroup of four waves per query row.  It finds the shares as they did; the
// weights of up to 256 pieces at a time are made by a thread each; then wave w
// adds pieces w, w + 4, ..., whose loads do not wait for one another, and the four
// sums meet in LDS.
template <int D, int RT>
__global__ __launch_bounds__(256) void kv_attn_join_kernel(KvAttnArgs a, int HW, int step, int urows, uint32_t wgs) {
  constexpr int C = D / 64;
  __shared__ float wt[256], red[8], sum[4][D];
  __shared__ uint32_t shares[2 * kMaxFlat];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int HG = a.Hkv / HW, G = a.Hq / a.Hkv;
  uint32_t id = blockIdx.x;
  const int hq = id % (uint32_t)a.Hq;
  id /= (uint32_t)a.Hq;
  const int qi = id % (uint32_t)a.max_queries, b = id / (uint32_t)a.max_queries;
  int q0;
  if (qi >= queries_of(a, b, &q0)) return;
  const Shares sh = scan_shares(a, wgs, HG, 16 * RT, step, lane, shares);
  const uint32_t before = shares[b], steps = shares[kMaxFlat + b];
  const int kvh = hq / G, row = qi * G + hq % G, row0 = row / (16 * RT) * (16 * RT);
  const uint32_t u0 = before + (uint32_t)(row0 / (16 * RT) * HG + kvh / HW) * steps, u1 = u0 + steps;
  // the workgroups of its first and last step
  const uint32_t w0 = (uint32_t)(((uint64_t)(u0 + 1) * sh.n - 1) / sh.total);
  const uint32_t w1 = (uint32_t)(((uint64_t)u1 * sh.n - 1) / sh.total);
  if (w0 == w1) return;  // one workgroup had all of it
  const int n = (int)(w1 - w0) + 1;
  const int late = share_start(sh.total, w0, sh.n) < u0;  // for w0 it was the last unit, for the others the first
  const float* ws = static_cast<const float*>(a.workspace);
  const float2* stats = reinterpret_cast<const float2*>(ws + (int64_t)2 * wgs * HW * urows * D);
  const int in_slot = kvh % HW * urows + (row - row0);
  auto slot = [&](int s) -> int64_t { return (int64_t)(2 * (w0 + s) + (s == 0 ? late : 0)) * HW * urows + in_slot; };
  float M = kNegInf;
  for (int s = threadIdx.x; s < n; s += 256) M = fmaxf(M, stats[slot(s)].x);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) M = fmaxf(M, __shfl_xor(M, d));
  if (lane == 0) red[wave] = M;
  __syncthreads();
  M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float o[C], L = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = 0.0f;
  for (int s0 = 0; s0 < n; s0 += 256) {
    const int here = min(256, n - s0);
    if (s0) __syncthreads();
    if ((int)threadIdx.x < here) {
      const float2 ml = stats[slot(s0 + threadIdx.x)];
      const float k = ml.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ml.x - M);  // 0: the piece saw nothing
      wt[threadIdx.x] = k;
      L += ml.y * k;
    }
    __syncthreads();
#pragma unroll 4
    for (int s = wave; s < here; s += 4) {
      const float k = wt[s];
      const float* p = ws + slot(s0 + s) * D + lane * C;
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] += p[i] * k;
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) L += __shfl_xor(L, d);
  if (lane == 0) red[4 + wave] = L;
#pragma unroll
  for (int i = 0; i < C; ++i) sum[wave][lane * C + i] = o[i];
  __syncthreads();
  L = red[4] + red[5] + red[6] + red[7];
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const int64_t orow = (int64_t)(q0 + qi) * a.Hq + hq;
  for (int x = threadIdx.x; x < D; x += 256) {
    const float v = (sum[0][x] + sum[1][x] + sum[2][x] + sum[3][x]) * inv;
    a.out[orow * D + x] = a.dtype == 1 ? f32_to_bf16_bits(v) : f32_to_f16_bits(v);
  }
  if (a.lse && threadIdx.x == 0) a.lse[orow] = L == 0.0f ? kNegInf : (M + __builtin_log2f(L)) * 0.6931471805599453f;
}

template <int D>
size_t lds_bytes(int W) {
  constexpr int DB = D < 128 ? D : 128;
  return ((size_t)W * (64 * Tile<D>::NB + 16 * DB + 32) + 2 * kMaxFlat) * 4;
}

template <int D, int RT, int W, bool P32>
hipError_t launch_main(const KvAttnArgs& a, const KvPlan& p, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  const size_t lds = lds_bytes<D>(W);
  hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&kv_attn_kernel<D, RT, W, P32>), lds, raised);
  if (e != hipSuccess) return e;
  kv_attn_kernel<D, RT, W, P32><<<(unsigned)p.grid, 64 * W, lds, stream>>>(a, p.HW, p.rtiles, p.urows, p.flat);
  e = hipGetLastError();
  if (e != hipSuccess || !p.flat) return e;
  const int64_t rows = (int64_t)a.B * a.max_queries * a.Hq;
  kv_attn_join_kernel<D, RT><<<(unsigned)rows, 256, 0, stream>>>(a, p.HW, 32 * (W / p.HW), p.urows, (uint32_t)p.grid);
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
  return p.flat ? (size_t)2 * p.grid * p.HW * p.urows * (D + 2) * 4 : 0;
}

int describe_kv_attn(int64_t T, int B, int Hq, int Hkv, int D, int page, int64_t max_context, int64_t max_queries,
                     char* buf, size_t len) {
  const KvPlan p = plan_kv(T, B, Hq, Hkv, D, page, max_context, max_queries);
  return snprintf(buf, len, "kv_attn_kernel<D=%d, RT=%d, W=%d, P32=%d> grid=%lld block=%d heads=%d %s", D, p.RT, p.W,
                  page % 32 == 0 ? 1 : 0, (long long)p.grid, 64 * p.W, p.HW, p.flat ? "shared steps" : "whole units");
}

hipError_t launch_kv_attn(const KvAttnArgs& a, hipStream_t stream) {
  const KvPlan p = plan_kv(a.T, a.B, a.Hq, a.Hkv, a.D, a.page, a.max_context, a.max_queries);
  if (a.D == 64) return launch_rt<64>(a, p, stream);
  if (a.D == 128) return launch_rt<128>(a, p, stream);
  return launch_rt<256>(a, p, stream);
}

}  // namespace wq
