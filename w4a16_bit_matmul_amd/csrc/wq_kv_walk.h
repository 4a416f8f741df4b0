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
// fp32 before that weight is rounded (V).  So nothing is rounded but q (rows are
// moved into fp16's range by a power of two: values below 2^-14 of the row's
// largest lose bits) and the weights w_t = p_t s_t, both to fp16, the widest type of
// the matrix instructions of full rate.  A weight is off by 2^-11 of itself at most
// down to 2^-20 of the row's largest: the reference point of w_t is the largest score +
// power of two above s_t among the tokens that the row sees, less kLift.  (The largest
// score and the largest scale, of two tokens perhaps, would hide the other weights:
// with 2^24 between scales all of them became 0.)  The two blocks of a head of 256 have
// a reference point each.  Leaving 64 + z of half of the codes to the fp32 sums saves a
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
// one channel in a lane while a cache word holds eight channels of one token, the
// even ones in its low half and the odd ones in its high half: ds_read_b64_tr_b16
// transposes half words as it reads them from LDS, so a lane gets words of the
// same four channels of two tokens each.
//
// Reading is the bound: 2 (D/2 + 2.5 D/128) bytes a token and KV head.  A wave
// walks 32-token tiles: codes come as whole rows, 16 bytes a lane, pass through
// LDS, and the next tile's are in flight while it computes.  It takes as many
// neighbouring KV heads as fill a 128-byte line (two of 128 values): what a CU
// can have in flight is bounded by the lines of its 32 KB cache, and half-used
// lines halve it.  Decoding and the softmax come next, so heads with few rows (a
// decode step of 8 query heads a KV head, say) share a tile's 16 columns: each
// head's product has zeros for the others' columns, all of them add up in one
// accumulator, and one softmax serves all (64 contexts of up to 8K: heads of 64 in
// groups of four 63 us, 79 with a tile each; of 128 in groups of eight 110 and 113).
// The waves of a workgroup take different tiles of the same heads and join in LDS.
// Where sequences and heads are too few to fill the GPU evenly, all steps of all
// units are shared out equally; units that end up in several workgroups leave fp32
// results which a second kernel joins.
//
// 64 contexts of 4-8K tokens, 64 / 8 heads of 128: the walk 95-102 us, 4.3 TB/s (a copy
// reaches 5.0, reads alone 6.2-7.0; vector units 44 % and matrix cores 12 % busy),
// the join 8.  One of 131072: 35 and 6 us.  One of 201 tokens: 7 us, all latency.  With
// 9-16 rows of heads of 64 a wave takes half a line and another workgroup the other:
// 16 contexts of 1-9K, 25 us and 5, half of the 25 for the second reading.
#pragma once
#include <stdio.h>

#include "wq_attn.h"

namespace wq {
namespace {

constexpr int kShares = 512;     // workgroups that steps are shared out to
constexpr int kMaxShared = 256;  // sequences that a wave scans for its share
// words of a wave's scales, zero-points and V scales' powers of a tile and block, and 32
// more, so that the same words of two blocks lie in different banks
constexpr int kMeta = 224;

constexpr int kWaves = 4;

struct KvPlan {
  int HP;        // KV heads of a wave
  int PK;        // of them, heads that share a tile of 16 rows
  int RT;        // 16-row tiles of a head
  int rtiles;    // units along the query rows of one KV head
  int urows;     // query rows of a unit and head that a call can use
  bool chunk;    // many rows: the kernel of wq_kv_chunk.hip, RT its 16-row tiles
  bool flat;     // the steps of all units are shared out equally (else one unit a workgroup)
  int64_t grid;  // workgroups launched
};

// A unit is HP heads of one sequence and one tile of query rows; its steps are
// the runs of 32 kWaves tokens that a workgroup's waves take together.
// tree: of a draft tree's nodes, which the walk of this file always takes.
KvPlan plan_kv(int B, int Hq, int Hkv, int D, int64_t max_context, int64_t max_queries, bool tree) {
  KvPlan p;
  const int64_t G = Hq / Hkv, rows = max_queries * G;
  p.HP = p.PK = 1;
  p.RT = 2 * kChunkWaves;
  p.rtiles = (int)((rows + 16 * p.RT - 1) / (16 * p.RT));
  p.urows = 16 * p.RT;
  p.grid = (int64_t)B * Hkv * p.rtiles;
  p.flat = false;
  // Tiles of 128 rows once two workgroups a CU come of it (512 tokens over 16K of one
  // sequence, one a CU: 510 us, 455-465 with tiles of 32 rows; of two sequences 585 and
  // 789) and nearly all of their rows are used (64 sequences, 128 rows a head: 97 us
  // and 133; 72 rows: 91 and 75).  With heads of 256 (two sequences over 7-8K, 32 / 4
  // heads) 660 us and 588: decoded tiles of 128 KB leave it one workgroup a CU.
  p.chunk = !tree && D != 256 && p.grid >= kShares && 5 * ((rows + 31) / 32) >= 16 * p.rtiles;
  if (p.chunk) return p;
  // more than 16 rows: two tiles share the decoded codes (4 contexts of up to 4K
  // with 32 rows: 29 us, 32 with one; with heads of 256 two spill 432 bytes or more)
  // Of trees only where codes are many.  A step is one tile's vector instructions after
  // another's, so one tile a wave, in twice the workgroups, is faster until decoding them again
  // bounds (us, one and two; tiles x steps, heads of 128: 16 x 3 9.1 and 13.3, 128 x 16 21 and 24,
  // 128 x 32 27 and 27, 128 x 63 57 and 41, 256 x 16 23 and 29, 256 x 32 40 and 36, 512 x 8 20.4 and 21.0,
  // 1024 x 3 19 and 19, 1024 x 8 32 and 29; of 64: 16 x 3 10.4 and 16.0, 256 x 32 30.6 and 31.6, 256 x 63 60
  // and 49, 512 x 16 29 and 36, 1024 x 8 25 and 28).
  const int64_t tiles = (int64_t)B * Hkv * ((rows + 15) / 16);
  const int64_t steps = (max_context + 32 * kWaves - 1) / (32 * kWaves);
  const bool few = tree && tiles <= 65536 / D && tiles * steps * D <= 1 << 19;
  p.RT = rows <= 16 || D == 256 || few ? 1 : 2;
  p.rtiles = (int)((rows + 16 * p.RT - 1) / (16 * p.RT));
  p.urows = (int)(rows < 16 * p.RT ? rows : 16 * p.RT);
  // Whole 128-byte lines to a wave (two heads of 128; four of 64 if two of them share
  // a tile, for registers) once there is work for all CUs that way: 64 contexts of up
  // to 512 tokens 15.7 us, 16.7 without; of up to 8K 109 and 152, with heads of 64 in
  // groups of eight 65 and 75; 32 of up to 4K (4096 steps) 40 and 47.  Below, twice
  // the workgroups count more: 32 of up to 2K 32 us and 28 without.
  p.HP = D == 64 ? 2 : 1;
  const int line = 256 / D;
  const int64_t full = (int64_t)B * (Hkv / line) * p.rtiles;
  if (rows <= (D == 128 ? 16 : 8) && D != 256 && Hkv % line == 0 && (full >= 256 || full * steps >= 4096)) p.HP = line;
  while (2 * p.PK <= p.HP && 2 * p.PK * rows <= 16) p.PK *= 2;
  const int64_t units = (int64_t)B * (Hkv / p.HP) * p.rtiles;
  // Shares cost a joining kernel and a start for each unit that a workgroup takes
  // part in; what they win grows with the steps (units x steps, whole and shared:
  // 8 x 4 9.1 and 11.0 us, 8 x 8 13.2 and 11.1, 8 x 64 69 and 14; 128 x 8 13.6 and
  // 18.8, 128 x 16 37 and 32; 256 x 16 39 and 43, 256 x 32 67 and 58, 256 x 64 154 and
  // 110; 800 x 16 98 and 108).  Two workgroups a CU.
  const int64_t n = units * steps < kShares ? units * steps : kShares;
  p.flat = units < 2 * kShares && steps >= 8 && 2 * units <= steps * steps && B <= kMaxShared &&
           units * steps < (int64_t)1 << 31;  // steps are counted in 32 bits
  p.grid = p.flat ? n : units;
  return p;
}

// Units of sequence b and steps of each (one at least: a row that sees nothing
// is written too).
__device__ __forceinline__ uint32_t units_of(int nq, int G, int HG, int row_tile) {
  return (uint32_t)HG * ((uint32_t)(nq * G + row_tile - 1) / (uint32_t)row_tile);
}
__device__ __forceinline__ uint32_t steps_of(int len, int step) {
  return max((uint32_t)(len + step - 1) / (uint32_t)step, 1u);
}

size_t walk_workspace_bytes(const KvPlan& p, int D) { return p.flat ? (size_t)2 * p.grid * p.HP * p.urows * (D + 2) * 4 : 0; }
int describe_walk(const KvPlan& p, int D, int page, char* buf, size_t len) {
  return snprintf(buf, len, "kv_attn_kernel<D=%d, HP=%d, RT=%d, PK=%d, P32=%d> grid=%lld block=%d %s", D, p.HP, p.RT, p.PK,
                  page % 32 == 0 ? 1 : 0, (long long)p.grid, 64 * kWaves, p.flat ? "shares" : "whole units");
}

// Equal shares of the steps of all units: with n workgroups and total = q n + r
// steps the first r take q + 1, the others q.  They follow from the lengths alone,
// which only the device knows: every wave scans all of them and writes the same
// words to LDS, so none waits for another.
struct Shares {
  uint32_t n, q, r;
};
struct ShareLds {  // of every sequence
  uint32_t before[kMaxShared];  // steps before its units
  uint32_t steps[kMaxShared];   // steps of each of them
  int32_t len[kMaxShared], q0[kMaxShared], nq[kMaxShared], all[kMaxShared];
};
__device__ __forceinline__ Shares scan_shares(const KvAttnArgs& a, uint32_t wgs, int HG, int row_tile, int step, int lane,
                                              ShareLds* lds) {
  uint32_t total = 0;
  const int G = a.Hq / a.Hkv;
  for (int w = 0; w < a.B; w += 64) {
    const int b = w + lane;
    uint32_t cost = 0, steps = 1;
    Queries qs{0, 0, 0};
    int len = 0;
    if (b < a.B) {
      qs = queries_of(a, b);
      len = length_of(a, b);
      steps = steps_of(len, step);
      cost = units_of(qs.n, G, HG, row_tile) * steps;
    }
    uint32_t run = cost;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t up = (uint32_t)__shfl_up((int)run, d);
      run += lane >= d ? up : 0u;
    }
    lds->before[b] = total + run - cost;
    lds->steps[b] = steps;
    lds->len[b] = len;
    lds->q0[b] = qs.q0;
    lds->nq[b] = qs.n;
    lds->all[b] = qs.all;
    total += (uint32_t)__builtin_amdgcn_readlane((int)run, 63);
  }
  Shares s;
  s.n = max(min(wgs, total), 1u);
  s.q = total / s.n;
  s.r = total - s.q * s.n;
  return s;
}
__device__ __forceinline__ uint32_t share_start(const Shares& s, uint32_t i) { return s.q * i + min(i, s.r); }
__device__ __forceinline__ uint32_t share_of(const Shares& s, uint32_t at) {  // the share that holds a step
  const uint32_t long_end = (s.q + 1) * s.r;
  return at < long_end ? at / (s.q + 1) : s.r + (at - long_end) / s.q;
}

// Over the lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_over_rows16(float v) {
  const uint32_t w = __builtin_bit_cast(uint32_t, max_over_halves(v));
  auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
__device__ __forceinline__ float sum_over_rows16(float v) {
  const uint32_t w = __builtin_bit_cast(uint32_t, sum_over_halves(v));
  auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return __builtin_bit_cast(float, (uint32_t)b[0]) + __builtin_bit_cast(float, (uint32_t)b[1]);
}

__device__ __forceinline__ void store_pair(const KvAttnArgs& a, int64_t at, float x, float y) {
  *reinterpret_cast<uint32_t*>(a.out + at) = pack_out(a.dtype, x, y);
}

// What a wave covers of a cache row, and one 32-token tile of it as loaded.
template <int D, int HP>
struct Tile {
  static constexpr int NB = HP * D / 128;         // cache blocks
  static constexpr int kChunks = HP * D / 32;     // 16-byte chunks of a token's codes
  static constexpr int kTok = 64 / kChunks;       // tokens of one 16-byte load a lane
  static constexpr int KL = 32 / kTok;            // such loads
  u4 k[KL], v[KL];
  uint32_t s;  // scales of the blocks (16 bits each): lanes 0..31 K's of token l, lanes 32..63 V's of token l - 32
  uint32_t z;  // the zero-point byte beside them
  bool ok;     // the tile's page (small pages: the page of the lane's token) exists
};

// The codes of a tile pass through LDS: they are loaded as whole rows (4 or 8
// lanes a token) and read as operands: K's 16 tokens of one chunk, V's 8 bytes of
// a token a lane, four tokens of 64 channels, which the reading instruction
// transposes.  Chunk j of token t sits where the lanes that read together fall in
// different banks.
template <int CHUNKS>
__device__ __forceinline__ int k_place(int t, int j) {
  return CHUNKS == 4 ? j ^ (t >> 2 & 3) : j ^ (t >> 1 & 7);
}
template <int CHUNKS>
__device__ __forceinline__ int v_place(int t, int j) {
  return CHUNKS == 4 ? j ^ 2 * (t >> 2 & 1) : j ^ 2 * (t >> 1 & 3);
}
// Words of LDS: a wave's scales, zero-points and codes of a tile; over them, at
// the end, its results of one row tile and block; then the waves' statistics and
// the shares.
template <int D, int HP>
constexpr int kWalk = kMeta * Tile<D, HP>::NB + 2 * 128 * Tile<D, HP>::kChunks;
template <int D>
constexpr int kSlabRow = (D < 128 ? D : 128) + 4;  // padded: rows in different banks
template <int D>
constexpr int kSlab = 16 * kSlabRow<D>;
template <int D, int HP>
constexpr int kPerWave = kWalk<D, HP> > kSlab<D> ? kWalk<D, HP> : kSlab<D>;
template <int D, int HP>
constexpr int lds_words = kWaves * (kPerWave<D, HP> + 32) + sizeof(ShareLds) / 4;

template <int D, int HP, int RT, int PK, bool P32, bool TREE>
__global__ __launch_bounds__(64 * kWaves, 2) void kv_attn_kernel(KvAttnArgs a, int rtiles, int urows, bool flat) {
  using T = Tile<D, HP>;
  constexpr int NB = T::NB;
  constexpr int X = HP / PK * RT;         // row tiles of a wave: tile x has rows of heads x / RT * PK + sub
  constexpr int PR = 16 / PK;             // rows of a head in a tile
  constexpr int NH = D == 256 ? 2 : 1;    // blocks of a head
  constexpr int NS = D / 32;              // MFMA steps of a score
  constexpr int NE = D / 16;              // MFMAs of an output tile: 16 channels each
  constexpr int kStep = 32 * kWaves;
  // Where a bound of a row's reference points is looked at first, the largest score plus
  // the largest power of V's scales so far: with the two points of a head of 256 (512
  // tokens each over 7-8K of two sequences, 32 / 4 heads: 639 us, 671 without).  Elsewhere
  // it costs as much as it saves (512 tokens over 16K of one sequence, 64 / 8 heads of 128:
  // 460 and 467; 4 contexts of up to 4K with 32 rows 28.1 and 27.0; one of 201 tokens 7.0
  // and 6.8 us).
  constexpr bool kBounded = D == 256;
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4, ml = lane & 31;
  const int sub = r / PR;  // (0 unless heads share a tile)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int HG = a.Hkv / HP, G = a.Hq / a.Hkv;
  const uint32_t rowb = (uint32_t)a.Hkv * (D / 2);  // code bytes of a cache row
  const uint32_t nbt = (uint32_t)a.Hkv * D / 128, zb = (nbt + 1) / 2;
  const int lg = 31 - __builtin_clz(a.page);
  const int pages = (int)(a.S >> lg);
  float* meta = reinterpret_cast<float*>(lds) + wave * kWalk<D, HP>;
  u4* kd = reinterpret_cast<u4*>(meta + kMeta * NB);
  u4* vd = kd + 32 * T::kChunks;
  float* slab = reinterpret_cast<float*>(lds);
  float* stat = slab + kWaves * kPerWave<D, HP>;  // [wave][2][16]
  ShareLds* shares = reinterpret_cast<ShareLds*>(lds + kWaves * (kPerWave<D, HP> + 32));
  const Magic magic;

  const uint32_t wg = blockIdx.x;

  // this workgroup's steps, counted over all units
  uint32_t at = 0, at_end = 1;
  Shares sh{1, 1, 0};
  if (flat) {
    sh = scan_shares(a, gridDim.x, HG, 16 * RT, kStep, lane, shares);
    if (wg >= sh.n) return;
    at = share_start(sh, wg);
    at_end = share_start(sh, wg + 1);
  }
  for (int seg = 0; at < at_end; ++seg) {
    int b, rt, hg, s0 = 0, s1;
    uint32_t u0 = 0, steps = 1;  // first step and steps of the unit
    if (flat) {
      // the last sequence whose units start at or before `at` (an empty one has
      // the start of the next)
      b = 0;
      for (int w = 0; w < a.B; w += 64) {
        const uint64_t le = __ballot(w + lane < a.B && shares->before[w + lane] <= at);
        if (le) b = w + 63 - __builtin_clzll(le);
      }
      const uint32_t first = __builtin_amdgcn_readfirstlane(shares->before[b]);
      steps = __builtin_amdgcn_readfirstlane(shares->steps[b]);
      const uint32_t unit = (at - first) / steps;
      rt = (int)(unit / (uint32_t)HG);
      hg = (int)(unit - (uint32_t)rt * HG);
      u0 = first + unit * steps;
      s0 = (int)(at - u0);
      s1 = (int)min(steps, (uint32_t)s0 + (at_end - at));
      at += s1 - s0;
    } else {
      const uint32_t x = wg / (uint32_t)HG;
      hg = (int)(wg - x * HG);
      b = (int)(x / (uint32_t)rtiles);
      rt = (int)(x - (uint32_t)b * rtiles);
      at = 1;
    }
    int q0, nq, before, len;  // before: the first query sees tokens 0..before
    if (flat) {
      q0 = __builtin_amdgcn_readfirstlane(shares->q0[b]);
      nq = __builtin_amdgcn_readfirstlane(shares->nq[b]);
      len = __builtin_amdgcn_readfirstlane(shares->len[b]);
      before = len - __builtin_amdgcn_readfirstlane(shares->all[b]);
    } else {
      const Queries qs = queries_of(a, b);
      q0 = qs.q0;
      nq = qs.n;
      len = length_of(a, b);
      before = len - qs.all;
      s1 = (int)(steps = steps_of(len, kStep));
    }
    const bool whole = s0 == 0 && s1 == (int)steps;
    const int row0 = rt * (16 * RT), rows = nq * G;
    if (row0 >= rows) return;
    const int row1 = min(row0 + 16 * RT, rows) - 1;
    // of these rows' tokens: what the last row sees ends the walk, what the first
    // sees ends the tiles that need no mask
    const int t_begin = s0 * kStep;
    const int t_end = TREE ? (int)min((int64_t)s1 * kStep, (int64_t)len)
                           : min((int)min((int64_t)s1 * kStep, (int64_t)len), before + (int)((uint32_t)row1 / (uint32_t)G) + 1);
    const int low = min(t_end, TREE ? max(before, 0) : before + (int)((uint32_t)row0 / (uint32_t)G) + 1);

    const uint32_t blk = (uint32_t)hg * HP * D / 128;  // first block of the wave's heads
    const int32_t* table = a.table + (int64_t)b * a.table_width;
    const uint8_t* kc = a.k_codes + (uint32_t)hg * (HP * D / 2);
    const uint8_t* vc = a.v_codes + (uint32_t)hg * (HP * D / 2);
    int ln = lane;  // per-lane offsets are made here for each unit, not kept through the loop over units
    asm volatile("" : "+v"(ln));
    const uint16_t* sp = (ln < 32 ? a.k_s : a.v_s) + blk + (P32 ? (ln & 31) * nbt : 0);
    const uint8_t* zp = (ln < 32 ? a.k_zp : a.v_zp) + blk / 2 + (P32 ? (ln & 31) * zb : 0);
    const uint32_t c_at = 16 * (ln % T::kChunks) + (P32 ? ln / T::kChunks * rowb : 0);

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
    auto load_codes = [&](u4 (&to)[T::KL], const uint8_t* from, int row) {
      uint32_t off = c_at;  // a lane's offset from a scalar address (not folded into a 64-bit one outside the loop)
      asm volatile("" : "+v"(off));
#pragma unroll
      for (int i = 0; i < T::KL; ++i) {
        const int at_row = P32 ? row + T::kTok * i : __shfl(row, T::kTok * i + lane / T::kChunks);
        const uint8_t* p = from + (int64_t)at_row * rowb;
        if constexpr (P32) asm volatile("" : "+s"(p));
        to[i] = *reinterpret_cast<const u4*>(p + off);
      }
    };
    auto load = [&](T& t, int row) {
      const uint16_t* s = sp + (int64_t)row * nbt;
      if constexpr (NB == 2) __builtin_memcpy(&t.s, s, 4);
      else t.s = *s;
      t.z = (zp + (int64_t)row * zb)[0];
      load_codes(t.k, kc, row);
      load_codes(t.v, vc, row);
    };

    T tile;
    int tk = t_begin + 32 * wave, row = 0, pg = 0;
    if (tk < t_end) {
      row = rows_of(tk, page_entry(tk), &tile.ok);
      load(tile, row);
      pg = page_entry(tk + kStep);
    }

    // the wave's queries, as the B operand of the scores: lane (r, c) channels
    // 32 c + 8 j (D = 64: 16 c + 8 j) of each block, brought into fp16's range by
    // the power of two that takes the row's largest value into [1, 2)
    h8 qf[HP * RT][NS];
    float f[X];   // score of a row in units of log2: raw * f
    int lim[RT];  // tokens the row sees, of those of this walk (TREE: the row's node, whose mask says which)
#pragma unroll
    for (int x = 0; x < HP * RT; ++x) {
      const int t = x % RT;
      const uint32_t qrow = min(row0 + 16 * t + r % PR, rows - 1);  // rows past the end repeat the last, not stored
      const uint32_t qi = qrow / (uint32_t)G;
      lim[t] = TREE ? (int)qi : min(t_end, before + (int)qi + 1);
      const int head = (hg * HP + x / RT) * G + (int)(qrow - qi * G);
      const uint16_t* qp = a.q + (int64_t)(q0 + qi) * a.q_stride + (int64_t)head * D;
      u4 raw[NS];
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const int ch = D == 64 ? 16 * c + 8 * j : 128 * (j / 4) + 32 * c + 8 * (j % 4);
        raw[j] = *reinterpret_cast<const u4*>(qp + ch);
      }
      float y[NS][8], top_q = 0.0f;
#pragma unroll
      for (int j = 0; j < NS; ++j) widen8(raw[j], a.dtype, y[j]);
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) top_q = fmaxf(top_q, fabsf(y[j][e]));
      const RowPower pw = row_power(max_over_rows16(top_q));
      // heads that share a tile: 0 in the columns of the others
      const bool mine = PK == 1 || x % PK == sub;
      if (mine) f[x / PK] = score_factor(a.scale, pw.up);
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) qf[x][j][e] = mine ? (_Float16)(y[j][e] * pw.down) : (_Float16)0.0f;
    }

    f4 acc[X][NE];
    // weights are 2^(score - m); m follows the largest score + V scale's power of each
    // block of the head, l goes by the first one's
    float m[X][NH], l[X];
#pragma unroll
    for (int x = 0; x < X; ++x) {
#pragma unroll
      for (int n = 0; n < NH; ++n) m[x][n] = kNegInf;
      l[x] = 0.0f;
#pragma unroll
      for (int e = 0; e < NE; ++e) acc[x][e] = f4{0, 0, 0, 0};
    }

    float v_top[NB];  // (kBounded) the largest power of each block so far
#pragma unroll
    for (int n = 0; n < NB; ++n) v_top[n] = kNoPower;

    // Works on tile tk; the next tile (rows `next`) is loaded as soon as this one
    // lies in LDS.
    auto compute = [&](int next, bool next_ok) {
      const bool ok = tile.ok;
      // scales and zero-points through LDS to the lanes that need them, in the
      // form they need; a token that is not attended has 0 for all, whatever its
      // cache row holds
      const bool off = !ok || tk + ml >= t_end;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const int zshift = NB == 2 ? 4 * n : (int)(blk & 1) * 4;
        const uint32_t z = off ? 0u : (tile.z >> zshift) & 15u;
        const uint32_t sb = off ? 0u : (tile.s >> (16 * n)) & 0xffffu;
        const float sv = f16_bits_to_f32((uint16_t)sb);
        float* mn = meta + kMeta * n;
        // K's, then V's.  TREE: an infinite K scale as NaN, a score that every row that sees the token takes over
        // (infinite, the score may be -inf and the token gone)
        mn[lane] = TREE && lane < 32 && !(fabsf(sv) <= 65504.0f) ? __builtin_nanf("") : sv;
        const uint32_t z10 = z | 0x6400u, z6 = (z << 4) | 0x5400u;  // 1024 + z, 64 + z
        if (lane < 32) {
          *reinterpret_cast<u2*>(mn + 64 + 2 * ml) = u2{z10 * 0x00010001u, z6 * 0x00010001u};
        } else {
          reinterpret_cast<uint16_t*>(mn + 128)[ml] = (uint16_t)z10;
          reinterpret_cast<uint16_t*>(mn + 144)[ml] = (uint16_t)z6;
          mn[160 + ml] = scale_power(sv);
        }
        if (kBounded) raise_top(v_top[n], lane < 32 ? kNoPower : scale_power(sv));
      }
      // tokens of small pages that do not exist, a bit each (P32: all or none)
      const uint32_t gone = P32 ? 0u : ~(uint32_t)__ballot(ok);
      const bool masked = tk + 32 > low || (P32 ? !ok : gone != 0);
#pragma unroll
      for (int i = 0; i < T::KL; ++i) {
        const int t = T::kTok * i + lane / T::kChunks;
        kd[t * T::kChunks + k_place<T::kChunks>(t, lane % T::kChunks)] = tile.k[i];
        vd[t * T::kChunks + v_place<T::kChunks>(t, lane % T::kChunks)] = tile.v[i];
      }
      __builtin_amdgcn_sched_barrier(0);
      load(tile, next);
      tile.ok = next_ok;
      // heads (those that share a tile together) in turn: scores, softmax of their row
      // tiles, then O^T += V^T P^T
#pragma unroll
      for (int hp = 0; hp < HP / PK; ++hp) {
        f4 sc[RT][2][NH];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int y = 0; y < PK; ++y)
#pragma unroll
            for (int n = 0; n < NH; ++n) {
              const int p = hp * PK + y, t16 = 16 * g + r, blkn = D == 64 ? p / 2 : p + n;
              uint32_t kw[NS / NH];
              if constexpr (D == 64) {
                const u4* at16 = kd + t16 * T::kChunks + k_place<T::kChunks>(t16, 2 * p + c / 2);
                const u2 w = reinterpret_cast<const u2*>(at16)[c % 2];
                kw[0] = w[0];
                kw[1] = w[1];
              } else {
                const u4 w = kd[t16 * T::kChunks + k_place<T::kChunks>(t16, 4 * (p + n) + c)];
#pragma unroll
                for (int j = 0; j < 4; ++j) kw[j] = w[j];
              }
              const u2 z = *reinterpret_cast<const u2*>(meta + kMeta * blkn + 64 + 2 * t16);
#pragma unroll
              for (int t = 0; t < RT; ++t)
                if (y == 0) sc[t][g][n] = f4{0, 0, 0, 0};
#pragma unroll
              for (int j = 0; j < NS / NH; ++j) {
                const u4 d = code_pairs(kw[j], z[0], z[1], magic);
#pragma unroll
                for (int t = 0; t < RT; ++t)
                  sc[t][g][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                      __builtin_bit_cast(h8, d), qf[p * RT + t][NS / NH * n + j], sc[t][g][n], 0, 0, 0);
              }
            }
        const int hb = D == 64 ? (hp * PK + sub) / 2 : hp * PK + sub;  // (first) block of the lane's head
        const float* mh = meta + kMeta * hb;
        h8 pf[RT][NH];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const int x = hp * RT + t;
          float s8[8];
          // scores times their token's scale
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int n = 0; n < NH; ++n) {
              const f4 ks = *reinterpret_cast<const f4*>(mh + kMeta * n + 16 * g + 4 * c);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float& v = s8[4 * g + i];
                v = n == 0 ? sc[t][g][n][i] * ks[i] : __builtin_fmaf(sc[t][g][n][i], ks[i], v);
              }
            }
          uint32_t miss = 0;  // TREE: bit i: the row does not see token i of the tile
          if (masked) {
            if constexpr (TREE) {
              miss = ~(uint32_t)tree_window(a, q0 + lim[t], tk - before) | gone;
              if (tk + 32 > t_end) miss |= 0xffffffffu << (t_end - tk);
              if (P32 && !ok) miss = 0xffffffffu;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int tok = 16 * (i / 4) + 4 * c + i % 4;
                if (miss >> tok & 1) s8[i] = kNegInf;
              }
            } else {
              const int seen = P32 && !ok ? 0 : lim[t] - tk;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int tok = 16 * (i / 4) + 4 * c + i % 4;
                if (tok >= seen || (!P32 && (gone >> tok & 1))) s8[i] = kNegInf;
              }
            }
          }
          // reference points: the largest score + power of its token's V scale
          float top = kNegInf;
          if (kBounded) {
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, s8[i]);
            top = max_over_rows16(top);
          }
#pragma unroll
          for (int n = 0; n < NH; ++n) {
            if (kBounded) {
              if (!__ballot(__builtin_fmaf(top, f[x], v_top[n]) > m[x][n] + (kLag + kLift))) continue;
            }
            float mx = kNegInf;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const f4 v = *reinterpret_cast<const f4*>(mh + kMeta * n + 160 + 16 * g + 4 * c);
#pragma unroll
              for (int i = 0; i < 4; ++i) mx = fmaxf(mx, __builtin_fmaf(s8[4 * g + i], f[x], v[i]));
            }
            mx = max_over_rows16(mx) - kLift;
            if (__ballot(mx > m[x][n] + kLag)) {
              const float mn = fmaxf(m[x][n], mx);
              const float al = m[x][n] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[x][n] - mn);
              m[x][n] = mn;
              if (n == 0) l[x] *= al;
#pragma unroll
              for (int e = 0; e < NE / NH; ++e) acc[x][NE / NH * n + e] *= al;
            }
          }
          const float ms = m[x][0] == kNegInf ? 0.0f : m[x][0];
          // the second block's weights, from the first one's
          const float up = NH == 1 || m[x][0] == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(ms - m[x][NH - 1]);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            f4 vs[NH];
#pragma unroll
            for (int n = 0; n < NH; ++n) vs[n] = *reinterpret_cast<const f4*>(mh + kMeta * n + 32 + 16 * g + 4 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s8[4 * g + i], f[x], -ms));
              l[x] += w;
#pragma unroll
              for (int n = 0; n < NH; ++n) pf[t][n][4 * g + i] = (_Float16)((n == 0 ? w : w * up) * vs[n][i]);
            }
          }
          if (TREE && masked) {  // a weight of 0 times the scale of a node of another branch, which may be infinite or NaN
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int n = 0; n < NH; ++n)
                if (miss >> (16 * (i / 4) + 4 * c + i % 4) & 1) pf[t][n][i] = (_Float16)0.0f;
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int y = 0; y < PK; ++y) {
          const int p = hp * PK + y;
          h8 pm[RT][NH];  // (a shared tile: the weights of this head's rows)
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int n = 0; n < NH; ++n) {
              u4 w = __builtin_bit_cast(u4, pf[t][n]);
              if (PK > 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = sub == y ? w[i] : 0u;
              pm[t][n] = __builtin_bit_cast(h8, w);
            }
#pragma unroll
          for (int n = 0; n < NH; ++n) {
            // 1024 + z and 64 + z of the token pairs
            const float* mn = meta + kMeta * (D == 64 ? p / 2 : p + n) + 128;
            uint32_t z10[4], z6[4];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const u2 w10 = *reinterpret_cast<const u2*>(mn + 8 * g + 2 * c);
              const u2 w6 = *reinterpret_cast<const u2*>(mn + 16 + 8 * g + 2 * c);
              z10[2 * g] = w10[0], z10[2 * g + 1] = w10[1], z6[2 * g] = w6[0], z6[2 * g + 1] = w6[1];
            }
#pragma unroll
            for (int j = 0; j < (D == 64 ? 1 : 2); ++j) {
              // 64 channels: lane m gets their half word m (four channels, every second
              // of eight) of its eight tokens, in pairs
              const int h = 2 * (n + p * NH) + j, q64 = D == 64 ? p : h, t4 = 4 * c + r / 4;
              const u4* at16 = vd + t4 * T::kChunks + v_place<T::kChunks>(t4, 2 * q64 + r % 4 / 2);
              const u2* at64 = reinterpret_cast<const u2*>(at16) + r % 2;
              const u2 y0 = read_transposed(at64), y1 = read_transposed(at64 + 2 * 16 * T::kChunks);
              const uint32_t yw[4] = {y0[0], y0[1], y1[0], y1[1]};
              u4 d[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const u4 w = code_pairs(yw[i], z10[i], z6[i], magic);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e][i] = w[e];
              }
              // MFMA k of them: row m is channel 8 (m / 2) + m % 2 + 2 k
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                  const int e = 8 * n + 4 * j + k;
                  acc[hp * RT + t][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, d[k]), pm[t][n],
                                                                              acc[hp * RT + t][e], 0, 0, 0);
                }
            }
          }
        }
      }
    };

    if (tk < t_end) {
      do {
        // past the end the next tile repeats real rows and is not used
        bool ok;
        row = rows_of(min(tk + kStep, (t_end - 1) & ~31), pg, &ok);
        pg = page_entry(tk + 2 * kStep);
        compute(row, ok);
        tk += kStep;
      } while (tk < t_end);
    }

    // The waves join through LDS: the largest reference point, every wave's sums
    // scaled to it, added in wave order.  Slab: the 16 rows of one row tile and
    // block, [row][channel] per wave, over what the waves walked with (they meet
    // before it is written).  A unit that is split leaves its sums, reference
    // points and sums of weights in the workspace: two slots a workgroup, of its
    // first and of its last unit.
    constexpr int DB = D < 128 ? D : 128;
    float* stats = static_cast<float*>(a.workspace);
    float* part = stats + (int64_t)4 * gridDim.x * HP * urows;
    int tid = threadIdx.x;  // indices made here, not kept in registers through the walk
    asm volatile("" : "+v"(tid));
    const int re = tid & 15, ce = (tid & 63) >> 4;
#pragma unroll
    for (int x = 0; x < X; ++x) {
      if (x) __syncthreads();
      const float lt = sum_over_rows16(l[x]);
      if (ce == 0) {
        stat[wave * 32 + re] = m[x][0];
        stat[wave * 32 + 16 + re] = lt;
      }
      __syncthreads();
      float M = kNegInf;
#pragma unroll
      for (int g = 0; g < kWaves; ++g) M = fmaxf(M, stat[g * 32 + re]);
      // a wave whose sum is 0 saw nothing (a NaN sum stays one)
      float k = lt == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m[x][0] - M);
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        if (n) {
          if (lt != 0.0f) k = __builtin_amdgcn_exp2f(m[x][n] - M);
          __syncthreads();
        }
        float* mine = slab + wave * kSlab<D> + re * kSlabRow<D>;
#pragma unroll
        for (int j = 0; j < DB / 64; ++j)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            // rows 2 w, 2 w + 1 of the product are the even and odd channels of eight
            const f4* v = &acc[x][8 * n + 4 * j];
            float* at8 = mine + 64 * j + 8 * (2 * ce + i / 2);
            *reinterpret_cast<f4*>(at8) = f4{v[0][i], v[0][i + 1], v[1][i], v[1][i + 1]} * k;
            *reinterpret_cast<f4*>(at8 + 4) = f4{v[2][i], v[2][i + 1], v[3][i], v[3][i + 1]} * k;
          }
        __syncthreads();
        // a thread: two channels of one row
        for (uint32_t y = tid; y < 16 * DB / 2; y += 64 * kWaves) {
          const int rr = y / (DB / 2), ch = 2 * (y % (DB / 2));
          const uint32_t qrow = row0 + 16 * (x % RT) + rr % PR;
          const int h = x / RT * PK + rr / PR;  // of the unit's heads
          if ((int)qrow > row1) continue;
          float o0 = 0.0f, o1 = 0.0f, Mr = kNegInf, L = 0.0f;
#pragma unroll
          for (int g = 0; g < kWaves; ++g) Mr = fmaxf(Mr, stat[g * 32 + rr]);
#pragma unroll
          for (int g = 0; g < kWaves; ++g) {
            const float lw = stat[g * 32 + 16 + rr];
            const float2 v = *reinterpret_cast<const float2*>(slab + g * kSlab<D> + rr * kSlabRow<D> + ch);
            o0 += v.x;
            o1 += v.y;
            L += lw == 0.0f ? 0.0f : lw * __builtin_amdgcn_exp2f(stat[g * 32 + rr] - Mr);
          }
          const uint32_t qi = qrow / (uint32_t)G;
          if (whole) {
            const int64_t orow = (int64_t)(q0 + qi) * a.Hq + (hg * HP + h) * G + (qrow - qi * G);
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            store_pair(a, orow * D + 128 * n + ch, o0 * inv, o1 * inv);
            if (a.lse && ch == 0 && n == 0) a.lse[orow] = lse_of(Mr, L);
          } else {
            const int64_t slot = ((int64_t)(2 * wg + (seg > 0)) * HP + h) * urows + (qrow - row0);
            *reinterpret_cast<float2*>(part + slot * D + 128 * n + ch) = make_float2(o0, o1);
            if (ch == 0 && n == 0) *reinterpret_cast<float2*>(stats + 2 * slot) = make_float2(Mr, L);
          }
        }
      }
    }
    __syncthreads();  // the next unit's walk is over this one's LDS
  }
}

// Joins the results of the units that several workgroups held, WPR waves a query
// row (the pieces of a row in turn), four waves a workgroup.  It finds the
// shares as they did.  D / 64 channels a lane, the loads of kBatch pieces in flight
// together.
template <int D, int HP, int RT, int WPR>
__global__ __launch_bounds__(256) void kv_attn_join_kernel(KvAttnArgs a, int urows, uint32_t wgs, int64_t nrows) {
  constexpr int C = D / 64, kBatch = D == 256 ? 8 : 16;
  __shared__ ShareLds shares;
  __shared__ float red[4][2], sum[4][D];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part_of = wave % WPR;
  const int HG = a.Hkv / HP, G = a.Hq / a.Hkv;
  const Shares sh = scan_shares(a, wgs, HG, 16 * RT, 32 * kWaves, lane, &shares);
  uint32_t id = min((int64_t)blockIdx.x * (4 / WPR) + wave / WPR, nrows - 1);
  const int hq = id % (uint32_t)a.Hq;
  id /= (uint32_t)a.Hq;
  const int b = id / (uint32_t)a.max_queries, qi = id - b * (uint32_t)a.max_queries;
  int q0, n = 1, late = 0;
  uint32_t w0 = 0;
  const int kvh = hq / G, row = qi * G + hq % G, row0 = row / (16 * RT) * (16 * RT);
  q0 = shares.q0[b];
  if (qi < shares.nq[b]) {
    const uint32_t steps = shares.steps[b];
    const uint32_t u0 = shares.before[b] + (uint32_t)(row0 / (16 * RT) * HG + kvh / HP) * steps;
    w0 = share_of(sh, u0);
    n = (int)(share_of(sh, u0 + steps - 1) - w0) + 1;
    late = share_start(sh, w0) < u0;  // for w0 it was the last unit, for the others the first
  }
  // n == 1: one workgroup had all of the unit (or there is no such query)
  const float* stats = static_cast<const float*>(a.workspace);
  const float* part = stats + (int64_t)4 * wgs * HP * urows;
  auto slot = [&](int k) -> int64_t {
    return ((int64_t)(2 * (w0 + k) + (k == 0 ? late : 0)) * HP + kvh % HP) * urows + (row - row0);
  };
  float M = kNegInf, o[C], L = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = 0.0f;
  if (n > 1) {
    for (int k0 = part_of; k0 < n; k0 += WPR * kBatch) {
      float2 ml[kBatch];
      float v[kBatch][C];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t sl = slot(min(k0 + WPR * j, n - 1));  // past the end: the last again, not added
        ml[j] = *reinterpret_cast<const float2*>(stats + 2 * sl);
#pragma unroll
        for (int i = 0; i < C; ++i) v[j][i] = part[sl * D + lane * C + i];
      }
      float top = M;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) top = fmaxf(top, ml[j].x);
      const float al = L == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(M - top);
      M = top;
      L *= al;
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] *= al;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        // 0: the piece saw nothing, or is past the end
        const float w = ml[j].y == 0.0f || k0 + WPR * j >= n ? 0.0f : __builtin_amdgcn_exp2f(ml[j].x - M);
        L += ml[j].y * w;
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] += v[j][i] * w;
      }
    }
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      red[wave][0] = M;
      red[wave][1] = L;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) sum[wave][lane * C + i] = o[i];
    __syncthreads();
    if (part_of != 0 || n == 1) return;
    M = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
    L = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = 0.0f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float w = red[g][1] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(red[g][0] - M);
      L += red[g][1] * w;
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] += sum[g][lane * C + i] * w;
    }
  }
  if (n == 1 || (int64_t)blockIdx.x * (4 / WPR) + wave / WPR >= nrows) return;
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const int64_t orow = (int64_t)(q0 + qi) * a.Hq + hq;
  if constexpr (C == 1) {
    a.out[orow * D + lane] = a.dtype == 1 ? f32_to_bf16_bits(o[0] * inv) : f32_to_f16_bits(o[0] * inv);
  } else {
#pragma unroll
    for (int i = 0; i < C; i += 2) store_pair(a, orow * D + lane * C + i, o[i] * inv, o[i + 1] * inv);
  }
  if (a.lse && lane == 0) a.lse[orow] = lse_of(M, L);
}

template <int D, int HP, int RT, int PK, bool P32, bool TREE>
hipError_t launch_main(const KvAttnArgs& a, const KvPlan& p, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  constexpr size_t lds = lds_words<D, HP> * 4;
  const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&kv_attn_kernel<D, HP, RT, PK, P32, TREE>), lds, raised);
  if (e != hipSuccess) return e;
  kv_attn_kernel<D, HP, RT, PK, P32, TREE><<<(unsigned)p.grid, 64 * kWaves, lds, stream>>>(a, p.rtiles, p.urows, p.flat);
  if (!p.flat) return hipGetLastError();
  const int64_t rows = (int64_t)a.B * a.max_queries * a.Hq, units = (int64_t)a.B * (a.Hkv / HP) * p.rtiles;
  // many pieces to a row: four waves share them (131072 tokens 42 us, 49 with one;
  // 64 contexts of up to 8K 119 us, 110 with one)
  if (p.grid > 8 * units)
    kv_attn_join_kernel<D, HP, RT, 4><<<(unsigned)rows, 256, 0, stream>>>(a, p.urows, (uint32_t)p.grid, rows);
  else
    kv_attn_join_kernel<D, HP, RT, 1><<<(unsigned)((rows + 3) / 4), 256, 0, stream>>>(a, p.urows, (uint32_t)p.grid, rows);
  return hipGetLastError();
}

template <int D, int HP, int RT, int PK, bool TREE>
hipError_t launch_p(const KvAttnArgs& a, const KvPlan& p, hipStream_t stream) {
  return a.page % 32 == 0 ? launch_main<D, HP, RT, PK, true, TREE>(a, p, stream)
                          : launch_main<D, HP, RT, PK, false, TREE>(a, p, stream);
}

template <bool TREE>
hipError_t launch_walk(const KvAttnArgs& a, const KvPlan& p, hipStream_t stream) {
  if (a.D == 256) return launch_p<256, 1, 1, 1, TREE>(a, p, stream);
  if (a.D == 128) {
    if (p.RT == 2) return launch_p<128, 1, 2, 1, TREE>(a, p, stream);
    if (p.HP == 1) return launch_p<128, 1, 1, 1, TREE>(a, p, stream);
    return p.PK == 2 ? launch_p<128, 2, 1, 2, TREE>(a, p, stream) : launch_p<128, 2, 1, 1, TREE>(a, p, stream);
  }
  if (p.RT == 2) return launch_p<64, 2, 2, 1, TREE>(a, p, stream);
  if (p.HP == 4) return p.PK == 4 ? launch_p<64, 4, 1, 4, TREE>(a, p, stream) : launch_p<64, 4, 1, 2, TREE>(a, p, stream);
  return p.PK == 2 ? launch_p<64, 2, 1, 2, TREE>(a, p, stream) : launch_p<64, 2, 1, 1, TREE>(a, p, stream);
}

}  // namespace
}  // namespace wq
