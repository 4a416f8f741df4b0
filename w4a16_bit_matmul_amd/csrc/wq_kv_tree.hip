// Attention over the INT4 KV cache for the nodes of draft trees (gfx950).
//
// A sequence's n queries are the nodes of a tree whose keys and values are its
// last n cached tokens.  Node i sees the tokens before them and of the nodes those
// whose bit of its mask is set, its ancestors and itself as a rule:
//   out_i = sum_t p_t v_t / sum_t p_t over t < len - n and over nodes j with bit j.
// All but the last n tokens are seen by every row, so the walks below are those of
// a causal attention with another mask: where a tile of tokens reaches the nodes,
// each row's lanes read the window of its mask that falls on the tile, one or two
// 64-bit words, in place of a comparison of token numbers.
//
// Up to 32 query rows of a KV head (a row is a node and a head of the group), and
// small calls, take the walk of wq_kv_walk.h, where every wave decodes its own tiles.
// With more rows and long contexts decoding and softmax bound, not the reading, and
// kv_tree_kernel below lets a workgroup of four waves decode each tile of 64 tokens
// once for 64 or 128 rows.  The mathematics and the two products are those of
// wq_kv_walk.h and wq_kv_chunk.hip: the integers c - z exactly in fp16, K's scale times
// the score and V's times the weight in fp32, S^T = K q^T and O^T = V^T P^T with
// v_mfma_f32_32x32x16_f16, 32 rows a wave.  For 128 rows each wave has its own; for 64
// two waves share rows and take half of a tile's tokens each, and join at the end.
// Waves whose rows do not exist (short trees in a batch) only decode.
//
// One sequence's or a batch's units (a sequence, KV head and tile of rows) are few, and
// contexts long and of different lengths: all steps of all units are shared out
// equally over two workgroups a CU, as in wq_kv_walk.h, and kv_tree_join_kernel joins the
// units that end up in several.
//
// 48 trees of 5-16 nodes over 3-6K tokens, 64 / 8 heads of 128: 170 us and 14 for the
// join (75 GFLOP, 440 TFLOP/s), matrix instructions 24 % and others 41 % of the
// cycles (a wave issues 38 % of its time, waits for operands or at a tile's barrier 43 %, and
// for the other wave of its SIMD 19 %); tiles decoded by each wave for itself, in the walk, took 260.  Four of
// 100-120 nodes over 7-12K, 32 / 8 heads of 64: 97 us and 7.5, 18 % and 48 % (126 in the
// walk).  One of 8 nodes over 308 tokens, in the walk: 9 us, all latency.
#include "wq_kv_walk.h"

namespace wq {
namespace {

constexpr int kTreeTok = 64;  // tokens of a tile
constexpr int kTreeStep = 128;  // tokens of a step that is shared out
template <int D>
constexpr int kTreeTile = 2 * kTreeTok * D / 8;  // 16-byte chunks of a decoded tile, K then V
// words beside it: K scales, V scales, and the powers of two above V's or a mark: the
// token is missing, or its V scale is infinite or NaN.  Such a one counts as 0, and as a NaN score in the
// rows that see it: the rows of other branches, whose weight for it is 0, would be NaN by it
// (weights set to 0 after the softmax part it from the reads of V: 102 us for 96 over four trees of 120 nodes).
constexpr int kTreeMeta = 3 * kTreeTok;
constexpr float kGone = 128.0f, kBad = 129.0f;

// 16-byte chunk j of token t in a tile's row: the lanes that read together (16 tokens of
// a chunk of K; 4 tokens of four chunks of V) fall in different banks.  Those that write
// decoded chunks (two tokens, every fourth or second chunk of each) meet in pairs: 16 cycles an
// instruction in place of 8, all of the kernel's bank conflicts, 8 % of its cycles with heads of 128 and
// 5 % with heads of 64, beside other waves' work.
template <int D>
__device__ __forceinline__ int place(int t, int j) {
  return D == 64 ? j ^ ((t >> 1) & 7) : j ^ ((t & 3) << 2 | (t >> 2 & 3));
}
template <int D>
__device__ __forceinline__ int place_v(int t, int j) {
  return D == 64 ? j ^ ((t & 2) << 1) : place<D>(t, j);
}

__device__ __forceinline__ f16v mfma32(const u4& x, const h8& y, const f16v& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, x), y, c, 0, 0, 0);
}

template <int D>
constexpr size_t tree_lds = 2 * (kTreeTile<D> * 16 + kTreeMeta * 4) + sizeof(ShareLds);

// RG: groups of 32 rows of a unit (4, or 2 whose waves take half of the tokens each).
template <int D, int RG>
__global__ __launch_bounds__(256, 2) void kv_tree_kernel(KvAttnArgs a, int rtiles, bool flat) {
  constexpr int NC = D / 8;       // chunks of a decoded row
  constexpr int NS = D / 16;      // MFMA steps of a score
  constexpr int NB = D / 32;      // output blocks of 32 channels
  constexpr int TPT = 256 / kTreeTok;  // threads that decode a token
  constexpr int NW = NC / TPT;    // code words of K, and of V, each decodes
  constexpr int TB = RG / 2;      // blocks of 32 tokens of a tile that a wave takes
  typedef uint32_t Words __attribute__((ext_vector_type(NW)));
  extern __shared__ __attribute__((aligned(16))) u4 tile[];  // [2] tiles, then [2][kTreeMeta] words, then the shares
  float* meta = reinterpret_cast<float*>(tile + 2 * kTreeTile<D>);
  ShareLds* shares = reinterpret_cast<ShareLds*>(meta + 2 * kTreeMeta);
  const int lane = threadIdx.x & 63, r = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // (the two workgroups of a CU, as a rule 256 apart, start their rows at different waves:
  // where a short tree leaves waves without rows, these are on different SIMDs)
  const int turned = RG == 4 ? (wave + (blockIdx.x >> 8 & 1) * 2) % 4 : wave;
  const int group = turned % RG, part = turned / RG, tb0 = part * TB;
  const int G = a.Hq / a.Hkv;
  // Neighbouring shares, the other heads of the same tokens as a rule, to one XCD and its L2: a
  // head has half or a quarter of a cache line (us, so and as the workgroups are numbered: 32 trees of 8 nodes
  // over 8K, heads of 128, 133 and 143, of 16 nodes over 8K 197 and 209, of heads of 64 93 and 100; 16 over 4K, heads of
  // 64, 34.4 and 33.9).
  const uint32_t wg = gridDim.x % 8 == 0 ? (blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8 : blockIdx.x;
  uint32_t at = 0, at_end = 1;  // this workgroup's steps, counted over all units
  if (flat) {
    const Shares sh = scan_shares(a, gridDim.x, a.Hkv, 32 * RG, kTreeStep, lane, shares);
    if (wg >= sh.n) return;
    at = share_start(sh, wg);
    at_end = share_start(sh, wg + 1);
  }

  // the thread's part of a tile: NW words of token t0, from chunk j0 on
  const int own = threadIdx.x / TPT, j0 = threadIdx.x % TPT * NW;
  const int t0 = D == 64 ? own : (own & ~15) | (own & 3) << 2 | (own >> 2 & 3);
  const uint32_t rowb = (uint32_t)a.Hkv * (D / 2), nbt = (uint32_t)a.Hkv * D / 128, zb = (nbt + 1) / 2;
  const int lg = 31 - __builtin_clz(a.page), pages = (int)(a.S >> lg);
  const Magic magic;
  // the lane's places in a tile: of K, chunk hf of token r (chunk 2 j + hf: bits of
  // the index turned); of V, the 8 bytes it hands to a transposed read of the first
  // 32 channels of tokens 4 hf.. (other channels, and 8 tokens further: alike)
  const int t4 = 4 * hf + (lane & 15) / 4;
  const int kat = (32 * tb0 + r) * NC + place<D>(r, hf);
  const int vat = 2 * ((32 * tb0 + t4) * NC + place_v<D>(t4, 2 * ((lane >> 4) & 1) + (lane & 3) / 2)) + (lane & 1);

  for (int seg = 0; at < at_end; ++seg) {
    int b = 0, rt, kvh, q0, len, rows, before;  // before: tokens before the nodes
    uint32_t s0 = 0, s1, steps;                 // this workgroup's steps of the unit
    if (flat) {
      // the last sequence whose units start at or before `at`
      for (int w = 0; w < a.B; w += 64) {
        const uint64_t le = __ballot(w + lane < a.B && shares->before[w + lane] <= at);
        if (le) b = w + 63 - __builtin_clzll(le);
      }
      const uint32_t first = __builtin_amdgcn_readfirstlane(shares->before[b]);
      steps = __builtin_amdgcn_readfirstlane(shares->steps[b]);
      q0 = __builtin_amdgcn_readfirstlane(shares->q0[b]);
      len = __builtin_amdgcn_readfirstlane(shares->len[b]);
      before = len - __builtin_amdgcn_readfirstlane(shares->all[b]);
      rows = __builtin_amdgcn_readfirstlane(shares->nq[b]) * G;
      const uint32_t unit = (at - first) / steps;
      rt = (int)(unit / (uint32_t)a.Hkv);
      kvh = (int)(unit - (uint32_t)rt * a.Hkv);
      s0 = at - (first + unit * steps);
      s1 = min(steps, s0 + (at_end - at));
      at += s1 - s0;
    } else {
      const uint32_t x = wg / (uint32_t)a.Hkv;
      kvh = (int)(wg - x * a.Hkv);
      b = (int)(x / (uint32_t)rtiles);
      rt = (int)(x - (uint32_t)b * rtiles);
      const Queries qs = queries_of(a, b);
      q0 = qs.q0;
      len = length_of(a, b);
      before = len - qs.all;
      rows = qs.n * G;
      if (rt * (32 * RG) >= rows) return;
      s1 = steps = steps_of(len, kTreeStep);
      at = 1;
    }
    const bool whole = s0 == 0 && s1 == steps;
    const int row0 = rt * (32 * RG), row1 = min(row0 + 32 * RG, rows) - 1;
    const int k0 = (int)s0 * 2;  // tiles of this walk
    const int k1 = min((int)s1 * 2, (len + kTreeTok - 1) / kTreeTok);
    const int low = max(before, 0);                // every row sees these
    const bool idle = row0 + 32 * group > row1;    // none of the wave's rows exists
    const uint32_t qrow = min(row0 + 32 * group + r, row1);  // past the end: the last row again, not stored
    const uint32_t qi = qrow / (uint32_t)G;
    const int head = kvh * G + (int)(qrow - qi * G);

    const uint32_t blk = (uint32_t)kvh * D / 128;  // the head's cache block
    const int32_t* table = a.table + (int64_t)b * a.table_width;
    const uint8_t* kc = a.k_codes + (uint32_t)kvh * (D / 2) + 4 * j0;
    const uint8_t* vc = a.v_codes + (uint32_t)kvh * (D / 2) + 4 * j0;
    struct Fetched {  // the thread's part of a tile on its way: two tiles are, each has several us to come
      Words kw, vw;
      // scales and zero-points as loaded: any use of them here would wait for them
      uint16_t ks, vs;
      uint8_t zk, zv;
      bool ok;
    };
    int pg = 0;  // page of the token of the next fetch
    auto page_entry = [&](int kt) { return table[min(kt * kTreeTok + t0, len - 1) >> lg]; };
    auto fetch = [&](Fetched& x, int kt) {
      const int t = min(kt * kTreeTok + t0, len - 1);  // past the end: the last token again, masked
      x.ok = (uint32_t)pg < (uint32_t)pages;
      const uint32_t row = ((uint32_t)(x.ok ? pg : 0) << lg) + (t & (a.page - 1));  // none: of the first page
      pg = page_entry(kt + 1);  // (before the tile's loads: waiting for it does not wait for them)
      __builtin_memcpy(&x.kw, __builtin_assume_aligned(kc + (uint64_t)row * rowb, 4 * NW), 4 * NW);
      __builtin_memcpy(&x.vw, __builtin_assume_aligned(vc + (uint64_t)row * rowb, 4 * NW), 4 * NW);
      const uint64_t at_s = (uint64_t)row * nbt + blk, at_z = (uint64_t)row * zb + blk / 2;
      x.ks = a.k_s[at_s];
      x.vs = a.v_s[at_s];
      x.zk = a.k_zp[at_z];
      x.zv = a.v_zp[at_z];
    };
    auto stage = [&](const Fetched& x, int buf) {
      u4* kd = tile + buf * kTreeTile<D> + t0 * NC;
      u4* vd = kd + kTreeTok * NC;
      const uint32_t zk = x.zk >> (blk & 1) * 4 & 15u, zv = x.zv >> (blk & 1) * 4 & 15u;
      const uint32_t k10 = (zk | 0x6400u) * 0x00010001u, k6 = (zk << 4 | 0x5400u) * 0x00010001u;
      const uint32_t v10 = (zv | 0x6400u) * 0x00010001u, v6 = (zv << 4 | 0x5400u) * 0x00010001u;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        kd[place<D>(t0, j0 + i)] = code_pairs(x.kw[i], k10, k6, magic);
        vd[place_v<D>(t0, j0 + i)] = code_pairs(x.vw[i], v10, v6, magic);
      }
      if (j0 == 0) {
        float* mt = meta + buf * kTreeMeta + t0;
        const float k = f16_bits_to_f32(x.ks), v = f16_bits_to_f32(x.vs);
        // (an infinite one as NaN: the score would be -inf where the product's sign is the other)
        mt[0] = !x.ok ? 0.0f : fabsf(k) <= 65504.0f ? k : __builtin_nanf("");
        const bool finite = fabsf(v) <= 65504.0f;
        mt[kTreeTok] = x.ok && finite ? v : 0.0f;
        mt[2 * kTreeTok] = !x.ok ? kGone : finite ? scale_power(v) : kBad;
      }
    };
    Fetched even, odd;
    if (k0 < k1) {
      pg = page_entry(k0);
      fetch(even, k0);
      if (k0 + 1 < k1) fetch(odd, k0 + 1);
    }

    // the wave's queries, B operand: lane (r, hf) channels 16 j + 8 hf, brought into
    // fp16's range by the power of two that takes the row's largest value into [1, 2)
    h8 qf[NS];
    float f;  // score of a row in units of log2: raw * f
    {
      const uint16_t* qp = a.q + (int64_t)(q0 + qi) * a.q_stride + (int64_t)head * D + 8 * hf;
      u4 raw[NS];
#pragma unroll
      for (int j = 0; j < NS; ++j) raw[j] = *reinterpret_cast<const u4*>(qp + 16 * j);
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        float y[8];
        widen8(raw[j], a.dtype, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
      }
      const RowPower pw = row_power(max_over_halves(top));
      f = score_factor(a.scale, pw.up);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        float y[8];
        widen8(raw[j], a.dtype, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) qf[j][e] = (_Float16)(y[e] * pw.down);
      }
    }
    f16v acc[NB];
#pragma unroll
    for (int d = 0; d < NB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    float m = kNegInf, l = 0.0f;  // weights are 2^(score - m); m follows the largest score + V scale's power
    float v_top = kNoPower;       // the largest such power so far

    auto work = [&](int kt, int buf) {
      const u4* kd = tile + buf * kTreeTile<D>;
      const u2* vd = reinterpret_cast<const u2*>(kd + kTreeTok * NC);
      const float* mt = meta + buf * kTreeMeta + 32 * tb0;
      const float power = mt[2 * kTreeTok + (TB == 2 ? lane : r)];
      const uint64_t marked = __ballot(power >= kGone);
      raise_top(v_top, power >= kGone ? kNoPower : power);
      int k = kat, v0 = vat;  // turned here: held, the places of all steps would fill the registers
      asm volatile("" : "+v"(k), "+v"(v0));
      f16v s[TB];
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[tb][i] = 0.0f;
      // operands are read kAhead products early (the compiler would read each just before
      // its product, and wait for it)
      constexpr int kAhead = 2;
      u4 kb[kAhead + 1][TB];
#pragma unroll
      for (int j = 0; j < NS + kAhead; ++j) {
        if (j < NS)
#pragma unroll
          for (int tb = 0; tb < TB; ++tb) kb[j % (kAhead + 1)][tb] = kd[32 * tb * NC + (k ^ 2 * j)];

        if (j >= kAhead)
#pragma unroll
          for (int tb = 0; tb < TB; ++tb)
            s[tb] = mfma32(kb[(j - kAhead) % (kAhead + 1)][tb], qf[j - kAhead], s[tb]);
      }
      // times the tokens' scales
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const f4 sc = *reinterpret_cast<const f4*>(mt + 32 * tb + 8 * y + 4 * hf);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[tb][4 * y + i] *= sc[i];
        }
      const int key0 = kt * kTreeTok + 32 * tb0;
      if (key0 + 32 * TB > low || marked != 0) {
        // bit i: the row does not see token i of the tile
        uint64_t off = __ballot(power == kGone) | ~tree_window(a, q0 + (int)qi, key0 - before);
        if (key0 + 64 > len) off |= len > key0 ? ~0ull << (len - key0) : ~0ull;
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
          const uint32_t miss = (uint32_t)(off >> 32 * tb) >> 4 * hf;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (miss >> (8 * (i / 4) + i % 4) & 1) s[tb][i] = kNegInf;
        }
        const uint64_t bad = __ballot(power == kBad);
        if (bad != 0)
#pragma unroll
          for (int tb = 0; tb < TB; ++tb) {
            const uint32_t hit = (uint32_t)((bad & ~off) >> 32 * tb) >> 4 * hf;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (hit >> (8 * (i / 4) + i % 4) & 1) s[tb][i] = __builtin_nanf("");
          }
      }
      float mx = kNegInf;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[tb][i]);
      mx = __builtin_fmaf(max_over_halves(mx), f, v_top);
      // that bounds score + power of every token; only where the bound calls for a new
      // reference point is the largest sum itself taken, token by token
      if (__ballot(mx > m + (kLag + kLift))) {
        mx = kNegInf;
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const f4 v = *reinterpret_cast<const f4*>(mt + 2 * kTreeTok + 32 * tb + 8 * y + 4 * hf);
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = fmaxf(mx, __builtin_fmaf(s[tb][4 * y + i], f, v[i]));
          }
        mx = max_over_halves(mx) - kLift;
        const float mn = fmaxf(m, mx);
        const float al = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= al;
#pragma unroll
        for (int d = 0; d < NB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[d][i] *= al;
      }
      const float ms = m == kNegInf ? 0.0f : m;
      h8 pf[2 * TB];
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const f4 v = *reinterpret_cast<const f4*>(mt + kTreeTok + 32 * tb + 8 * y + 4 * hf);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][4 * y + i], f, -ms));
            l += p;
            pf[2 * tb + y / 2][y % 2 * 4 + i] = (_Float16)(p * v[i]);
          }
        }
      u2 vb[kAhead + 1][2];
#pragma unroll
      for (int x = 0; x < 2 * TB * NB + kAhead; ++x) {
        if (x < 2 * TB * NB) {
          const int kk = x / NB, d = x % NB;
          vb[x % (kAhead + 1)][0] = read_transposed(vd + 32 * kk * NC + (v0 ^ 8 * d));
          vb[x % (kAhead + 1)][1] = read_transposed(vd + 32 * kk * NC + 16 * NC + (v0 ^ (8 * d + (D == 64 ? 0 : 4))));
        }

        if (x >= kAhead) {
          const int y = x - kAhead;
          const u2 *lo = &vb[y % (kAhead + 1)][0], *hi = &vb[y % (kAhead + 1)][1];
          acc[y % NB] = mfma32(u4{(*lo)[0], (*lo)[1], (*hi)[0], (*hi)[1]}, pf[y / NB], acc[y % NB]);
        }
      }
    };
    // tile kt is worked on while tile kt + 2 starts out and tile kt + 1 arrives
    auto step = [&](int kt, int buf, Fetched& mine, const Fetched& next) {
      if (kt + 2 < k1) fetch(mine, kt + 2);
      if (!idle) work(kt, buf);
      if (kt + 1 < k1) stage(next, buf ^ 1);
      __syncthreads();
    };

    if (k0 < k1) stage(even, 0);
    __syncthreads();
    for (int kt = k0; kt < k1; kt += 2) {
      step(kt, 0, even, odd);
      if (kt + 1 < k1) step(kt + 1, 1, odd, even);
    }
    l = sum_over_halves(l);
    if constexpr (RG == 2) {
      // the second half's waves hand their results over, in LDS where the tiles were
      f4* slab = reinterpret_cast<f4*>(tile) + group * (NB * 4 * 64) + lane;
      float* stat = meta + group * 128 + lane;
      if (part == 1) {
#pragma unroll
        for (int d = 0; d < NB; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            slab[(4 * d + i / 4) * 64] = f4{acc[d][i], acc[d][i + 1], acc[d][i + 2], acc[d][i + 3]};
        stat[0] = m;
        stat[64] = l;
      }
      __syncthreads();
      if (part == 0) {
        const float m1 = stat[0], l1 = stat[64], top = fmaxf(m, m1);
        // a wave whose sum is 0 saw nothing (a NaN sum stays one)
        const float x = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        const float y = l1 == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m1 - top);
        l = (l == 0.0f ? 0.0f : l * x) + (l1 == 0.0f ? 0.0f : l1 * y);
        m = top;
#pragma unroll
        for (int d = 0; d < NB; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const f4 o = slab[(4 * d + i / 4) * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[d][i + e] = acc[d][i + e] * x + o[e] * y;
          }
      }
    }
    if (part == 0 && row0 + 32 * group + r <= row1) {
      if (whole) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t orow = (int64_t)(q0 + qi) * a.Hq + head;
        uint16_t* o = a.out + orow * D + 4 * hf;
#pragma unroll
        for (int d = 0; d < NB; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<u2*>(o + 32 * d + 2 * i) = u2{pack_out(a.dtype, acc[d][i] * inv, acc[d][i + 1] * inv),
                                                            pack_out(a.dtype, acc[d][i + 2] * inv, acc[d][i + 3] * inv)};
        if (a.lse && hf == 0) a.lse[orow] = lse_of(m, l);
      } else {
        // two slots a workgroup, of its first and of its last unit
        float* stats = static_cast<float*>(a.workspace);
        const int64_t slot = (int64_t)(2 * wg + (seg > 0)) * (32 * RG) + (qrow - row0);
        float* to = stats + (int64_t)4 * gridDim.x * (32 * RG) + slot * D + 4 * hf;
#pragma unroll
        for (int d = 0; d < NB; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f4*>(to + 32 * d + 2 * i) = f4{acc[d][i], acc[d][i + 1], acc[d][i + 2], acc[d][i + 3]};
        if (hf == 0) *reinterpret_cast<float2*>(stats + 2 * slot) = make_float2(m, l);
      }
    }
    __syncthreads();  // the next unit's tiles go over this one's
  }
}

// Joins the units that several workgroups held: D / 4 lanes a row, four channels a lane.
// A workgroup has 32 rows of a unit, a few at a time, or (PG = 4, where a row has many
// pieces) a few, whose pieces four groups of lanes take in turn.  It finds the shares as
// they did.
template <int D, int PG>
constexpr int kJoinRows = PG == 1 ? 32 : 256 / PG / (D / 4);  // of a workgroup
template <int D, int RG, int PG>
__global__ __launch_bounds__(256) void kv_tree_join_kernel(KvAttnArgs a, uint32_t wgs, int rtiles) {
  constexpr int LPR = D / 4, RPP = 256 / PG / LPR, kBatch = 4;  // lanes of a row, rows at a time
  constexpr int kRows = kJoinRows<D, PG>;
  __shared__ ShareLds shares;
  __shared__ f4 red[PG][256 / PG];
  __shared__ float2 red_ml[PG][256 / PG];
  const int lane = threadIdx.x & 63;
  const Shares sh = scan_shares(a, wgs, a.Hkv, 32 * RG, kTreeStep, lane, &shares);
  const int G = a.Hq / a.Hkv;
  uint32_t id = blockIdx.x;
  const int part = id % (32 * RG / kRows);
  id /= 32 * RG / kRows;
  const int kvh = id % (uint32_t)a.Hkv;
  id /= (uint32_t)a.Hkv;
  const int b = id / (uint32_t)rtiles, rt = id - b * (uint32_t)rtiles;
  const int rows = shares.nq[b] * G, first = rt * (32 * RG), row0 = first + kRows * part;
  if (row0 >= rows) return;
  const uint32_t steps = shares.steps[b], u0 = shares.before[b] + (uint32_t)(rt * a.Hkv + kvh) * steps;
  const uint32_t w0 = share_of(sh, u0);
  const int n = (int)(share_of(sh, u0 + steps - 1) - w0) + 1;
  if (n == 1) return;  // one workgroup had all of it
  const int late = share_start(sh, w0) < u0;  // for w0 it was the last unit, for the others the first
  const float* stats = static_cast<const float*>(a.workspace);
  const float* partial = stats + (int64_t)4 * wgs * (32 * RG);
  const int in = threadIdx.x % (256 / PG), pg = threadIdx.x / (256 / PG), ch = 4 * (in % LPR);
  const int end = min(row0 + kRows, rows);
#pragma unroll 1
  for (int r0 = row0; r0 < end; r0 += RPP) {
    const int row = min(r0 + in / LPR, rows - 1), qi = row / G;  // past the end: the last again, not stored
    auto slot = [&](int k) { return (int64_t)(2 * (w0 + k) + (k == 0 ? late : 0)) * (32 * RG) + (row - first); };
    float M = kNegInf, L = 0.0f;
    f4 o = f4{0, 0, 0, 0};
    // 0: the piece saw nothing
    auto add = [&](float m, float l, const f4& v) {
      if (l == 0.0f) return;
      const float top = fmaxf(M, m), x = L == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(M - top), y = __builtin_amdgcn_exp2f(m - top);
      M = top;
      L = L * x + l * y;
      o = o * x + v * y;
    };
    for (int k0 = pg; k0 < n; k0 += PG * kBatch) {
      float2 ml[kBatch];
      f4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + PG * k >= n) break;
        ml[k] = *reinterpret_cast<const float2*>(stats + 2 * slot(k0 + PG * k));
        v[k] = *reinterpret_cast<const f4*>(partial + slot(k0 + PG * k) * D + ch);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + PG * k < n) add(ml[k].x, ml[k].y, v[k]);
    }
    if constexpr (PG > 1) {  // (one turn of the loop)
      red[pg][in] = o;
      red_ml[pg][in] = make_float2(M, L);
      __syncthreads();
      if (pg != 0) return;
#pragma unroll
      for (int g = 1; g < PG; ++g) add(red_ml[g][in].x, red_ml[g][in].y, red[g][in]);
    }
    if (r0 + in / LPR >= end) return;
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int64_t orow = (int64_t)(shares.q0[b] + qi) * a.Hq + kvh * G + (row - qi * G);
    *reinterpret_cast<u2*>(a.out + orow * D + ch) = u2{pack_out(a.dtype, o[0] * inv, o[1] * inv), pack_out(a.dtype, o[2] * inv, o[3] * inv)};
    if (a.lse && ch == 0) a.lse[orow] = lse_of(M, L);
  }
}

struct TreePlan {
  bool wide;     // kv_tree_kernel (else the walk of wq_kv_walk.h)
  bool flat;     // the steps of all units are shared out (else a unit a workgroup)
  int RG, rtiles;
  int64_t grid;  // workgroups
};

TreePlan plan_tree(int B, int Hq, int Hkv, int D, int64_t max_context, int64_t max_queries) {
  TreePlan p;
  const int64_t rows = max_queries * (Hq / Hkv);
  // 64 rows in workgroups for 128 would leave half of the waves without any (48 trees of
  // up to 16 nodes, up to 128 rows: 166 us, 184 in units of 64)
  p.RG = rows <= 64 ? 2 : 4;
  p.rtiles = (int)((rows + 32 * p.RG - 1) / (32 * p.RG));
  const int64_t units = (int64_t)B * Hkv * p.rtiles;
  const int64_t steps = max_context > kTreeStep ? (max_context + kTreeStep - 1) / kTreeStep : 1;
  // Shared out, units leave their results in fp32 for the join, 64 KB a piece at 128 rows of
  // 128: worth it for long contexts and few units (units x steps, shared out and whole, heads of
  // 128: 256 x 10 38-52 us and 34-47, 256 x 20 56-79 and 60-84, 256 x 40 88-132 and 107-154,
  // 512 x 40 168-253 and 164-245).
  p.flat = B <= kMaxShared && steps > 1 && (units < 256 || (units < kShares && steps >= 16)) &&
           units * steps < (int64_t)1 << 31;  // (steps are counted in 32 bits)
  // Where units and steps are few, pieces are small or CUs idle, and the walk with its tiles of 16
  // rows is faster (tiles x steps, this and the walk, us.  Heads of 128: 64 x 1 8.2 and 7.1, 512 x 1
  // 9.4 and 8.4, 1024 x 1 9.8 and 12.5; 64 x 3 17 and 9.2, 512 x 8 31 and 20, 1024 x 8 35 and 29; 128 x 16 27 and
  // 21, 512 x 16 35.5 and 31.5, 1024 x 16 46 and 43; 64 x 32 27 and 21, 256 x 32 34 and 36, 512 x 32 46 and 56, 1024 x
  // 32 66 and 80; 32 x 63 27 and 25, 64 x 63 31 and 30, 128 x 63 38 and 41, 256 x 63 49 and 67.  Of 64: 64 x 1 6.6 and
  // 7.8; 64 x 3 12.6 and 10.6, 512 x 3 17 and 11; 64 x 5 12.5 and 12.9, 128 x 8 14.2 and 17.0, 256 x 5 16.9 and
  // 13.5, 512 x 8 20.7 and 18.7; 128 x 16 18.7 and 18.8, 256 x 16 21 and 24, 512 x 16 26 and 29).  Units for all
  // CUs: this (heads of 128 2048 x 3 19 and 33, 2048 x 16 67 and 78; of 64 1024 x 3 11.2 and 14.1).  Heads of 256
  // always take the walk: a tile would fill the LDS.
  const int64_t tiles = (int64_t)B * Hkv * ((rows + 15) / 16);
  const bool much = units >= 256 || (D == 64 ? steps == 1 || steps > 8 || (steps > 4 && tiles <= 128)
                                             : steps == 1 ? tiles > 512 : steps >= 24 && tiles * steps > 4096);
  p.wide = rows > 32 && D != 256 && much;
  p.grid = !p.flat ? units : units * steps < kShares ? units * steps : kShares;
  return p;
}

template <int D, int RG>
hipError_t launch_tree(const KvAttnArgs& a, const TreePlan& p, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&kv_tree_kernel<D, RG>), tree_lds<D>, raised);
  if (e != hipSuccess) return e;
  kv_tree_kernel<D, RG><<<(unsigned)p.grid, 256, tree_lds<D>, stream>>>(a, p.rtiles, p.flat);
  if (!p.flat) return hipGetLastError();
  const int64_t units = (int64_t)a.B * a.Hkv * p.rtiles;
  if (p.grid > 4 * units)
    kv_tree_join_kernel<D, RG, 4><<<(unsigned)(units * (32 * RG / kJoinRows<D, 4>)), 256, 0, stream>>>(a, (uint32_t)p.grid, p.rtiles);
  else
    kv_tree_join_kernel<D, RG, 1><<<(unsigned)(units * (32 * RG / kJoinRows<D, 1>)), 256, 0, stream>>>(a, (uint32_t)p.grid, p.rtiles);
  return hipGetLastError();
}

}  // namespace

size_t kv_tree_workspace_bytes(int B, int Hq, int Hkv, int D, int64_t max_context, int64_t max_queries) {
  const TreePlan p = plan_tree(B, Hq, Hkv, D, max_context, max_queries);
  return p.wide ? (p.flat ? (size_t)2 * p.grid * (32 * p.RG) * (D + 2) * 4 : 0)
                : walk_workspace_bytes(plan_kv(B, Hq, Hkv, D, max_context, max_queries, true), D);
}

int describe_kv_tree(int B, int Hq, int Hkv, int D, int page, int64_t max_context, int64_t max_queries, char* buf,
                     size_t len) {
  const TreePlan p = plan_tree(B, Hq, Hkv, D, max_context, max_queries);
  if (p.wide) return snprintf(buf, len, "kv_tree_kernel<D=%d, RG=%d> grid=%lld block=256 %s", D, p.RG, (long long)p.grid,
                    p.flat ? "shares" : "whole units");
  const int n = describe_walk(plan_kv(B, Hq, Hkv, D, max_context, max_queries, true), D, page, buf, len);
  if (n >= 0 && (size_t)n < len) snprintf(buf + n, len - n, ", tree masks");
  return n;
}

hipError_t launch_kv_tree(const KvAttnArgs& a, hipStream_t stream) {
  const TreePlan t = plan_tree(a.B, a.Hq, a.Hkv, a.D, a.max_context, a.max_queries);
  if (t.wide) {
    if (a.D == 64) return t.RG == 2 ? launch_tree<64, 2>(a, t, stream) : launch_tree<64, 4>(a, t, stream);
    return t.RG == 2 ? launch_tree<128, 2>(a, t, stream) : launch_tree<128, 4>(a, t, stream);
  }
  return launch_walk<true>(a, plan_kv(a.B, a.Hq, a.Hkv, a.D, a.max_context, a.max_queries, true), stream);
}

}  // namespace wq
