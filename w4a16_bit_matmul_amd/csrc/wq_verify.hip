// Drafted tokens against the target's distributions, from given random numbers
// (gfx950).
//
// A row of logits l at temperature t is the distribution p(x) = w(x) / sum w,
// w(x) = exp((l(x) - max l) / t); at t = 0 it is its likeliest token.  A token is
// taken from it with one number u in [0, 1): the first x whose cumulated weight is
// above u sum w.  u counts as 2^-60 at least, so that weights too small to add up, or
// to be told from 0, decide nothing (32-bit generators give multiples of 2^-24 or so, and
// with u = 0 the first weight would be taken, however far below the others).
//   Trees of given tokens: every row's token is taken with its own u, and a drafted
// token is accepted if it is what its parent's row took and the parent is accepted.
// The answer is then what taking token after token from the target alone would have
// given, and a token x is accepted with probability p(x).
//   Chains drawn from a draft model's distributions q: token x is accepted if
// u q(x) < p(x); behind the first refusal comes a token from max(p - q, 0), behind
// the last token one from p.
//
// Which token that is changes where a cumulated weight passes u sum w, so weights and
// sums are 64-bit: with 100,000 tokens, 2^-24 of error in the weights would move one
// pick in a few hundred, their 2^-44.6 less than one in 10^8.  The 64-bit exponential is 2^f by a
// polynomial on [-1/2, 1/2] (Chebyshev interpolation) times 2^n; 64-bit operations
// have the rate of 32-bit ones here.
//
// A row is cut into chunks of kChunk logits, a wave's.  The first kernel reads all rows
// once and leaves each chunk's maximum and its sum of weights relative to that; it is
// bound by the exponentials, 17 instructions a logit.  The next ones join the chunks of a row,
// find the one in which the row's threshold falls, and read a quarter of that again.
// Every sum has a fixed order.
//
// 1024 rows of 131072 fp16 logits (64 trees): 100 us, the vector units 94 % busy, 2.7 TB/s,
// and 9 us for the picks; 128 fp32 rows of 100003: 18.6 and 5.2 us; one tree of 12 rows of
// 32768: 5.2 and 6.6; 33 chains of up to 6 rows of 50001, with drafts: 14.5, 9.9 and 5.4.
#include "wq_attn.h"

namespace wq {
namespace {

constexpr int kChunk = 2048;
constexpr int kFewNodes = 64;    // trees that one workgroup takes
constexpr int kFewDrafts = 16;   // chains whose rows every workgroup joins for itself

struct Partial {  // of a chunk: sum of weights relative to max, first token with max (greedy)
  double sum;
  float max;
  int top;
};
struct Quarters {  // the sum, by quarters of the chunk
  double sum[4];
};

// Parts of the workspace, in order of alignment.
struct Parts {
  Partial* chunks;      // [rows][C]
  Quarters* quarters;   // [rows][C]
  Partial* rows;        // [rows]: sum relative to the row's maximum
  Quarters* left;       // [B][C]: sums of max(p - q, 0)
  int* pick;            // [T]: the rows' tokens; chains: [B] the first refused draft
};
__host__ __device__ inline Parts parts_of(void* ws, int64_t T, int64_t rows, int64_t B, int C, bool chain) {
  Parts p;
  p.chunks = static_cast<Partial*>(ws);
  p.quarters = reinterpret_cast<Quarters*>(p.chunks + rows * C);
  p.rows = reinterpret_cast<Partial*>(p.quarters + rows * C);
  p.left = reinterpret_cast<Quarters*>(p.rows + rows);
  p.pick = reinterpret_cast<int*>(p.left + (chain ? B * C : 0));
  return p;
}

constexpr double kLog2e = 1.4426950408889634;
constexpr double kLeastU = 0x1p-60;
// A chunk's blocks whose weights all lie below 2^kFar of its largest are left out of its sums:
// 2048 of them are below 2^-49 of kLeastU.
constexpr double kFar = -120.0;
// The least factor between weights relative to a chunk's maximum and to the row's with which
// the chunk is taken from: the largest of each block that its sums hold is then no subnormal.
constexpr double kLeastFactor = 0x1p-900;

// Weights at one temperature, k = log2(e) / temperature: of a logit l relative to a
// finite maximum m, 2^y with y = (l - m) k.  Adding 1.5 * 2^52 leaves the integer n
// nearest to y in the low word; 2^(y - n) is the polynomial, 3.8e-14 of it off at most
// (degree 10 3e-16, degree 8 1.1e-12): half of that is the interpolation's, as much comes of its
// value at 0, set to 1 so that equal logits have whole weights.  y stops at -1100, whose power
// is 0: masked logits weigh nothing (NaN neither: they are looked for apart).
struct Weights {
  double k, low;
  // in vector registers: an instruction takes one constant from scalar ones, and copying
  // another each time would be two more
  double whole = 0x1.8p52, c8 = 0x1.63ef969a64d3cp-20;
  __device__ __forceinline__ explicit Weights(double k) : k(k), low(-1100.0 / k) {
    asm("" : "+v"(whole));
    asm("" : "+v"(c8));
  }
  __device__ __forceinline__ double operator()(float l, double m) const {
    const double d = fmax((double)l - m, low), t = fma(d, k, whole), f = fma(d, k, whole - t);
    double p = fma(0x1.b6571de2f2351p-24, f, c8);
    p = fma(p, f, 0x1.ffcb76789860fp-17);
    p = fma(p, f, 0x1.43088e257f341p-13);
    p = fma(p, f, 0x1.5d87fe908f88ap-10);
    p = fma(p, f, 0x1.3b2ab72b175eep-7);
    p = fma(p, f, 0x1.c6b08d7044119p-5);
    p = fma(p, f, 0x1.ebfbdff8149f2p-3);
    p = fma(p, f, 0x1.62e42fefa39f7p-1);
    p = fma(p, f, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)(uint32_t)__builtin_bit_cast(uint64_t, t));
  }
};

template <int DT>  // 0 fp32, 1 bf16, 2 fp16
struct Logits {
  static constexpr int E = DT == 0 ? 4 : 8;  // of 16 bytes
  static constexpr int K = kChunk / (64 * E);
  static __device__ __forceinline__ float one(const void* base, int64_t at) {
    if constexpr (DT == 0) return static_cast<const float*>(base)[at];
    const uint16_t b = static_cast<const uint16_t*>(base)[at];
    if constexpr (DT == 1) return __builtin_bit_cast(float, (uint32_t)b << 16);
    return f16_bits_to_f32(b);
  }
  // Logits x..x+E-1 of a row (rows lie at any multiple of the type's size).
  static __device__ __forceinline__ void load_whole(const void* base, int64_t at, float (&l)[E]) {
    u4 w;
    __builtin_memcpy(&w, static_cast<const char*>(base) + at * (DT == 0 ? 4 : 2), 16);
    if constexpr (DT == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) l[i] = __builtin_bit_cast(float, (uint32_t)w[i]);
    } else {
      widen8(w, DT, l);
    }
  }
  // N neighbouring blocks of 64 E logits from x on, E a lane of each: chunk c is K of them,
  // quarter q of it KQ.  -inf past the row's end.
  template <int N>
  static __device__ __forceinline__ void load_blocks(const void* base, int64_t row_at, int x, int V, int lane, float (&l)[N][E]) {
    if (x + N * 64 * E <= V) {
#pragma unroll
      for (int i = 0; i < N; ++i) load_whole(base, row_at + (x + lane * E) + 64 * i * E, l[i]);
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = x + (64 * i + lane) * E;
      if (at + E <= V) {
        load_whole(base, row_at + at, l[i]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) l[i][e] = one(base, row_at + min(at + e, V - 1));  // all in flight together
#pragma unroll
        for (int e = 0; e < E; ++e) l[i][e] = at + e < V ? l[i][e] : kNegInf;
      }
    }
  }
  static constexpr int KQ = K / 4;
  static __device__ __forceinline__ void load_chunk(const void* base, int64_t row_at, int c, int64_t V, int lane,
                                                    float (&l)[K][E]) {
    load_blocks<K>(base, row_at, c * kChunk, (int)V, lane, l);
  }
  static __device__ __forceinline__ void load_quarter(const void* base, int64_t row_at, int c, int q, int64_t V, int lane,
                                                      float (&l)[KQ][E]) {
    load_blocks<KQ>(base, row_at, c * kChunk + q * (kChunk / 4), (int)V, lane, l);
  }
};

// log2(e) / temperature of sequence b (at least 2^-1000: its inverse is a number).
__device__ __forceinline__ double sharpness(const VerifyArgs& a, int b) {
  const float t = a.temperature ? a.temperature[b] : 1.0f;
  return t > 0.0f ? fmax(kLog2e / (double)t, 0x1p-1000) : 1.0;
}
__device__ __forceinline__ bool is_greedy(const VerifyArgs& a, int b) {
  return a.temperature && !(a.temperature[b] > 0.0f);
}

__device__ __forceinline__ int read_lane(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ float read_lane(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ double read_lane(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)u, l), hi = __builtin_amdgcn_readlane((int)(u >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// op over the lanes up to each one; lane 63 has it of all.
template <class T, class Op>
__device__ __forceinline__ T wave_scan(T v, T none, Op op) {
  v = op(v, dpp<0x111, 0xf>(none, v));
  v = op(v, dpp<0x112, 0xf>(none, v));
  v = op(v, dpp<0x114, 0xf>(none, v));
  v = op(v, dpp<0x118, 0xf>(none, v));
  v = op(v, dpp<0x142, 0xa>(none, v));
  return op(v, dpp<0x143, 0xc>(none, v));
}
__device__ __forceinline__ double scan_sum(double v) {
  return wave_scan(v, 0.0, [](double x, double y) { return x + y; });
}
__device__ __forceinline__ double wave_sum(double v) { return read_lane(scan_sum(v), 63); }
// Four sums over the wave at once: lane l gets the one of s[l % 4].
__device__ __forceinline__ double wave_sum4(const double (&s)[4], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
  const double x = (b0 ? s[1] : s[0]) + dpp<0xB1, 0xf>(0.0, b0 ? s[0] : s[1]);  // lane l ^ 1
  const double y = (b0 ? s[3] : s[2]) + dpp<0xB1, 0xf>(0.0, b0 ? s[2] : s[3]);
  double v = (b1 ? y : x) + dpp<0x4E, 0xf>(0.0, b1 ? x : y);  // lane l ^ 2
  v += dpp<0x128, 0xf>(0.0, v);                               // rotated by 8 and by 4 within 16 lanes
  v += dpp<0x124, 0xf>(0.0, v);
  return add_swapped(add_swapped(v, false), true);
}
// A lane's v and those of the three others of its four lanes.
__device__ __forceinline__ double quad_sum(double v) {
  v += dpp<0xB1, 0xf>(0.0, v);
  return v + dpp<0x4E, 0xf>(0.0, v);
}
__device__ __forceinline__ float wave_max(float v) {
  return read_lane(wave_scan(v, kNegInf, [](float x, float y) { return fmaxf(x, y); }), 63);
}
__device__ __forceinline__ int wave_min(int v) {
  return read_lane(wave_scan(v, 0x7fffffff, [](int x, int y) { return min(x, y); }), 63);
}
__device__ __forceinline__ bool is_distribution(const Partial& p) {
  return fabsf(p.max) <= 3.4028235e38f && p.sum == p.sum;
}

// The nodes of sequence b that count.
__device__ __forceinline__ Place nodes_of(const VerifyArgs& a, int b) {
  if (!a.q_starts) return {b, b, 1};
  const int q0 = max(a.q_starts[b], 0);
  return {b, q0, (int)max((int64_t)0, min(min((int64_t)a.q_starts[b + 1], a.T) - q0, a.max_queries))};
}

template <int DT>
__global__ __launch_bounds__(256) void verify_chunks_kernel(VerifyArgs a, int C, uint32_t waves) {
  using L = Logits<DT>;
  const int lane = threadIdx.x & 63;
  const uint32_t id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= waves) return;
  const uint32_t r = id / (uint32_t)C;
  const int c = (int)(id - r * C);
  const bool drafted = r >= a.T;
  const int t = (int)(drafted ? r - a.T : r);
  float l[L::K][L::E];
  L::load_chunk(drafted ? a.draft : a.logits, (int64_t)t * (drafted ? a.draft_stride : a.stride), c, a.V, lane, l);
  const Place pl = place_of(a.q_starts, a.B, a.T, t, lane);
  if (pl.b < 0) return;
  const bool greedy = is_greedy(a, pl.b);
  if (drafted && (greedy || t + 1 == pl.q0 + pl.n)) return;  // no token was drawn from it
  float m = kNegInf, mb[L::K];  // largest of the chunk, and of the lane's blocks
  bool odd = false;
#pragma unroll
  for (int i = 0; i < L::K; ++i) {
    mb[i] = kNegInf;
#pragma unroll
    for (int e = 0; e < L::E; e += 2) {
      mb[i] = fmaxf(fmaxf(mb[i], l[i][e]), l[i][e + 1]);
      odd |= __builtin_isunordered(l[i][e], l[i][e + 1]);
    }
    m = fmaxf(m, mb[i]);
  }
  m = wave_max(m);
  double sum = 0.0, quarter = 0.0;
  int top = 0x7fffffff;
  if (greedy) {
#pragma unroll
    for (int i = L::K - 1; i >= 0; --i)
#pragma unroll
      for (int e = L::E - 1; e >= 0; --e)
        if (l[i][e] == m) top = c * kChunk + (64 * i + lane) * L::E + e;
    top = wave_min(top);
  } else if (m != kNegInf) {
    const Weights weight(sharpness(a, pl.b));
    const double md = m;
    double s4[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < L::K; ++i) {
      if (!__ballot(((double)mb[i] - md) * weight.k > kFar)) continue;  // nothing beside the largest (masked, say)
#pragma unroll
      for (int e = 0; e < L::E; ++e) s4[i / L::KQ] += weight(l[i][e], md);
    }
    quarter = wave_sum4(s4, lane);
    sum = quad_sum(quarter);
  }
  if (__ballot(odd)) sum = __builtin_nan("");
  const Parts p = parts_of(a.workspace, a.T, a.draft ? 2 * a.T : a.T, a.B, C, a.draft != nullptr);
  if (lane == 0) p.chunks[(int64_t)r * C + c] = {sum, m, top};
  if (lane < 4) p.quarters[(int64_t)r * C + c].sum[lane] = quarter;
}

// A row's chunks joined, one wave.
__device__ __forceinline__ Partial join_chunks(const Partial* ch, int C, const Weights& weight, int lane) {
  Partial p{0.0, kNegInf, 0x7fffffff};
  for (int c = lane; c < C; c += 64)
    if (ch[c].max > p.max) {
      p.max = ch[c].max;
      p.top = ch[c].top;
    }
  const float m = wave_max(p.max);
  p.top = wave_min(p.max == m ? p.top : 0x7fffffff);
  p.max = m;
  for (int c = lane; c < C; c += 64) p.sum += ch[c].sum == 0.0 ? 0.0 : ch[c].sum * weight(ch[c].max, p.max);
  p.sum = wave_sum(p.sum);
  return p;
}

// The first lane whose inclusive sum of s is above `limit`, or the last one with
// s > 0 where none is (-1: no such lane); `before`: the sum of the lanes before it.
__device__ __forceinline__ int wave_pick(double s, double limit, int lane, double* before, bool* hit, double* all) {
  const double run = scan_sum(s), ex = dpp<0x138, 0xf>(0.0, run);
  const uint64_t above = __ballot(run > limit && s > 0.0), some = __ballot(s > 0.0);
  const int at = above ? __builtin_ctzll(above) : some ? 63 - __builtin_clzll(some) : -1;
  *hit = above != 0;
  *before = read_lane(ex, max(at, 0));
  *all = read_lane(run, 63);
  return at;
}

// The token in which u of a row's weights is passed, one wave: chunk_sum(c) and
// quarter_sum(c, q) are the weights of a chunk and of a quarter of it, weights(c, q, w)
// those of the quarter's tokens.  -1 if no token has any.
template <int KQ, int E, class ChunkSum, class QuarterSum, class Weights>
__device__ __forceinline__ int pick_token(int C, double u, int lane, ChunkSum chunk_sum, QuarterSum quarter_sum,
                                          Weights weights) {
  double total = 0.0;
  for (int c0 = 0; c0 < C; c0 += 64) total += wave_sum(c0 + lane < C ? chunk_sum(c0 + lane) : 0.0);
  const double limit = fmax(u, kLeastU) * total;
  double carry = 0.0, rest = 0.0, before, all;
  bool hit;
  int chunk = -1;
  for (int c0 = 0; c0 < C; c0 += 64) {
    const int at = wave_pick(c0 + lane < C ? chunk_sum(c0 + lane) : 0.0, limit - carry, lane, &before, &hit, &all);
    if (at >= 0) {
      chunk = c0 + at;
      rest = limit - carry - before;
    }
    if (hit) break;
    carry += all;
  }
  if (chunk < 0) return -1;
  const int q = wave_pick(lane < 4 ? quarter_sum(chunk, lane) : 0.0, rest, lane, &before, &hit, &all);
  if (q < 0) return -1;
  rest -= before;
  double w[KQ][E], s[KQ], sums = 0.0;
  weights(chunk, q, w);
#pragma unroll
  for (int i = 0; i < KQ; ++i) {
    s[i] = 0.0;
#pragma unroll
    for (int e = 0; e < E; ++e) s[i] += w[i][e];
    if (KQ > 1) {
      const double ws = wave_sum(s[i]);
      sums = lane == i ? ws : sums;
    }
  }
  int i0 = 0;  // block of all lanes
  if (KQ > 1) {
    i0 = wave_pick(sums, rest, lane, &before, &hit, &all);
    if (i0 < 0) return -1;
    rest -= before;
  }
  double mine = 0.0, own[E];
#pragma unroll
  for (int i = 0; i < KQ; ++i) {
    mine = i == i0 ? s[i] : mine;
#pragma unroll
    for (int e = 0; e < E; ++e) own[e] = i == 0 || i == i0 ? w[i][e] : own[e];
  }
  const int l0 = wave_pick(mine, rest, lane, &before, &hit, &all);
  if (l0 < 0) return -1;
  rest -= before;
  int token = -1;
  double run = 0.0;
  bool done = false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    run += own[e];
    if (!done && own[e] > 0.0) {
      token = chunk * kChunk + (64 * (q * KQ + i0) + lane) * E + e;
      done = run > rest;
    }
  }
  return read_lane(token, l0);
}

// A row's token from its own weights; row: its chunks joined.
template <int DT>
__device__ __forceinline__ int pick_of_row(const VerifyArgs& a, const Partial* ch, const Quarters* qs, int C, int64_t t,
                                           const Partial& row, const Weights& weight, double u, int lane) {
  using L = Logits<DT>;
  auto factor = [&](int c) {
    const double f = weight(ch[c].max, row.max);
    return f < kLeastFactor ? 0.0 : f;
  };
  return pick_token<L::KQ, L::E>(
      C, u, lane, [&](int c) { return ch[c].sum == 0.0 ? 0.0 : ch[c].sum * factor(c); },
      [&](int c, int q) { return qs[c].sum[q] * factor(c); },
      [&](int c, int q, double(&w)[L::KQ][L::E]) {
        float l[L::KQ][L::E];
        L::load_quarter(a.logits, t * a.stride, c, q, a.V, lane, l);
#pragma unroll
        for (int i = 0; i < L::KQ; ++i)
#pragma unroll
          for (int e = 0; e < L::E; ++e) w[i][e] = weight(l[i][e], row.max);
      });
}

// The token that row t of sequence b gives, one wave.
template <int DT>
__device__ __forceinline__ int token_of_row(const VerifyArgs& a, const Parts& p, int C, int b, int t, int lane) {
  const Partial* ch = p.chunks + (int64_t)t * C;
  const Weights weight(sharpness(a, b));
  const Partial row = join_chunks(ch, C, weight, lane);
  if (!is_distribution(row)) return -1;
  return is_greedy(a, b) ? row.top : pick_of_row<DT>(a, ch, p.quarters + (int64_t)t * C, C, t, row, weight, (double)a.uniform[t], lane);
}

// The way down a tree of n nodes whose parents, tokens and rows' picks lie in LDS, one wave.
__device__ __forceinline__ void walk(const VerifyArgs& a, int b, int n, const int* parent, const int* token,
                                     const int* pick, int lane) {
  const int N = (int)a.max_queries;
  int32_t *out = a.out_tokens + (int64_t)b * N, *path = a.path + (int64_t)b * N;
  int count = 0, node = 0;
  while (node < n) {
    const int x = pick[node];
    if (lane == 0) {
      out[count] = x;
      path[count] = node;
    }
    ++count;
    int next = n;
    if (x >= 0)
      for (int i0 = node + 1; i0 < n; i0 += 64) {
        const int i = min(i0 + lane, n - 1);
        const uint64_t yes = __ballot(i0 + lane < n && parent[i] == node && token[i] == x);
        if (yes) {
          next = i0 + __builtin_ctzll(yes);
          break;
        }
      }
    node = next;
  }
  for (int i = count + lane; i < N; i += 64) out[i] = path[i] = -1;
  if (lane == 0) a.counts[b] = count;
}

// Small trees: a workgroup a sequence, its waves take the rows in turn.
template <int DT>
__global__ __launch_bounds__(1024) void verify_tree_kernel(VerifyArgs a, int C) {
  __shared__ int parent[kFewNodes], token[kFewNodes], pick[kFewNodes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), b = blockIdx.x;
  const Parts p = parts_of(a.workspace, a.T, a.T, a.B, C, false);
  const Place pl = nodes_of(a, b);
  if ((int)threadIdx.x < pl.n) {
    parent[threadIdx.x] = a.parents ? a.parents[pl.q0 + threadIdx.x] : (int)threadIdx.x - 1;
    token[threadIdx.x] = a.tokens[pl.q0 + threadIdx.x];
  }
  for (int i = wave; i < pl.n; i += blockDim.x / 64) {
    const int x = token_of_row<DT>(a, p, C, b, pl.q0 + i, lane);
    if (lane == 0) pick[i] = x;
  }
  __syncthreads();
  if (wave == 0) walk(a, b, pl.n, parent, token, pick, lane);
}

// Larger ones: a wave a row, then a wave a sequence.
template <int DT>
__global__ __launch_bounds__(256) void verify_pick_kernel(VerifyArgs a, int C) {
  const int lane = threadIdx.x & 63;
  const int t = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  const Place pl = place_of(a.q_starts, a.B, a.T, t, lane);
  if (pl.b < 0) return;
  const Parts p = parts_of(a.workspace, a.T, a.T, a.B, C, false);
  const int x = token_of_row<DT>(a, p, C, pl.b, t, lane);
  if (lane == 0) p.pick[t] = x;
}

__global__ __launch_bounds__(64) void verify_walk_kernel(VerifyArgs a, int C) {
  extern __shared__ int nodes[];
  const int lane = threadIdx.x, b = blockIdx.x, N = (int)a.max_queries;
  const Parts p = parts_of(a.workspace, a.T, a.T, a.B, C, false);
  const Place pl = nodes_of(a, b);
  int *parent = nodes, *token = nodes + N, *pick = nodes + 2 * N;
  for (int i = lane; i < pl.n; i += 64) {
    parent[i] = a.parents ? a.parents[pl.q0 + i] : i - 1;
    token[i] = a.tokens[pl.q0 + i];
    pick[i] = p.pick[pl.q0 + i];
  }
  __syncthreads();
  walk(a, b, pl.n, parent, token, pick, lane);
}

// Chains of many nodes: their rows joined beforehand, a wave each.
__global__ __launch_bounds__(256) void verify_rows_kernel(VerifyArgs a, int C, uint32_t rows) {
  const int lane = threadIdx.x & 63;
  const uint32_t r = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (r >= rows) return;
  const bool drafted = r >= a.T;
  const int t = (int)(drafted ? r - a.T : r);
  const Place pl = place_of(a.q_starts, a.B, a.T, t, lane);
  if (pl.b < 0 || (drafted && (is_greedy(a, pl.b) || t + 1 == pl.q0 + pl.n))) return;
  const Parts p = parts_of(a.workspace, a.T, rows, a.B, C, true);
  const Partial j = join_chunks(p.chunks + (int64_t)r * C, C, Weights(sharpness(a, pl.b)), lane);
  if (lane == 0) p.rows[r] = j;
}

// Weights max(p - q, 0) of the tokens whose logits are l and d; pr, qr: the rows' chunks joined.
template <int K, int E>
__device__ __forceinline__ void left_weights(const float (&l)[K][E], const float (&d)[K][E], const Partial& pr,
                                             const Partial& qr, const Weights& weight, double (&w)[K][E]) {
  const double ip = 1.0 / pr.sum, iq = 1.0 / qr.sum;
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e)
      w[i][e] = fmax(weight(l[i][e], pr.max) * ip - weight(d[i][e], qr.max) * iq, 0.0);
}

// Chains: which draft is refused first, and the sums of what that leaves to take from.
// Four chunks of a sequence's refused row a workgroup; every one finds that row for
// itself.  JOIN: short chains, whose rows each workgroup joins too.
template <int DT, bool JOIN>
__global__ __launch_bounds__(256) void verify_left_kernel(VerifyArgs a, int C) {
  using L = Logits<DT>;
  __shared__ int stop;
  __shared__ Partial joined[JOIN ? 2 * kFewDrafts : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = (C + 3) / 4, b = blockIdx.x / (uint32_t)per, c = (blockIdx.x % (uint32_t)per) * 4 + wave;
  const Parts p = parts_of(a.workspace, a.T, 2 * a.T, a.B, C, true);
  const Place pl = nodes_of(a, b);
  if (pl.n == 0) return;
  const bool greedy = is_greedy(a, b);
  const Weights weight(sharpness(a, b));
  // rows of a node: the target's, then the draft's
  auto row_at = [&](int i, int drafted) -> const Partial& {
    if constexpr (JOIN) return joined[2 * i + drafted];
    return p.rows[(drafted ? a.T : 0) + pl.q0 + i];
  };
  if constexpr (JOIN) {
    for (int i = wave; i < 2 * pl.n - 1; i += 4) {
      if (i % 2 && greedy) continue;
      const int64_t r = (i % 2 ? a.T : 0) + pl.q0 + i / 2;
      const Partial j = join_chunks(p.chunks + r * C, C, weight, lane);
      if (lane == 0) joined[i] = j;
    }
  }
  if (threadIdx.x == 0) stop = pl.n - 1;
  __syncthreads();
  for (int i = threadIdx.x; i < pl.n - 1; i += 256) {
    const int64_t r = pl.q0 + i;
    const int x = a.tokens[r + 1];
    const Partial pr = row_at(i, 0);
    bool yes = is_distribution(pr);
    if (greedy) {
      yes &= x == pr.top;
    } else {
      const Partial qr = row_at(i, 1);
      yes &= is_distribution(qr) && x >= 0 && x < a.V;
      if (yes) {
        const double pw = weight(L::one(a.logits, r * a.stride + x), pr.max) / pr.sum;
        const double qw = weight(L::one(a.draft, r * a.draft_stride + x), qr.max) / qr.sum;
        yes = (double)a.uniform[r + 1] * qw < pw;
      }
    }
    if (!yes) atomicMin(&stop, i);
  }
  __syncthreads();
  const int j = stop;
  const bool whole = greedy || j == pl.n - 1;
  const int64_t r = pl.q0 + j;
  if (c == 0 && lane == 0) {
    p.pick[b] = j;
    if (JOIN) {
      p.rows[r] = row_at(j, 0);
      if (!whole) p.rows[a.T + r] = row_at(j, 1);
    }
  }
  if (whole || c >= C) return;
  const Partial pr = row_at(j, 0), qr = row_at(j, 1);
  double s4[4] = {0.0, 0.0, 0.0, 0.0};
  if (is_distribution(pr) && is_distribution(qr)) {
    float l[L::K][L::E], d[L::K][L::E];
    L::load_chunk(a.logits, r * a.stride, c, a.V, lane, l);
    L::load_chunk(a.draft, r * a.draft_stride, c, a.V, lane, d);
    double w[L::K][L::E];
    left_weights(l, d, pr, qr, weight, w);
#pragma unroll
    for (int i = 0; i < L::K; ++i)
#pragma unroll
      for (int e = 0; e < L::E; ++e) s4[i / L::KQ] += w[i][e];
  }
  const double quarter = wave_sum4(s4, lane);
  if (lane < 4) p.left[(int64_t)b * C + c].sum[lane] = quarter;
}

// The end of a chain: its last token and what is written, a wave a sequence.
template <int DT>
__global__ __launch_bounds__(64) void verify_end_kernel(VerifyArgs a, int C) {
  using L = Logits<DT>;
  const int lane = threadIdx.x, b = blockIdx.x, N = (int)a.max_queries;
  const Parts p = parts_of(a.workspace, a.T, 2 * a.T, a.B, C, true);
  const Place pl = nodes_of(a, b);
  int32_t *out = a.out_tokens + (int64_t)b * N, *path = a.path + (int64_t)b * N;
  int count = 0;
  if (pl.n > 0) {
    const bool greedy = is_greedy(a, b);
    const Weights weight(sharpness(a, b));
    const double u = (double)a.uniform[pl.q0];
    const int j = p.pick[b];
    const int64_t r = pl.q0 + j;
    const Partial pr = p.rows[r];
    int token = -1;
    if (!is_distribution(pr)) {
    } else if (greedy) {
      token = pr.top;
    } else {
      bool whole = j == pl.n - 1;
      if (!whole) {
        const Partial qr = p.rows[a.T + r];
        if (is_distribution(qr)) {
          const Quarters* left = p.left + (int64_t)b * C;
          token = pick_token<L::KQ, L::E>(
              C, u, lane, [&](int c) { return left[c].sum[0] + left[c].sum[1] + left[c].sum[2] + left[c].sum[3]; },
              [&](int c, int q) { return left[c].sum[q]; },
              [&](int c, int q, double(&w)[L::KQ][L::E]) {
                float l[L::KQ][L::E], d[L::KQ][L::E];
                L::load_quarter(a.logits, r * a.stride, c, q, a.V, lane, l);
                L::load_quarter(a.draft, r * a.draft_stride, c, q, a.V, lane, d);
                left_weights(l, d, pr, qr, weight, w);
              });
          whole = token < 0;  // nothing is left: p and q are one
        }
      }
      if (whole) token = pick_of_row<DT>(a, p.chunks + r * C, p.quarters + r * C, C, r, pr, weight, u, lane);
    }
    count = j + 1;
    for (int i = lane; i < count; i += 64) {
      out[i] = i < j ? a.tokens[pl.q0 + i + 1] : token;
      path[i] = i;
    }
  }
  for (int i = count + lane; i < N; i += 64) out[i] = path[i] = -1;
  if (lane == 0) a.counts[b] = count;
}

template <int DT>
hipError_t launch_dt(const VerifyArgs& a, hipStream_t stream) {
  const int C = verify_chunks(a.V);
  const int64_t rows = a.draft ? 2 * a.T : a.T;
  const size_t lds = 3 * a.max_queries * sizeof(int);
  const unsigned tree_threads = 64 * (unsigned)(a.max_queries < 16 ? a.max_queries : 16);
  if (rows == 0) {  // sequences without nodes
    verify_walk_kernel<<<(unsigned)a.B, 64, lds, stream>>>(a, C);
    return hipGetLastError();
  }
  const uint32_t waves = (uint32_t)(rows * C);
  verify_chunks_kernel<DT><<<(waves + 3) / 4, 256, 0, stream>>>(a, C, waves);
  if (a.draft) {
    const unsigned grid = (unsigned)((int64_t)a.B * ((C + 3) / 4));
    if (a.max_queries <= kFewDrafts) {
      verify_left_kernel<DT, true><<<grid, 256, 0, stream>>>(a, C);
    } else {
      verify_rows_kernel<<<(unsigned)((rows + 3) / 4), 256, 0, stream>>>(a, C, (uint32_t)rows);
      verify_left_kernel<DT, false><<<grid, 256, 0, stream>>>(a, C);
    }
    verify_end_kernel<DT><<<(unsigned)a.B, 64, 0, stream>>>(a, C);
  } else if (a.max_queries <= kFewNodes && (uint64_t)a.B * tree_threads < (uint64_t)1 << 32) {  // (threads of a grid)
    verify_tree_kernel<DT><<<(unsigned)a.B, tree_threads, 0, stream>>>(a, C);
  } else {
    verify_pick_kernel<DT><<<(unsigned)((a.T + 3) / 4), 256, 0, stream>>>(a, C);
    verify_walk_kernel<<<(unsigned)a.B, 64, lds, stream>>>(a, C);
  }
  return hipGetLastError();
}

}  // namespace

int verify_chunks(int64_t V) { return (int)((V + kChunk - 1) / kChunk); }

size_t verify_workspace_bytes(int64_t T, int64_t V, int64_t B, bool draft) {
  const int C = verify_chunks(V);
  const int64_t rows = draft ? 2 * T : T;
  const Parts p = parts_of(nullptr, T, rows, B, C, draft);
  return reinterpret_cast<size_t>(p.pick) + 4 * (size_t)(draft ? B : T);
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream) {
  return a.dtype == 0 ? launch_dt<0>(a, stream) : a.dtype == 1 ? launch_dt<1>(a, stream) : launch_dt<2>(a, stream);
}

}  // namespace wq
