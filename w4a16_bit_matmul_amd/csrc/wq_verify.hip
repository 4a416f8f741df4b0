// Drafted tokens against the target's distributions, from given random numbers
// (gfx950).
//
// A row of logits l at temperature t is the distribution p(x) = w(x) / sum w,
// w(x) = exp((l(x) - max l) / t); at t = 0 it is its likeliest token.  A token is
// taken from it with one number u in [0, 1): the first x whose cumulated weight is
// above u sum w.
//   Trees of given tokens: every row's token is taken with its own u, and a drafted
// token is accepted if it is what its parent's row took and the parent is accepted.
// The answer is then what taking token after token from the target alone would have
// given, and a token x is accepted with probability p(x).
//   Chains drawn from a draft model's distributions q: token x is accepted if
// u q(x) < p(x); behind the first refusal comes a token from max(p - q, 0), behind
// the last token one from p.
//
// Which token that is changes where a cumulated weight passes u sum w, so weights and
// sums are 64-bit: with 100,000 tokens, 2^-24 of error in the sums would move one
// pick in a few hundred, 2^-50 none in 10^9.  The 64-bit exponential is 2^f by a
// polynomial of degree 10 on [-1/2, 1/2] (Chebyshev interpolation, 3e-16 off) times
// 2^n; 64-bit operations have the rate of 32-bit ones here.
//
// A row is cut into chunks of kChunk logits.  The first kernel reads all rows once:
// each chunk's maximum and its sum of weights relative to that.  The next ones join
// them, find the chunk in which a row's threshold falls, and read that chunk again.
// Every sum has a fixed order.
#include "wq_attn.h"

namespace wq {
namespace {

constexpr int kChunk = 8192;

struct Partial {  // of a chunk: sum of weights relative to max, first token with max
  double sum;
  float max;
  int top;
};

// Parts of the workspace, in order of alignment.
struct Parts {
  Partial* chunks;  // [rows][C]
  Partial* rows;    // [rows]: sum relative to the row's maximum
  double* left;     // [B][C]: sums of max(p - q, 0)
  int* pick;        // [T]: the rows' tokens; chains: [B] the first refused draft
};
__host__ __device__ inline Parts parts_of(void* ws, int64_t T, int64_t rows, int64_t B, int C, bool chain) {
  Parts p;
  p.chunks = static_cast<Partial*>(ws);
  p.rows = p.chunks + rows * C;
  p.left = reinterpret_cast<double*>(p.rows + rows);
  p.pick = reinterpret_cast<int*>(p.left + (chain ? B * C : 0));
  return p;
}

// 2^y for y <= 0 (NaN stays); below 2^-1100 zero.
__device__ __forceinline__ double exp2_64(double y) {
  y = y < -1100.0 ? -1100.0 : y;
  const double n = rint(y), f = y - n;
  double p = 0x1.e6063f7217bc6p-28;
  p = fma(p, f, 0x1.b675bca4eeebbp-24);
  p = fma(p, f, 0x1.62bfd47773353p-20);
  p = fma(p, f, 0x1.ffcb54062e698p-17);
  p = fma(p, f, 0x1.430913096fd9fp-13);
  p = fma(p, f, 0x1.5d87fe9d7a584p-10);
  p = fma(p, f, 0x1.3b2ab6fba1ddap-7);
  p = fma(p, f, 0x1.c6b08d703ce49p-5);
  p = fma(p, f, 0x1.ebfbdff82c598p-3);
  p = fma(p, f, 0x1.62e42fefa3a19p-1);
  p = fma(p, f, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}

constexpr double kLog2e = 1.4426950408889634;

// A logit's weight relative to a finite maximum m; k = log2(e) / temperature.
__device__ __forceinline__ double weight(float l, float m, double k) {
  return l == kNegInf ? 0.0 : exp2_64(((double)l - (double)m) * k);
}

template <int DT>  // 0 fp32, 1 bf16, 2 fp16
struct Logits {
  static constexpr int E = DT == 0 ? 4 : 8;  // of 16 bytes
  static constexpr int K = kChunk / (256 * E);
  static __device__ __forceinline__ float one(const void* base, int64_t at) {
    if constexpr (DT == 0) return static_cast<const float*>(base)[at];
    const uint16_t b = static_cast<const uint16_t*>(base)[at];
    if constexpr (DT == 1) return __builtin_bit_cast(float, (uint32_t)b << 16);
    return f16_bits_to_f32(b);
  }
  // Logits x..x+E-1 of a row (rows lie at any multiple of the type's size); -inf past the end.
  static __device__ __forceinline__ void load(const void* base, int64_t row_at, int64_t x, int64_t V, float (&l)[E]) {
    if (x + E <= V) {
      u4 w;
      __builtin_memcpy(&w, static_cast<const char*>(base) + (row_at + x) * (DT == 0 ? 4 : 2), 16);
      if constexpr (DT == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[i] = __builtin_bit_cast(float, (uint32_t)w[i]);
      } else {
        widen8(w, DT, l);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) l[i] = x + i < V ? one(base, row_at + x + i) : kNegInf;
    }
  }
};

// log2(e) / temperature of sequence b; 0: the likeliest token alone.
__device__ __forceinline__ double sharpness(const VerifyArgs& a, int b) {
  const float t = a.temperature ? a.temperature[b] : 1.0f;
  return t > 0.0f ? kLog2e / (double)t : 0.0;
}
__device__ __forceinline__ bool is_greedy(const VerifyArgs& a, int b) {
  return a.temperature && !(a.temperature[b] > 0.0f);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
// The larger maximum; of equal ones the lower token.
__device__ __forceinline__ void take_larger(float& m, int& top, float om, int otop) {
  if (om > m || (om == m && otop < top)) {
    m = om;
    top = otop;
  }
}
__device__ __forceinline__ void wave_larger(float& m, int& top) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) take_larger(m, top, __shfl_xor(m, d), __shfl_xor(top, d));
}
__device__ __forceinline__ bool is_distribution(const Partial& p) {
  return fabsf(p.max) <= 3.4028235e38f && p.sum == p.sum;
}

template <int DT>
__global__ __launch_bounds__(256) void verify_chunks_kernel(VerifyArgs a, int C) {
  using L = Logits<DT>;
  __shared__ float s_max[4];
  __shared__ int s_top[4];
  __shared__ double s_sum[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t r = blockIdx.x / (uint32_t)C;
  const int c = (int)(blockIdx.x - r * C);
  const bool drafted = r >= a.T;
  const int t = (int)(drafted ? r - a.T : r);
  const Place pl = place_of(a.q_starts, a.B, a.T, t, lane);
  if (pl.b < 0) return;
  const bool greedy = is_greedy(a, pl.b);
  if (drafted && (greedy || t + 1 == pl.q0 + pl.n)) return;  // no token was drawn from it
  const double k = sharpness(a, pl.b);
  const void* base = drafted ? a.draft : a.logits;
  const int64_t at = (int64_t)t * (drafted ? a.draft_stride : a.stride);
  float l[L::K][L::E];
#pragma unroll
  for (int i = 0; i < L::K; ++i)
    L::load(base, at, (int64_t)c * kChunk + (int64_t)(i * 256 + threadIdx.x) * L::E, a.V, l[i]);
  float m = kNegInf;
  int top = 0x7fffffff;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < L::K; ++i)
#pragma unroll
    for (int e = 0; e < L::E; ++e) {
      const int x = c * kChunk + (i * 256 + (int)threadIdx.x) * L::E + e;
      if (l[i][e] > m) {
        m = l[i][e];
        top = x;
      }
      odd |= l[i][e] != l[i][e];
    }
  wave_larger(m, top);
  if (lane == 0) {
    s_max[wave] = m;
    s_top[wave] = top;
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 4; ++g) take_larger(m, top, s_max[g], s_top[g]);
  double sum = odd ? __builtin_nan("") : 0.0;
  if (!greedy && m != kNegInf) {
#pragma unroll
    for (int i = 0; i < L::K; ++i)
#pragma unroll
      for (int e = 0; e < L::E; ++e) sum += weight(l[i][e], m, k);
  }
  sum = wave_sum(sum);
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    const Parts p = parts_of(a.workspace, a.T, a.draft ? 2 * a.T : a.T, a.B, C, a.draft != nullptr);
    p.chunks[(int64_t)r * C + c] = {s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3], m, top};
  }
}

// A row's chunks joined, one wave.
__device__ __forceinline__ Partial join_chunks(const Partial* ch, int C, double k, int lane) {
  Partial p{0.0, kNegInf, 0x7fffffff};
  for (int c = lane; c < C; c += 64) take_larger(p.max, p.top, ch[c].max, ch[c].top);
  wave_larger(p.max, p.top);
  for (int c = lane; c < C; c += 64) p.sum += ch[c].sum == 0.0 ? 0.0 : ch[c].sum * weight(ch[c].max, p.max, k);
  p.sum = wave_sum(p.sum);
  return p;
}

__global__ __launch_bounds__(256) void verify_rows_kernel(VerifyArgs a, int C, uint32_t rows) {
  const int lane = threadIdx.x & 63;
  const uint32_t r = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= rows) return;
  const bool drafted = r >= a.T;
  const int t = (int)(drafted ? r - a.T : r);
  const Place pl = place_of(a.q_starts, a.B, a.T, t, lane);
  if (pl.b < 0 || (drafted && (is_greedy(a, pl.b) || t + 1 == pl.q0 + pl.n))) return;
  const Parts p = parts_of(a.workspace, a.T, a.draft ? 2 * a.T : a.T, a.B, C, a.draft != nullptr);
  const Partial j = join_chunks(p.chunks + (int64_t)r * C, C, sharpness(a, pl.b), lane);
  if (lane == 0) p.rows[r] = j;
}

// The first lane whose inclusive sum of s is above `limit`, or the last one with
// s > 0 where none is (-1: no such lane); `before`: the sum of the lanes before it.
__device__ __forceinline__ int wave_pick(double s, double limit, int lane, double* before, bool* hit, double* all) {
  double run = s;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double up = __shfl_up(run, d);
    run += lane >= d ? up : 0.0;
  }
  double ex = __shfl_up(run, 1);
  if (lane == 0) ex = 0.0;
  const uint64_t above = __ballot(run > limit && s > 0.0), some = __ballot(s > 0.0);
  const int at = above ? __builtin_ctzll(above) : some ? 63 - __builtin_clzll(some) : -1;
  *hit = above != 0;
  *before = __shfl(ex, max(at, 0));
  *all = __shfl(run, 63);
  return at;
}

struct PickLds {
  double sums[64];
  int token;
};

// The token in which u of the row's weights is passed: chunk_sum(c) the weights of a
// chunk, weights(x, w) those of the E tokens from x on.  One workgroup; -1 if no
// token has any weight.
template <int E, int K, class ChunkSum, class Weights>
__device__ __forceinline__ int pick_token(int C, double u, PickLds* lds, ChunkSum chunk_sum, Weights weights) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // every wave finds the chunk
  double total = 0.0;
  for (int c0 = 0; c0 < C; c0 += 64) total += wave_sum(c0 + lane < C ? chunk_sum(c0 + lane) : 0.0);
  const double limit = u * total;
  double carry = 0.0, rest = 0.0;
  int chunk = -1;
  for (int c0 = 0; c0 < C; c0 += 64) {
    double before, all;
    bool hit;
    const int at = wave_pick(c0 + lane < C ? chunk_sum(c0 + lane) : 0.0, limit - carry, lane, &before, &hit, &all);
    if (at >= 0) {
      chunk = c0 + at;
      rest = limit - carry - before;
    }
    if (hit) break;
    carry += all;
  }
  if (chunk < 0) return -1;
  double s[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    double w[E];
    weights((int64_t)chunk * kChunk + (int64_t)(i * 256 + threadIdx.x) * E, w);
    s[i] = 0.0;
#pragma unroll
    for (int e = 0; e < E; ++e) s[i] += w[e];
    const double ws = wave_sum(s[i]);
    if (lane == 0) lds->sums[4 * i + wave] = ws;
  }
  if (threadIdx.x == 0) lds->token = -1;
  __syncthreads();
  double before, all;
  bool hit;
  const int at = wave_pick(lane < 4 * K ? lds->sums[lane] : 0.0, rest, lane, &before, &hit, &all);
  if (at >= 0 && at % 4 == wave) {
    const int i0 = at / 4;
    rest -= before;
    double mine = 0.0;
#pragma unroll
    for (int i = 0; i < K; ++i) mine = i == i0 ? s[i] : mine;
    const int l = wave_pick(mine, rest, lane, &before, &hit, &all);
    if (lane == l) {
      rest -= before;
      const int64_t x = (int64_t)chunk * kChunk + (int64_t)(i0 * 256 + threadIdx.x) * E;
      double w[E], run = 0.0;
      weights(x, w);
      int token = -1;
      bool done = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        run += w[e];
        if (!done && w[e] > 0.0) {
          token = (int)x + e;
          done = run > rest;
        }
      }
      lds->token = token;
    }
  }
  __syncthreads();
  return lds->token;
}

template <int DT>
__global__ __launch_bounds__(256) void verify_pick_kernel(VerifyArgs a, int C) {
  using L = Logits<DT>;
  __shared__ PickLds lds;
  const int t = (int)blockIdx.x;
  const Place pl = place_of(a.q_starts, a.B, a.T, t, threadIdx.x & 63);
  if (pl.b < 0) return;
  const Parts p = parts_of(a.workspace, a.T, a.T, a.B, C, false);
  const double k = sharpness(a, pl.b);
  const Partial row = p.rows[t];
  int token = -1;
  if (!is_distribution(row)) {
  } else if (is_greedy(a, pl.b)) {
    token = row.top;
  } else {
    const Partial* ch = p.chunks + (int64_t)t * C;
    const int64_t at = (int64_t)t * a.stride;
    token = pick_token<L::E, L::K>(
        C, (double)a.uniform[t], &lds,
        [&](int c) { return ch[c].sum == 0.0 ? 0.0 : ch[c].sum * weight(ch[c].max, row.max, k); },
        [&](int64_t x, double(&w)[L::E]) {
          float l[L::E];
          L::load(a.logits, at, x, a.V, l);
#pragma unroll
          for (int e = 0; e < L::E; ++e) w[e] = weight(l[e], row.max, k);
        });
  }
  if (threadIdx.x == 0) p.pick[t] = token;
}

// The way down the tree, a wave a sequence: the nodes' parents and tokens and the
// rows' picks lie in LDS.
__global__ __launch_bounds__(64) void verify_walk_kernel(VerifyArgs a, int C) {
  extern __shared__ int nodes[];
  const int lane = threadIdx.x, b = blockIdx.x, N = (int)a.max_queries;
  const Parts p = parts_of(a.workspace, a.T, a.T, a.B, C, false);
  int q0 = b, n = 1;
  if (a.q_starts) {
    q0 = max(a.q_starts[b], 0);
    n = (int)max((int64_t)0, min(min((int64_t)a.q_starts[b + 1], a.T) - q0, a.max_queries));
  }
  int *parent = nodes, *token = nodes + N, *pick = nodes + 2 * N;
  for (int i = lane; i < n; i += 64) {
    parent[i] = a.parents ? a.parents[q0 + i] : i - 1;
    token[i] = a.tokens[q0 + i];
    pick[i] = p.pick[q0 + i];
  }
  __syncthreads();
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
        const int i = i0 + lane;
        const uint64_t yes = __ballot(i < n && parent[min(i, n - 1)] == node && token[min(i, n - 1)] == x);
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

// Chains: the first refused draft of the sequence (n - 1: none), one workgroup.
template <int DT>
__device__ __forceinline__ int first_refused(const VerifyArgs& a, const Parts& p, int q0, int n, double k, bool greedy,
                                             int* lds) {
  if (threadIdx.x == 0) *lds = n - 1;
  __syncthreads();
  for (int i = threadIdx.x; i < n - 1; i += 256) {
    const int r = q0 + i, x = a.tokens[r + 1];
    const Partial pr = p.rows[r];
    bool yes = is_distribution(pr);
    if (greedy) {
      yes &= x == pr.top;
    } else {
      const Partial qr = p.rows[a.T + r];
      yes &= is_distribution(qr) && x >= 0 && x < a.V;
      if (yes) {
        const double pw = weight(Logits<DT>::one(a.logits, (int64_t)r * a.stride + x), pr.max, k) / pr.sum;
        const double qw = weight(Logits<DT>::one(a.draft, (int64_t)r * a.draft_stride + x), qr.max, k) / qr.sum;
        yes = (double)a.uniform[r + 1] * qw < pw;
      }
    }
    if (!yes) atomicMin(lds, i);
  }
  __syncthreads();
  return *lds;
}

// Weights max(p - q, 0) of a row's tokens.
template <int DT>
__device__ __forceinline__ void left_weights(const VerifyArgs& a, int64_t r, int64_t x, const Partial& pr, const Partial& qr,
                                             double k, double (&w)[Logits<DT>::E]) {
  using L = Logits<DT>;
  float l[L::E], d[L::E];
  L::load(a.logits, r * a.stride, x, a.V, l);
  L::load(a.draft, r * a.draft_stride, x, a.V, d);
  const double ip = 1.0 / pr.sum, iq = 1.0 / qr.sum;
#pragma unroll
  for (int e = 0; e < L::E; ++e) w[e] = fmax(weight(l[e], pr.max, k) * ip - weight(d[e], qr.max, k) * iq, 0.0);
}

__device__ __forceinline__ Place chain_of(const VerifyArgs& a, int b) {
  if (!a.q_starts) return {b, b, 1};
  const int q0 = max(a.q_starts[b], 0);
  return {b, q0, (int)max((int64_t)0, min(min((int64_t)a.q_starts[b + 1], a.T) - q0, a.max_queries))};
}

template <int DT>
__global__ __launch_bounds__(256) void verify_left_kernel(VerifyArgs a, int C) {
  using L = Logits<DT>;
  __shared__ int stop;
  __shared__ double s_sum[4];
  const int b = blockIdx.x / (uint32_t)C, c = blockIdx.x % (uint32_t)C;
  const Parts p = parts_of(a.workspace, a.T, 2 * a.T, a.B, C, true);
  const Place pl = chain_of(a, b);
  if (pl.n == 0) return;
  const bool greedy = is_greedy(a, b);
  const double k = sharpness(a, b);
  const int j = first_refused<DT>(a, p, pl.q0, pl.n, k, greedy, &stop);
  if (c == 0 && threadIdx.x == 0) p.pick[b] = j;
  if (greedy || j == pl.n - 1) return;
  const int64_t r = pl.q0 + j;
  const Partial pr = p.rows[r], qr = p.rows[a.T + r];
  double sum = 0.0;
  if (is_distribution(pr) && is_distribution(qr)) {
#pragma unroll
    for (int i = 0; i < L::K; ++i) {
      double w[L::E];
      left_weights<DT>(a, r, (int64_t)c * kChunk + (int64_t)(i * 256 + threadIdx.x) * L::E, pr, qr, k, w);
#pragma unroll
      for (int e = 0; e < L::E; ++e) sum += w[e];
    }
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) p.left[(int64_t)b * C + c] = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
}

template <int DT>
__global__ __launch_bounds__(256) void verify_end_kernel(VerifyArgs a, int C) {
  using L = Logits<DT>;
  __shared__ PickLds lds;
  const int b = blockIdx.x, N = (int)a.max_queries;
  const Parts p = parts_of(a.workspace, a.T, 2 * a.T, a.B, C, true);
  const Place pl = chain_of(a, b);
  int32_t *out = a.out_tokens + (int64_t)b * N, *path = a.path + (int64_t)b * N;
  int count = 0;
  if (pl.n > 0) {
    const bool greedy = is_greedy(a, b);
    const double k = sharpness(a, b), u = (double)a.uniform[pl.q0];
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
          const double* left = p.left + (int64_t)b * C;
          token = pick_token<L::E, L::K>(C, u, &lds, [&](int c) { return left[c]; },
                                         [&](int64_t x, double(&w)[L::E]) { left_weights<DT>(a, r, x, pr, qr, k, w); });
          whole = token < 0;  // nothing left over: the two are one
        }
      }
      if (whole) {
        const Partial* ch = p.chunks + r * C;
        token = pick_token<L::E, L::K>(
            C, u, &lds, [&](int c) { return ch[c].sum == 0.0 ? 0.0 : ch[c].sum * weight(ch[c].max, pr.max, k); },
            [&](int64_t x, double(&w)[L::E]) {
              float l[L::E];
              L::load(a.logits, r * a.stride, x, a.V, l);
#pragma unroll
              for (int e = 0; e < L::E; ++e) w[e] = weight(l[e], pr.max, k);
            });
      }
    }
    count = j + 1;
    for (int i = threadIdx.x; i < count; i += 256) {
      out[i] = i < j ? a.tokens[pl.q0 + i + 1] : token;
      path[i] = i;
    }
  }
  for (int i = count + threadIdx.x; i < N; i += 256) out[i] = path[i] = -1;
  if (threadIdx.x == 0) a.counts[b] = count;
}

template <int DT>
hipError_t launch_dt(const VerifyArgs& a, hipStream_t stream) {
  const int C = verify_chunks(a.V);
  const int64_t rows = a.draft ? 2 * a.T : a.T;
  if (rows == 0) {  // sequences without nodes
    verify_walk_kernel<<<(unsigned)a.B, 64, 3 * a.max_queries * sizeof(int), stream>>>(a, C);
    return hipGetLastError();
  }
  verify_chunks_kernel<DT><<<(unsigned)(rows * C), 256, 0, stream>>>(a, C);
  verify_rows_kernel<<<(unsigned)((rows + 3) / 4), 256, 0, stream>>>(a, C, (uint32_t)rows);
  if (a.draft) {
    verify_left_kernel<DT><<<(unsigned)((int64_t)a.B * C), 256, 0, stream>>>(a, C);
    verify_end_kernel<DT><<<(unsigned)a.B, 256, 0, stream>>>(a, C);
  } else {
    verify_pick_kernel<DT><<<(unsigned)a.T, 256, 0, stream>>>(a, C);
    verify_walk_kernel<<<(unsigned)a.B, 64, 3 * a.max_queries * sizeof(int), stream>>>(a, C);
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
