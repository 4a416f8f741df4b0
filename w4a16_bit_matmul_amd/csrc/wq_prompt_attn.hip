// Causal attention over whole prompts, packed one after another, with grouped
// heads (gfx950).
//
// For query i of a sequence and head h of KV head h / G:
//   out = sum_{t <= i} p_t v_t / sum p_t,  p_t = exp(scale * q.k_t - max),
// in one pass over the keys with a running reference point and sum in fp32.
//
// A workgroup owns 128 rows of one KV head, a row being (token, head of the
// group): its 128 / G tokens share every K and V tile it reads, and a short
// sequence still fills its rows.  Four waves of 32 rows walk tiles of keys that
// the workgroup keeps in LDS, double buffered, the next tile's loads in flight.
// Both products are computed transposed, S^T = K q^T and O^T = V^T P^T, with
// v_mfma_f32_32x32x16: a row is a column there, all its scores lie in lanes r
// and r + 32 (one lane swap for its maximum), and a lane's scores are, in order,
// its operand of the second product (tokens {8a + 4h .. + 3} of half h).  V^T
// comes out of the row-major tile by ds_read_b64_tr_b16, which transposes 4 x 16
// blocks as it reads.
//
// The weights are rounded to the inputs' type, the operand type of the matrix
// instructions of full rate: off by half a step of themselves (bf16 2^-8, fp16 2^-11) in
// a sum of hundreds of them.  fp16 ones would be subnormal from 2^-14 of the largest on,
// and behind a key that takes the weight and has little value, as a first token often is,
// all of the output comes from such; so their reference point lies kLift below the
// largest score, which keeps their bits down to 2^-21 of it (with the point at the
// largest score, 3000 keys of weight e^-17 came out 43 % off).
//
// LDS rows hold D values as 16-byte chunks; chunk j of K's token t sits at
// j ^ (t mod 16) (the 16 tokens a b128 read takes at once then fall in
// different banks), V's at j ^ 4 (t mod 4) (the four rows of a transposed read).
//
// A weight of exactly 0 does not hide a value that is no number (0 * inf), and
// one V operand serves rows that see a key and rows that do not.  So a tile that
// some rows see only in part is looked through as it is staged: an infinity or
// a NaN in its values enters the product as 0 and is added, after the outputs are
// stored, to the rows that do see it.
//
// Bound by the matrix cores for long prompts: 8K tokens with 64 / 8 heads of 128 in
// 1.1 ms, 980-1,020 TFLOP/s (a library product of bf16 reaches 1,415 in a burst), matrix
// instructions half of the cycles and the softmax a third; with heads of 64 the
// softmax comes first (16 prompts of up to 1500: 66 us, 556 TFLOP/s); short prompts
// are bound by the latency of a workgroup's start (48 of up to 300 tokens: 77-84 us,
// 3.2-3.5 TB/s).  Two workgroups a CU: while one waits the other works.  128 rows keep
// four waves in step; 256, or two groups of four waves half a tile apart (one
// multiplies while the other takes its softmax), measured 1,200 and 1,316 us where
// the kernel of that time took 1,183.
//
// Workgroups find their sequence from the device's starts: sequence b owns the
// tile slots from floor(start_b G / 128) + b on, at least as many as it has
// tiles and increasing in b, so no host needs the lengths.  Later (longer) tiles
// go first.
#include "wq_attn.h"

namespace wq {
namespace {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 128;
constexpr int kSplitRows = 32;

template <bool BF>
__device__ __forceinline__ f16v mfma32(u4 x, u4 y, f16v c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, x), __builtin_bit_cast(b8, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, x), __builtin_bit_cast(h8, y), c, 0, 0, 0);
}

// Ones over each 16-bit half of a word that holds a finite value.
template <bool BF>
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
  constexpr uint32_t lo = BF ? 0x7f80u : 0x7c00u, hi = lo << 16;
  return ((w & lo) == lo ? 0u : 0xffffu) | ((w & hi) == hi ? 0u : 0xffff0000u);
}
template <bool BF>
__device__ __forceinline__ float to_f32(uint32_t h) {
  return BF ? __builtin_bit_cast(float, h << 16) : f16_bits_to_f32((uint16_t)h);
}

template <int D>
__device__ __forceinline__ int k_chunk(int t, int j) {
  return D == 64 ? j ^ ((t >> 1) & 7) : j ^ (t & 15);
}
template <int D>
__device__ __forceinline__ int v_chunk(int t, int j) {
  return D == 64 ? j ^ ((t & 2) << 1) : j ^ ((t & 3) << 2);
}

// The reference point of weights whose largest score is mx (bf16 has fp32's exponents).
template <bool BF>
__device__ __forceinline__ float lowered(float mx) {
  return BF ? mx : mx - kLift;
}

// First sequence whose slots start past i, less one: the sequence of slot i.
// Every lane takes part; starts are clamped to [0, T].
__device__ __forceinline__ int64_t clamp_start(const int32_t* starts, int b, int64_t T) {
  return min(max((int64_t)starts[b], (int64_t)0), T);
}
template <int ROWS>
__device__ __forceinline__ int find_sequence(const int32_t* starts, int B, int64_t T, int64_t G, int64_t i, int lane) {
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int b = lo + lane * step;
    const bool le = lane * step < n && clamp_start(starts, b, T) * G / ROWS + b <= i;
    const int k = __builtin_popcountll(__ballot(le));
    if (k == 0) return lo;  // the slot lies before the first sequence's
    lo += (k - 1) * step;
    n = min(step, n - (k - 1) * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Infinities and NaNs of the tiles that rows R0..last see only in part: a thread per
// channel adds them, key by key, to the stored rows that see the key (`any`: the
// workgroup found one; every row sees keys 0..first).
template <int D, int KT, bool BF>
__device__ __forceinline__ void add_odd_values(const PromptAttnArgs& a, const uint16_t* vp, int64_t q0, int kvh, int G,
                                               int64_t R0, int first, int64_t last, int any) {
  if (!any || threadIdx.x >= D) return;
  const int ch = threadIdx.x;
  for (int64_t t = (int64_t)(first + 1) / KT * KT; t <= last / G; ++t) {
    const uint32_t v = vp[t * a.v_stride + ch];
    if (finite_halves<BF>(v) == 0xffffffffu) continue;
    for (int64_t x = max(t * G, R0); x <= last; ++x) {
      uint16_t* o = a.out + ((q0 + x / G) * a.Hq + (int64_t)kvh * G + x % G) * D + ch;
      *o = (uint16_t)pack_pair<BF>(to_f32<BF>(*o) + to_f32<BF>(v), 0.0f);
    }
  }
}

// KT: keys of a tile
template <int D, int KT, bool BF>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void prompt_attn_kernel(PromptAttnArgs a, int64_t slots) {
  constexpr int TB = KT / 32;               // 32-key MFMA blocks
  constexpr int NC = D / 8;                 // 16-byte chunks of a row
  constexpr int NS = D / 16;                // MFMA steps of a score
  constexpr int NB = D / 32;                // output blocks of 32 channels
  constexpr int LD = KT * NC / 256;         // chunks a thread stages of K, and of V
  extern __shared__ __attribute__((aligned(16))) u4 tile[];  // [2][K, V][KT * NC]
  const int lane = threadIdx.x & 63, r = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  const int kvh = (int)(blockIdx.x % a.Hkv);
  const int64_t slot = slots - 1 - blockIdx.x / a.Hkv;
  const int b = find_sequence<kRows>(a.starts, a.B, a.T, G, slot, lane);
  const int64_t q0 = clamp_start(a.starts, b, a.T);
  const int64_t n = clamp_start(a.starts, b + 1, a.T) - q0;
  const int64_t R0 = (slot - (q0 * G / kRows + b)) * kRows;
  if (R0 < 0 || R0 >= n * G) return;
  const int64_t Rw = R0 + 32 * wave;                        // the wave's first row
  const int64_t row = min(Rw + r, n * G - 1);               // past the end: the last row again, not stored
  const int64_t qi = row / G;                               // the row's token; it sees keys 0..qi
  const int64_t head = (int64_t)kvh * G + row % G;
  const int qi32 = (int)qi;
  const int first = (int)(min(Rw, n * G - 1) / G);          // fewest keys of the wave's rows, less one
  const int64_t last = min(R0 + kRows, n * G) - 1;
  const int tiles = (int)((last / G) / KT) + 1;

  // the wave's queries, B operand: lane (r, hf) channels 16 j + 8 hf
  u4 qf[NS];
  {
    const uint16_t* qp = a.q + (q0 + qi) * a.q_stride + head * D + 8 * hf;
#pragma unroll
    for (int j = 0; j < NS; ++j) qf[j] = *reinterpret_cast<const u4*>(qp + 16 * j);
  }
  const float f = a.scale * 1.4426950408889634f;

  f16v acc[NB];
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
  float m = kNegInf, l = 0.0f;

  const uint16_t* kp = a.k + q0 * a.k_stride + (int64_t)kvh * D;
  const uint16_t* vp = a.v + q0 * a.v_stride + (int64_t)kvh * D;
  const int wg_first = (int)(R0 / G);  // every row of the workgroup sees keys 0..wg_first
  const int keys = (int)n;
  // the thread's 16 bytes of a tile's load x: token t0 + x (256 / NC), chunk j0, as
  // 32-bit offsets from the tile's first key (strides are below 2^23 values)
  const int t0 = threadIdx.x / NC, j0 = threadIdx.x % NC;
  const uint32_t ks = (uint32_t)a.k_stride, vs = (uint32_t)a.v_stride;
  uint32_t k_at = (t0 * ks + 8 * j0) * 2, v_at = (t0 * vs + 8 * j0) * 2;
  u4 kreg[LD], vreg[LD];
  uint32_t odd = 0;
  auto fetch = [&](int kt) {
    const int key0 = kt * KT;
    const char* kb = reinterpret_cast<const char*>(kp + (int64_t)key0 * a.k_stride);
    const char* vb = reinterpret_cast<const char*>(vp + (int64_t)key0 * a.v_stride);
    if (key0 + KT <= keys) {
#pragma unroll
      for (int x = 0; x < LD; ++x) {
        kreg[x] = *reinterpret_cast<const u4*>(kb + x * (512 / NC) * (int64_t)ks + k_at);
        vreg[x] = *reinterpret_cast<const u4*>(vb + x * (512 / NC) * (int64_t)vs + v_at);
      }
    } else {
#pragma unroll
      for (int x = 0; x < LD; ++x) {
        const uint32_t t = min(t0 + x * (256 / NC), keys - 1 - key0);  // past the sequence: its last key again
        kreg[x] = *reinterpret_cast<const u4*>(kb + (t * ks + 8 * j0) * 2);
        vreg[x] = *reinterpret_cast<const u4*>(vb + (t * vs + 8 * j0) * 2);
      }
    }
  };
  auto stage = [&](int kt, int buf) {
    if (kt * KT + KT - 1 > wg_first) {
#pragma unroll
      for (int x = 0; x < LD; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t keep = finite_halves<BF>(vreg[x][i]);
          odd |= ~keep;
          vreg[x][i] &= keep;
        }
    }
    u4* kd = tile + buf * (2 * KT * NC);
    u4* vd = kd + KT * NC;
#pragma unroll
    for (int x = 0; x < LD; ++x) {
      const int p = x * 256 + threadIdx.x, t = p / NC, j = p % NC;
      kd[t * NC + k_chunk<D>(t, j)] = kreg[x];
      vd[t * NC + v_chunk<D>(t, j)] = vreg[x];
    }
  };
  // the lane's places in a tile: of K, chunk 2 j + hf of token r (a block of 32
  // tokens further on: the same chunk); of V, the 8 bytes it hands to a
  // transposed read of channels 32 d.. (16 kk + 8 x tokens further on: the same)
  int kat[NS], vat[NB];
#pragma unroll
  for (int j = 0; j < NS; ++j) kat[j] = r * NC + k_chunk<D>(r, 2 * j + hf);
#pragma unroll
  for (int d = 0; d < NB; ++d) {
    const int t = 4 * hf + (lane & 15) / 4;
    vat[d] = 2 * (t * NC + v_chunk<D>(t, 4 * d + 2 * ((lane >> 4) & 1) + (lane & 3) / 2)) + (lane & 1);
  }

  auto step = [&](int kt, int buf) {
    if (kt + 1 < tiles) fetch(kt + 1);
    const u4* kd = tile + buf * (2 * KT * NC);
    const u2* vd = reinterpret_cast<const u2*>(kd + KT * NC);
    f16v s[TB];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[tb][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) s[tb] = mfma32<BF>(kd[32 * tb * NC + kat[j]], qf[j], s[tb]);
    // three steps' reads ahead of the products (left alone, a read waits for the
    // products before it: 4K tokens with 32 / 4 heads of 256 450 us, 416 so (408 now); 8K with 64 / 8
    // of 128 1240, 1224)
    constexpr int kAhead = 3 * TB;
    __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
    for (int i = 0; i < NS * TB - kAhead; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
    const int key0 = kt * KT;
    if (key0 + KT - 1 > first) {
      const int seen = qi32 - key0 - 4 * hf;  // the row sees the tile's keys 0..seen + 4 hf
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * tb + 8 * (i / 4) + i % 4 > seen) s[tb][i] = kNegInf;
    }
    float mx = kNegInf;
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[tb][i]);
    mx = lowered<BF>(max_over_halves(mx) * f);
    // the reference point in use may lag the true one by kLag: weights up to 2^kLag (bf16) or
    // 2^(kLag + kLift)
    if (__ballot(mx > m + kLag)) {
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
    u4 pf[2 * TB];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][i], f, -ms));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][i + 1], f, -ms));
        l += p0 + p1;
        pf[2 * tb + i / 8][(i % 8) / 2] = pack_pair<BF>(p0, p1);
      }
#pragma unroll
    for (int kk = 0; kk < 2 * TB; ++kk)
#pragma unroll
      for (int d = 0; d < NB; ++d) {
        const u2 lo = read_transposed(vd + 2 * (16 * kk * NC) + vat[d]);
        const u2 hi = read_transposed(vd + 2 * ((16 * kk + 8) * NC) + vat[d]);
        acc[d] = mfma32<BF>(u4{lo[0], lo[1], hi[0], hi[1]}, pf[kk], acc[d]);
      }
    if (kt + 1 < tiles) stage(kt + 1, buf ^ 1);
    __syncthreads();
  };

  fetch(0);
  stage(0, 0);
  __syncthreads();
  for (int kt = 0; kt < tiles; kt += 2) {
    step(kt, 0);
    if (kt + 1 < tiles) step(kt + 1, 1);
  }
  l = sum_over_halves(l);
  // The outputs leave through LDS as whole rows, 16 bytes a lane: a lane holds 8 bytes
  // here and there of its row, and the cache takes a write of 16 bytes no faster than
  // one of a line.
  {
    const float inv = 1.0f / l;
    const uint32_t at = (uint32_t)(qi * a.Hq + head);  // the row among the sequence's
    if (a.lse && hf == 0 && Rw + r < n * G) a.lse[q0 * a.Hq + at] = (m + __builtin_log2f(l)) * 0.6931471805599453f;
    u4* ob = tile + wave * (32 * NC);
    constexpr int kTurn = NC < 16 ? NC - 1 : 15;
#pragma unroll
    for (int d = 0; d < NB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<u2*>(ob + r * NC + ((4 * d + i) ^ (r & kTurn)))[hf] =
            u2{pack_pair<BF>(acc[d][4 * i] * inv, acc[d][4 * i + 1] * inv),
               pack_pair<BF>(acc[d][4 * i + 2] * inv, acc[d][4 * i + 3] * inv)};
#pragma unroll
    for (int x = 0; x < NC / 2; ++x) {
      const int rr = (64 * x + lane) / NC, j = lane % NC;
      const u4 v = ob[rr * NC + (j ^ (rr & kTurn))];
      const uint32_t to = (uint32_t)__shfl((int)at, rr);
      if (Rw + rr < n * G) *reinterpret_cast<u4*>(a.out + (q0 * a.Hq + to) * D + 8 * j) = v;
    }
  }
  add_odd_values<D, KT, BF>(a, vp, q0, kvh, G, R0, wg_first, last, __syncthreads_or(odd != 0));
}

// The same for prompts that give few workgroups: bound by the walk over the keys of
// the last rows, so a workgroup owns 32 rows, its four waves take every fourth tile
// of 32 keys each, in LDS of their own, and join at the end (the largest reference
// point, sums scaled to it, in wave order).
template <int D, bool BF>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void prompt_split_kernel(PromptAttnArgs a, int64_t slots) {
  constexpr int KT = 32;
  constexpr int NC = D / 8, NS = D / 16, NB = D / 32;
  constexpr int LD = KT * NC / 64;  // chunks a lane stages of K, and of V
  extern __shared__ __attribute__((aligned(16))) u4 tile[];  // [wave][K, V][KT * NC], then [wave][row][D] fp32
  __shared__ float stat[4][2][kSplitRows];
  const int lane = threadIdx.x & 63, r = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  const int kvh = (int)(blockIdx.x % a.Hkv);
  const int64_t slot = slots - 1 - blockIdx.x / a.Hkv;
  const int b = find_sequence<kSplitRows>(a.starts, a.B, a.T, G, slot, lane);
  const int64_t q0 = clamp_start(a.starts, b, a.T);
  const int64_t n = clamp_start(a.starts, b + 1, a.T) - q0;
  const int64_t R0 = (slot - (q0 * G / kSplitRows + b)) * kSplitRows;
  if (R0 < 0 || R0 >= n * G) return;
  const int64_t row = min(R0 + r, n * G - 1);  // past the end: the last row again, not stored
  const int64_t qi = row / G;
  const int64_t head = (int64_t)kvh * G + row % G;
  const int qi32 = (int)qi, first = (int)(R0 / G);  // every row sees keys 0..first
  const int64_t last = min(R0 + kSplitRows, n * G) - 1;
  const int tiles = (int)((last / G) / KT) + 1, keys = (int)n;

  u4 qf[NS];
  {
    const uint16_t* qp = a.q + (q0 + qi) * a.q_stride + head * D + 8 * hf;
#pragma unroll
    for (int j = 0; j < NS; ++j) qf[j] = *reinterpret_cast<const u4*>(qp + 16 * j);
  }
  const float f = a.scale * 1.4426950408889634f;
  const uint16_t* kp = a.k + q0 * a.k_stride + (int64_t)kvh * D;
  const uint16_t* vp = a.v + q0 * a.v_stride + (int64_t)kvh * D;
  u4* kd = tile + wave * (2 * KT * NC);
  u4* vd = kd + KT * NC;
  u4 kreg[LD], vreg[LD];
  uint32_t odd = 0;
  auto fetch = [&](int kt) {
#pragma unroll
    for (int x = 0; x < LD; ++x) {
      const int p = 64 * x + lane;
      const int64_t t = min(kt * KT + p / NC, keys - 1);  // past the sequence: its last key again
      kreg[x] = *reinterpret_cast<const u4*>(kp + t * a.k_stride + 8 * (p % NC));
      vreg[x] = *reinterpret_cast<const u4*>(vp + t * a.v_stride + 8 * (p % NC));
    }
  };
  auto stage = [&](int kt) {
    const bool part = kt * KT + KT - 1 > first;
#pragma unroll
    for (int x = 0; x < LD; ++x) {
      if (part) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t keep = finite_halves<BF>(vreg[x][i]);
          odd |= ~keep;
          vreg[x][i] &= keep;
        }
      }
      const int p = 64 * x + lane, t = p / NC, j = p % NC;
      kd[t * NC + k_chunk<D>(t, j)] = kreg[x];
      vd[t * NC + v_chunk<D>(t, j)] = vreg[x];
    }
  };

  f16v acc[NB];
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
  float m = kNegInf, l = 0.0f;
  if (wave < tiles) fetch(wave);
  for (int kt = wave; kt < tiles; kt += 4) {
    stage(kt);
    if (kt + 4 < tiles) fetch(kt + 4);
    f16v s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < NS; ++j) s = mfma32<BF>(kd[r * NC + k_chunk<D>(r, 2 * j + hf)], qf[j], s);
    const int key0 = kt * KT;
    if (key0 + KT - 1 > first) {
      const int seen = qi32 - key0 - 4 * hf;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (8 * (i / 4) + i % 4 > seen) s[i] = kNegInf;
    }
    float mx = kNegInf;
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[i]);
    mx = lowered<BF>(max_over_halves(mx) * f);
    if (__ballot(mx > m + kLag)) {
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
    u4 pf[2];
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], f, -ms));
      const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i + 1], f, -ms));
      l += p0 + p1;
      pf[i / 8][(i % 8) / 2] = pack_pair<BF>(p0, p1);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int d = 0; d < NB; ++d) {
        const int t = 4 * hf + (lane & 15) / 4;
        const u2* at = reinterpret_cast<const u2*>(vd + 16 * kk * NC) + (lane & 1) +
                       2 * (t * NC + v_chunk<D>(t, 4 * d + 2 * ((lane >> 4) & 1) + (lane & 3) / 2));
        const u2 lo = read_transposed(at), hi = read_transposed(at + 2 * 8 * NC);
        acc[d] = mfma32<BF>(u4{lo[0], lo[1], hi[0], hi[1]}, pf[kk], acc[d]);
      }
  }
  l = sum_over_halves(l);
  if (hf == 0) {
    stat[wave][0][r] = m;
    stat[wave][1][r] = l;
  }
  __syncthreads();  // (and the waves are done with their tiles)
  float top = kNegInf;
#pragma unroll
  for (int g = 0; g < 4; ++g) top = fmaxf(top, stat[g][0][r]);
  // a wave whose sum is 0 saw nothing (a NaN sum stays one)
  const float k = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m - top);
  // fp32 quads of a row turned by the row, so that a quad of all rows spans the banks
  constexpr int NQ = D / 4;
  f4* slab = reinterpret_cast<f4*>(kd);
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      slab[r * NQ + ((8 * d + 2 * i + hf) ^ (r & 15))] =
          f4{acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]} * k;
  __syncthreads();
  for (uint32_t x = threadIdx.x; x < kSplitRows * NC; x += 256) {
    const uint32_t rr = x / NC, j = x % NC;
    const int64_t rw = R0 + rr;
    if (rw >= n * G) continue;
    float M = kNegInf, L = 0.0f;
#pragma unroll
    for (int g = 0; g < 4; ++g) M = fmaxf(M, stat[g][0][rr]);
    f4 o0 = {0, 0, 0, 0}, o1 = {0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float lw = stat[g][1][rr];
      L += lw == 0.0f ? 0.0f : lw * __builtin_amdgcn_exp2f(stat[g][0][rr] - M);
      const f4* sl = reinterpret_cast<const f4*>(tile + g * (2 * KT * NC)) + rr * NQ;
      o0 += sl[(2 * j) ^ (rr & 15)];
      o1 += sl[(2 * j + 1) ^ (rr & 15)];
    }
    const float inv = 1.0f / L;
    const uint32_t tok = (uint32_t)rw / (uint32_t)G;
    const int64_t at = (q0 + tok) * a.Hq + (int64_t)kvh * G + ((uint32_t)rw - tok * G);
    *reinterpret_cast<u4*>(a.out + at * D + 8 * j) =
        u4{pack_pair<BF>(o0[0] * inv, o0[1] * inv), pack_pair<BF>(o0[2] * inv, o0[3] * inv),
           pack_pair<BF>(o1[0] * inv, o1[1] * inv), pack_pair<BF>(o1[2] * inv, o1[3] * inv)};
    if (a.lse && j == 0) a.lse[at] = (M + __builtin_log2f(L)) * 0.6931471805599453f;
  }
  add_odd_values<D, KT, BF>(a, vp, q0, kvh, G, R0, first, last, __syncthreads_or(odd != 0));
}

template <int D, bool BF>
hipError_t launch_split(const PromptAttnArgs& a, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  constexpr size_t lds = (size_t)4 * 2 * 32 * D * 2;
  const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&prompt_split_kernel<D, BF>), lds, raised);
  if (e != hipSuccess) return e;
  const int64_t slots = a.T * (a.Hq / a.Hkv) / kSplitRows + a.B;
  prompt_split_kernel<D, BF><<<(unsigned)(slots * a.Hkv), 256, lds, stream>>>(a, slots);
  return hipGetLastError();
}

template <int D, int KT, bool BF>
hipError_t launch_one(const PromptAttnArgs& a, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  constexpr size_t lds = (size_t)2 * 2 * KT * D * 2;
  const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&prompt_attn_kernel<D, KT, BF>), lds, raised);
  if (e != hipSuccess) return e;
  const int64_t slots = a.T * (a.Hq / a.Hkv) / kRows + a.B;
  prompt_attn_kernel<D, KT, BF><<<(unsigned)(slots * a.Hkv), 256, lds, stream>>>(a, slots);
  return hipGetLastError();
}

template <int D, int KT>
hipError_t launch_d(const PromptAttnArgs& a, hipStream_t stream) {
  // fewer workgroups than half the CUs: one prompt of 500 / 1000 / 2000 tokens with
  // 8 / 1 heads of 128 10.3 / 15.1 / 28.5 us, 16.1 / 25.3 / 44.5 with 128 rows; with
  // 182 workgroups (four of 700) 22.9 and 20.0.  With heads of 256 this
  // tiling spills 204 bytes out of 512 registers.
  if constexpr (D != 256)
    if ((a.T * (a.Hq / a.Hkv) / kRows + a.B) * a.Hkv < 128)
      return a.dtype == 1 ? launch_split<D, true>(a, stream) : launch_split<D, false>(a, stream);
  return a.dtype == 1 ? launch_one<D, KT, true>(a, stream) : launch_one<D, KT, false>(a, stream);
}

}  // namespace

hipError_t launch_prompt_attn(const PromptAttnArgs& a, hipStream_t stream) {
  if (a.D == 64) return launch_d<64, 64>(a, stream);
  // short prompts: less of a tile lies behind their last key (48 prompts of up to 300
  // tokens 84 us, 89 with 64 keys; 16 of up to 1000 160 and 160; one of 8K 1143 and 1111)
  if (a.D == 128 && a.T < 512 * (int64_t)a.B) return launch_d<128, 32>(a, stream);
  return a.D == 128 ? launch_d<128, 64>(a, stream) : launch_d<256, 32>(a, stream);
}

}  // namespace wq
