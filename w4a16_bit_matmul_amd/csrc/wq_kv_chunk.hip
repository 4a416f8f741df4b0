// Attention over the INT4 KV cache for many query rows at once (gfx950): the next
// part of a prompt over what is already cached.
//
// The mathematics of wq_kv_attn.hip: k_t = s_t (c_t - z_t), v_t alike, a running
// maximum and sum per row; the matrix cores take c - z exactly in fp16, K's scale
// multiplies the score and V's the softmax weight in fp32, and only q and that
// weight are rounded (fp16, with the reference point of wq_kv_attn.hip).
//
// With many rows the decoding and the softmax bound, not the reading.  So a
// workgroup of four waves owns 128 rows of one KV head (a row is a token and a head
// of the group), decodes each tile of tokens once into LDS, double buffered, and
// its waves, 32 rows each, take both products transposed from there with
// v_mfma_f32_32x32x16_f16: S^T = K q^T and O^T = V^T P^T.  All scores of a row lie
// in lanes r and r + 32, a lane's scores are in order its operand of the second
// product (tokens {8a + 4h .. + 3} of half h), and V^T comes out of the row-major
// tile by ds_read_b64_tr_b16.
//
// Two sequences' next 512 tokens over 12-16K cached ones, 64 / 8 heads of 128: 582
// us, 837 TFLOP/s (matrix instructions 36 % of the cycles, decoding and softmax 52 %),
// where tiles of 32 rows decoded by each wave took 789.  256 rows a workgroup halve
// the decoding again but tie eight waves together: 631 us where this took 583.
#include "wq_attn.h"

namespace wq {
namespace {

// 16-byte chunk j of token t in a tile's row: the lanes that write or read
// together (16 tokens of a chunk of K; 4 tokens of four chunks of V; four tokens,
// four apart, as decoded) fall in different banks.
template <int D>
__device__ __forceinline__ int place(int t, int j) {
  return D == 64 ? j ^ ((t >> 1) & 7) : j ^ ((t & 3) << 2 | (t >> 2 & 3));
}
template <int D>
__device__ __forceinline__ int place_v(int t, int j) {
  return D == 64 ? j ^ ((t & 2) << 1) : place<D>(t, j);
}

constexpr int kTok = 64;  // tokens of a tile
template <int D>
constexpr int kTile = 2 * kTok * D / 8;  // 16-byte chunks of a decoded tile, K then V
// words beside it: K scales, V scales, and the powers of two above V's or the mark of a
// missing token
constexpr int kMeta = 3 * kTok;
constexpr float kGone = 128.0f;

__device__ __forceinline__ f16v mfma32(const u4& x, const h8& y, const f16v& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, x), y, c, 0, 0, 0);
}

template <int D>
__global__ __launch_bounds__(64 * kChunkWaves, 2) void kv_chunk_kernel(KvAttnArgs a, int rtiles) {
  constexpr int NC = D / 8;            // chunks of a decoded row
  constexpr int NS = D / 16;           // MFMA steps of a score
  constexpr int NB = D / 32;           // output blocks of 32 channels
  constexpr int TPT = 64 * kChunkWaves / kTok;  // threads that decode a token
  constexpr int NW = NC / TPT;         // code words of K, and of V, each decodes
  typedef uint32_t Words __attribute__((ext_vector_type(NW)));
  extern __shared__ __attribute__((aligned(16))) u4 tile[];  // [2] tiles, then [2][kMeta] words
  float* meta = reinterpret_cast<float*>(tile + 2 * kTile<D>);
  const int lane = threadIdx.x & 63, r = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  const uint32_t x = blockIdx.x / (uint32_t)a.Hkv;
  const int kvh = (int)(blockIdx.x - x * a.Hkv);
  const int b = (int)(x / (uint32_t)rtiles), rt = (int)(x - (uint32_t)b * rtiles);
  const Queries qs = queries_of(a, b);
  const int q0 = qs.q0, len = length_of(a, b);
  const int rows = qs.n * G, row0 = rt * (32 * kChunkWaves);
  if (row0 >= rows) return;
  const int row1 = min(row0 + 32 * kChunkWaves, rows) - 1;
  const int before = len - qs.all + 1;  // query i sees tokens below before + i
  const int t_end = min(len, before + (int)((uint32_t)row1 / (uint32_t)G));
  const int tiles = t_end > 0 ? (t_end + kTok - 1) / kTok : 0;
  const int wrow = min(row0 + 32 * wave, row1);
  const int low = min(t_end, before + (int)((uint32_t)wrow / (uint32_t)G));  // every row of the wave sees these
  const uint32_t qrow = min(row0 + 32 * wave + r, row1);  // past the end: the last row again, not stored
  const uint32_t qi = qrow / (uint32_t)G;
  const int head = kvh * G + (int)(qrow - qi * G);
  const int lim = min(t_end, before + (int)qi);

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

  // the thread's part of a tile: NW words of token t0, from chunk j0 on
  const int own = threadIdx.x / TPT, j0 = threadIdx.x % TPT * NW;
  const int t0 = D == 64 ? own : (own & ~15) | (own & 3) << 2 | (own >> 2 & 3);
  const uint32_t rowb = (uint32_t)a.Hkv * (D / 2), nbt = (uint32_t)a.Hkv * D / 128, zb = (nbt + 1) / 2;
  const uint32_t blk = (uint32_t)kvh * D / 128;  // the head's cache block
  const int lg = 31 - __builtin_clz(a.page), pages = (int)(a.S >> lg);
  const int32_t* table = a.table + (int64_t)b * a.table_width;
  const uint8_t* kc = a.k_codes + (uint32_t)kvh * (D / 2) + 4 * j0;
  const uint8_t* vc = a.v_codes + (uint32_t)kvh * (D / 2) + 4 * j0;
  Words kw, vw;
  uint32_t ks, vs, zs;  // scales (0 for a token whose page does not exist), zero-points (K's, V's in bits 4..)
  bool ok;
  int pg = 0;  // page of the token of the next fetch
  auto page_entry = [&](int kt) { return table[min(kt * kTok + t0, t_end - 1) >> lg]; };
  auto fetch = [&](int kt) {
    const int t = min(kt * kTok + t0, t_end - 1);  // past the end: the last token again, masked
    ok = pg >= 0 && pg < pages;
    const int64_t row = ok ? ((int64_t)pg << lg) + (t & (a.page - 1)) : 0;
    __builtin_memcpy(&kw, __builtin_assume_aligned(kc + row * rowb, 4 * NW), 4 * NW);
    __builtin_memcpy(&vw, __builtin_assume_aligned(vc + row * rowb, 4 * NW), 4 * NW);
    ks = a.k_s[row * nbt + blk];
    vs = a.v_s[row * nbt + blk];
    zs = a.k_zp[row * zb + blk / 2] | (uint32_t)a.v_zp[row * zb + blk / 2] << 8;
    pg = page_entry(kt + 1);
  };
  const Magic magic;
  auto stage = [&](int buf) {
    u4* kd = tile + buf * kTile<D> + t0 * NC;
    u4* vd = kd + kTok * NC;
    const uint32_t z = zs >> (blk & 1) * 4;
    const uint32_t zk = z & 15u, zv = z >> 8 & 15u;
    const uint32_t k10 = (zk | 0x6400u) * 0x00010001u, k6 = (zk << 4 | 0x5400u) * 0x00010001u;
    const uint32_t v10 = (zv | 0x6400u) * 0x00010001u, v6 = (zv << 4 | 0x5400u) * 0x00010001u;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      kd[place<D>(t0, j0 + i)] = code_pairs(kw[i], k10, k6, magic);
      vd[place_v<D>(t0, j0 + i)] = code_pairs(vw[i], v10, v6, magic);
    }
    if (j0 == 0) {
      float* mt = meta + buf * kMeta + t0;
      const float v = f16_bits_to_f32((uint16_t)vs);
      mt[0] = ok ? f16_bits_to_f32((uint16_t)ks) : 0.0f;
      mt[kTok] = ok ? v : 0.0f;
      mt[2 * kTok] = ok ? scale_power(v) : kGone;
    }
  };
  // the lane's places in a tile: of K, chunk hf of token r (chunk 2 j + hf: bits of
  // the index turned); of V, the 8 bytes it hands to a transposed read of the first
  // 32 channels of tokens 4 hf.. (other channels, and 8 tokens further: alike)
  const int t4 = 4 * hf + (lane & 15) / 4;
  const int kat = r * NC + place<D>(r, hf);
  const int vat = 2 * (t4 * NC + place_v<D>(t4, 2 * ((lane >> 4) & 1) + (lane & 3) / 2)) + (lane & 1);

  auto step = [&](int kt, int buf) {
    if (kt + 1 < tiles) fetch(kt + 1);
    const u4* kd = tile + buf * kTile<D>;
    const u2* vd = reinterpret_cast<const u2*>(kd + kTok * NC);
    const float* mt = meta + buf * kMeta;
    const float power = mt[2 * kTok + lane];
    const uint64_t gone = __ballot(power == kGone);
    raise_top(v_top, power == kGone ? kNoPower : power);
    int k0 = kat, v0 = vat;  // turned here: held, the places of all steps would fill the registers
    asm volatile("" : "+v"(k0), "+v"(v0));
    f16v s[2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[tb][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) s[tb] = mfma32(kd[32 * tb * NC + (k0 ^ 2 * j)], qf[j], s[tb]);
    // times the tokens' scales
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const f4 k = *reinterpret_cast<const f4*>(mt + 32 * tb + 8 * y + 4 * hf);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[tb][4 * y + i] *= k[i];
      }
    const int key0 = kt * kTok;
    if (key0 + kTok > low || gone != 0) {
      const int seen = lim - key0 - 4 * hf;
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
        const uint32_t miss = (uint32_t)(gone >> 32 * tb) >> 4 * hf;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = 8 * (i / 4) + i % 4;
          if (32 * tb + t >= seen || (miss >> t & 1)) s[tb][i] = kNegInf;
        }
      }
    }
    float mx = kNegInf;
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[tb][i]);
    mx = __builtin_fmaf(max_over_halves(mx), f, v_top);
    // that bounds score + power of every token; only where the bound calls for a new
    // reference point is the largest sum itself taken, token by token (taken always, 631
    // us in turn with 605)
    if (__ballot(mx > m + (kLag + kLift))) {
      mx = kNegInf;
#pragma unroll
      for (int tb = 0; tb < 2; ++tb)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const f4 v = *reinterpret_cast<const f4*>(mt + 2 * kTok + 32 * tb + 8 * y + 4 * hf);
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
    h8 pf[4];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const f4 v = *reinterpret_cast<const f4*>(mt + kTok + 32 * tb + 8 * y + 4 * hf);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][4 * y + i], f, -ms));
          l += p;
          pf[2 * tb + y / 2][y % 2 * 4 + i] = (_Float16)(p * v[i]);
        }
      }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int d = 0; d < NB; ++d) {
        const u2 lo = read_transposed(vd + 32 * kk * NC + (v0 ^ 8 * d));
        const u2 hi = read_transposed(vd + 32 * kk * NC + 16 * NC + (v0 ^ (8 * d + (D == 64 ? 0 : 4))));
        acc[d] = mfma32(u4{lo[0], lo[1], hi[0], hi[1]}, pf[kk], acc[d]);
      }
    if (kt + 1 < tiles) stage(buf ^ 1);
    __syncthreads();
  };

  if (tiles > 0) {
    pg = page_entry(0);
    fetch(0);
    stage(0);
  }
  __syncthreads();
  for (int kt = 0; kt < tiles; kt += 2) {
    step(kt, 0);
    if (kt + 1 < tiles) step(kt + 1, 1);
  }
  l = sum_over_halves(l);
  if (row0 + 32 * wave + r > row1) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t at = (int64_t)(q0 + qi) * a.Hq + head;
  uint16_t* o = a.out + at * D + 4 * hf;
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<u2*>(o + 32 * d + 2 * i) = u2{pack_out(a.dtype, acc[d][i] * inv, acc[d][i + 1] * inv),
                                                      pack_out(a.dtype, acc[d][i + 2] * inv, acc[d][i + 3] * inv)};
  if (a.lse && hf == 0) a.lse[at] = lse_of(m, l);
}

template <int D>
hipError_t launch_one(const KvAttnArgs& a, int64_t grid, int rtiles, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  constexpr size_t lds = 2 * (kTile<D> * 16 + kMeta * 4);
  const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&kv_chunk_kernel<D>), lds, raised);
  if (e != hipSuccess) return e;
  kv_chunk_kernel<D><<<(unsigned)grid, 64 * kChunkWaves, lds, stream>>>(a, rtiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_chunk(const KvAttnArgs& a, int64_t grid, int rtiles, hipStream_t stream) {
  return a.D == 64 ? launch_one<64>(a, grid, rtiles, stream) : launch_one<128>(a, grid, rtiles, stream);
}

}  // namespace wq
