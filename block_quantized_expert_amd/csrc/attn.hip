// attn.hip -- attention of new columns over the FP4 cache, and the weight
// that every cached token has gathered.
//
// Mathematics.  With codes c and scales 2^e, a value is (c - 7.5) 2^(e-127).
// A code masked into the mantissa of 2^(e-127) is the bf16 number (1 + c/16)
// 2^(e-127), exactly, so that
//   (c - 7.5) 2^(e-127) / 16 = word - 1.46875 * 2^(e-127):
// a product of codes runs on the bf16 matrix instruction with one more
// product that takes the offset off, and the factor 16 goes into the scale
// of the scores and the last division.  Nothing of the cache is rounded.
//   Scores:  S^T = K Q^T, a 16-token tile at a time: D/32 products of code
//   words, and one of the blocks' 2^(e-127) with -1.46875 times the sums of
//   q over the blocks (three bf16 terms: 24 bits).
//   Output:  O^T += V^T P^T, 32 tokens at a time: two products for each
//   block of 32 values (even and odd ones), and products of 2^(e-127) that
//   take the offsets off.  Row sums of P: one product with ones.
// Both are transposed, so that lane (m = lane & 15, g = lane >> 4) holds of
// query row m the scores of tokens 4g .. 4g+3 and 16+4g .. 16+4g+3, which
// are the eight k-values that the second product takes from that very lane:
// P never leaves its registers.  Softmax is the running kind: row maximum
// and sum in fp32, the maximum moved (and everything rescaled) only when a
// score exceeds it by 2^8.
//
// Bases.  Maxima are kept as the products give them (raw), so that comparing
// them rounds nothing.  What a row's numerators stand against is base =
// fl(maximum * sc): 2^(s sc - base) is one fma a score.  What base was rounded
// by (half a step of it at most) is a factor that their sums share; a wave
// takes it out of them at its end, so that joins and lse see sums against the
// maximum itself.  At a base of 2^31 that factor can be 2^64, so from |base| =
// kWide on numerators are 2^((s - maximum) sc) to begin with.  A wave with such
// a row has a threshold of -inf, so that all its tiles come by the block where
// maxima move, and other waves pay nothing for it.
#include "rfpx_attn.hpp"

namespace rfpx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;         // waves of a workgroup whose work is split over several
constexpr int kWavesOne = 8;      // ... and of one that has a sequence's head to itself
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 32;          // tokens of one step of a wave
constexpr float kOffset = 1.46875f;  // (16 + 7.5) / 16
constexpr uint32_t kCodeMask = 0x00780078u;
constexpr uint32_t kNegOffset = 0x803C803Cu;  // sign and mantissa of -1.46875, twice
constexpr float kNegInf = -__builtin_inff();

struct AttnArgs {
  KvView v;
  const void *q;
  void *out;
  float *lse;
  float *part;    // [rows * heads][splits][D] numerators (splits > 1)
  float *part_ml; // [rows * heads][splits][4]: raw maximum, sum, exact sum
  long long q_stride, out_stride;
  int xtype, heads, group, n_rows, splits, row_blocks;
  float sc;       // 16 * scale * log2(e)
};

__device__ __forceinline__ floatx4 mfma(const u32x4v &a, const u32x4v &b, const floatx4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  const floatx2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float max_across_g(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  const uint32_t w = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Half a step of a base of 2^24 is 1, a factor of two at most (and scores of
// that size have lost as much to their own rounding).
constexpr float kWide = 16777216.f;

// What numerators against the raw maximum `from` are multiplied by (as a power
// of two) to stand against `to`, which is no smaller: the difference of the
// bases as they were rounded, or of the maxima where they are wide.
__device__ __forceinline__ float base_step(float from, float to, float sc) {
#pragma clang fp contract(off)
  if (to == kNegInf) to = 0.f;  // nothing seen yet: numerators against 0
  const float base = to * sc, was = from * sc;
  return fabsf(base) < kWide ? was - base : (from - to) * sc;
}
// What base was rounded by; 0 where numerators stand against the maximum
// itself, for which base is 0.
__device__ __forceinline__ float rounded_by(float top, float base, float sc) {
  return base == 0.f ? 0.f : -fmaf(top, sc, -base);
}
// From one raw maximum to another, no smaller, as a power of two (to 0 while
// nothing has been seen).
__device__ __forceinline__ float down_to(float from, float to, float sc) {
  return (from - (to == kNegInf ? 0.f : to)) * sc;
}
// Log of a row's sum `ex` of numerators against its raw maximum.
__device__ __forceinline__ float lse_of(float top, float ex, float sc) {
  return fmaf(top, sc, log2f(ex)) * 0.69314718055994531f;
}

// N dwords from p (aligned to their size, at most 16 bytes a load).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
    }
  }
}

// ------------------------------------------------------------ the query side

// Operand words of row m's values for every block: terms t = 0 .. VX-1 of
// pairs (j, j + 4) of the lane's octet, and the offset operand (see top).
template <int NB, int VX>
struct QTile {
  u32x4v w[VX][NB];
  u32x4v off;
};
// ... of a tile in LDS, where all waves read it.
template <int NB, int VX>
struct QShared {
  u32x4v at[VX * NB + 1][64];
};

template <int NB, int VX>
__device__ __forceinline__ void load_q(const void *q, size_t at, bool live, int g,
                                       QTile<NB, VX> &t) {
  float sum[NB];
#pragma unroll
  for (int kb = 0; kb < NB; ++kb) {
    float s = 0.f;
    if constexpr (VX == 1) {
      uint4 d = make_uint4(0, 0, 0, 0);
      if (live)
        d = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(q) + at + 32 * kb + 8 * g);
      // pairs (0,1) (2,3) (4,5) (6,7) -> (0,4) (1,5) (2,6) (3,7)
      t.w[0][kb][0] = __builtin_amdgcn_perm(d.z, d.x, 0x05040100u);
      t.w[0][kb][1] = __builtin_amdgcn_perm(d.z, d.x, 0x07060302u);
      t.w[0][kb][2] = __builtin_amdgcn_perm(d.w, d.y, 0x05040100u);
      t.w[0][kb][3] = __builtin_amdgcn_perm(d.w, d.y, 0x07060302u);
#pragma unroll
      for (int i = 0; i < 4; ++i) s += lo_f(t.w[0][kb][i]) + hi_f(t.w[0][kb][i]);
    } else {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(q) + at + 32 * kb + 8 * g);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
#pragma unroll
      for (int x = 0; x < VX; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t h = pk_bf16(v[i], v[i + 4]);
          t.w[x][kb][i] = h;
          v[i] -= lo_f(h);
          v[i + 4] -= hi_f(h);
        }
    }
    sum[kb] = cross_row_sum(s) * -kOffset;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = 2 * i < NB ? sum[2 * i] : 0.f, b = 2 * i + 1 < NB ? sum[2 * i + 1] : 0.f;
    uint32_t h = pk_bf16(a, b), mine = g == 0 ? h : 0u;
#pragma unroll
    for (int x = 1; x < 3; ++x) {
      a -= lo_f(h);
      b -= hi_f(h);
      h = pk_bf16(a, b);
      mine = g == x ? h : mine;
    }
    t.off[i] = mine;
  }
}

// ------------------------------------------------------------- the key side

template <int NB>
struct KTile {  // a 16-token tile as loaded
  uint32_t c[NB];
  uint32_t s[(NB + 3) / 4];
};

template <int NB>
__device__ __forceinline__ void load_k(const uint8_t *slab, const KvGeo &g, int t0, int lane,
                                       KTile<NB> &k) {
  const int t = t0 + (lane & 15);
  load_words<NB>(slab + g.kc + t * (16 * NB) + (lane >> 4) * (4 * NB), k.c);
  const uint8_t *s = slab + g.ks + t * NB;
  if constexpr (NB == 2) k.s[0] = *reinterpret_cast<const uint16_t *>(s);
  else if constexpr (NB == 4) k.s[0] = *reinterpret_cast<const uint32_t *>(s);
  else load_words<2>(s, k.s);
}

template <int NB>
struct KWords {  // its operands
  u32x4v w[NB];
  u32x4v e;
};

template <int NB>
__device__ __forceinline__ void decode_k(const KTile<NB> &k, KWords<NB> &o) {
  uint32_t base[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint32_t sel = 0x0C000C00u | (b & 3) | (b & 3) << 16;
    base[b] = __builtin_amdgcn_perm(0u, k.s[b >> 2], sel) << 7;
    o.w[b][0] = and_or(k.c[b] << 3, kCodeMask, base[b]);
    o.w[b][1] = and_or(k.c[b] >> 1, kCodeMask, base[b]);
    o.w[b][2] = and_or(k.c[b] >> 5, kCodeMask, base[b]);
    o.w[b][3] = and_or(k.c[b] >> 9, kCodeMask, base[b]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o.e[i] = 2 * i < NB ? __builtin_amdgcn_perm(base[2 * i + 1 < NB ? 2 * i + 1 : 0],
                                                base[2 * i < NB ? 2 * i : 0], 0x05040100u)
                        : 0u;
}

template <int NB, int VX>
__device__ __forceinline__ floatx4 scores(const KWords<NB> &k, const QShared<NB, VX> &q, int lane) {
  floatx4 s = {0.f, 0.f, 0.f, 0.f};
  // the offsets and the leading terms first: the sum is back at its own size
  // before the smaller terms come
  s = mfma(k.e, q.at[VX * NB][lane], s);
#pragma unroll
  for (int x = 0; x < VX; ++x)
#pragma unroll
    for (int b = 0; b < NB; ++b) s = mfma(k.w[b], q.at[x * NB + b][lane], s);
  return s;
}

// ----------------------------------------------------------- the value side

template <int NB>
struct VTile {  // 32 tokens as loaded: tokens 4g .. of the two 16-token tiles
  uint32_t c[2][NB];
  uint32_t s[2][NB];
};

template <int NB>
__device__ __forceinline__ void load_v(const uint8_t *slab, const KvGeo &g, int t0, int lane,
                                       VTile<NB> &v) {
  const int r = lane & 15, grp = lane >> 4;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int t = t0 + 16 * u + 4 * grp;
    load_words<NB>(slab + g.vc + (t * 4 + r) * (4 * NB), v.c[u]);
    load_words<NB>(slab + g.vs + t * NB, v.s[u]);
  }
}

// The scale of page token i (0..3) of half u, block b.
template <int NB>
__device__ __forceinline__ uint32_t v_scale(const VTile<NB> &v, int u, int i, int b) {
  const int at = i * NB + b;
  return (v.s[u][at >> 2] >> (8 * (at & 3))) & 0xFFu;
}

// The offsets come off in one of two ways.  With three terms (fp32), in the
// same sums: a product of -1.46875 * 2^(e-127) for every product of words, so
// that a sum never grows past its own size.  With one (bf16), in a sum of
// their own: rows 4 g + i of one product hold sum p 2^(e-127) of block i (mod
// D/32), taken off the others every 2048 tokens of a wave and at its end; that
// costs a product a tile and four blocks instead of two a block, and rounding
// errors below 2^-24 * 24 a step, far under the numerators' own.
template <int NB, int RT>
struct Offsets {
  floatx4 sum[RT][(NB + 3) / 4];
};

template <int NB, int RT, int VX>
__device__ __forceinline__ void add_values(const VTile<NB> &v, const u32x4v (&p)[RT][VX],
                                           floatx4 (&acc)[RT][NB][2], floatx4 (&l)[RT],
                                           Offsets<NB, RT> &offs, int lane) {
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    u32x4v even, odd, off;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // token pairs
      const int u = i >> 1, a0 = (2 * (i & 1)) * NB + b, a1 = a0 + NB;
      const uint32_t sel = 0x0C000C00u | (a0 & 3) | (4 + (a1 & 3)) << 16;
      const uint32_t base = __builtin_amdgcn_perm(v.s[u][a1 >> 2], v.s[u][a0 >> 2], sel) << 7;
      const uint32_t w = v.c[u][(i & 1) * (NB / 2) + (b >> 1)];
      even[i] = and_or(b & 1 ? w >> 5 : w << 3, kCodeMask, base);
      odd[i] = and_or(b & 1 ? w >> 9 : w >> 1, kCodeMask, base);
      off[i] = base | kNegOffset;
    }
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int x = 0; x < VX; ++x) {
        if (VX > 1) {
          acc[t][b][0] = mfma(off, p[t][x], acc[t][b][0]);
          acc[t][b][1] = mfma(off, p[t][x], acc[t][b][1]);
        }
        acc[t][b][0] = mfma(even, p[t][x], acc[t][b][0]);
        acc[t][b][1] = mfma(odd, p[t][x], acc[t][b][1]);
      }
  }
  if constexpr (VX == 1) {
    // row r = lane & 15 takes block r mod 4 (or 2) of every token
    const int r = lane & (NB == 2 ? 1 : 3);
    const uint32_t sel = 0x0C000C00u | r | ((NB == 2 ? 2 : 4) + r) << 16;
#pragma unroll
    for (int j = 0; j < (NB + 3) / 4; ++j) {
      u32x4v e;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = i >> 1, d0 = NB == 2 ? i & 1 : (2 * (i & 1) * NB) / 4 + j;
        e[i] = __builtin_amdgcn_perm(v.s[u][NB == 2 ? d0 : d0 + NB / 4], v.s[u][d0], sel) << 7;
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) offs.sum[t][j] = mfma(e, p[t][0], offs.sum[t][j]);
    }
  }
  const u32x4v ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int x = 0; x < VX; ++x) l[t] = mfma(ones, p[t][x], l[t]);
}

// ------------------------------------------------------------------ forward
//
// What bounds it: instruction issue, then HBM.  A wave's 32-token tile of a
// head of 128 is 4352 bytes, about 290 vector instructions (two thirds of
// them the two decodes) and, at 32 rows, 40 matrix instructions.  Measured on
// an MI355X: 5 columns of 32 heads over 131071 tokens (143 MB) 37 us, 3.8
// TB/s, 79% of a large copy's rate; 64 sequences of up to 4096 tokens 4.0
// TB/s; one column over 1021 tokens 11.7 us, a chain of loads.  Tried and not
// kept: 256, 768, 1024 and 2048 workgroups instead of 512 (22, 15, 12 and 33%
// slower at 16 ragged sequences: a second round of workgroups costs more than
// it evens out).

// Workgroup (x, y, z): kv head and row block x, split y, sequence z.  A row
// block is 16 RT of the sequence's rows (column, head of the group); its W waves
// share out the split's 32-token tiles and join their sums in LDS.
template <int NB, int VX, int RT, int W>
__global__ __launch_bounds__(64 * W, NB == 8 ? 1 : 2) void k_attn(AttnArgs a) {
  constexpr int D = 32 * NB;
  constexpr int LD = D + 4;
  __shared__ float sh_ml[W][RT * 16][3];
  __shared__ __align__(16) float sh_o[W][16][LD];
  __shared__ QShared<NB, VX> sh_q[RT];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  // The last rows see most: they start first (a chunk over its own 2048 tokens,
  // fp32: 169 -> 162 us).
  const int head = blockIdx.x % a.v.hk, rb0 = a.row_blocks - 1 - blockIdx.x / a.v.hk;
  const int split = blockIdx.y, seq = blockIdx.z;
  const int s0 = a.v.starts[seq];
  const int n = min(a.v.starts[seq + 1], a.n_rows) - s0;
  const int n_all = a.v.starts[seq + 1] - s0;
  if (s0 < 0 || n <= 0) return;
  const int len = kv_len(a.v, seq);
  const long long rows = (long long)n * a.group;
  const KvGeo geo = a.v.g;
  const int32_t *table = a.v.table + (size_t)seq * a.v.pages_per_seq;

  for (long long r0 = (long long)rb0 * (16 * RT); r0 < rows; r0 += (long long)a.row_blocks * (16 * RT)) {
    int vis[RT];
    int first_vis, last_vis;
    {
      const int c0 = (int)(r0 / a.group);
      long long e = r0 + 16 * RT - 1;
      if (e >= rows) e = rows - 1;
      const int c1 = (int)(e / a.group);
      first_vis = min(len, max(0, len - n_all + c0 + 1));
      last_vis = min(len, max(0, len - n_all + c1 + 1));
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      long long r = r0 + 16 * t + m;
      const bool live = r < rows;
      if (!live) r = rows - 1;
      const int col = (int)(r / a.group), hd = head * a.group + (int)(r % a.group);
      vis[t] = min(len, max(0, len - n_all + col + 1));
      if (wave == t) {
        QTile<NB, VX> q;
        load_q<NB, VX>(a.q, (size_t)(s0 + col) * a.q_stride + (size_t)hd * D, live, g, q);
#pragma unroll
        for (int x = 0; x < VX; ++x)
#pragma unroll
          for (int b = 0; b < NB; ++b) sh_q[t].at[x * NB + b][lane] = q.w[x][b];
        sh_q[t].at[VX * NB][lane] = q.off;
      }
    }
    const int tiles = (last_vis + kTile - 1) / kTile;
    const int per = (tiles + a.splits - 1) / a.splits;
    const int t_first = min(tiles, split * per), t_last = min(tiles, t_first + per);

    floatx4 acc[RT][NB][2], l[RT];
    Offsets<NB, RT> offs;
    // l is the sum of the numerators as they enter the second product, the
    // output's denominator (so that rounding them to bf16 cancels where one
    // token has the weight); exact the one before bf16 rounding, for lse
    // mx: raw maximum; a score above thr moves it; numerators are 2^(s sc -
    // base), with a wide base against 0 and mx taken off s before
    float mx[RT], thr[RT], base[RT], exact[RT];
    // (finite, so that a row without a maximum stays without)
    const float room = fminf(8.f / a.sc, 3.0e38f);
    uint32_t poison[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      l[t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < (NB + 3) / 4; ++j) offs.sum[t][j] = floatx4{0.f, 0.f, 0.f, 0.f};
      mx[t] = thr[t] = kNegInf;
      base[t] = 0.f;
      exact[t] = 0.f;
      poison[t] = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[t][b][0] = acc[t][b][1] = floatx4{0.f, 0.f, 0.f, 0.f};
    }

    // a wave's loads run two tiles ahead of what it computes, and the page of a
    // tile is looked up one tile before that
    struct Raw {
      KTile<NB> k[2];
      VTile<NB> v;
      bool held;
    } raw0, raw1;
    const auto page_of = [&](int tile) {
      return scalar_read(table + ((min(tile, t_last - 1) * kTile) >> geo.page_log));
    };
    const auto load = [&](int tile, int page, Raw &r) {
      const int tp = (min(tile, t_last - 1) * kTile) & (geo.page_tokens - 1);
      r.held = (unsigned)page < (unsigned)a.v.n_pages;
      const uint8_t *slab = a.v.pool + ((size_t)(r.held ? page : 0) * a.v.hk + head) * geo.slab;
      load_k<NB>(slab, geo, tp, lane, r.k[0]);
      load_k<NB>(slab, geo, tp + 16, lane, r.k[1]);
      load_v<NB>(slab, geo, tp, lane, r.v);
    };
    int tile = t_first + wave, next_page = 0;
    if (tile < t_last) {
      load(tile, page_of(tile), raw0);
      load(tile + W, page_of(tile + W), raw1);
      next_page = page_of(tile + 2 * W);
    }
    __syncthreads();  // the queries are in LDS
    const auto take_off = [&]() {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float o = -kOffset * offs.sum[t][b >> 2][NB == 2 ? b : b & 3];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[t][b][0][i] += o;
            acc[t][b][1][i] += o;
          }
        }
#pragma unroll
        for (int j = 0; j < (NB + 3) / 4; ++j) offs.sum[t][j] = floatx4{0.f, 0.f, 0.f, 0.f};
      }
    };
    const auto step = [&](Raw &raw) {
      asm volatile("" ::: "memory");  // the queries are read from LDS again, not kept in registers
      const int t0 = tile * kTile;
      KTile<NB> k[2] = {raw.k[0], raw.k[1]};
      VTile<NB> v = raw.v;
      const bool held = raw.held;
      floatx4 s[RT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        KWords<NB> kw;
        decode_k<NB>(k[u], kw);
#pragma unroll
        for (int t = 0; t < RT; ++t) s[t][u] = scores<NB, VX>(kw, sh_q[t], lane);
      }
      if (!held || t0 + kTile > first_vis) {
        // some row does not see some token: its score is -inf, and what its
        // scale says must not reach any row
        const int lim = held ? len : 0;
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (t0 + 16 * u + 4 * g + i >= min(vis[t], lim)) s[t][u][i] = kNegInf;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int slot = t0 + 16 * u + 4 * g + i;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const int at = i * NB + b;
              const bool bad = v_scale<NB>(v, u, i, b) == 255u;
              if (slot >= lim || bad) {
                // a NaN block reaches the rows that see its token, no other
                v.s[u][at >> 2] &= ~(0xFFu << (8 * (at & 3)));
#pragma unroll
                for (int t = 0; t < RT; ++t)
                  if (bad && slot < min(vis[t], lim)) poison[t] |= 1u << b;
              }
            }
          }
      }
      u32x4v p[RT][VX];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float top = fmaxf(fmaxf(fmaxf(s[t][0][0], s[t][0][1]), fmaxf(s[t][0][2], s[t][0][3])),
                          fmaxf(fmaxf(s[t][1][0], s[t][1][1]), fmaxf(s[t][1][2], s[t][1][3])));
        if (__builtin_expect(__ballot(top > thr[t]) != 0, 0)) {
          top = fmaxf(mx[t], max_across_g(top));
          const float f = __builtin_amdgcn_exp2f(base_step(mx[t], top, a.sc));
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            acc[t][b][0] *= f;
            acc[t][b][1] *= f;
          }
#pragma unroll
          for (int j = 0; j < (NB + 3) / 4; ++j) offs.sum[t][j] *= f;
          l[t] *= f;
          exact[t] *= f;
          mx[t] = top;
          const float ref = top == kNegInf ? 0.f : top;
          thr[t] = top + room;
          base[t] = ref * a.sc;
          if (__builtin_expect(__ballot(!(fabsf(base[t]) < kWide)) != 0, 0)) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[t][u][i] -= ref;
            thr[t] = kNegInf;
            base[t] = 0.f;
          }
        }
        float e[8];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            e[4 * u + i] = __builtin_amdgcn_exp2f(fmaf(s[t][u][i], a.sc, -base[t]));
        if (VX == 1)
          exact[t] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
        for (int x = 0; x < VX; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t h = pk_bf16(e[2 * i], e[2 * i + 1]);
            p[t][x][i] = h;
            if (x + 1 < VX) {
              e[2 * i] -= lo_f(h);
              e[2 * i + 1] -= hi_f(h);
            }
          }
      }
      add_values<NB, RT, VX>(v, p, acc, l, offs, lane);
      load(tile + 2 * W, next_page, raw);
      next_page = page_of(tile + 3 * W);
      tile += W;
    };
    for (int turn = 1; tile < t_last; ++turn) {
      step(raw0);
      if (tile >= t_last) break;
      step(raw1);
      if (VX == 1 && (turn & 31) == 0) take_off();
    }
    if (VX == 1) take_off();

    // join the waves: every one scales its sums to the common maximum
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      poison[t] |= __shfl_xor(poison[t], 16);
      poison[t] |= __shfl_xor(poison[t], 32);
      if (VX == 1) exact[t] = cross_row_sum(exact[t]);
      if (g == 0) sh_ml[wave][16 * t + m][0] = mx[t];
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float top = kNegInf;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, sh_ml[w][16 * t + m][0]);
      const float f = __builtin_amdgcn_exp2f(down_to(mx[t], top, a.sc) +
                                             rounded_by(mx[t], base[t], a.sc));
      if (g == 0) {
        sh_ml[wave][16 * t + m][1] = l[t][0] * f;
        sh_ml[wave][16 * t + m][2] = (VX == 1 ? exact[t] : l[t][0]) * f;
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float h = (poison[t] >> b) & 1 ? __builtin_nanf("") : f;
        float4 *o = reinterpret_cast<float4 *>(&sh_o[wave][m][32 * b + 8 * g]);
        o[0] = make_float4(acc[t][b][0][0] * h, acc[t][b][1][0] * h, acc[t][b][0][1] * h,
                           acc[t][b][1][1] * h);
        o[1] = make_float4(acc[t][b][0][2] * h, acc[t][b][1][2] * h, acc[t][b][0][3] * h,
                           acc[t][b][1][3] * h);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * (D / 4); i += 64 * W) {
        const int row = i / (D / 4), d = 4 * (i % (D / 4));
        const long long r = r0 + 16 * t + row;
        if (r < rows) {
          float rt = kNegInf, sum = 0.f, ex = 0.f;
#pragma unroll
          for (int w = 0; w < W; ++w) rt = fmaxf(rt, sh_ml[w][16 * t + row][0]);
          floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < W; ++w) {
            sum += sh_ml[w][16 * t + row][1];
            ex += sh_ml[w][16 * t + row][2];
            o += *reinterpret_cast<const floatx4 *>(&sh_o[w][row][d]);
          }
          const int col = (int)(r / a.group), hd = head * a.group + (int)(r % a.group);
          const size_t rh = (size_t)(s0 + col) * a.heads + hd;
          if (a.splits == 1) {
            if (rt == kNegInf && sum == 0.f) o = floatx4{0.f, 0.f, 0.f, 0.f};
            else o *= 16.f / sum;
            const size_t at = (size_t)(s0 + col) * a.out_stride + (size_t)hd * D + d;
            if (VX == 1)
              *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
                  make_uint2(pk_bf16(o[0], o[1]), pk_bf16(o[2], o[3]));
            else
              *reinterpret_cast<floatx4 *>(static_cast<float *>(a.out) + at) = o;
            if (a.lse && d == 0) a.lse[rh] = lse_of(rt, ex, a.sc);
          } else {
            const size_t at = rh * a.splits + split;
            if (rt != kNegInf || sum != 0.f) *reinterpret_cast<floatx4 *>(a.part + at * D + d) = o;
            if (d == 0) *reinterpret_cast<float4 *>(a.part_ml + 4 * at) = make_float4(rt, sum, ex, 0.f);
          }
        }
      }
      __syncthreads();
    }
  }
}

// Four joined values of a (row, head), and its log of the sum once.
template <int NB, int VX>
__device__ __forceinline__ void join_write(const AttnArgs &a, long long rh, int d, float top,
                                           float sum, float ex, floatx4 o) {
  if (top == kNegInf && sum == 0.f) o = floatx4{0.f, 0.f, 0.f, 0.f};
  else o *= 16.f / sum;
  const size_t at = (size_t)(rh / a.heads) * a.out_stride + (size_t)(rh % a.heads) * (32 * NB) + d;
  if (VX == 1)
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
        make_uint2(pk_bf16(o[0], o[1]), pk_bf16(o[2], o[3]));
  else
    *reinterpret_cast<floatx4 *>(static_cast<float *>(a.out) + at) = o;
  if (a.lse && d == 0) a.lse[rh] = lse_of(top, ex, a.sc);
}

// Joins the splits of a (row, head): a workgroup each, four values a thread,
// the splits dealt out over the 1024/D groups of threads.
template <int NB, int VX>
__global__ __launch_bounds__(kThreads) void k_attn_join(AttnArgs a) {
  constexpr int D = 32 * NB, TG = D / 4, NG = kThreads / TG;
  __shared__ __align__(16) float sh_o[NG][D];
  __shared__ float sh_s[NG][2];
  const int g = threadIdx.x / TG, d = 4 * (threadIdx.x % TG), lane = threadIdx.x & 63;
  const long long last = (long long)min(a.v.starts[a.v.n_seqs], a.n_rows) * a.heads;
  for (long long rh = blockIdx.x; rh < last; rh += gridDim.x) {
    if (rh / a.heads < a.v.starts[0]) continue;
    const float4 *ml = reinterpret_cast<const float4 *>(a.part_ml) + rh * a.splits;
    float top = kNegInf;
    for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, ml[s].x);
#pragma unroll
    for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    float sum = 0.f, ex = 0.f;
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = g; s < a.splits; s += NG) {
      const float4 w = ml[s];
      if (w.x == kNegInf && w.y == 0.f) continue;  // no tokens: its numerators were not written
      const float f = __builtin_amdgcn_exp2f(down_to(w.x, top, a.sc));
      sum += w.y * f;
      ex += w.z * f;
      o += *reinterpret_cast<const floatx4 *>(a.part + (rh * a.splits + s) * D + d) * f;
    }
    *reinterpret_cast<floatx4 *>(&sh_o[g][d]) = o;
    if (d == 0) {
      sh_s[g][0] = sum;
      sh_s[g][1] = ex;
    }
    __syncthreads();
    if (g == 0) {
      for (int i = 1; i < NG; ++i) {
        sum += sh_s[i][0];
        ex += sh_s[i][1];
        o += *reinterpret_cast<const floatx4 *>(&sh_o[i][d]);
      }
      join_write<NB, VX>(a, rh, d, top, sum, ex, o);
    }
    __syncthreads();
  }
}

// The same for few splits: D/4 threads a (row, head) take all of them, and
// nothing is shared.  A split without tokens has written no numerators: what
// stands in their place is read and not taken.  Measured, k_attn_join and this
// in us: 16384 (row, head) of 64 values in 4 splits 29.6, 5.0, of 128 values
// 23.1, 8.4; 640 of 256 values in 12 splits 5.2, 4.8; and beyond, 288 of 128
// values in 16 splits 4.0, 4.6, 320 in 32 splits 5.0, 7.0.
constexpr int kJoinFew = 12;
template <int NB, int VX>
__global__ __launch_bounds__(kThreads) void k_attn_join_few(AttnArgs a) {
  constexpr int D = 32 * NB, TG = D / 4, NG = kThreads / TG;
  const int d = 4 * (threadIdx.x % TG);
  const long long last = (long long)min(a.v.starts[a.v.n_seqs], a.n_rows) * a.heads;
  for (long long rh = (long long)blockIdx.x * NG + threadIdx.x / TG; rh < last;
       rh += (long long)gridDim.x * NG) {
    if (rh / a.heads < a.v.starts[0]) continue;
    const float4 *ml = reinterpret_cast<const float4 *>(a.part_ml) + rh * a.splits;
    float top = kNegInf;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) top = fmaxf(top, ml[s].x);
    float sum = 0.f, ex = 0.f;
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const float4 w = ml[s];
      floatx4 v = *reinterpret_cast<const floatx4 *>(a.part + (rh * a.splits + s) * D + d);
      const bool none = w.x == kNegInf && w.y == 0.f;
      const float f = none ? 0.f : __builtin_amdgcn_exp2f(down_to(w.x, top, a.sc));
      if (none) v = floatx4{0.f, 0.f, 0.f, 0.f};
      sum += w.y * f;
      ex += w.z * f;
      o += v * f;
    }
    join_write<NB, VX>(a, rh, d, top, sum, ex, o);
  }
}

// ------------------------------------------------------- forward, many rows
//
// Where a sequence brings many rows, decoding is shared: a workgroup of eight
// waves, 32 rows each, decodes 64 tokens at a time to exact bf16 values in
// LDS, in the order in which the 32x32x16 matrix instruction's operands are
// read (16 bytes a lane, adjacent lanes adjacent), while it computes the 64
// before.  The offset comes off in the decoding (one mixed-precision fma a
// value, exact_pair), so no product is spent on it.  Lane (row m
// = lane & 31, h = lane >> 5) holds of its row the scores of tokens 8 j + 4 h
// + i (i < 4, j < 4) of 32, and the second product takes j = 2 s and 2 s + 1
// as its step s from that very lane.
constexpr int kChunkWaves = 8;
constexpr int kChunkRows = 32 * kChunkWaves;
constexpr int kChunkTile = 64;
// A score may exceed a row's base by this much (as a power of two) before the
// base moves: rarely reached by scores that rise along a sequence, and little
// of fp32's range, which values as large as 2^100 need as well.
constexpr float kChunkRoom = 16.f;

typedef float floatx16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ floatx16 mfma32(const u32x4v &a, const u32x4v &b, const floatx16 &c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A block's scale 2^(e-127) and offset -1.46875 * 2^(e-127) (NaN for e = 255).
struct Unit {
  float scale, offset;
};
__device__ __forceinline__ Unit unit_of(uint32_t e) {
  return {__uint_as_float(e << 23), __uint_as_float(0x803C0000u | e << 23)};
}

// The values of a pair of codes, each nibble `at` (0..3) of a half-word of w,
// as bf16, exactly: the code in the mantissa of the fp16 number 1 + c/16, one
// mixed-precision fma a value with its block's scale and offset, and the upper
// halves of the two results.
__device__ __forceinline__ uint32_t exact_pair(uint32_t w, int at, Unit lo, Unit hi) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  const uint32_t x = at == 0 ? w << 6 : at == 1 ? w << 2 : at == 2 ? w >> 2 : w >> 6;
  const f16x2 v = __builtin_bit_cast(f16x2, and_or(x, 0x03C003C0u, 0x3C003C00u));
  const float a = __builtin_fmaf((float)v[0], lo.scale, lo.offset);
  const float b = __builtin_fmaf((float)v[1], hi.scale, hi.offset);
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// A lane's share of 64 tokens, of which wave w decodes tokens 8 w .. 8 w + 7:
// of the keys, half the blocks of one token's octet (lane = octet, half,
// token: eight neighbouring lanes write 128 neighbouring bytes of LDS); of the
// values, byte r of every block of a pair of tokens (lane =
// group of four, r, pair).
template <int NB>
struct ChunkRaw {
  uint32_t k[NB / 2], v[NB / 2];
  uint32_t ks;          // the half's scales
  uint32_t vs[NB / 2];  // the pair's scales
};

template <int NB>
__device__ __forceinline__ void chunk_load(const uint8_t *slab, const KvGeo &g, int tp, int lane,
                                           ChunkRaw<NB> &r) {
  const uint8_t *k = slab + g.kc + (tp + (lane & 7)) * (16 * NB) + (lane >> 3) * (2 * NB);
  const uint8_t *v = slab + g.vc + tp * (16 * NB) + lane * (2 * NB);
  const uint8_t *ks = slab + g.ks + (tp + (lane & 7)) * NB + ((lane >> 3) & 1) * (NB / 2);
  const uint8_t *vs = slab + g.vs + (tp + 4 * (lane >> 5) + 2 * (lane & 1)) * NB;
  if constexpr (NB == 2) {
    r.k[0] = *reinterpret_cast<const uint32_t *>(k);
    r.v[0] = *reinterpret_cast<const uint32_t *>(v);
    r.ks = *ks;
    r.vs[0] = *reinterpret_cast<const uint32_t *>(vs);
  } else {
    load_words<NB / 2>(k, r.k);
    load_words<NB / 2>(v, r.v);
    if constexpr (NB == 4) r.ks = *reinterpret_cast<const uint16_t *>(ks);
    else r.ks = *reinterpret_cast<const uint32_t *>(ks);
    load_words<NB / 2>(vs, r.vs);
  }
}

// Decoded keys [32-token half][step of 16 values][h][token][16 bytes] and
// values [step of 16 tokens][block][h][value][16 bytes] of one tile.
template <int NB>
struct ChunkK {
  u32x4v at[2][2 * NB][2][32];
};
template <int NB>
struct ChunkV {
  u32x4v at[4][NB][2][32];
};

template <int NB>
__device__ __forceinline__ void chunk_decode(const ChunkRaw<NB> &r, int wave, int lane,
                                             ChunkK<NB> &tk, ChunkV<NB> &tv) {
  const int tok = 8 * wave + (lane & 7), g = lane >> 4, half = (lane >> 3) & 1;
#pragma unroll
  for (int i = 0; i < NB / 2; ++i) {
    const Unit e = unit_of((r.ks >> (8 * i)) & 0xFFu);
    u32x4v o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = exact_pair(r.k[i], j, e, e);
    tk.at[tok >> 5][2 * (half * (NB / 2) + i) + (g >> 1)][g & 1][tok & 31] = o;
  }
  const int grp = 2 * wave + (lane >> 5), rr = (lane >> 1) & 15;  // group of four tokens, byte
  uint32_t *u = reinterpret_cast<uint32_t *>(&tv.at[grp >> 2][0][grp & 1][2 * rr]) +
                2 * ((grp >> 1) & 1) + (lane & 1);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const Unit e0 = unit_of((r.vs[b >> 2] >> (8 * (b & 3))) & 0xFFu);
    const Unit e1 = unit_of((r.vs[(NB + b) >> 2] >> (8 * ((NB + b) & 3))) & 0xFFu);
    u[b * 256] = exact_pair(r.v[b >> 1], 2 * (b & 1), e0, e1);
    u[b * 256 + 4] = exact_pair(r.v[b >> 1], 2 * (b & 1) + 1, e0, e1);
  }
}

// One barrier a tile: while a tile is computed from one pair of buffers, the
// next is decoded into the other.
//
// Measured on an MI355X: 2048 columns of 32 heads of 128 at the end of 8192
// tokens 276 us, 871 TFLOP/s, 77% of a library's 8192^3 bf16 product (1126); by
// its counters matrix units 41% busy, vector instructions issuing 56% of the
// time.  Tried and not kept, all within 3%: operands read six products ahead,
// both halves' score chains in turn, pages read three tiles ahead, rows written
// through LDS; the scores of a tile beside the exps of the tile before it
// spills (355 us).
template <int NB>
__global__ __launch_bounds__(64 * kChunkWaves) void k_attn_chunk(AttnArgs a) {
  constexpr int D = 32 * NB;
  extern __shared__ __align__(16) uint8_t lds[];
  ChunkK<NB> *buf_k = reinterpret_cast<ChunkK<NB> *>(lds);
  ChunkV<NB> *buf_v = reinterpret_cast<ChunkV<NB> *>(buf_k + 2);
  uint8_t *bad = reinterpret_cast<uint8_t *>(buf_v + 2);  // [2][NB][8 waves]: a bit a token
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int m = lane & 31, h = lane >> 5;
  // The last rows see most: they start first (4096 columns over their own
  // tokens 237 -> 198 us).
  const int head = blockIdx.x % a.v.hk, rb0 = a.row_blocks - 1 - blockIdx.x / a.v.hk;
  const int split = blockIdx.y, seq = blockIdx.z;
  const int s0 = a.v.starts[seq];
  const int n_all = a.v.starts[seq + 1] - s0;
  const int n = min(a.v.starts[seq + 1], a.n_rows) - s0;
  if (s0 < 0 || n <= 0) return;
  const int len = kv_len(a.v, seq);
  const long long rows = (long long)n * a.group;
  const KvGeo geo = a.v.g;
  const int32_t *table = a.v.table + (size_t)seq * a.v.pages_per_seq;

  for (long long r0 = (long long)rb0 * kChunkRows; r0 < rows;
       r0 += (long long)a.row_blocks * kChunkRows) {
    const auto sees = [&](long long r) {  // slots that a row sees
      if (r >= rows) r = rows - 1;
      return min(len, max(0, len - n_all + (int)(r / a.group) + 1));
    };
    const int first_vis = sees(r0), last_vis = sees(r0 + kChunkRows - 1);
    long long r = r0 + 32 * wave + m;
    const bool live = r < rows;
    if (!live) r = rows - 1;
    const int col = (int)(r / a.group), hd = head * a.group + (int)(r % a.group);
    const int vis = sees(r);
    u32x4v q[2 * NB];
    {
      const uint16_t *p = static_cast<const uint16_t *>(a.q) + (size_t)(s0 + col) * a.q_stride +
                          (size_t)hd * D + 8 * h;
#pragma unroll
      for (int ks = 0; ks < 2 * NB; ++ks) {
        const uint4 d = *reinterpret_cast<const uint4 *>(p + 16 * ks);
        q[ks][0] = __builtin_amdgcn_perm(d.z, d.x, 0x05040100u);
        q[ks][1] = __builtin_amdgcn_perm(d.z, d.x, 0x07060302u);
        q[ks][2] = __builtin_amdgcn_perm(d.w, d.y, 0x05040100u);
        q[ks][3] = __builtin_amdgcn_perm(d.w, d.y, 0x07060302u);
      }
    }
    const int all = (last_vis + kChunkTile - 1) / kChunkTile;
    const int per = (all + a.splits - 1) / a.splits;
    const int t_first = min(all, split * per), t_last = min(all, t_first + per);
    // tiles that this wave's rows see
    const int wave_vis = r0 + 32 * wave < rows ? sees(r0 + 32 * wave + 31) : 0;
    const int t_wave = min(t_last, (wave_vis + kChunkTile - 1) / kChunkTile);

    floatx16 acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[b][i] = 0.f;
    // as in k_attn; sum is of the numerators before bf16 rounding, the output's
    // denominator and lse's: one of the rounded ones besides would cost a
    // vector instruction a score more
    float mx = kNegInf, base = 0.f, thr = kNegInf, sum = 0.f;
    const float room = fminf(kChunkRoom / a.sc, 3.0e38f);  // finite, as in k_attn
    uint32_t poison = 0;

    // the page of a token (of the table's last token, past its end)
    const auto page_at = [&](int token) {
      return scalar_read(table + min(token >> geo.page_log, a.v.pages_per_seq - 1));
    };
    const auto is_page = [&](int page) { return (unsigned)page < (unsigned)a.v.n_pages; };
    // every row sees every token of the tile
    const auto is_whole = [&](int tile) {
      const int t0 = tile * kChunkTile;
      return t0 + kChunkTile <= first_vis && is_page(page_at(t0)) && is_page(page_at(t0 + 32));
    };
    // the page of this wave's 8 tokens of a tile (of the last, past its end)
    const auto page_of = [&](int tile) {
      return page_at(min(tile, t_last - 1) * kChunkTile + 8 * wave);
    };
    const auto load = [&](int tile, int page, ChunkRaw<NB> &raw) {
      const int tp = (min(tile, t_last - 1) * kChunkTile + 8 * wave) & (geo.page_tokens - 1);
      chunk_load<NB>(a.v.pool + ((size_t)(is_page(page) ? page : 0) * a.v.hk + head) * geo.slab,
                     geo, tp, lane, raw);
    };
    // In a tile that some row sees only a part of, tokens that no row may read
    // lose their scales, and value blocks marked NaN become 0 and a bit in
    // `bad`, from which each row takes what it sees.
    const auto screen = [&](int tile, int page, ChunkRaw<NB> &raw, int at) {
      const int first = tile * kChunkTile + 8 * wave;
      const int lim = is_page(page) ? len : 0;
      if (first + (lane & 7) >= lim) raw.ks = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int by = i * NB + b;
          const bool out = first + 4 * (lane >> 5) + 2 * (lane & 1) + i >= lim;
          const bool nan = !out && ((raw.vs[by >> 2] >> (8 * (by & 3))) & 0xFFu) == 255u;
          if (out || nan) raw.vs[by >> 2] &= ~(0xFFu << (8 * (by & 3)));
          const uint64_t v = __ballot(nan);
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int pr = 0; pr < 2; ++pr)
              mask |= (uint32_t)((v >> (32 * g + pr)) & 1) << (4 * g + 2 * pr + i);
        }
        if (lane == 0) bad[(at * NB + b) * kChunkWaves + wave] = (uint8_t)mask;
      }
    };
    // scores of one half of a tile
    const auto scores_of = [&](const ChunkK<NB> &t, int u, floatx16 &o) {
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 2 * NB; ++ks) o = mfma32(t.at[u][ks][h][m], q[ks], o);
    };
    const auto hide = [&](int tile, int u, int at, floatx16 &o) {
      const int t0 = tile * kChunkTile + 32 * u;
      const int lim = is_page(page_at(t0)) ? vis : 0;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t0 + 8 * (i >> 2) + 4 * h + (i & 3) >= lim) o[i] = kNegInf;
      const int seen = lim - t0;
      const uint32_t in = seen <= 0 ? 0u : seen >= 32 ? 0xFFFFFFFFu : (1u << seen) - 1u;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (*reinterpret_cast<const uint32_t *>(&bad[(at * NB + b) * kChunkWaves + 4 * u]) & in)
          poison |= 1u << b;
    };
    const auto top_of = [&](const floatx16 &o) {
      float t = o[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) t = fmaxf(t, o[i]);
      return t;
    };
    const auto numerators = [&](floatx16 &o, u32x4v (&p)[2]) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        o[i] = __builtin_amdgcn_exp2f(fmaf(o[i], a.sc, -base));
        x += o[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i >> 2][i & 3] = pk_bf16(o[2 * i], o[2 * i + 1]);
      sum += x;
    };
    const auto add_up = [&](const ChunkV<NB> &t, int u, const u32x4v (&p)[2]) {
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = mfma32(t.at[2 * u + st][b][h][m], p[st], acc[b]);
    };

    ChunkRaw<NB> raw;
    int page = 0;
    if (t_first < t_last) {
      page = page_of(t_first);
      load(t_first, page, raw);
      if (!is_whole(t_first)) screen(t_first, page, raw, 0);
      chunk_decode<NB>(raw, wave, lane, buf_k[0], buf_v[0]);
      page = page_of(t_first + 1);
      load(t_first + 1, page, raw);
    }
    // Decode the tile behind (past the last, that one again, into a free
    // buffer), and load the one after it.
    const auto next = [&](int tile, int at) {
      chunk_decode<NB>(raw, wave, lane, buf_k[at], buf_v[at]);
      page = page_of(tile + 2);
      load(tile + 2, page, raw);
    };
    // Of the two waves of a SIMD one decodes before its products and one
    // after them, so that one's vector work stands beside the other's matrix
    // work.
    const bool early = wave >= 4;

    // The inner loop keeps the base that numerators are relative to.  A score
    // far above it leaves it (so does the first tile); everything summed up so
    // far is scaled to a new base, and that tile is computed here, whatever its
    // scores.
    const auto scores_at = [&](int tile, int at, floatx16 &s0, floatx16 &s1) {
      scores_of(buf_k[at], 0, s0);
      scores_of(buf_k[at], 1, s1);
      if (!is_whole(tile)) {
        hide(tile, 0, at, s0);
        hide(tile, 1, at, s1);
      }
      return fmaxf(top_of(s0), top_of(s1));
    };
    const auto take = [&](int at, floatx16 &s0, floatx16 &s1) {
      u32x4v p0[2], p1[2];
      numerators(s0, p0);
      add_up(buf_v[at], 0, p0);
      numerators(s1, p1);
      add_up(buf_v[at], 1, p1);
    };
    for (int tile = t_first; tile < t_last; ++tile) {
      float top = kNegInf;
      for (; tile < t_last; ++tile) {
        const int at = (tile - t_first) & 1;
        __syncthreads();
        if (tile + 1 < t_last && !is_whole(tile + 1)) screen(tile + 1, page, raw, at ^ 1);
        if (early) next(tile, at ^ 1);
        if (tile < t_wave) {
          floatx16 s0, s1;
          top = scores_at(tile, at, s0, s1);
          if (__ballot(top > thr)) break;
          take(at, s0, s1);
        }
        if (!early) next(tile, at ^ 1);
      }
      if (tile < t_last) {
        const int at = (tile - t_first) & 1;
        const uint32_t x = __float_as_uint(top);
        const auto sw = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        top = fmaxf(mx, fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1])));
        const float f = __builtin_amdgcn_exp2f(base_step(mx, top, a.sc));
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] *= f;
        sum *= f;
        mx = top;
        const float ref = top == kNegInf ? 0.f : top;
        base = ref * a.sc;
        thr = top + room;
        floatx16 s0, s1;
        scores_at(tile, at, s0, s1);
        if (__ballot(!(fabsf(base) < kWide))) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            s0[i] -= ref;
            s1[i] -= ref;
          }
          thr = kNegInf;
          base = 0.f;
        }
        take(at, s0, s1);
        if (!early) next(tile, at ^ 1);
      }
    }
    __syncthreads();

    sum += __shfl_xor(sum, 32);
    poison |= __shfl_xor(poison, 32);
    if (live) {
      const size_t rh = (size_t)(s0 + col) * a.heads + hd;
      const bool empty = mx == kNegInf && sum == 0.f;
      const float whole = __builtin_amdgcn_exp2f(rounded_by(mx, base, a.sc));
      const float inv = a.splits > 1 ? whole : empty ? 0.f : 16.f / sum;
      sum *= whole;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float f = (poison >> b) & 1 ? __builtin_nanf("") : inv;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          floatx4 o = {acc[b][4 * j], acc[b][4 * j + 1], acc[b][4 * j + 2], acc[b][4 * j + 3]};
          o *= f;
          const int d = 32 * b + 8 * j + 4 * h;
          if (a.splits == 1)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) +
                                       (size_t)(s0 + col) * a.out_stride + (size_t)hd * D + d) =
                make_uint2(pk_bf16(o[0], o[1]), pk_bf16(o[2], o[3]));
          else
            *reinterpret_cast<floatx4 *>(a.part + (rh * a.splits + split) * D + d) = o;
        }
      }
      if (h == 0) {
        if (a.splits > 1)
          *reinterpret_cast<float4 *>(a.part_ml + 4 * (rh * a.splits + split)) =
              make_float4(mx, sum, sum, 0.f);
        else if (a.lse)
          a.lse[rh] = lse_of(mx, sum, a.sc);
      }
    }
  }
}

// ------------------------------------------------------------------ weights

struct WeightArgs {
  KvView v;
  const void *q;
  const float *lse, *acc;
  float *acc_out;
  long long q_stride;
  int heads, group, n_rows;
  float sc, decay;
};

// Sums of eight values over the 16 lanes of a row, all at once: the lanes m
// with bit 0 clear then hold the total of value ms_index<8>(m).
__device__ __forceinline__ float row_sums(const float (&v)[8], int lane) {
  float a[4], b[2], c[1];
  ms_step<0x140, 3, 8>(v, a, lane);
  ms_step<0x141, 2, 4>(a, b, lane);
  ms_step<0x4E, 1, 2>(b, c, lane);
  return c[0] + dpp_f<0xB1>(c[0]);
}

// Workgroup (x, y, z): kv head x of sequence z, 32-token tiles shared out over
// the waves of all y.  The rows' operands stand in LDS, QB tiles of 16 at a
// time, while the keys pass, the next tile's loads in flight.  Measured: 4
// sequences of up to 16384 tokens, 4 columns of 32 heads, 14.1 us.
template <int NB, int VX>
__global__ __launch_bounds__(kThreads) void k_attn_weights(WeightArgs a) {
  constexpr int D = 32 * NB, QB = VX == 1 ? 4 : 2;
  __shared__ QShared<NB, VX> sh_q[QB];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int head = blockIdx.x, seq = blockIdx.z;
  const int len = kv_len(a.v, seq);
  const KvGeo geo = a.v.g;
  const int s0 = a.v.starts[seq];
  const int n_all = a.v.starts[seq + 1] - s0;
  const int n = s0 < 0 ? 0 : min(a.v.starts[seq + 1], a.n_rows) - s0;
  const long long rows = n > 0 ? (long long)n * a.group : 0;
  const size_t base = ((size_t)seq * a.v.hk + head) * kv_capacity(a.v);
  const int32_t *table = a.v.table + (size_t)seq * a.v.pages_per_seq;
  const int tiles = (len + kTile - 1) / kTile, step = gridDim.y * kWaves;
  const int first = blockIdx.y * kWaves + wave;
  const int mine = ms_index<8>(m);  // the value that this lane writes
  for (long long r0 = 0; r0 == 0 || r0 < rows; r0 += 16 * QB) {
    float z[QB];
    int vis[QB];
    if (r0) __syncthreads();
#pragma unroll
    for (int t = 0; t < QB; ++t) {
      const long long r = r0 + 16 * t + m;
      const bool live = r < rows;
      const int col = live ? (int)(r / a.group) : 0;
      const int hd = head * a.group + (live ? (int)(r % a.group) : 0);
      z[t] = live ? a.lse[(size_t)(s0 + col) * a.heads + hd] : 0.f;
      vis[t] = live ? min(len, max(0, len - n_all + col + 1)) : 0;
      if (z[t] == kNegInf) vis[t] = 0, z[t] = 0.f;
      z[t] *= 1.4426950408889634f;
      if (wave == t && r0 + 16 * t < rows) {
        QTile<NB, VX> q;
        load_q<NB, VX>(a.q, (size_t)(s0 + col) * a.q_stride + (size_t)hd * D, live, g, q);
#pragma unroll
        for (int x = 0; x < VX; ++x)
#pragma unroll
          for (int b = 0; b < NB; ++b) sh_q[t].at[x * NB + b][lane] = q.w[x][b];
        sh_q[t].at[VX * NB][lane] = q.off;
      }
    }
    const int live_tiles = (int)min((long long)QB, (rows - r0 + 15) / 16);
    KTile<NB> next[2];
    bool next_held = false;
    const auto load = [&](int tile) {
      const int t0 = min(tile, tiles - 1) * kTile;
      const int page = scalar_read(table + (t0 >> geo.page_log));
      next_held = (unsigned)page < (unsigned)a.v.n_pages;
      const uint8_t *slab = a.v.pool + ((size_t)(next_held ? page : 0) * a.v.hk + head) * geo.slab;
      const int tp = t0 & (geo.page_tokens - 1);
      load_k<NB>(slab, geo, tp, lane, next[0]);
      load_k<NB>(slab, geo, tp + 16, lane, next[1]);
    };
    if (first < tiles) load(first);
    __syncthreads();
    for (int tile = first; tile < tiles; tile += step) {
      const int t0 = tile * kTile;
      const int slot = t0 + 16 * (mine >> 2) + 4 * g + (mine & 3);
      const bool writes = !(m & 1) && slot < len;
      float old = 0.f;
      if (writes) old = r0 ? a.acc_out[base + slot] : a.acc[base + slot] * a.decay;
      const bool held = next_held;
      KWords<NB> kw[2];
      decode_k<NB>(next[0], kw[0]);
      decode_k<NB>(next[1], kw[1]);
      load(tile + step);
      float sum[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = 0.f;
#pragma unroll
      for (int t = 0; t < QB; ++t) {
        if (held && t < live_tiles) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const floatx4 s = scores<NB, VX>(kw[u], sh_q[t], lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float e = __builtin_amdgcn_exp2f(fmaf(s[i], a.sc, -z[t]));
              sum[4 * u + i] += t0 + 16 * u + 4 * g + i < vis[t] ? e : 0.f;
            }
          }
        }
      }
      const float r = row_sums(sum, lane);
      if (writes) a.acc_out[base + slot] = old + r;
    }
  }
}

// Between a wave's own stores to LDS and its lanes' reads of each other's.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

// Many rows.  A workgroup takes two 32-token tiles, one from each end of the
// sequence, one after the other: rows see early tokens more than late ones,
// and so every workgroup has about the same to do.  A tile's keys are decoded
// to exact bf16 operands once, by every wave for itself, and stay in registers
// while the eight waves share out the rows, 32 at a time.  Every workgroup
// reads all rows that see its tiles, from the caches: a wave reads them whole,
// neighbouring lanes a row, and turns them over in its own part of
// LDS (pieces of 16 bytes, a row's exchanged by its number, so that both sides
// are free of bank conflicts).  Each lane reading its own row from memory was
// bound by a cache line a lane: 64 us.  The waves' sums meet in LDS.
// Measured: 2048 columns of 32 heads of 128 over their own 2048 tokens 47 us.
template <int NB, int VX>
__global__ __launch_bounds__(64 * kChunkWaves) void k_attn_weights_chunk(WeightArgs a) {
  constexpr int D = 32 * NB, KS = 2 * NB;
  constexpr int kBytes = D * (VX == 1 ? 2 : 4);     // of a row
  constexpr int SEG = kBytes >= 256 ? 16 : 8;       // 16-byte pieces of a row staged at a time
  constexpr int STEPS = VX == 1 ? SEG / 2 : SEG / 4;  // products of a stage
  // Loads a stage ahead: 4096 rows over 2048 tokens in bf16 48.5 -> 46.5 us,
  // but fp32 92.7 -> 98.5 us, whose three terms leave fewer registers.
  constexpr bool kAhead = VX == 1;
  __shared__ __align__(16) u32x4v stage[kChunkWaves][32 * SEG];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int m = lane & 31, h = lane >> 5;
  u32x4v *const mine = stage[wave];
  const auto red = [&](int w) { return reinterpret_cast<float *>(stage[w]); };
  const auto piece = [](int row, int at) { return row * SEG + (at ^ (row & (SEG - 1))); };
  const int head = blockIdx.x, seq = blockIdx.z;
  const int len = kv_len(a.v, seq);
  const KvGeo geo = a.v.g;
  const int s0 = a.v.starts[seq];
  const int n_all = a.v.starts[seq + 1] - s0;
  const int n = s0 < 0 ? 0 : min(a.v.starts[seq + 1], a.n_rows) - s0;
  const long long rows = n > 0 ? (long long)n * a.group : 0;
  const size_t cap = kv_capacity(a.v);
  const int tiles = (len + 31) / 32;
  for (int turn = 2 * blockIdx.y; turn < tiles;
       turn = turn & 1 ? turn + 2 * (int)gridDim.y - 1 : turn + 1) {
    const int t0 = 32 * (turn & 1 ? tiles - 1 - (turn >> 1) : turn >> 1);
    const int page = scalar_read(a.v.table + (size_t)seq * a.v.pages_per_seq + (t0 >> geo.page_log));
    const bool held = (unsigned)page < (unsigned)a.v.n_pages;
    const uint8_t *slab = a.v.pool + ((size_t)(held ? page : 0) * a.v.hk + head) * geo.slab;
    const int tp = (t0 & (geo.page_tokens - 1)) + m;
    uint32_t c[2][NB], sb[(NB + 3) / 4];
    load_words<NB>(slab + geo.kc + tp * (16 * NB) + h * (4 * NB), c[0]);
    load_words<NB>(slab + geo.kc + tp * (16 * NB) + (2 + h) * (4 * NB), c[1]);
    const uint8_t *sp = slab + geo.ks + tp * NB;
    if constexpr (NB == 2) sb[0] = *reinterpret_cast<const uint16_t *>(sp);
    else if constexpr (NB == 4) sb[0] = *reinterpret_cast<const uint32_t *>(sp);
    else load_words<2>(sp, sb);
    u32x4v k[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int b = ks >> 1;
      const Unit e = unit_of((sb[b >> 2] >> (8 * (b & 3))) & 0xFFu);
#pragma unroll
      for (int j = 0; j < 4; ++j) k[ks][j] = exact_pair(c[ks & 1][b], j, e, e);
    }
    float sum[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[i] = 0.f;
    // columns that see none of the tile's tokens add nothing
    const long long first = (long long)max(0, t0 - (len - n_all)) * a.group / 32;
    int col, hd;    // of row r0 + m, or of the last one
    long long off;  // and where it begins
    const auto locate = [&](long long r0) {
      const unsigned r = (unsigned)min(r0 + m, rows - 1);  // rows are 2^30 at most
      col = (int)(r / (unsigned)a.group);
      hd = (head - col) * a.group + (int)r;
      off = ((long long)(s0 + col) * a.q_stride + (long long)hd * D) * (VX == 1 ? 2 : 4);
    };
    u32x4v d[SEG / 2];
    const auto fetch = [&](int st) {
#pragma unroll
      for (int i = 0; i < SEG / 2; ++i)
        d[i] = *reinterpret_cast<const u32x4v *>(static_cast<const uint8_t *>(a.q) +
                                                __shfl(off, (64 * i + lane) / SEG) +
                                                16 * (SEG * st + lane % SEG));
    };
    long long r0 = 32 * (first + wave);
    if (kAhead && held && r0 < rows) {
      locate(r0);
      fetch(0);
    }
    for (; held && r0 < rows; r0 += 32 * kChunkWaves) {
      if (!kAhead) locate(r0);
      float z = a.lse[(size_t)(s0 + col) * a.heads + hd];
      int vis = r0 + m < rows ? min(len, max(0, len - n_all + col + 1)) : 0;
      floatx16 s;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
      for (int st = 0; st < kBytes / (16 * SEG); ++st) {
        if (!kAhead) fetch(st);
        wave_fence();  // the stage before has been read
#pragma unroll
        for (int i = 0; i < SEG / 2; ++i) mine[piece((64 * i + lane) / SEG, lane % SEG)] = d[i];
        wave_fence();
        // the next piece, or the next rows' first (past the end, the last row's)
        if (kAhead && st + 1 < kBytes / (16 * SEG)) {
          fetch(st + 1);
        } else if (kAhead) {
          locate(r0 + 32 * kChunkWaves);
          fetch(0);
        }
#pragma unroll
        for (int step = 0; step < STEPS; ++step) {
          const int ks = st * STEPS + step;
          if constexpr (VX == 1) {
            const u32x4v x = mine[piece(m, 2 * step + h)];
            const u32x4v q = {__builtin_amdgcn_perm(x[2], x[0], 0x05040100u),
                              __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                              __builtin_amdgcn_perm(x[3], x[1], 0x05040100u),
                              __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
            s = mfma32(k[ks], q, s);
          } else {
            const float4 x = __builtin_bit_cast(float4, mine[piece(m, 4 * step + 2 * h)]);
            const float4 y = __builtin_bit_cast(float4, mine[piece(m, 4 * step + 2 * h + 1)]);
            float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int t = 0; t < VX; ++t) {
              u32x4v q;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                q[i] = pk_bf16(v[i], v[i + 4]);
                v[i] -= lo_f(q[i]);
                v[i + 4] -= hi_f(q[i]);
              }
              s = mfma32(k[ks], q, s);
            }
          }
        }
      }
      if (z == kNegInf) vis = 0, z = 0.f;
      z *= 1.4426950408889634f;
      if (__ballot(t0 + 32 > vis)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float e = __builtin_amdgcn_exp2f(fmaf(s[i], a.sc, -z));
          sum[i] += t0 + 8 * (i >> 2) + 4 * h + (i & 3) < vis ? e : 0.f;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] += __builtin_amdgcn_exp2f(fmaf(s[i], a.sc, -z));
      }
    }
    {
      // all sixteen sums over the 32 lanes at once: lane m < 16 has number
      // ms_index<16>(m)
      float v8[8], v4[4], v2[2], v1[1];
      ms_step<0x140, 3, 16>(sum, v8, lane);
      ms_step<0x141, 2, 8>(v8, v4, lane);
      ms_step<0x4E, 1, 4>(v4, v2, lane);
      ms_step<0xB1, 0, 2>(v2, v1, lane);
      const uint32_t u = __float_as_uint(v1[0]);
      const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
      const int i = ms_index<16>(m & 15);
      wave_fence();  // the sums lie over the stage, which lanes of this wave have just read
      if (m < 16)
        red(wave)[8 * (i >> 2) + 4 * h + (i & 3)] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    __syncthreads();
    if (threadIdx.x < 32 && t0 + (int)threadIdx.x < len) {
      float r = 0.f;
#pragma unroll
      for (int w = 0; w < kChunkWaves; ++w) r += red(w)[threadIdx.x];
      const size_t at = ((size_t)seq * a.v.hk + head) * cap + t0 + threadIdx.x;
      a.acc_out[at] = fmaf(a.acc[at], a.decay, r);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- host side

constexpr int kChunkMin = 64;    // rows of a sequence that count as many
constexpr int kWeightsMin = 256;  // ... for k_attn_weights_chunk
constexpr int kChunkSplit = 16;  // tiles of a split of k_attn_chunk, at least

struct AttnPlan {
  int rt, row_blocks, splits, waves;
  bool chunk;
  size_t part, ml, total;
};

// Rows of a block: 16 where a sequence has no more, or fp32 is computed in
// three terms; 32 otherwise.  A short sequence is one workgroup's, with no
// second launch; a longer one is split so that the workgroups fill the chip
// once (two a compute unit), each wave with a tile at least.
//
// Many rows of bf16 go to k_attn_chunk, one workgroup a compute unit, where
// splits of 16 tiles (1024 tokens) or more give it half the chip: 8 kv heads
// of 128, rows of a sequence x tokens, k_attn and k_attn_chunk in us: 8192 x
// 8192 422, 293; 8192 x 2048 95, 82; 512 x 16384 77, 61; and without that
// 256 x 4096 (two sequences) 36, 43; 256 x 500 16, 30.
AttnPlan attn_plan(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int heads, int n_rows,
                   int xtype) {
  AttnPlan p;
  const int group = heads / c->n_kv_heads;
  const long long rows = (long long)(b->max_cols > 1 ? b->max_cols : 1) * group;
  const long long cap = (long long)b->pages_per_seq * c->page_tokens;
  const long long len = b->max_len < cap ? b->max_len : cap;
  const long long pairs = (long long)b->n_seqs * c->n_kv_heads;
  const long long most_rb = (1 << 20) / c->n_kv_heads;  // a workgroup takes several beyond that
  const auto clamp = [](long long v, long long lo, long long hi) {
    return v > hi ? hi : v < lo ? lo : v;
  };
  p.rt = rows <= 16 || xtype == RFPX_X_F32 || c->head_dim == 256 ? 1 : 2;
  p.chunk = false;
  if (rows > kChunkMin && xtype == RFPX_X_BF16 && c->head_dim <= 128) {
    const long long tiles = (len + kChunkTile - 1) / kChunkTile;
    const long long wgs = pairs * ((rows + kChunkRows - 1) / kChunkRows);
    const long long s = clamp(clamp(256 / wgs, 1, 64), 1, tiles / kChunkSplit);
    if (tiles >= kChunkSplit && wgs * s >= 128) {
      p.chunk = true;
      p.waves = kChunkWaves;
      p.splits = (int)s;
    }
  }
  const long long block = p.chunk ? kChunkRows : 16 * p.rt;
  p.row_blocks = (int)clamp((rows + block - 1) / block, 1, most_rb);
  if (!p.chunk) {
    const long long wgs = pairs * p.row_blocks, tiles = (len + kTile - 1) / kTile;
    if (tiles <= 4 * kWavesOne && wgs < 512 && c->head_dim < 256) {
      p.waves = kWavesOne;
      p.splits = 1;
    } else {
      p.waves = kWaves;
      p.splits = (int)clamp(clamp(512 / wgs, 1, 128), 1, (tiles + kWaves - 1) / kWaves);
      if (p.splits < 1) p.splits = 1;
    }
  }
  const size_t rh = (size_t)n_rows * heads;
  p.part = 0;
  p.ml = align_up(p.splits > 1 ? rh * p.splits * c->head_dim * 4 : 0, 256);
  p.total = p.ml + align_up(p.splits > 1 ? rh * p.splits * 16 : 0, 256);
  if (p.total < 256) p.total = 256;  // a supported shape never reads as "unsupported"
  return p;
}

rfpx_status check_heads(const char *fn, const rfpx_kv_cache *c, int heads, int n_rows, int xtype,
                        float scale) {
  if (!valid_xtype(xtype)) return fail(RFPX_E_ARG, "%s: xtype=%d", fn, xtype);
  if (heads < 1 || heads > RFPX_HEADS_MAX || heads % c->n_kv_heads)
    return fail(RFPX_E_SHAPE, "%s: %d query heads over %d kv heads", fn, heads, c->n_kv_heads);
  if (n_rows < 0 || n_rows > RFPX_ROWS_MAX)
    return fail(RFPX_E_SHAPE, "%s: n_rows=%d: must be in [0, %d]", fn, n_rows, RFPX_ROWS_MAX);
  if (!(scale > 0.f) || !(scale < 1e30f)) return fail(RFPX_E_ARG, "%s: scale=%g", fn, scale);
  return RFPX_OK;
}

template <int NB>
hipError_t launch_attn(const AttnPlan &p, const AttnArgs &a, hipStream_t s) {
  const dim3 grid(a.v.hk * p.row_blocks, p.splits, a.v.n_seqs), block(64 * p.waves);
  constexpr int RT = NB == 8 ? 1 : 2;
  constexpr int W1 = NB == 8 ? kWaves : kWavesOne;  // heads of 256 leave no registers for more
  const bool one = p.waves == kWavesOne;
  void (*k)(AttnArgs) =
      p.chunk               ? k_attn_chunk<NB == 8 ? 4 : NB>
      : a.xtype == RFPX_X_F32 ? (one ? k_attn<NB, 3, 1, W1> : k_attn<NB, 3, 1, kWaves>)
      : p.rt == 1           ? (one ? k_attn<NB, 1, 1, W1> : k_attn<NB, 1, 1, kWaves>)
                            : (one ? k_attn<NB, 1, RT, W1> : k_attn<NB, 1, RT, kWaves>);
  const size_t lds =
      p.chunk ? 2 * sizeof(ChunkK<NB>) + 2 * sizeof(ChunkV<NB>) + 2 * NB * kChunkWaves : 0;
  const hipError_t e = launch_k(k, grid, block, lds, s, a);
  if (e != hipSuccess || p.splits == 1) return e;
  const long long rh = (long long)a.n_rows * a.heads;
  const bool few = p.splits <= kJoinFew;
  constexpr int NG = 4 * kThreads / (32 * NB);
  const long long wgs = few ? (rh + NG - 1) / NG : rh;
  const dim3 jg((unsigned)(wgs < (1 << 20) ? wgs : 1 << 20));
  void (*j)(AttnArgs) =
      a.xtype == RFPX_X_F32 ? (few ? k_attn_join_few<NB, 3> : k_attn_join<NB, 3>)
                            : (few ? k_attn_join_few<NB, 1> : k_attn_join<NB, 1>);
  return launch_k(j, jg, dim3(kThreads), 0, s, a);
}

}  // namespace
}  // namespace rfpx

using namespace rfpx;

extern "C" {

size_t rfpx_attn_workspace_bytes(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int n_heads,
                                 int n_rows) {
  const char *fn = "rfpx_attn_workspace_bytes";
  if (check_kv(fn, c, b, false) || check_heads(fn, c, n_heads, n_rows, RFPX_X_F32, 1.f)) return 0;
  const size_t f = attn_plan(c, b, n_heads, n_rows, RFPX_X_F32).total;
  const size_t h = attn_plan(c, b, n_heads, n_rows, RFPX_X_BF16).total;
  return f > h ? f : h;
}

rfpx_status rfpx_attn_forward(const rfpx_kv_cache *c, const rfpx_kv_batch *b, const void *q,
                              long long q_stride, int xtype, int n_heads, int n_rows, float scale,
                              void *out, long long out_stride, float *lse, void *ws,
                              size_t ws_bytes, void *stream) {
  const char *fn = "rfpx_attn_forward";
  rfpx_status st = check_kv(fn, c, b, true);
  if (st) return st;
  if ((st = check_heads(fn, c, n_heads, n_rows, xtype, scale))) return st;
  if (n_rows == 0) return RFPX_OK;
  if ((st = check_rows(fn, "q", q, q_stride, n_heads, c->head_dim, xtype))) return st;
  if ((st = check_rows(fn, "out", out, out_stride, n_heads, c->head_dim, xtype))) return st;
  if (q == out) return fail(RFPX_E_ARG, "%s: out is q", fn);
  if ((uintptr_t)lse % 4) return fail(RFPX_E_ALIGN, "%s: lse not 4-byte aligned", fn);
  if (!ws) return fail(RFPX_E_ARG, "%s: workspace is null", fn);
  if ((uintptr_t)ws % 256) return fail(RFPX_E_ALIGN, "%s: workspace not 256-byte aligned", fn);
  const AttnPlan p = attn_plan(c, b, n_heads, n_rows, xtype);
  if (ws_bytes < p.total)
    return fail(RFPX_E_WORKSPACE, "%s: workspace holds %zu bytes, needs %zu", fn, ws_bytes, p.total);
  AttnArgs a{};
  a.v = kv_view(c, b);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + p.part);
  a.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + p.ml);
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.xtype = xtype;
  a.heads = n_heads;
  a.group = n_heads / c->n_kv_heads;
  a.n_rows = n_rows;
  a.splits = p.splits;
  a.row_blocks = p.row_blocks;
  a.sc = 16.f * scale * 1.4426950408889634f;
  hipStream_t s = (hipStream_t)stream;
  hipError_t e = c->head_dim == 64    ? launch_attn<2>(p, a, s)
                 : c->head_dim == 128 ? launch_attn<4>(p, a, s)
                                      : launch_attn<8>(p, a, s);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

rfpx_status rfpx_attn_weights(const rfpx_kv_cache *c, const rfpx_kv_batch *b, const void *q,
                              long long q_stride, int xtype, int n_heads, int n_rows, float scale,
                              const float *lse, float decay, const float *acc, float *acc_out,
                              void *stream) {
  const char *fn = "rfpx_attn_weights";
  rfpx_status st = check_kv(fn, c, b, true);
  if (st) return st;
  if ((st = check_heads(fn, c, n_heads, n_rows, xtype, scale))) return st;
  if (n_rows && (st = check_rows(fn, "q", q, q_stride, n_heads, c->head_dim, xtype))) return st;
  if ((n_rows && !lse) || !acc || !acc_out)
    return fail(RFPX_E_ARG, "%s: lse, acc or acc_out is null", fn);
  if ((uintptr_t)lse % 4 || (uintptr_t)acc % 4 || (uintptr_t)acc_out % 4)
    return fail(RFPX_E_ALIGN, "%s: lse, acc and acc_out must be 4-byte aligned", fn);
  if (!(decay - decay == 0.f)) return fail(RFPX_E_ARG, "%s: decay=%g", fn, decay);
  WeightArgs a{};
  a.v = kv_view(c, b);
  a.q = q;
  a.lse = lse;
  a.acc = acc;
  a.acc_out = acc_out;
  a.q_stride = q_stride;
  a.heads = n_heads;
  a.group = n_heads / c->n_kv_heads;
  a.n_rows = n_rows;
  a.sc = 16.f * scale * 1.4426950408889634f;
  a.decay = decay;
  const long long cap = (long long)b->pages_per_seq * c->page_tokens;
  const long long len = b->max_len < cap ? b->max_len : cap;
  // k_attn_weights_chunk has every wave decode every tile of its workgroup,
  // for which many rows pay, the fewer the shorter the sequence: there
  // k_attn_weights has few tiles a wave.  k_attn_weights and
  // k_attn_weights_chunk in us, 8 kv heads of 128, bf16, rows x tokens: 80 x
  // 9594 13, 29; 256 x 4096 17, 16; 256 x 8192 20, 28; 512 x 8192 38, 40; 1024
  // x 8192 73, 59; 512 x 16384 65, 76; 1024 x 16384 129, 115; 1024 x 32768
  // 194, 237; of 64: 256 x 8192 16.5, 15.7; 512 x 16384 45, 40; 512 x 32768
  // 69, 75; 1024 x 32768 134, 115.
  const long long many = (long long)b->max_cols * a.group;
  const bool chunk = many >= kWeightsMin && many * (c->head_dim == 64 ? 32 : 16) >= len;
  const int per = chunk ? 64 : kTile * kWaves;  // tokens of a workgroup's turn
  long long gy = (len + per - 1) / per;
  if (!chunk) {  // about four workgroups a compute unit, with several turns each
    const long long most = 1024 / ((long long)c->n_kv_heads * b->n_seqs);
    if (gy > most) gy = most;
  }
  if (gy < 1) gy = 1;
  if (gy > 65535) gy = 65535;
  const dim3 grid(c->n_kv_heads, (unsigned)gy, b->n_seqs);
  hipStream_t s = (hipStream_t)stream;
  const bool f = xtype == RFPX_X_F32;
  if (chunk) {
    void (*k)(WeightArgs) =
        c->head_dim == 64    ? (f ? k_attn_weights_chunk<2, 3> : k_attn_weights_chunk<2, 1>)
        : c->head_dim == 128 ? (f ? k_attn_weights_chunk<4, 3> : k_attn_weights_chunk<4, 1>)
                             : (f ? k_attn_weights_chunk<8, 3> : k_attn_weights_chunk<8, 1>);
    const hipError_t e = launch_k(k, grid, dim3(64 * kChunkWaves), 0, s, a);
    return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
  }
  void (*k)(WeightArgs) =
      c->head_dim == 64    ? (f ? k_attn_weights<2, 3> : k_attn_weights<2, 1>)
      : c->head_dim == 128 ? (f ? k_attn_weights<4, 3> : k_attn_weights<4, 1>)
                           : (f ? k_attn_weights<8, 3> : k_attn_weights<8, 1>);
  const hipError_t e = launch_k(k, grid, dim3(kThreads), 0, s, a);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

}  // extern "C"
