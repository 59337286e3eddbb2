// kvcache.hip -- rows of a qkv projection on their way into attention: norm
// and rotation of the heads, the FP4 cache's append and unpack, and the host
// checks that the attention entry points share.
#include "rfpx_attn.hpp"

namespace rfpx {

rfpx_status check_kv(const char *fn, const rfpx_kv_cache *c, const rfpx_kv_batch *b,
                     bool pointers) {
  if (!c || !b) return fail(RFPX_E_ARG, "%s: cache or batch is null", fn);
  const size_t need = rfpx_kv_pool_bytes(c->n_kv_heads, c->head_dim, c->page_tokens, c->n_pages);
  if (!need)
    return fail(RFPX_E_SHAPE,
                "%s: cache of %d kv heads of %d, %d pages of %d tokens: heads 1..%d, head_dim 64, "
                "128 or 256, pages of 32, 64, 128 or 256 tokens", fn, c->n_kv_heads, c->head_dim,
                c->n_pages, c->page_tokens, RFPX_HEADS_MAX);
  if (b->n_seqs < 1 || b->n_seqs > RFPX_SEQS_MAX)
    return fail(RFPX_E_SHAPE, "%s: n_seqs=%d: must be in [1, %d]", fn, b->n_seqs, RFPX_SEQS_MAX);
  if (b->pages_per_seq < 1 || (long long)b->pages_per_seq * c->page_tokens > (1 << 30))
    return fail(RFPX_E_SHAPE, "%s: pages_per_seq=%d: 1 or more, up to 2^30 tokens", fn,
                b->pages_per_seq);
  if (b->max_cols < 0 || b->max_cols > RFPX_ROWS_MAX)
    return fail(RFPX_E_SHAPE, "%s: max_cols=%d: must be in [0, %d]", fn, b->max_cols,
                RFPX_ROWS_MAX);
  if (b->max_len < 0) return fail(RFPX_E_SHAPE, "%s: max_len=%d is negative", fn, b->max_len);
  if (!pointers) return RFPX_OK;
  if (!c->pool || !b->page_table || !b->lens || !b->starts)
    return fail(RFPX_E_ARG, "%s: pool, page_table, lens or starts is null", fn);
  if ((uintptr_t)c->pool % 256) return fail(RFPX_E_ALIGN, "%s: pool not 256-byte aligned", fn);
  if ((uintptr_t)b->page_table % 4 || (uintptr_t)b->lens % 4 || (uintptr_t)b->starts % 4)
    return fail(RFPX_E_ALIGN, "%s: page_table, lens or starts not 4-byte aligned", fn);
  if (c->pool_bytes < need)
    return fail(RFPX_E_WORKSPACE, "%s: pool holds %zu bytes, needs %zu", fn, c->pool_bytes, need);
  return RFPX_OK;
}

rfpx_status check_rows(const char *fn, const char *what, const void *p, long long stride, int heads,
                       int head_dim, int xtype) {
  if (!p) return fail(RFPX_E_ARG, "%s: %s is null", fn, what);
  if ((uintptr_t)p % 16 || stride * xtype_size(xtype) % 16)
    return fail(RFPX_E_ALIGN, "%s: %s and its rows must be 16-byte aligned", fn, what);
  if (stride < (long long)heads * head_dim || stride > (1ll << 40))
    return fail(RFPX_E_SHAPE, "%s: rows of %s are %lld elements apart, %d heads of %d need %lld",
                fn, what, stride, heads, head_dim, (long long)heads * head_dim);
  return RFPX_OK;
}

namespace {

constexpr int kThreads = 256;

// Eight neighbouring values as fp32.
__device__ __forceinline__ void load8(const void *p, size_t i, int xtype, float *v) {
  if (xtype == RFPX_X_BF16) {
    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(d[j] << 16);
      v[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
    }
  } else {
    const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

__device__ __forceinline__ void store8(void *p, size_t i, int otype, const float *v) {
  if (otype == RFPX_X_BF16) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
        make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                   bf16_pair(v[6], v[7]));
  } else {
    float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// ------------------------------------------------------ norm and rotation

constexpr int kRopeRows = 4;  // rows whose angles a workgroup holds

struct NormRopeArgs {
  const void *x[2];            // q, k
  void *out[2];
  const float *weight[2];
  long long stride[2], out_stride[2];
  int heads[2];
  const int32_t *positions;
  int n_rows, xtype, otype, half, style, per;  // per: head rows of a workgroup
  float eps;
  double turns[128];           // inv_freq / 2 pi
};

// Where a rotation finds a value's mate: in the lane's own eight values
// (neighbouring pairs), in another lane's register of the same number (halves
// of a multiple of eight), or anywhere, through LDS.
enum { kRopeNone, kRopeLane, kRopeShuffle, kRopeLds };

// Workgroup (x, y): rows 4x .. 4x+3, their head rows per * y .. (per a
// multiple of what a pass takes).  Eight values to a lane, D/8 lanes to a
// head.  cos and sin of the rows' angles are computed once a workgroup: the
// angle in turns, its whole turns taken off in 64 bits, the rest (below half
// a turn) in 32.  A pass's loads are issued before the pass ahead of it is
// computed.  2048 rows of 40 heads of 128 in bf16 (42 MB, each byte moved once)
// 12.6 us, 3.3 TB/s, where a plain copy of as much takes 8.1: waves wait 57% of
// their time, for a row's position and then for the row.  Five rows 3.9 us,
// which is a launch and two chains of loads.
template <int D, int MODE>
__global__ __launch_bounds__(kThreads) void k_norm_rope(NormRopeArgs a) {
  constexpr int LPH = D / 8, HPP = kThreads / LPH;
  __shared__ __align__(16) float cs[kRopeRows][128], sn[kRopeRows][128];
  __shared__ __align__(16) float xn[MODE == kRopeLds ? HPP : 1][D];
  const int row0 = blockIdx.x * kRopeRows;
  const int slot = threadIdx.x / LPH, l = threadIdx.x % LPH;
  const int heads = a.heads[0] + a.heads[1], rot = 2 * a.half;
  const int first = blockIdx.y * a.per;
  const int last = min(first + a.per, kRopeRows * heads);
  struct Pass {
    float v[8];
    int r, w, head;
    bool live;
  };
  const auto fetch = [&](int hr, Pass &p) {
    p.r = min(hr / heads, kRopeRows - 1);  // (a lane past the last head row computes nothing)
    const int hd = hr - p.r * heads, row = row0 + p.r;
    p.live = hr < last && row < a.n_rows && a.positions[row] >= 0;
    p.w = hd >= a.heads[0];
    p.head = hd - (p.w ? a.heads[0] : 0);
    if (p.live)
      load8(p.w ? a.x[1] : a.x[0],
            (size_t)row * (p.w ? a.stride[1] : a.stride[0]) + p.head * D + 8 * l, a.xtype, p.v);
  };
  Pass next;
  fetch(first + slot, next);
  if (MODE != kRopeNone) {
    for (int i = threadIdx.x; i < kRopeRows * a.half; i += kThreads) {
      const int r = i / a.half, j = i - r * a.half;
      const int row = row0 + r;
      const double t = row < a.n_rows ? (double)a.positions[row] * a.turns[j] : 0.0;
      float s, c;
      sincospif(2.0f * (float)(t - rint(t)), &s, &c);
      cs[r][j] = c;
      sn[r][j] = s;
    }
    __syncthreads();
  }
  for (int base = first; base < last; base += HPP) {
    Pass p = next;
    if (base + HPP < last) fetch(base + HPP + slot, next);
    float *v = p.v;
    const float *weight = p.w ? a.weight[1] : a.weight[0];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
    for (int off = 1; off < LPH; off <<= 1) ss += __shfl_xor(ss, off, LPH);
    if (p.live && weight) {
      const float rn = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
      const float4 w0 = reinterpret_cast<const float4 *>(weight)[2 * l];
      const float4 w1 = reinterpret_cast<const float4 *>(weight)[2 * l + 1];
      const float g[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * rn * g[j];
    }
    if (MODE == kRopeLane) {
      if (8 * l < rot) {
        const float4 c4 = *reinterpret_cast<const float4 *>(&cs[p.r][4 * l]);
        const float4 s4 = *reinterpret_cast<const float4 *>(&sn[p.r][4 * l]);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (8 * l + 2 * j < rot) {
            const float x = v[2 * j], y = v[2 * j + 1];
            v[2 * j] = fmaf(-y, s[j], x * c[j]);
            v[2 * j + 1] = fmaf(x, s[j], y * c[j]);
          }
      }
    } else if (MODE == kRopeShuffle) {
      const int far = a.half / 8;  // lanes to the mate
      const bool second = l >= far;
      const int mate = second ? l - far : l + far;
      const int at = 8 * (second ? l - far : l);  // of the angles
      float m[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = __shfl(v[j], mate, LPH);
      if (8 * l < rot) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float c = cs[p.r][at + j], s = sn[p.r][at + j];
          v[j] = fmaf(second ? m[j] : -m[j], s, v[j] * c);
        }
      }
    } else if (MODE == kRopeLds) {
      __syncthreads();
      if (p.live) {
        float4 *d = reinterpret_cast<float4 *>(&xn[slot][8 * l]);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
      __syncthreads();
      if (p.live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 8 * l + j;
          if (i < rot) {  // halves
            const bool second = i >= a.half;
            const int q = second ? i - a.half : i;
            const float m = xn[slot][second ? q : i + a.half], c = cs[p.r][q], s = sn[p.r][q];
            v[j] = second ? fmaf(m, s, v[j] * c) : fmaf(-m, s, v[j] * c);
          }
        }
      }
    }
    if (p.live)
      store8(p.w ? a.out[1] : a.out[0],
             (size_t)(row0 + p.r) * (p.w ? a.out_stride[1] : a.out_stride[0]) + p.head * D + 8 * l,
             a.otype, v);
  }
}

template <int D>
void (*norm_rope_kernel(int half, int style))(NormRopeArgs) {
  if (half == 0) return k_norm_rope<D, kRopeNone>;
  if (style == RFPX_ROPE_PAIRS) return k_norm_rope<D, kRopeLane>;
  return half % 8 == 0 ? k_norm_rope<D, kRopeShuffle> : k_norm_rope<D, kRopeLds>;
}

// ----------------------------------------------------- append and unpack

struct AppendArgs {
  KvView v;
  const void *x[2];  // k, v
  long long stride[2];
  int xtype, n_rows;
  const int32_t *positions;
  int32_t *pos;
  float *acc;
};

// The FP4 scale of a block of largest magnitude a (finite, > 0): the least e
// with a <= 7.5 * 2^(e-127), at least 1.  7.5 = 1.875 * 4, so e is a's own
// exponent - 2, plus one where its significand is over 1.875.
__device__ __forceinline__ int fp4_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 2 + ((u & 0x7FFFFFu) > 0x700000u);
  return e < 1 ? 1 : e;
}

// One row a workgroup; eight values to a lane, four lanes to a block.  64-bit
// arithmetic for the codes costs nothing that shows: 2048 rows of 8 heads of
// 128 in fp32 (17 MB in, 2.2 MB of blocks out) 8 us; 38 rows 4.1 us.
__global__ __launch_bounds__(kThreads) void k_kv_append(AppendArgs a) {
  const KvGeo &g = a.v.g;
  const int row = blockIdx.x, lane = threadIdx.x & 63;
  int b;
  const int slot = kv_slot_of(a.v, row, lane, &b);
  if (slot < 0) return;
  const int lph = g.head_dim / 8;
  const int t = slot & (g.page_tokens - 1);
  const int per = a.v.hk * lph;  // lanes of k, and of v
  for (int i = threadIdx.x; i < 2 * per; i += kThreads) {
    const int w = i >= per;
    const int head = (i - w * per) / lph, o = (i - w * per) % lph;
    uint8_t *slab = kv_slab(a.v, b, slot, head);
    float v[8];
    load8(a.x[w], (size_t)row * a.stride[w] + head * g.head_dim + 8 * o, a.xtype, v);
    float m = 0.f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bad |= !(fabsf(v[j]) < __builtin_inff());
      m = fmaxf(m, fabsf(v[j]));
    }
    m = fmaxf(m, __shfl_xor(m, 1, 4));
    m = fmaxf(m, __shfl_xor(m, 2, 4));
    int any = bad;
    any |= __shfl_xor(any, 1, 4);
    any |= __shfl_xor(any, 2, 4);
    uint32_t codes = 0;
    int e = 0;
    if (any) {
      e = 255;
      codes = 0xFFFFFFFFu;
    } else if (m > 0.f) {
      e = fp4_exponent(m);
      const double unit = __longlong_as_double((long long)(1023 + 127 - e) << 52);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // in 64 bits, as rfpx_pack rounds
        const double c = rint((double)v[j] * unit + 7.5);
        const int q = c < 0.0 ? 0 : c > 15.0 ? 15 : (int)c;
        codes |= (uint32_t)q << (4 * j);
      }
    }
    const uint32_t mate = __shfl_xor(codes, 4, 8);  // the same octet of block b ^ 1
    if (!slab) continue;
    const int oct = o & 3, blk = o >> 2;
    if (!w) {
      *reinterpret_cast<uint32_t *>(slab + g.kc + t * (g.head_dim / 2) + (oct * g.nb + blk) * 4) =
          codes;
    } else {
      const uint32_t even = blk & 1 ? mate : codes, odd = blk & 1 ? codes : mate;
      const int sh = blk & 1 ? 16 : 0;  // the even block's lane stores bytes 0, 1, the odd one's 2, 3
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t h = ((even >> (sh + 8 * j)) & 0xFFu) | (((odd >> (sh + 8 * j)) & 0xFFu) << 8);
        *reinterpret_cast<uint16_t *>(
            slab + g.vc + v_byte(g.nb, t, blk & ~1, 4 * oct + (sh >> 3) + j)) = (uint16_t)h;
      }
    }
    if (oct == 0) slab[(w ? g.vs : g.ks) + t * g.nb + blk] = (uint8_t)e;
    if (!w && o == 0) {
      const size_t at = ((size_t)b * a.v.hk + head) * kv_capacity(a.v) + slot;
      if (a.pos) a.pos[at] = a.positions[row];
      if (a.acc) a.acc[at] = 0.f;
    }
  }
}

struct UnpackArgs {
  KvView v;
  void *out[2];
  int otype, n_rows;
};

__global__ __launch_bounds__(kThreads) void k_kv_unpack(UnpackArgs a) {
  const KvGeo &g = a.v.g;
  const int row = blockIdx.x, lane = threadIdx.x & 63;
  int b;
  const int slot = kv_slot_of(a.v, row, lane, &b);
  if (slot < 0) return;
  const int lph = g.head_dim / 8;
  const int t = slot & (g.page_tokens - 1);
  const int per = a.v.hk * lph;
  for (int i = threadIdx.x; i < 2 * per; i += kThreads) {
    const int w = i >= per;
    const int head = (i - w * per) / lph, o = (i - w * per) % lph;
    const uint8_t *slab = kv_slab(a.v, b, slot, head);
    if (!slab) continue;
    const int oct = o & 3, blk = o >> 2;
    uint32_t codes = 0;
    if (!w) {
      codes = *reinterpret_cast<const uint32_t *>(slab + g.kc + t * (g.head_dim / 2) +
                                                  (oct * g.nb + blk) * 4);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        codes |= (uint32_t)slab[g.vc + v_byte(g.nb, t, blk, 4 * oct + j)] << (8 * j);
    }
    const int e = slab[(w ? g.vs : g.ks) + t * g.nb + blk];
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = e == 255 ? __builtin_nanf("")
                      : ldexpf((float)((codes >> (4 * j)) & 15u) - 7.5f, e - 127);
    store8(a.out[w], ((size_t)row * a.v.hk + head) * g.head_dim + 8 * o, a.otype, v);
  }
}

}  // namespace
}  // namespace rfpx

using namespace rfpx;

extern "C" {

size_t rfpx_kv_pool_bytes(int n_kv_heads, int head_dim, int page_tokens, int n_pages) {
  if (n_kv_heads < 1 || n_kv_heads > RFPX_HEADS_MAX || n_pages < 1) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  if (page_tokens != 32 && page_tokens != 64 && page_tokens != 128 && page_tokens != 256) return 0;
  return (size_t)n_pages * n_kv_heads * kv_geo(head_dim, page_tokens).slab;
}

rfpx_status rfpx_qk_norm_rope(const void *q, long long q_stride, int n_heads, const void *k,
                              long long k_stride, int n_kv_heads, int head_dim, int xtype,
                              int n_rows, const int32_t *positions, const float *q_weight,
                              const float *k_weight, float eps, const rfpx_rope *rope, void *q_out,
                              long long q_out_stride, void *k_out, long long k_out_stride,
                              int otype, void *stream) {
  const char *fn = "rfpx_qk_norm_rope";
  if (!valid_xtype(xtype) || !valid_xtype(otype))
    return fail(RFPX_E_ARG, "%s: xtype=%d, otype=%d", fn, xtype, otype);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(RFPX_E_SHAPE, "%s: head_dim=%d: must be 64, 128 or 256", fn, head_dim);
  if (n_heads < 0 || n_heads > RFPX_HEADS_MAX || n_kv_heads < 0 || n_kv_heads > RFPX_HEADS_MAX ||
      n_heads + n_kv_heads < 1)
    return fail(RFPX_E_SHAPE, "%s: %d query and %d key heads", fn, n_heads, n_kv_heads);
  if (n_rows < 0 || n_rows > RFPX_ROWS_MAX)
    return fail(RFPX_E_SHAPE, "%s: n_rows=%d: must be in [0, %d]", fn, n_rows, RFPX_ROWS_MAX);
  if (!(eps >= 0.f) || !(eps < __builtin_inff())) return fail(RFPX_E_ARG, "%s: eps=%g", fn, eps);
  if (rope) {
    if (rope->dim < 0 || rope->dim % 2 || rope->dim > head_dim)
      return fail(RFPX_E_SHAPE, "%s: %d rotated values of %d: must be even", fn, rope->dim, head_dim);
    if (rope->style != RFPX_ROPE_HALF && rope->style != RFPX_ROPE_PAIRS)
      return fail(RFPX_E_ARG, "%s: rope style %d", fn, rope->style);
    if (rope->dim && !rope->inv_freq_host)
      return fail(RFPX_E_ARG, "%s: inv_freq is null", fn);
  }
  if (n_rows == 0) return RFPX_OK;
  if (!positions) return fail(RFPX_E_ARG, "%s: positions is null", fn);
  if ((uintptr_t)positions % 4 || (uintptr_t)q_weight % 16 || (uintptr_t)k_weight % 16)
    return fail(RFPX_E_ALIGN, "%s: positions must be 4-byte, weights 16-byte aligned", fn);
  rfpx_status st;
  if (n_heads) {
    if ((st = check_rows(fn, "q", q, q_stride, n_heads, head_dim, xtype))) return st;
    if ((st = check_rows(fn, "q_out", q_out, q_out_stride, n_heads, head_dim, otype))) return st;
    if (q == q_out && (xtype != otype || q_stride != q_out_stride))
      return fail(RFPX_E_ARG, "%s: q_out is q with another stride or type", fn);
  }
  if (n_kv_heads) {
    if ((st = check_rows(fn, "k", k, k_stride, n_kv_heads, head_dim, xtype))) return st;
    if ((st = check_rows(fn, "k_out", k_out, k_out_stride, n_kv_heads, head_dim, otype))) return st;
    if (k == k_out && (xtype != otype || k_stride != k_out_stride))
      return fail(RFPX_E_ARG, "%s: k_out is k with another stride or type", fn);
  }
  NormRopeArgs a{};
  a.x[0] = q;
  a.x[1] = k;
  a.out[0] = q_out;
  a.out[1] = k_out;
  a.weight[0] = q_weight;
  a.weight[1] = k_weight;
  a.stride[0] = q_stride;
  a.stride[1] = k_stride;
  a.out_stride[0] = q_out_stride;
  a.out_stride[1] = k_out_stride;
  a.heads[0] = n_heads;
  a.heads[1] = n_kv_heads;
  a.positions = positions;
  a.n_rows = n_rows;
  a.xtype = xtype;
  a.otype = otype;
  a.eps = eps;
  a.half = rope ? rope->dim / 2 : 0;
  a.style = rope ? rope->style : RFPX_ROPE_HALF;
  for (int j = 0; j < a.half; ++j) {
    if (!(rope->inv_freq_host[j] >= -1e9 && rope->inv_freq_host[j] <= 1e9))
      return fail(RFPX_E_ARG, "%s: inv_freq[%d] is not a finite frequency", fn, j);
    a.turns[j] = rope->inv_freq_host[j] / 6.283185307179586476925286766559;
  }
  const int gx = (n_rows + kRopeRows - 1) / kRopeRows;
  const int hpp = kThreads / (head_dim / 8), all = kRopeRows * (n_heads + n_kv_heads);
  // few rows: one pass a workgroup, the angles computed again in each; many:
  // about ten workgroups a compute unit
  int gy = (all + hpp - 1) / hpp;
  const int most = gx >= 2560 ? 1 : 2560 / gx;
  if (gy > most) gy = most;
  a.per = ((all + gy - 1) / gy + hpp - 1) / hpp * hpp;
  gy = (all + a.per - 1) / a.per;
  hipStream_t s = (hipStream_t)stream;
  const dim3 grid(gx, gy);
  void (*kernel)(NormRopeArgs) = head_dim == 64    ? norm_rope_kernel<64>(a.half, a.style)
                                 : head_dim == 128 ? norm_rope_kernel<128>(a.half, a.style)
                                                   : norm_rope_kernel<256>(a.half, a.style);
  const hipError_t e = launch_k(kernel, grid, dim3(kThreads), 0, s, a);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

rfpx_status rfpx_kv_append(const rfpx_kv_cache *c, const rfpx_kv_batch *b, const void *k,
                           long long k_stride, const void *v, long long v_stride, int xtype,
                           int n_rows, const int32_t *positions, int32_t *pos, float *acc,
                           void *stream) {
  const char *fn = "rfpx_kv_append";
  rfpx_status st = check_kv(fn, c, b, true);
  if (st) return st;
  if (!valid_xtype(xtype)) return fail(RFPX_E_ARG, "%s: xtype=%d", fn, xtype);
  if (n_rows < 0 || n_rows > RFPX_ROWS_MAX)
    return fail(RFPX_E_SHAPE, "%s: n_rows=%d: must be in [0, %d]", fn, n_rows, RFPX_ROWS_MAX);
  if (n_rows == 0) return RFPX_OK;
  if ((st = check_rows(fn, "k", k, k_stride, c->n_kv_heads, c->head_dim, xtype))) return st;
  if ((st = check_rows(fn, "v", v, v_stride, c->n_kv_heads, c->head_dim, xtype))) return st;
  if (pos && !positions) return fail(RFPX_E_ARG, "%s: pos without positions", fn);
  if ((uintptr_t)positions % 4 || (uintptr_t)pos % 4 || (uintptr_t)acc % 4)
    return fail(RFPX_E_ALIGN, "%s: positions, pos and acc must be 4-byte aligned", fn);
  AppendArgs a{};
  a.v = kv_view(c, b);
  a.x[0] = k;
  a.x[1] = v;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.xtype = xtype;
  a.n_rows = n_rows;
  a.positions = positions;
  a.pos = pos;
  a.acc = acc;
  hipError_t e = launch_k(k_kv_append, dim3(n_rows), dim3(kThreads), 0, (hipStream_t)stream, a);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

rfpx_status rfpx_kv_unpack(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int n_rows, void *k,
                           void *v, int otype, void *stream) {
  const char *fn = "rfpx_kv_unpack";
  rfpx_status st = check_kv(fn, c, b, true);
  if (st) return st;
  if (!valid_xtype(otype)) return fail(RFPX_E_ARG, "%s: otype=%d", fn, otype);
  if (n_rows < 0 || n_rows > RFPX_ROWS_MAX)
    return fail(RFPX_E_SHAPE, "%s: n_rows=%d: must be in [0, %d]", fn, n_rows, RFPX_ROWS_MAX);
  if (n_rows == 0) return RFPX_OK;
  const long long stride = (long long)c->n_kv_heads * c->head_dim;
  if ((st = check_rows(fn, "k", k, stride, c->n_kv_heads, c->head_dim, otype))) return st;
  if ((st = check_rows(fn, "v", v, stride, c->n_kv_heads, c->head_dim, otype))) return st;
  UnpackArgs a{};
  a.v = kv_view(c, b);
  a.out[0] = k;
  a.out[1] = v;
  a.otype = otype;
  a.n_rows = n_rows;
  hipError_t e = launch_k(k_kv_unpack, dim3(n_rows), dim3(kThreads), 0, (hipStream_t)stream, a);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

}  // extern "C"
