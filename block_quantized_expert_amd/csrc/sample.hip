// sample.hip -- a token of every row of logits: temperature, top-k, top-p,
// min-p, and a draw by a given number.
//
// Mathematics.  In the order (logit descending, index ascending) every cut
// leaves a beginning of the row, so that what stays is known by its weight:
//   M_k  of the first top_k tokens,
//   M_p  of the shortest beginning that reaches top_p M_k,
//   M_m  of the tokens of weight min_p or more,
//   W = min(M_k, M_p, M_m),
// and the token is the first one whose running sum exceeds u W.  M_k, M_p and
// the token are one question, find(): the first token of the order at which
// a running sum, of weights or of ones, exceeds a number.
//
// Weights are whole multiples of 2^-s (from a polynomial in 64 bits), and
// sums, targets and comparisons whole numbers: no order of additions changes
// a choice, LDS atomics may have any, and tokens of equal logits weigh the
// same, so that a place among them is a division.
//
// find() narrows: a histogram over 256 bins of the distance from the largest
// logit, 5 an octave of weight (the row is read for the largest, for the
// histogram, and once more for the tokens of the bins that the three
// questions fall into, which go into a list in LDS), then digits of the keys
// in the list, until at most 64 tokens are left, which one wave ranks, or
// tokens of one logit.  A list that is too short for its bins (flat rows) is
// replaced by the row itself.
#include "../../include/rfpx_verify.h"
#include "rfpx_impl.hpp"

namespace rfpx {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 256;
constexpr int kCopies = 4;   // of a histogram, by lane: neighbours often share a bin
constexpr int kList = 4096;
constexpr int kSmall = 64;   // tokens that one wave ranks
constexpr float kBinsPerOctave = 5.f;
constexpr uint32_t kNoToken = 0x007FFFFFu;  // key of -inf, which NaN gets too
constexpr float kNegInf = -__builtin_inff();

struct SampleArgs {
  const void *logits;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
  float *probs;
  long long stride;
  int n_rows, vocab, bits;  // weights are multiples of 2^-bits
};

// Keys order as floats do.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// NaN is no token, and -0 is 0.
__device__ __forceinline__ float logit_of(float x) { return x > kNegInf ? x + 0.0f : kNegInf; }

// A row's settings.
struct Row {
  float largest;
  double rate;    // log2(e) / temperature
  float bin_rate; // bins a logit
  int bits;
};

__device__ __forceinline__ double below(const Row &r, float v) {  // 0 or less
  return v == r.largest ? 0.0 : (double)v - (double)r.largest;
}

// exp(below / temperature) in units of 2^-bits, rounded to the nearest: 2^f by
// its Taylor series to f^11 (|f| <= 1/2: 7e-15), the rounding by adding 2^52.
__device__ __forceinline__ u64 weight(const Row &r, float v) {
#pragma clang fp contract(off)
  const double x = below(r, v) * r.rate;
  if (!(x > -64.0)) return 0;  // (also 0 times an infinite distance)
  const double n = __builtin_rint(x), f = x - n;
  double p = 4.4455382718708100e-10;                     // ln2^11 / 11!
  p = __builtin_fma(p, f, 7.0549116208011208e-09);
  p = __builtin_fma(p, f, 1.0178086009239700e-07);
  p = __builtin_fma(p, f, 1.3215486790144307e-06);
  p = __builtin_fma(p, f, 1.5252733804059841e-05);
  p = __builtin_fma(p, f, 1.5403530393381610e-04);
  p = __builtin_fma(p, f, 1.3333558146428441e-03);
  p = __builtin_fma(p, f, 9.6181291076284769e-03);
  p = __builtin_fma(p, f, 5.5504108664821580e-02);
  p = __builtin_fma(p, f, 2.4022650695910069e-01);
  p = __builtin_fma(p, f, 6.9314718055994529e-01);
  p = __builtin_fma(p, f, 1.0);
  const double y = __builtin_ldexp(p, (int)n + r.bits) + 4503599627370496.0;
  return __builtin_bit_cast(u64, y) & 0xFFFFFFFFFFFFFull;
}

// The bin of a logit: no larger for a larger one.
__device__ __forceinline__ int bin_of(const Row &r, float v) {
  const float y = v == r.largest ? 0.f : (r.largest - v) * r.bin_rate;
  return y < (float)(kBins - 1) ? (int)y : kBins - 1;
}

// x as a fraction of 2^64, below 1.
__device__ __forceinline__ u64 fraction(float x) {
  if (!(x > 0.f)) return 0;
  if (x >= 1.f) return ~0ull;
  return (u64)__builtin_ldexp((double)x, 64);
}
// The smallest sum that reaches `part` of `whole`, less one.
__device__ __forceinline__ u64 just_below(u64 whole, u64 part) {
  const u64 hi = __umul64hi(whole, part);
  return whole * part ? hi : hi ? hi - 1 : 0;
}

__device__ __forceinline__ u64 shfl_u64(u64 v, int lane) {
  return ((u64)(uint32_t)__shfl((int)(v >> 32), lane) << 32) | (uint32_t)__shfl((int)v, lane);
}
__device__ __forceinline__ u64 shfl_up_u64(u64 v, int off) {
  return ((u64)(uint32_t)__shfl_up((int)(v >> 32), off) << 32) | (uint32_t)__shfl_up((int)v, off);
}

struct Sums {  // of a bin and those before it
  u64 mass[kBins];
  uint32_t count[kBins];
};

// What a workgroup shares.
struct Shared {
  u64 mass[kBins * kCopies];
  uint32_t count[kBins * kCopies];
  Sums bins;                // of the row
  Sums digits;              // of what find() is narrowing
  uint32_t key[kList];
  int32_t index[kList];
  u64 sum[kWaves];
  uint32_t best[kWaves];
  int32_t first[kWaves];
  uint32_t small_key[kSmall];
  int32_t small_index[kSmall];
  // answers of wave 0
  u64 upto, own;
  uint32_t in_count, key_lo, key_hi;
  int n_list, n_small, token;
};

// -------------------------------------------------------- sources of tokens

// The logits of a row, 16 bytes a lane: f(logit, index) for each.
template <typename T>
struct RowSource {
  const T *p;
  int n;
  template <typename F>
  __device__ __forceinline__ void each(F &&f) const {
    constexpr int E = 16 / sizeof(T);
    const int skip = (int)(((uintptr_t)p & 15) / sizeof(T));
    const int chunks = (n + skip + E - 1) / E;
    for (int c = threadIdx.x; c < chunks; c += kThreads) {
      const int at = c * E - skip;
      float v[E];
      if (at >= 0 && at + E <= n) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p + at);
        const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < E; ++j)
          v[j] = sizeof(T) == 4 ? __uint_as_float(d[j * sizeof(T) / 4])
                 : j & 1        ? __uint_as_float(d[j / 2] & 0xFFFF0000u)
                                : __uint_as_float(d[j / 2] << 16);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const bool in = at + j >= 0 && at + j < n;
          const T x = in ? p[at + j] : T(0);
          v[j] = !in ? kNegInf
                 : sizeof(T) == 4 ? __builtin_bit_cast(float, (uint32_t)x)
                                  : __uint_as_float((uint32_t)x << 16);
        }
      }
#pragma unroll
      for (int j = 0; j < E; ++j) f(logit_of(v[j]), at + j);
    }
  }
};

struct ListSource {
  const Shared &sh;
  int n;
  template <typename F>
  __device__ __forceinline__ void each(F &&f) const {
    for (int i = threadIdx.x; i < n; i += kThreads) f(value_of(sh.key[i]), sh.index[i]);
  }
};

// --------------------------------------------------------------- histograms

__device__ __forceinline__ void clear_histogram(Shared &sh) {
  for (int i = threadIdx.x; i < kBins * kCopies; i += kThreads) {
    sh.mass[i] = 0;
    sh.count[i] = 0;
  }
}
__device__ __forceinline__ void add_to_bin(Shared &sh, int bin, u64 w, bool counts) {
  const int at = bin * kCopies + (threadIdx.x & (kCopies - 1));
  if (w) atomicAdd(&sh.mass[at], w);
  if (counts) atomicAdd(&sh.count[at], 1u);
}
// Running sums over the histogram's bins (between barriers of its own).
__device__ __forceinline__ void sum_histogram(const Shared &sh, Sums &to) {
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    u64 m = 0;
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      m += sh.mass[i * kCopies + k];
      c += sh.count[i * kCopies + k];
    }
    to.mass[i] = m;
    to.count[i] = c;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    u64 m[4];
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = to.mass[4 * lane + i] + (i ? m[i - 1] : 0);
      c[i] = to.count[4 * lane + i] + (i ? c[i - 1] : 0);
    }
    u64 ms = m[3];
    uint32_t cs = c[3];
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const u64 mo = shfl_up_u64(ms, off);
      const uint32_t co = (uint32_t)__shfl_up((int)cs, off);
      if (lane >= off) {
        ms += mo;
        cs += co;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      to.mass[4 * lane + i] = ms - m[3] + m[i];
      to.count[4 * lane + i] = cs - c[3] + c[i];
    }
  }
  __syncthreads();
}
// The first bin whose running sum exceeds r (the last, if none does); every
// wave finds it for itself.
__device__ __forceinline__ int bin_over(const Sums &to, u64 r, bool by_count) {
  const int lane = threadIdx.x & 63;
  int over = kBins;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const int b = 4 * lane + i;
    if ((by_count ? (u64)to.count[b] : to.mass[b]) > r) over = b;
  }
  const uint64_t lanes = __ballot(over < kBins);
  return lanes ? __shfl(over, __builtin_ctzll(lanes)) : kBins - 1;
}

// ------------------------------------------------------------------- find()

struct Found {
  u64 upto;   // weights up to the token, with it
  u64 own;    // its weight
  int token;  // its index, if that was asked for
};

// Among the tokens of bin `bin`, before which the order has weights `above`:
// the first one at which the running sum (of weights, or of ones) within the
// bin exceeds r.  Every thread of the workgroup takes part.
template <typename S>
__device__ Found find(const S &src, Shared &sh, const Row &row, int bin, bool by_count, u64 r,
                      u64 above, bool want_token) {
  const int lane = threadIdx.x & 63;
  // the bin's keys and how many tokens it has
  uint32_t lo = 0xFFFFFFFFu, hi = 0, n = 0;
  src.each([&](float v, int) {
    if (v > kNegInf && bin_of(row, v) == bin) {
      const uint32_t k = key_of(v);
      lo = min(lo, k);
      hi = max(hi, k);
      ++n;
    }
  });
  __syncthreads();  // the answers of an earlier call have been read
  if (threadIdx.x == 0) {
    sh.key_lo = 0xFFFFFFFFu;
    sh.key_hi = 0;
    sh.in_count = 0;
  }
  __syncthreads();
#pragma unroll
  for (int off = 32; off; off >>= 1) {
    lo = min(lo, (uint32_t)__shfl_xor((int)lo, off));
    hi = max(hi, (uint32_t)__shfl_xor((int)hi, off));
    n += (uint32_t)__shfl_xor((int)n, off);
  }
  if (lane == 0 && n) {
    atomicMin(&sh.key_lo, lo);
    atomicMax(&sh.key_hi, hi);
    atomicAdd(&sh.in_count, n);
  }
  __syncthreads();
  lo = sh.key_lo;
  hi = sh.key_hi;
  n = sh.in_count;
  int first = 0, last = 0x7FFFFFFF;  // indices that count: all, until the logit is known
  // digits of the distance from the bin's largest key, then of the index
  while (n > kSmall && (lo < hi || (want_token && first < last))) {
    const bool keys = lo < hi;
    if (!keys && last == 0x7FFFFFFF) {
      // all have one logit: the place among them is a division, and now ones
      // are summed
      const u64 w = weight(row, value_of(lo));
      if (!by_count && w) {
        const u64 place = r / w;
        above += place * w;
        r = place;
      } else {
        above += r * w;
      }
      by_count = true;
      first = 0;
      last = RFPX_VOCAB_MAX - 1;
    }
    const uint32_t span = keys ? hi - lo : (uint32_t)(last - first);
    const int shift = max(0, 24 - __builtin_clz(span));
    __syncthreads();
    clear_histogram(sh);
    __syncthreads();
    src.each([&](float v, int i) {
      const uint32_t k = key_of(v);
      if (k < lo || k > hi || i < first || i > last) return;
      if (keys) add_to_bin(sh, (hi - k) >> shift, weight(row, v), true);
      else add_to_bin(sh, (i - first) >> shift, 0, true);
    });
    sum_histogram(sh, sh.digits);
    const int d = bin_over(sh.digits, r, by_count);
    const u64 m0 = d ? sh.digits.mass[d - 1] : 0;
    const uint32_t c0 = d ? sh.digits.count[d - 1] : 0;
    n = sh.digits.count[d] - c0;
    r -= by_count ? (u64)c0 : m0;
    if (keys) {
      above += m0;
      hi -= (uint32_t)d << shift;
      lo = max(lo, hi - min(hi, (1u << shift) - 1u));
    } else {
      first += d << shift;
      last = min(last, first + (int)((1u << shift) - 1u));
    }
  }
  Found f{above, 0, -1};
  if (n > kSmall) {  // many of one logit, and no index asked for
    const u64 w = weight(row, value_of(lo));
    f.own = w;
    f.upto = above + ((by_count ? r : w ? r / w : 0) + 1) * w;
    return f;
  }
  // One wave ranks what is left.  (Where indices were counted, the weights
  // before are in `above` already, and all weigh the same.)
  const bool by_index = last != 0x7FFFFFFF;
  __syncthreads();
  if (threadIdx.x == 0) sh.n_small = 0;
  __syncthreads();
  src.each([&](float v, int i) {
    const uint32_t k = key_of(v);
    if (k < lo || k > hi || k <= kNoToken || i < first || i > last) return;
    const int at = atomicAdd(&sh.n_small, 1);
    if (at < kSmall) {
      sh.small_key[at] = k;
      sh.small_index[at] = i;
    }
  });
  __syncthreads();
  if (threadIdx.x < 64) {
    const int m = min(sh.n_small, kSmall);
    const uint32_t k = lane < m ? sh.small_key[lane] : 0;
    const int i = lane < m ? sh.small_index[lane] : 0x7FFFFFFF;
    const u64 w = lane < m ? weight(row, value_of(k)) : 0;
    u64 upto = 0;
    uint32_t rank = 0;  // with itself
    for (int j = 0; j < m; ++j) {
      const uint32_t kj = (uint32_t)__shfl((int)k, j);
      const int ij = __shfl(i, j);
      const u64 wj = shfl_u64(w, j);
      if (kj > k || (kj == k && ij <= i)) {
        upto += wj;
        ++rank;
      }
    }
    const u64 sum = by_count ? (u64)rank : upto, own = by_count ? 1 : w;
    const bool it = lane < m && sum > r && sum - own <= r;
    const uint64_t lanes = __ballot(it);
    if (lanes ? lane == __builtin_ctzll(lanes) : lane == 0) {
      sh.upto = by_index ? above + w : above + upto;
      sh.own = w;
      sh.token = i;
    }
  }
  __syncthreads();
  f.upto = sh.upto;
  f.own = sh.own;
  f.token = sh.token;
  return f;
}

// ------------------------------------------------------------------- a row

// What a row asks for.
struct Ask {
  int top_k;         // 0: no cut
  bool nucleus;      // a cut by top_p
  u64 top_p, u;      // fractions of 2^64
  u64 least;         // weights of min_p
};

__device__ __forceinline__ Ask ask_of(const SampleArgs &a, int at, int bits) {
  Ask q;
  const int k = a.top_k ? a.top_k[at] : 0;
  q.top_k = k > 0 && k < a.vocab ? k : 0;
  const float p = a.top_p ? a.top_p[at] : 1.f;
  q.nucleus = p < 1.f;
  q.top_p = fraction(p);
  q.u = fraction(a.u[at]);
  const float m = a.min_p ? a.min_p[at] : 0.f;
  q.least = !(m > 0.f) ? 0
            : m >= 1.f ? 1ull << bits
                       : (u64)__builtin_ceil(__builtin_ldexp((double)m, bits));
  return q;
}

// Bins of whose tokens a question may need each by itself: of top_k's, and
// ranges for the two that depend on an answer that is known to its bin.
struct Need {
  int k, p0, p1, r0, r1;
  __device__ __forceinline__ bool operator()(int b) const {
    return b == k || (b >= p0 && b <= p1) || (b >= r0 && b <= r1);
  }
};

__device__ __forceinline__ u64 before(const Sums &s, int bin) { return bin ? s.mass[bin - 1] : 0; }

__device__ __forceinline__ Need need_of(const Sums &s, const Ask &q, u64 mass_min) {
  Need n{-1, 0, -1, 0, -1};
  u64 lo = s.mass[kBins - 1], hi = lo;
  if (q.top_k && s.count[kBins - 1] > (uint32_t)q.top_k) {
    n.k = bin_over(s, (u64)(q.top_k - 1), true);
    lo = before(s, n.k);
    hi = s.mass[n.k];
  }
  if (q.nucleus) {
    n.p0 = bin_over(s, just_below(lo, q.top_p), false);
    n.p1 = bin_over(s, just_below(hi, q.top_p), false);
    lo = min(lo, before(s, n.p0));
    hi = min(hi, s.mass[n.p1]);
  }
  n.r0 = bin_over(s, __umul64hi(min(lo, mass_min), q.u), false);
  n.r1 = bin_over(s, __umul64hi(min(hi, mass_min), q.u), false);
  return n;
}

// The questions in turn; `whole` gets the weight of all that stays.
template <typename S>
__device__ __forceinline__ Found answer(const S &src, Shared &sh, const Row &row, const Ask &q,
                                        u64 mass_min, u64 *whole) {
  const Sums &s = sh.bins;
  u64 m = s.mass[kBins - 1];
  if (q.top_k && s.count[kBins - 1] > (uint32_t)q.top_k) {
    const int b = bin_over(s, (u64)(q.top_k - 1), true);
    const u64 m0 = before(s, b);
    m = s.mass[b] == m0 ? m0
                        : find(src, sh, row, b, true,
                               (u64)(q.top_k - 1) - (b ? s.count[b - 1] : 0), m0, false).upto;
  }
  if (q.nucleus) {
    const u64 r = just_below(m, q.top_p);
    const int b = bin_over(s, r, false);
    const u64 m0 = before(s, b);
    // (where min_p leaves less than the bins before, it alone counts)
    if (m0 < mass_min) m = min(m, find(src, sh, row, b, false, r - m0, m0, false).upto);
  }
  m = min(m, mass_min);
  *whole = m;
  const u64 r = __umul64hi(m, q.u);
  const int b = bin_over(s, r, false);
  const u64 m0 = before(s, b);
  return find(src, sh, row, b, false, r - m0, m0, true);
}

// A workgroup a row.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_sample_row(SampleArgs a) {
  __shared__ Shared sh;
  const int at = blockIdx.x, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const RowSource<T> src{static_cast<const T *>(a.logits) + (size_t)at * a.stride, a.vocab};

  // the largest logit and its first place
  float best = kNegInf;
  int first = 0x7FFFFFFF;
  src.each([&](float v, int i) {
    if (v > best) {
      best = v;
      first = i;
    }
  });
  const auto join = [&](float v, int i) {
    if (v > best || (v == best && i < first)) {
      best = v;
      first = i;
    }
  };
#pragma unroll
  for (int off = 32; off; off >>= 1) join(__shfl_xor(best, off), __shfl_xor(first, off));
  if (lane == 0) {
    sh.best[wave] = __float_as_uint(best);
    sh.first[wave] = first;
  }
  clear_histogram(sh);
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w) join(__uint_as_float(sh.best[w]), sh.first[w]);
  const float t = a.temperature ? a.temperature[at] : 1.f;
  const Ask q = ask_of(a, at, a.bits);
  if (best == kNegInf || !(t > 0.f) || q.top_k == 1) {
    if (threadIdx.x == 0) {
      a.tokens[at] = best == kNegInf ? -1 : first;
      if (a.probs) a.probs[at] = best == kNegInf ? 0.f : 1.f;
    }
    return;
  }
  Row row;
  row.largest = best;
  row.rate = 1.4426950408889634 / (double)t;
  row.bin_rate = fminf((float)row.rate * kBinsPerOctave, 3.0e38f);
  row.bits = a.bits;

  // weights by bin, and of those that min_p leaves
  u64 mass_min = 0;
  src.each([&](float v, int) {
    if (v > kNegInf) {
      const u64 w = weight(row, v);
      add_to_bin(sh, bin_of(row, v), w, q.top_k != 0);
      if (w >= q.least) mass_min += w;
    }
  });
#pragma unroll
  for (int off = 32; off; off >>= 1) mass_min += shfl_u64(mass_min, lane ^ off);
  if (lane == 0) sh.sum[wave] = mass_min;
  sum_histogram(sh, sh.bins);
  mass_min = 0;
  for (int w = 0; w < kWaves; ++w) mass_min += sh.sum[w];

  // the tokens of the bins in question
  const Need need = need_of(sh.bins, q, mass_min);
  src.each([&](float v, int i) {
    if (v > kNegInf && need(bin_of(row, v))) {
      const int j = atomicAdd(&sh.n_list, 1);
      if (j < kList) {
        sh.key[j] = key_of(v);
        sh.index[j] = i;
      }
    }
  });
  __syncthreads();
  u64 whole;
  const Found f = sh.n_list <= kList
                      ? answer(ListSource{sh, sh.n_list}, sh, row, q, mass_min, &whole)
                      : answer(src, sh, row, q, mass_min, &whole);
  if (threadIdx.x == 0) {
    a.tokens[at] = f.token;
    if (a.probs) a.probs[at] = (float)((double)f.own / (double)whole);
  }
}

int weight_bits(int vocab) {
  int log = 12;
  while (1 << log < vocab) ++log;
  return 62 - log;
}

rfpx_status check_sample(const char *fn, int n_rows, int vocab, int xtype) {
  if (xtype != RFPX_X_F32 && xtype != RFPX_X_BF16)
    return fail(RFPX_E_ARG, "%s: xtype=%d", fn, xtype);
  if (n_rows < 0 || n_rows > (1 << 20))
    return fail(RFPX_E_SHAPE, "%s: n_rows=%d: must be in [0, %d]", fn, n_rows, 1 << 20);
  if (vocab < 1 || vocab > RFPX_VOCAB_MAX)
    return fail(RFPX_E_SHAPE, "%s: vocab=%d: must be in [1, %d]", fn, vocab, RFPX_VOCAB_MAX);
  return RFPX_OK;
}

}  // namespace
}  // namespace rfpx

using namespace rfpx;

extern "C" {

size_t rfpx_sample_workspace_bytes(int n_rows, int vocab, int xtype) {
  if (check_sample("rfpx_sample_workspace_bytes", n_rows, vocab, xtype)) return 0;
  return 256;
}

rfpx_status rfpx_sample(const void *logits, long long stride, int xtype, int n_rows, int vocab,
                        const float *u, const float *temperature, const int32_t *top_k,
                        const float *top_p, const float *min_p, int32_t *tokens, float *probs,
                        void *ws, size_t ws_bytes, void *stream) {
  const char *fn = "rfpx_sample";
  const rfpx_status st = check_sample(fn, n_rows, vocab, xtype);
  if (st) return st;
  if (n_rows == 0) return RFPX_OK;
  if (!logits || !u || !tokens) return fail(RFPX_E_ARG, "%s: logits, u or tokens is null", fn);
  if (n_rows > 1 && (stride < vocab || stride > (1ll << 40)))
    return fail(RFPX_E_SHAPE, "%s: rows are %lld elements apart, %d logits need as many", fn,
                stride, vocab);
  if ((uintptr_t)logits % (xtype == RFPX_X_BF16 ? 2 : 4) || (uintptr_t)u % 4 ||
      (uintptr_t)temperature % 4 || (uintptr_t)top_k % 4 || (uintptr_t)top_p % 4 ||
      (uintptr_t)min_p % 4 || (uintptr_t)tokens % 4 || (uintptr_t)probs % 4)
    return fail(RFPX_E_ALIGN, "%s: logits must be aligned to an element, the others to 4 bytes", fn);
  if (!ws) return fail(RFPX_E_ARG, "%s: workspace is null", fn);
  if ((uintptr_t)ws % 256) return fail(RFPX_E_ALIGN, "%s: workspace not 256-byte aligned", fn);
  const size_t need = rfpx_sample_workspace_bytes(n_rows, vocab, xtype);
  if (ws_bytes < need)
    return fail(RFPX_E_WORKSPACE, "%s: workspace holds %zu bytes, needs %zu", fn, ws_bytes, need);
  SampleArgs a{};
  a.logits = logits;
  a.u = u;
  a.temperature = temperature;
  a.top_p = top_p;
  a.min_p = min_p;
  a.top_k = top_k;
  a.tokens = tokens;
  a.probs = probs;
  a.stride = stride;
  a.n_rows = n_rows;
  a.vocab = vocab;
  a.bits = weight_bits(vocab);
  const hipError_t e =
      launch_k(xtype == RFPX_X_BF16 ? k_sample_row<uint16_t> : k_sample_row<uint32_t>,
               dim3(n_rows), dim3(kThreads), 0, (hipStream_t)stream, a);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

}  // extern "C"
