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
// find() narrows: bins of the distance from the largest logit, 10 an octave of
// weight, then digits of the keys in one bin, until at most 256 tokens are left,
// which are ranked by comparing each with all, or tokens of one logit.
//
// Rows of up to 32765 fp32 or 32761 bf16 logits (32768, less what one that begins off
// 16 bytes costs) are a workgroup's each, in registers (k_sample_row).  Longer ones are
// cut into slices:
//   k_sample_slices   a workgroup holds its slice in registers: its largest
//                     logit; and, if the row keeps the first of few, or tokens
//                     of some weight, all of the slice that can be among them,
//                     a list; or else the slice's weights by bin
//   k_sample_decide   a workgroup a row: of rows of the second kind the bins
//                     that the questions fall into
//   k_sample_collect  the tokens of those bins (these rows are read once more)
//   k_sample_pick     a workgroup a row: the questions
// A slice's weights are relative to a power of two of its own, and shifted where
// the slices of a row come together (which rounds down: less than 2^-s a bin).
//
// Why not one workgroup for a row of any length: 64 rows would read through 64
// compute units.  Why not slices for every row: four launches instead of one.
// Measured on an MI355X, us a call in a graph, a workgroup a row / slices: 1 row of
// 32000 fp32 logits by top_p 23.5 / 27.5, by top_k 14.0 / 22.2, greedy 7.3 / 10.5; 512
// rows 67 / 81, 32 / 41, 20 / 23; 512 rows of 8000 37 / 47; one row of 4000 13.4 / 26.5.
// Above those the registers of a workgroup do not hold a row.
#include "../../include/rfpx_verify.h"
#include "rfpx_impl.hpp"

namespace rfpx {
namespace {

typedef unsigned long long u64;

constexpr int kWide = 1024;    // threads of a workgroup that has a row's logits
constexpr int kNarrow = 256;   // ... a slice's
constexpr int kMiddle = 512;   // ... or what is left of a row
constexpr int kMostWaves = 16;
constexpr int kBins = 512;
constexpr int kLaneBins = kBins / 64;
constexpr int kSumWaves = 4;  // that sum up a histogram, two bins a lane
static_assert(kBins == 2 * 64 * kSumWaves, "two bins a lane");
constexpr int kCopyLog = 1;  // copies of a histogram, by lane: neighbours often share a bin
constexpr int kCopies = 1 << kCopyLog;
constexpr int kFewLog = 4;   // ... of one of few bins, where most of them do
constexpr int kFewBins = kBins * kCopies >> kFewLog;
constexpr int kList = 6144;  // tokens that answer() has in LDS
// Tokens that find() ranks by comparing each with all (64: one more digit, 4 us, for
// most bins; 512: the same time as 256).
constexpr int kRank = 256;
constexpr float kBinsPerOctave = 10.f;  // 51 octaves; what is below weighs a unit at most
constexpr uint32_t kNoToken = 0x007FFFFFu;  // key of -inf, which NaN gets too
constexpr float kNegInf = -__builtin_inff();
constexpr int kRowMost = 32 * kWide;  // logits of a row that is not cut into slices
constexpr int kSlice = 32 * kNarrow;  // logits of a slice
constexpr int kSliceList = kMiddle;   // tokens that a slice may list
static_assert(kBins == kMiddle, "a thread a bin");
constexpr int kBatch = 4;       // loads of lists that are in flight at once
constexpr int kBinsBatch = 24;  // ... of slices' bins
constexpr int kMostSlices = RFPX_VOCAB_MAX / kSlice + 1;
constexpr int kTopMost = 256;     // top_k of rows whose slices list their tokens
constexpr int kRowsAtOnce = 512;  // rows of one set of launches, which bounds the workspace

// What k_sample_slices says of a slice.
struct SliceHead {
  double ref;  // of its weights
  u64 total;   // their sum, where they stand by bin
  float largest;
  int first;   // its first place
  float base;  // of its bins
  int binned;  // its weights stand by bin
  int listed;  // tokens that had to be listed (more than kSliceList: the list is not whole)
  int last;    // the first top_k are in bins up to this one
  int collected;  // tokens that k_sample_collect had to list
  int none;
};

// Bins whose tokens the questions need one by one: of min_p's and top_k's, and
// ranges for the two that depend on an answer that is known to its bin.
struct Need {
  int m0, m1, k0, k1, p0, p1, r0, r1;
};

struct Sums {  // of a bin and those before it
  u64 mass[kBins];
  uint32_t count[kBins];
};

// What k_sample_decide says of a row without lists.
struct RowState {
  float largest;
  Need need;
  Sums bins;
};

struct SampleArgs {
  const void *logits;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
  float *probs;
  long long stride;
  int n_rows, vocab, bits;  // weights are multiples of 2^-bits
  int row0, rows, slices;
  int *active;       // [1 + rows]: how many rows have no lists, and which
  RowState *state;   // [rows]
  SliceHead *heads;  // [rows][slices]
  u64 *mass;         // [rows][slices][kBins]
  uint32_t *count;   // [rows][slices][kBins]
  uint2 *list;       // [rows][slices][kSliceList]: key, index
};

// Keys order as floats do, and -0 is 0.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// NaN is no token, as -inf; +inf counts as the type's largest number, so that
// all that is computed of tokens is one.
template <typename T>
__device__ __forceinline__ float logit_of(float x) {
  return x > kNegInf ? fminf(x, __uint_as_float(sizeof(T) == 2 ? 0x7F7F0000u : 0x7F7FFFFFu)) : kNegInf;
}

// What weights and bins of a row, or a slice of it, are relative to.
struct Row {
  float largest;
  float bin_rate;  // bins a logit
  float base;      // the largest logit's bin, counted from 0
  float lowest;    // what is below weighs nothing
  int bits;
  int key_zeros;   // low bits in which keys of one sign do not differ
  bool far;        // nothing but the largest logit weighs anything
  double rate;     // log2(e) / temperature
  double ref;      // a whole number, the largest logit times rate or above
  // Of a key without those bits (which are ones below 0).
  __device__ __forceinline__ float value(uint32_t k) const {
    return value_of(key_zeros ? k << 16 | (k & 0x8000u ? 0u : 0xFFFFu) : k);
  }
};

template <typename T>
__device__ __forceinline__ Row row_of(float largest, float temperature, int bits) {
  Row r;
  r.key_zeros = sizeof(T) == 2 ? 16 : 0;
  r.largest = largest;
  r.rate = 1.4426950408889634 / (double)temperature;
  // (above 0, so that -inf is in the last bin at any temperature)
  r.bin_rate = fmaxf(fminf((float)r.rate * kBinsPerOctave, 3.0e38f), 1.17549435e-38f);
  r.base = floorf(largest * r.bin_rate);
  r.bits = bits;
  r.ref = __builtin_ceil((double)largest * r.rate);
  // (from 2^30 on the next smaller logit, 2^-24 of it or more away, is 64 octaves or
  // more below; and rates stay below what fp32 holds)
  r.far = !(__builtin_fabs(r.ref) < 1073741824.0) || !(temperature >= 7.888609052210118e-31f);
  // (bits + 2 octaves below, where less than a quarter of a unit is left; rounded
  // down, and above -inf; a scalar, since rows in registers have no vector register
  // left: with one k_sample_row takes 24.3 us for 32000 bf16 logits by top_p, not 23.4)
  const double lowest = (double)largest - (bits + 2) * 0.6931471805599453 * (double)temperature;
  r.lowest = __int_as_float(uniform(__float_as_int(fmaxf(__double2float_rd(lowest), -3.4028234663852886e38f))));
  return r;
}

// The bin of a logit: no larger for a larger one.  Whole numbers of the logit
// itself, so that bins of slices differ by a whole number too.  Where products
// overflow, and what is left of two of them is no number, it is the first.
// Products of large logits are rounded, by more than a bin from 2^24 bins on: a
// bin says where a logit stands among others, and not what it weighs.
__device__ __forceinline__ int bin_of(const Row &r, float v) {
  const float b = r.base - floorf(v * r.bin_rate);
  return (int)fminf(fmaxf(b, 0.f), (float)(kBins - 1));
}
// Bin `i` of a slice, among the row's.
__device__ __forceinline__ int row_bin(const Row &r, float slice_base, int i) {
  return slice_base == r.base ? i : (int)fminf((float)i + (r.base - slice_base), (float)(kBins - 1));
}

// 2^(v rate - ref) in units of 2^-bits, rounded to the nearest, of a logit of
// `lowest` or more in a row that is not far (which is less than 200 octaves below the
// largest, bits + 2 and one step of fp32, so that the exponent is one).  With v rate = m
// + f, m whole and |f| <= 1/2, 2^f is the polynomial 1 + f q(f) of degree 10 of
// least relative error (3e-16, by Remez' exchange); the product is never rounded.
// Adding 1.5 * 2^52, less ref and plus bits, leaves the exponent in the low bits;
// adding 2^52 leaves the result there.
__device__ __forceinline__ u64 near_weight(const Row &r, float v) {
#pragma clang fp contract(off)
  const double whole = 6755399441055744.0 + ((double)r.bits - r.ref);
  const double t = __builtin_fma((double)v, r.rate, whole);
  const double f = __builtin_fma((double)v, r.rate, -(t - whole));
  double p = 7.11174936174289645e-09;
  p = __builtin_fma(p, f, 1.02105059849407951e-07);
  p = __builtin_fma(p, f, 1.32152356871880181e-06);
  p = __builtin_fma(p, f, 1.52526477502981718e-05);
  p = __builtin_fma(p, f, 1.54035308007198697e-04);
  p = __builtin_fma(p, f, 1.33335582464760177e-03);
  p = __builtin_fma(p, f, 9.61812910738078439e-03);
  p = __builtin_fma(p, f, 5.55041086643466158e-02);
  p = __builtin_fma(p, f, 2.40226506959104719e-01);
  p = __builtin_fma(p, f, 6.93147180559951614e-01);
  p = __builtin_fma(p, f, 1.0);
  typedef uint32_t words_t __attribute__((ext_vector_type(2)));
  words_t u = __builtin_bit_cast(words_t, p);
  u[1] += __builtin_bit_cast(words_t, t)[0] << 20;
  words_t y = __builtin_bit_cast(words_t, __builtin_bit_cast(double, u) + 4503599627370496.0);
  y[1] &= 0xFFFFFu;
  return __builtin_bit_cast(u64, y);
}
__device__ __forceinline__ u64 weight(const Row &r, float v) {
  if (r.far) return v == r.largest ? 1ull << r.bits : 0;
  return v >= r.lowest ? near_weight(r, v) : 0;
}

// v >> n, of a lane's own n below 64, by operations of 32 bits.  (A 64-bit shift
// whose amount lies in the last register that a wave has been given shifts some
// lanes by something else when waves share a SIMD.  Amounts that all lanes share
// are scalars.)
__device__ __forceinline__ u64 shifted(u64 v, int n) {
  const uint32_t lo = (uint32_t)v, hi = (uint32_t)(v >> 32);
  const uint32_t low = __builtin_amdgcn_alignbit(hi, lo, (uint32_t)n & 31), high = hi >> (n & 31);
  return n < 32 ? (u64)high << 32 | low : high;
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

// Over the lanes of a wave by data-parallel moves, within rows of 16 lanes and
// then from row to row: the last lane has seen all of them.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 moved(u64 v, u64 none) {
  return ((u64)moved<CTRL, ROWS>((uint32_t)(v >> 32), (uint32_t)(none >> 32)) << 32) |
         moved<CTRL, ROWS>((uint32_t)v, (uint32_t)none);
}
template <typename U, typename F>
__device__ __forceinline__ U running(U v, U none, F &&f) {
  v = f(v, moved<0x111, 0xF>(v, none));  // from 1, 2, 4, 8 lanes below
  v = f(v, moved<0x112, 0xF>(v, none));
  v = f(v, moved<0x114, 0xF>(v, none));
  v = f(v, moved<0x118, 0xF>(v, none));
  v = f(v, moved<0x142, 0xA>(v, none));  // the last lane of row 0 to row 1, of 2 to 3
  v = f(v, moved<0x143, 0xC>(v, none));  // the last lane of row 1 to rows 2 and 3
  return v;
}
template <typename U>
__device__ __forceinline__ U running_sum(U v) {
  return running(v, (U)0, [](U a, U b) { return a + b; });
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ u64 lane_of(u64 v, int lane) {
  return (u64)lane_of((uint32_t)(v >> 32), lane) << 32 | lane_of((uint32_t)v, lane);
}
template <typename U>
__device__ __forceinline__ U wave_sum(U v) {
  return lane_of(running_sum(v), 63);
}
template <typename U>
__device__ __forceinline__ U wave_max(U v) {
  return lane_of(running(v, (U)0, [](U a, U b) { return a > b ? a : b; }), 63);
}
template <typename U>
__device__ __forceinline__ U wave_min(U v) {
  return ~wave_max((U)~v);
}

struct Hist {
  alignas(16) u64 mass[kBins * kCopies];
  alignas(16) uint32_t count[kBins * kCopies];
  u64 wave_mass[kSumWaves];
  uint32_t wave_count[kSumWaves];
};
// What a workgroup that answers a row's questions shares.
struct Shared {
  Hist hist;
  Sums bins;    // of the row
  Sums digits;  // of what find() is narrowing
  uint32_t key[kList];
  int32_t index[kList];
  u64 sum[kMostWaves];
  // answers, and what is found out for them
  u64 upto, own;
  uint32_t key_lo, key_hi;
  int n_list, n_in, token;
  uint32_t ranks[kWide];
  int length[kMostSlices];  // of the slices' lists
};

// What one that joins a row's slices shares.
struct Joining {
  Hist hist;
  Sums bins;
  int length[kMostSlices + kBinsBatch];  // of lists (-1: weights by bin)
  float base[kMostSlices + kBinsBatch];
  int shift[kMostSlices + kBinsBatch];
};

// -------------------------------------------------------- sources of tokens

// 16 bytes of a row's logits as floats, -inf outside of it.
template <typename T>
struct RowSource {
  static constexpr int E = 16 / sizeof(T);
  const T *p;
  int n;
  // The row in pieces of 16 aligned bytes: how many, and where piece c begins.
  __device__ __forceinline__ int skip() const { return (int)(((uintptr_t)p & 15) / sizeof(T)); }
  __device__ __forceinline__ int pieces() const { return (n + skip() + E - 1) / E; }
  __device__ __forceinline__ int begin(int c) const { return c * E - skip(); }
  __device__ __forceinline__ float one(int i) const {
    return sizeof(T) == 4 ? __builtin_bit_cast(float, (uint32_t)p[i])
                          : __uint_as_float((uint32_t)p[i] << 16);
  }
  __device__ __forceinline__ bool inside(int c) const { return begin(c) >= 0 && begin(c) + E <= n; }
  __device__ __forceinline__ uint4 words(int c) const {  // of a piece that is inside
    return *reinterpret_cast<const uint4 *>(p + begin(c));
  }
  static __device__ __forceinline__ float logit(const uint4 &w, int j) {
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
    return logit_of<T>(sizeof(T) == 4 ? __uint_as_float(d[j * sizeof(T) / 4])
                    : j & 1        ? __uint_as_float(d[j / 2] & 0xFFFF0000u)
                                   : __uint_as_float(d[j / 2] << 16));
  }
  __device__ __forceinline__ void load(int c, float (&v)[E]) const {
    if (inside(c)) {
      const uint4 w = words(c);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = logit(w, j);
    } else {
      const int at = begin(c);
#pragma unroll
      for (int j = 0; j < E; ++j)
        v[j] = at + j >= 0 && at + j < n ? logit_of<T>(one(at + j)) : kNegInf;
    }
  }
  // f(logit, index) for each; also for -inf.
  template <typename F>
  __device__ __forceinline__ void each(F &&f) const {
    for (int c = threadIdx.x; c < pieces(); c += blockDim.x) {
      float v[E];
      load(c, v);
#pragma unroll
      for (int j = 0; j < E; ++j) f(v[j], begin(c) + j);
    }
  }
};

// Logits in registers: pieces first + N threads' ones of a row.  Loops over them
// are not unrolled (registers are indexed): a workgroup goes through them once or
// twice, and would wait for its instructions.
template <typename T, int N>
struct HeldSource {
  static constexpr int E = RowSource<T>::E;
  typedef float held_t __attribute__((ext_vector_type(N * E)));
  held_t v;
  int at;  // of the first
  __device__ __forceinline__ void load(const RowSource<T> &src, int slice) {
    const int first = slice * N * (int)blockDim.x, c0 = first + threadIdx.x;
    at = src.begin(c0);
    if (src.inside(first) && src.inside(first + N * (int)blockDim.x - 1)) {
      uint4 w[N];  // all loads in flight at once
#pragma unroll
      for (int j = 0; j < N; ++j) w[j] = src.words(c0 + j * (int)blockDim.x);
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) v[j * E + i] = src.logit(w[j], i);
      return;
    }
    // the row begins or ends within: pieces outside are replaced by the last
    // one inside, if there is one, and then by nothing
    const int lo = src.inside(0) ? 0 : 1, hi = (src.n + src.skip()) / E - 1;
    if (hi >= lo) {
      uint4 w[N];
#pragma unroll
      for (int j = 0; j < N; ++j)
        w[j] = src.words(min(max(c0 + j * (int)blockDim.x, lo), hi));
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int c = c0 + j * (int)blockDim.x;
#pragma unroll
        for (int i = 0; i < E; ++i) v[j * E + i] = c >= lo && c <= hi ? src.logit(w[j], i) : kNegInf;
      }
    } else {
      v = held_t(kNegInf);
    }
    // the pieces of which only a part is inside: the row's first and last
    const int edge[2] = {0, src.pieces() - 1};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 1 && edge[1] == 0) break;
      const int j = (edge[k] - c0) / (int)blockDim.x;
      if (src.inside(edge[k]) || edge[k] < c0 || (edge[k] - c0) % (int)blockDim.x || j >= N) continue;
      float x[E];
      src.load(edge[k], x);
#pragma unroll
      for (int b = 0; b < N; ++b)
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (b == j) v[b * E + i] = x[i];
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F &&f) const {
#pragma unroll 1
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (int i = 0; i < E; ++i) f(v[j * E + i], at + j * (int)blockDim.x * E + i);
    }
  }
  // f(place, key, index) for those that `in` picks: a wave takes its places from
  // `counter` at once.  They are few, and read again.
  template <typename In, typename F>
  __device__ __forceinline__ void pick(const RowSource<T> &src, int *counter, In &&in, F &&f) const {
    static_assert(N * E <= 32, "a bit each");
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) mask |= in(v[j * E + i]) ? 1u << (j * E + i) : 0u;
    if (!__any(mask != 0)) return;
    const uint32_t mine = __popc(mask), upto = running_sum(mine);
    int place = 0;
    if ((threadIdx.x & 63) == 63) place = atomicAdd(counter, (int)upto);
    place = __builtin_amdgcn_readlane(place, 63) + (int)(upto - mine);
    for (; mask; mask &= mask - 1, ++place) {
      const int bit = __builtin_ctz(mask);
      const int index = at + bit / E * (int)blockDim.x * E + bit % E;
      f(place, key_of(logit_of<T>(src.one(index))), index);
    }
  }
};

struct ListSource {
  const Shared &sh;
  int n;
  template <typename F>
  __device__ __forceinline__ void each(F &&f) const {
    for (int i = threadIdx.x; i < n; i += blockDim.x) f(value_of(sh.key[i]), sh.index[i]);
  }
};

// The lists of a row's slices, whose lengths are in LDS (below 0: none): a wave
// takes 64 tokens of a list, kBatch times at once.
struct GatherSource {
  const uint2 *list;
  const int *lengths;
  int slices;
  // f(kBatch entries), kNoToken where there is none
  template <typename F>
  __device__ __forceinline__ void batches(F &&f) const {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6;
#pragma unroll 1
    for (int s0 = 0; s0 < slices; s0 += 64) {
      const int len = s0 + lane < slices ? max(lengths[s0 + lane], 0) : 0;
      const uint32_t upto = running_sum((uint32_t)(len + 63) / 64);
      const int all = (int)lane_of(upto, 63);
#pragma unroll 1
      for (int k0 = wave; k0 < all; k0 += kBatch * waves) {
        uint2 e[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int k = k0 + j * waves;
          const int s = __popcll(__ballot((int)upto <= k));  // (64: there is none)
          const int at = (k - (s ? (int)lane_of(upto, s - 1) : 0)) * 64 + lane;
          e[j] = s < 64 && at < (int)lane_of((uint32_t)len, s & 63)
                     ? list[(size_t)(s0 + s) * kSliceList + at]
                     : make_uint2(kNoToken, 0);
        }
        f(e);
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F &&f) const {
    batches([&](uint2 (&e)[kBatch]) {
#pragma unroll 1
      for (int j = 0; j < kBatch; ++j) {
        if (e[0].x > kNoToken) f(value_of(e[0].x), (int)e[0].y);
#pragma unroll
        for (int i = 0; i < kBatch - 1; ++i) e[i] = e[i + 1];
      }
    });
  }
  // f(place, key, index) for those that `in` picks: a wave takes its places from
  // `counter` a batch at a time.
  template <typename In, typename F>
  __device__ __forceinline__ void pick(int *counter, In &&in, F &&f) const {
    batches([&](uint2 (&e)[kBatch]) {
      uint32_t mask = 0;
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        mask |= e[j].x > kNoToken && in(value_of(e[j].x)) ? 1u << j : 0u;
      const uint32_t mine = __popc(mask), upto = running_sum(mine);
      int place = 0;
      if ((threadIdx.x & 63) == 63 && upto) place = atomicAdd(counter, (int)upto);
      place = __builtin_amdgcn_readlane(place, 63) + (int)(upto - mine);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (mask >> j & 1u) f(place++, e[j].x, (int)e[j].y);
    });
  }
};

// --------------------------------------------------------------- histograms

__device__ __forceinline__ void clear_histogram(Hist &h) {
  for (int i = threadIdx.x; i < kBins * kCopies; i += blockDim.x) {
    h.mass[i] = 0;
    h.count[i] = 0;
  }
}
__device__ __forceinline__ void add_to_bin(Hist &h, int bin, u64 w, uint32_t n, int log = kCopyLog) {
  const int at = bin << log | (threadIdx.x & ((1 << log) - 1));
  if (w) atomicAdd(&h.mass[at], w);
  if (n) atomicAdd(&h.count[at], n);
}
// The weights of a source by bin, in a row that is not far.  (The branch is an
// addition's alone: the polynomial in it costs a move a step.)
template <typename S>
__device__ __forceinline__ void add_weights(const S &src, Hist &h, const Row &row) {
  const int copy = threadIdx.x & (kCopies - 1);
  src.each([&](float v, int) {
    const int b = bin_of(row, v);
    u64 w = near_weight(row, v);
    asm volatile("" : "+v"(w));
    if (v >= row.lowest) atomicAdd(&h.mass[b * kCopies + copy], w);
  });
}
// Running sums over the histogram's bins (between barriers of its own).
__device__ __forceinline__ void sum_histogram(Hist &h, Sums &to, int log = kCopyLog) {
  __syncthreads();
  const int t = threadIdx.x, wave = uniform(t >> 6);
  u64 m0 = 0, m1 = 0, m = 0;
  uint32_t c0 = 0, c1 = 0, c = 0;
  if (wave < kSumWaves) {
    if ((2 * t + 1) << log < kBins * kCopies) {
      static_assert(kCopies == 2 && (1 << kFewLog) % kCopies == 0, "copies in pairs");
#pragma unroll 4
      for (int k = 0; k < 1 << log; k += 2) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(&h.mass[(2 * t << log) + k]);
        const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(&h.mass[((2 * t + 1) << log) + k]);
        const uint2 u = *reinterpret_cast<const uint2 *>(&h.count[(2 * t << log) + k]);
        const uint2 v = *reinterpret_cast<const uint2 *>(&h.count[((2 * t + 1) << log) + k]);
        m0 += x.x + x.y;
        m1 += y.x + y.y;
        c0 += u.x + u.y;
        c1 += v.x + v.y;
      }
    }
    m = running_sum(m0 + m1);
    c = running_sum(c0 + c1);
    if ((t & 63) == 63) {
      h.wave_mass[wave] = m;
      h.wave_count[wave] = c;
    }
  }
  __syncthreads();
  if (wave < kSumWaves) {
    for (int w = 0; w < wave; ++w) {
      m += h.wave_mass[w];
      c += h.wave_count[w];
    }
    to.mass[2 * t] = m - m1;
    to.mass[2 * t + 1] = m;
    to.count[2 * t] = c - c1;
    to.count[2 * t + 1] = c;
  }
  __syncthreads();
}
// The first bin whose running sum exceeds r (the last, if none does); every
// wave finds it for itself.
__device__ __forceinline__ int bin_over(const Sums &to, u64 r, bool by_count) {
  const int lane = threadIdx.x & 63;
  const auto over = [&](int b) { return (by_count ? (u64)to.count[b] : to.mass[b]) > r; };
  const uint64_t lanes = __ballot(over(kLaneBins * lane + kLaneBins - 1));
  if (!lanes) return kBins - 1;
  const int first = kLaneBins * __builtin_ctzll(lanes);
  const uint64_t bins = __ballot(lane < kLaneBins && over(first + (lane & (kLaneBins - 1))));
  return uniform(first + __builtin_ctzll(bins));
}

// ------------------------------------------------------------------- find()

struct Found {
  u64 upto;   // weights up to the token, with it
  u64 own;    // its weight
  int token;  // its index, if that was asked for
};

// Ranks of n codes, no more than there are threads, by comparing each with all:
// `ranks` (0s) gets how many are larger.  Behind the codes are 0s up to the next
// power of two, from 64 on.  Where that is less than the workgroup, threads share
// a code's comparisons.  (Between barriers of the caller.)
__device__ __forceinline__ void rank_codes(const u64 *code, int n, uint32_t *ranks) {
  const int t = threadIdx.x;
  int log = 6;
  while (1 << log < n) ++log;
  const int part = uniform(t >> log), i = t & ((1 << log) - 1), parts = (int)blockDim.x >> log;
  if (uniform(i & ~63) >= n) return;
  const int each = ((n + parts - 1) / parts + 7) & ~7;
  const int from = part * each, to = min(from + each, n);
  const u64 mine = code[i];
  uint32_t rank = 0;
#pragma unroll 1
  for (int j = from; j < to; j += 8) {
    ulonglong2 c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = reinterpret_cast<const ulonglong2 *>(code + j)[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) rank += (c[k].x > mine) + (c[k].y > mine);
  }
  if (i < n && rank) atomicAdd(&ranks[i], rank);
}

// A place in a sum: the last one, if it is past that (sums of slices that came
// together are off by their rounding).
__device__ __forceinline__ u64 within(u64 r, u64 sum) { return r < sum ? r : sum ? sum - 1 : 0; }

// Among the tokens of bin `bin`, before which the order has weights `above`:
// the first one at which the running sum (of weights, or of ones) within the
// bin exceeds r.  Every thread of the workgroup takes part.
template <typename S>
__device__ Found find(const S &src, Shared &sh, const Row &row, int bin, bool by_count, u64 r,
                      u64 above, bool want_token) {
  const int t = threadIdx.x, wave = uniform(t >> 6);
  u64 *const code = sh.hist.mass;      // of the tokens in question: logit, then the lower index
  u64 *const sorted = sh.digits.mass;  // the same by rank
  const auto begin = [&] {
    __syncthreads();  // what was shared has been read
    if (t < kRank) {
      code[t] = 0;
      sh.ranks[t] = 0;
    }
    if (t == 0) sh.n_in = 0;
    __syncthreads();
  };
  const auto take = [&](float v, int i) {
    const int at = atomicAdd(&sh.n_in, 1);
    if (at < kRank) code[at] = (u64)key_of(v) << 32 | (uint32_t)~i;
  };
  // the bin's tokens, and their keys (without the bits in which they do not differ)
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  begin();
  src.each([&](float v, int i) {
    if (v > kNegInf && bin_of(row, v) == bin) {
      const uint32_t k = key_of(v) >> row.key_zeros;
      lo = min(lo, k);
      hi = max(hi, k);
      take(v, i);
    }
  });
  if (t == 0) {
    sh.key_lo = 0xFFFFFFFFu;
    sh.key_hi = 0;
  }
  __syncthreads();
  uint32_t n = (uint32_t)sh.n_in;
  const bool narrow = n > kRank;
  if (narrow) {
    lo = wave_min(lo);
    hi = wave_max(hi);
    if ((t & 63) == 0) {
      atomicMin(&sh.key_lo, lo);
      atomicMax(&sh.key_hi, hi);
    }
    __syncthreads();
    lo = sh.key_lo;
    hi = sh.key_hi;
  }
  int first = 0, last = 0x7FFFFFFF;  // indices that count: all, until the logit is known
  // digits of the distance from the bin's largest key, then of the index
  while (n > kRank && (lo < hi || (want_token && first < last))) {
    const bool keys = lo < hi;
    if (!keys && last == 0x7FFFFFFF) {
      // all have one logit: the place among them is a division, and now ones
      // are summed
      const u64 w = weight(row, row.value(lo));
      if (!by_count && w) {
        const u64 place = within(r / w, n);
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
    const int shift = max(0, 23 - __builtin_clz(span));
    const int log = (span >> shift) < kFewBins ? kFewLog : kCopyLog;
    __syncthreads();
    clear_histogram(sh.hist);
    __syncthreads();
    src.each([&](float v, int i) {
      const uint32_t k = key_of(v) >> row.key_zeros;
      if (k < lo || k > hi || !(v > kNegInf) || i < first || i > last) return;
      if (keys) add_to_bin(sh.hist, (hi - k) >> shift, weight(row, v), 1, log);
      else add_to_bin(sh.hist, (i - first) >> shift, 0, 1, log);
    });
    sum_histogram(sh.hist, sh.digits, log);
    r = within(r, by_count ? (u64)sh.digits.count[kBins - 1] : sh.digits.mass[kBins - 1]);
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
  if (n > kRank) {  // many of one logit, and no index asked for
    const u64 w = weight(row, row.value(lo));
    f.own = w;
    f.upto = above + (within(by_count ? r : w ? r / w : 0, n) + 1) * w;
    return f;
  }
  if (narrow) {
    begin();
    src.each([&](float v, int i) {
      const uint32_t k = key_of(v) >> row.key_zeros;
      if (k >= lo && k <= hi && v > kNegInf && i >= first && i <= last) take(v, i);
    });
    __syncthreads();
    n = (uint32_t)min(sh.n_in, kRank);
  }
  // They are ranked, and summed in that order by a thread each.
  // (Where indices were counted, the weights before are in `above` already, and
  // all weigh the same.)
  const bool by_index = last != 0x7FFFFFFF;
  rank_codes(code, (int)n, sh.ranks);
  __syncthreads();
  if (t < (int)n) sorted[sh.ranks[t]] = code[t];
  __syncthreads();
  const u64 mine = t < (int)n ? sorted[t] : 0;
  const u64 w = t < (int)n ? weight(row, value_of((uint32_t)(mine >> 32))) : 0;
  u64 sum = running_sum(w);
  if ((t & 63) == 63) sh.sum[wave] = sum;
  __syncthreads();
  u64 all = 0;
  for (int i = 0; i < (int)(n + 63) / 64; ++i) {
    if (i == wave) sum += all;
    all += sh.sum[i];
  }
  r = within(r, by_count ? (u64)n : all);
  if (by_count || !all ? t == (int)r : t < (int)n && sum > r && sum - w <= r) {
    sh.upto = by_index ? above + w : above + sum;
    sh.own = w;
    sh.token = n ? (int)~(uint32_t)mine : -1;
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
  float temperature;
  int top_k;         // 0: no cut
  bool nucleus;      // a cut by top_p
  u64 top_p, u;      // fractions of 2^64
  float min_p;       // 0: no cut
  __device__ __forceinline__ bool greedy() const { return !(temperature > 0.f) || top_k == 1; }
  // Slices list their tokens: the first top_k, or those of min_p
  __device__ __forceinline__ bool few() const { return top_k > 0 && top_k <= kTopMost; }
  // (with a longer top_k and top_p besides, tokens that min_p cuts count too)
  __device__ __forceinline__ bool listed() const {
    return few() || (min_p > 0.f && !(top_k > 0 && nucleus));
  }
  // The sum of all tokens counts
  __device__ __forceinline__ bool all() const { return !few() && (nucleus || !(min_p > 0.f)); }
};

__device__ __forceinline__ Ask ask_of(const SampleArgs &a, int at) {
  // all loads at once, u's in place of one that is not given
  const auto given = [&](const float *x) { return (x ? x : a.u)[at]; };
  const float u = a.u[at], t = given(a.temperature), p0 = given(a.top_p), m0 = given(a.min_p);
  const int k0 = __float_as_int(given(reinterpret_cast<const float *>(a.top_k)));
  Ask q;
  q.temperature = a.temperature ? t : 1.f;
  const int k = a.top_k ? k0 : 0;
  q.top_k = k > 0 && k < a.vocab ? k : 0;
  const float p = a.top_p ? p0 : 1.f;
  q.nucleus = p < 1.f;
  q.top_p = fraction(p);
  q.u = fraction(u);
  const float m = a.min_p ? m0 : 0.f;
  q.min_p = !(m > 0.f) ? 0.f : fminf(m, 1.f);
  return q;
}

// How far from the largest logit one of min_p lies (0 or less, the logarithm within
// 1e-5 of it).  At an infinite temperature all tokens weigh the same, and none is too
// far: there the product with the logarithm of 1 is no number.
__device__ __forceinline__ double depth_of_min_p(const Ask &q) {
  const double d = (double)__logf(q.min_p) * (double)q.temperature;
  return d == d ? d : -__builtin_inf();
}

// What a token of min_p weighs.
__device__ __forceinline__ u64 least_weight(const Row &row, const Ask &q) {
  return (u64)__builtin_ceil((double)weight(row, row.largest) * (double)q.min_p);
}

__device__ __forceinline__ u64 before(const Sums &s, int bin) { return bin ? s.mass[bin - 1] : 0; }

// Whether a logit is in one of the bins of a Need.  A bin is b or less just
// where logit * bin_rate >= base - b, which most logits are not for any.
struct Needed {
  Row row;
  Need n;
  float least;
  __device__ __forceinline__ Needed(const Row &r, const Need &need) : row(r), n(need) {
    const int last = max(max(n.m1, n.k1), max(n.p1, n.r1));
    least = last == kBins - 1 ? kNegInf : r.base - (float)last;
  }
  __device__ __forceinline__ bool operator()(float v) const {
    if (v * row.bin_rate < least) return false;
    const int b = bin_of(row, v);
    return v > kNegInf && ((b >= n.m0 && b <= n.m1) || (b >= n.k0 && b <= n.k1) ||
                           (b >= n.p0 && b <= n.p1) || (b >= n.r0 && b <= n.r1));
  }
};

// mass_min: the weights that min_p leaves, where they are known (else those
// of the bins up to its own, in which it then has to be found out).
__device__ __forceinline__ Need need_of(const Sums &s, const Row &row, const Ask &q, u64 all,
                                        u64 mass_min, bool known) {
  Need n{0, -1, 0, -1, 0, -1, 0, -1};
  u64 min_lo = mass_min, min_hi = mass_min;
  if (!known && q.min_p > 0.f) {
    // (its place within a bin, 0.07 of a temperature, of what min_p says)
    const int b = bin_of(row, (float)((double)row.largest + depth_of_min_p(q)));
    n.m0 = max(0, b - 1);
    n.m1 = min(kBins - 1, b + 1);
    min_lo = before(s, n.m0);
    min_hi = s.mass[n.m1];
  }
  u64 lo = all, hi = all;
  if (q.top_k && s.count[kBins - 1] > (uint32_t)q.top_k) {
    n.k0 = n.k1 = bin_over(s, (u64)(q.top_k - 1), true);
    lo = before(s, n.k0);
    hi = s.mass[n.k0];
  }
  if (q.nucleus) {
    n.p0 = bin_over(s, just_below(lo, q.top_p), false);
    n.p1 = bin_over(s, just_below(hi, q.top_p), false);
    lo = min(lo, before(s, n.p0));
    hi = min(hi, s.mass[n.p1]);
  }
  n.r0 = bin_over(s, __umul64hi(min(lo, min_lo), q.u), false);
  n.r1 = bin_over(s, __umul64hi(min(hi, min_hi), q.u), false);
  return n;
}

// The questions in turn: of top_k, of top_p, and of u.  `all` is the sum of the
// row's weights, `whole` gets the sum of those that stay.
template <typename S>
__device__ __forceinline__ Found answer(const S &src, Shared &sh, const Row &row, const Ask &q,
                                        u64 all, u64 mass_min, u64 *whole) {
  const Sums &s = sh.bins;
  u64 m = all;
  Found f{0, 0, -1};
  for (int turn = 0; turn < 3; ++turn) {
    u64 r = (u64)(q.top_k - 1);
    if (turn == 0 && !(q.top_k && s.count[kBins - 1] > (uint32_t)q.top_k)) continue;
    if (turn == 1) {
      r = just_below(m, q.top_p);
      if (!q.nucleus || r >= s.mass[kBins - 1]) continue;
    }
    if (turn == 2) {
      m = min(m, mass_min);
      *whole = m;
      r = __umul64hi(m, q.u);
    }
    const int b = bin_over(s, r, turn == 0);
    const u64 m0 = before(s, b);
    // no weight in the bin; or min_p leaves no more than the bins before, and
    // nothing else is to be taken of the sum
    if (turn < 2 && (s.mass[b] == m0 || (m0 >= mass_min && (turn == 1 || !q.nucleus)))) {
      m = min(m, m0);
      continue;
    }
    f = find(src, sh, row, b, turn == 0, r - (turn ? m0 : b ? s.count[b - 1] : 0), m0, turn == 2);
    if (turn < 2) m = min(m, min(f.upto, s.mass[b]));
  }
  return f;
}

// f(place, key, index) for the tokens of a source that `in` picks.
template <typename T, int N, typename In, typename F>
__device__ __forceinline__ void pick(const HeldSource<T, N> &src, const RowSource<T> &again, int *counter,
                                     In &&in, F &&f) {
  src.pick(again, counter, in, f);
}
template <typename L, typename In, typename F>
__device__ __forceinline__ void pick(const GatherSource &src, const L &, int *counter, In &&in, F &&f) {
  src.pick(counter, in, f);
}
template <typename T, typename L, typename In, typename F>
__device__ __forceinline__ void pick(const RowSource<T> &src, const L &, int *counter, In &&in, F &&f) {
  src.each([&](float v, int i) {
    if (in(v)) f(atomicAdd(counter, 1), key_of(v), i);
  });
}

// Those tokens into the list.  Their number: where it is more than kList, the
// list is of no use.
template <typename S, typename L, typename In>
__device__ __forceinline__ int list_tokens(const S &src, const L &again, Shared &sh, In &&in) {
  __syncthreads();
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  pick(src, again, &sh.n_list, in, [&](int j, uint32_t key, int i) {
    if (j < kList) {
      sh.key[j] = key;
      sh.index[j] = i;
    }
  });
  __syncthreads();
  return sh.n_list;
}

// The bins of all that may stay, from a source that has it; and what min_p
// leaves of it.
template <typename S>
__device__ __forceinline__ u64 bins_of(const S &src, Shared &sh, const Row &row, const Ask &q) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  clear_histogram(sh.hist);
  __syncthreads();
  u64 mass_min = 0;
  const bool counts = q.top_k != 0;
  const u64 least = least_weight(row, q);
  const bool plain = !row.far && !counts && least == 0;
  if (plain) {
    add_weights(src, sh.hist, row);
  } else {
    src.each([&](float v, int) {
      const int b = bin_of(row, v);
      const u64 w = weight(row, v);
      add_to_bin(sh.hist, b, w, counts && v > kNegInf);
      if (w >= least) mass_min += w;
    });
    mass_min = running_sum(mass_min);
    if (lane == 63) sh.sum[wave] = mass_min;
  }
  sum_histogram(sh.hist, sh.bins);
  if (plain) return sh.bins.mass[kBins - 1];
  mass_min = 0;
  for (int w = 0; w < waves; ++w) mass_min += sh.sum[w];
  return mass_min;
}

// The same where the list is no longer than a workgroup: a thread a token finds
// its rank by comparing with all of them, and with weights and running sums in
// that order every question is one comparison a thread.
__device__ __forceinline__ Found sorted_row(Shared &sh, int n, const Row &row, const Ask &q,
                                            bool all_here, u64 all, u64 *whole) {
  const int t = threadIdx.x, wave = uniform(t >> 6);
  u64 *const code = sh.hist.mass;   // logit, then the lower index
  u64 *const upto = sh.bins.mass;   // (both sums' arrays: 1024 of them)
  static_assert(kBins * kCopies >= kWide && 2 * sizeof(Sums) >= 8 * kWide, "a token a thread");
  __syncthreads();
  const uint32_t key = t < n ? sh.key[t] : 0;
  const int index = t < n ? sh.index[t] : 0;
  const u64 mine = (u64)key << 32 | (uint32_t)~index;
  code[t] = t < n ? mine : 0;
  sh.ranks[t] = 0;
  if (t == 0) sh.upto = 0;
  __syncthreads();
  rank_codes(code, n, sh.ranks);
  __syncthreads();
  if (t < n) {
    const uint32_t rank = sh.ranks[t];
    sh.key[rank] = key;
    sh.index[rank] = index;
  }
  __syncthreads();
  const u64 w = t < n ? weight(row, value_of(sh.key[t])) : 0;
  const int place = t < n ? sh.index[t] : 0;
  u64 sum = running_sum(w);
  if ((t & 63) == 63) sh.sum[wave] = sum;
  __syncthreads();
  for (int i = 0; i < wave; ++i) sum += sh.sum[i];
  upto[t] = sum;
  // the last that weighs min_p (weights fall with the order, but for their rounding)
  const uint64_t heavy = __ballot(t < n && w >= least_weight(row, q));
  if (heavy && (t & 63) == 63 - __builtin_clzll(heavy)) atomicMax(&sh.upto, sum);
  __syncthreads();
  const u64 here = upto[n - 1], mass_min = sh.upto;
  u64 m = all_here ? here : all;
  if (q.top_k && n > q.top_k) m = upto[q.top_k - 1];
  if (q.nucleus) {
    const u64 r = just_below(m, q.top_p);
    if (sum > r && sum - w <= r) sh.own = sum;
    __syncthreads();
    m = min(m, r < here ? sh.own : here);
  }
  m = min(m, mass_min);
  *whole = m;
  const u64 r = __umul64hi(m, q.u);
  __syncthreads();
  if (sum > r && sum - w <= r) {
    sh.own = w;
    sh.token = place;
  }
  __syncthreads();
  return Found{0, sh.own, sh.token};
}

// A row of which all that may stay is in the list.
__device__ __forceinline__ Found listed_row(Shared &sh, int n, const Row &row, const Ask &q,
                                            bool all_here, u64 all, u64 *whole) {
  if (n <= (int)blockDim.x) return sorted_row(sh, n, row, q, all_here, all, whole);
  const ListSource list{sh, n};
  const u64 mass_min = bins_of(list, sh, row, q);
  return answer(list, sh, row, q, all_here ? sh.bins.mass[kBins - 1] : all, mass_min, whole);
}

// Any row, from a source that has all of it (or all that may stay).
// `long_way` has the same tokens, and need not be fast.
template <typename S, typename L>
__device__ __forceinline__ Found whole_row(const S &src, const L &long_way, Shared &sh,
                                           const Row &row, const Ask &q, bool all_here, u64 all,
                                           u64 *whole) {
  const u64 mass_min = bins_of(src, sh, row, q);
  if (all_here) all = sh.bins.mass[kBins - 1];
  const int n = list_tokens(src, long_way, sh, Needed(row, need_of(sh.bins, row, q, all, mass_min, true)));
  return n <= kList ? answer(ListSource{sh, n}, sh, row, q, all, mass_min, whole)
                    : answer(long_way, sh, row, q, all, mass_min, whole);
}

// What can be among the first top_k, or weigh min_p: logits of which `scale`
// times is `least` or more.  Of the first top_k of a row its part in this workgroup
// has at most its own first top_k, and where so many of its threads' largest
// logits (of each half of what a thread holds) lie in the bins to `last`, they
// do.  (min_p is taken a little lower than it is, by far more than anything is
// rounded.)  The largest logit is always among them.
struct Limits {
  float scale, least;
  int last;
  __device__ __forceinline__ bool operator()(float v) const {
    return v > kNegInf && v * scale >= least;
  }
};
__device__ __forceinline__ Limits limits_of(const Row &row, const Ask &q, int last) {
  if (q.few()) return {row.bin_rate, last == kBins - 1 ? kNegInf : row.base - (float)last, last};
  if (!(q.min_p > 0.f)) return {1.f, kNegInf, kBins - 1};
  return {1.f,
          __double2float_rd((double)row.largest + depth_of_min_p(q) * (1.0 + 1e-4) -
                            1e-4 * (double)q.temperature),
          kBins - 1};
}
template <typename T, int N>
__device__ __forceinline__ Limits limits_of(const HeldSource<T, N> &src, const Row &row,
                                            const Ask &q, Hist &hist, Sums &sums) {
  if (!q.few()) return limits_of(row, q, kBins - 1);
  clear_histogram(hist);
  __syncthreads();
  constexpr int E = RowSource<T>::E;
  float top[2] = {kNegInf, kNegInf};
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int h = N > 1 ? 2 * j / N : 2 * i / E;
      top[h] = fmaxf(top[h], src.v[j * E + i]);
    }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (top[h] > kNegInf) add_to_bin(hist, bin_of(row, top[h]), 0, 1);
  sum_histogram(hist, sums);
  return limits_of(row, q, bin_over(sums, (u64)(q.top_k - 1), true));
}

__device__ __forceinline__ void write(const SampleArgs &a, int at, int token, float prob) {
  if (threadIdx.x) return;
  a.tokens[at] = token;
  if (a.probs) a.probs[at] = prob;
}

// The largest of (v, i) over the workgroup, the smallest i among equals: as
// one number, key and ~i.
__device__ __forceinline__ void first_largest(u64 (&best)[kMostWaves], float &v, int &i) {
  const u64 mine = wave_max((u64)key_of(v) << 32 | (uint32_t)~i);
  if ((threadIdx.x & 63) == 0) best[threadIdx.x >> 6] = mine;
  __syncthreads();
  u64 most = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) most = max(most, best[w]);
  v = value_of((uint32_t)(most >> 32));
  i = (int)~(uint32_t)most;
}
template <typename T, int N>
__device__ __forceinline__ void first_of(const HeldSource<T, N> &src, float &best, int &first) {
  best = kNegInf;
  first = 0x7FFFFFFF;
  src.each([&](float v, int i) {
    if (v > best) {
      best = v;
      first = i;
    }
  });
}

template <typename T>
__device__ __forceinline__ RowSource<T> logits_of(const SampleArgs &a, int at) {
  return RowSource<T>{static_cast<const T *>(a.logits) + (size_t)at * a.stride, a.vocab};
}

// A workgroup a row, whose logits it holds.
//
// What bounds it: one compute unit.  A row of 32000 fp32 logits by top_p is 23 us:
// 3.4 until the largest logit is known (128 KB through one compute unit), 7.5 for
// the weights by bin (32 logits a thread, 15 operations of 64 bits each, four
// cycles an operation and four waves on a SIMD), 2.3 for the list of the tokens in
// question, and the questions of 2 to 4 us, chains of barriers and LDS reads.  Loops
// over the registers are rolled: unrolled ones wait for their instructions.  A wave
// has 128 registers, which 16 waves leave it, and keeps 8 in scratch (36 bytes a lane)
// in rows above 16384 logits, 2 in rows of bf16 above 8192.
template <typename T, int N>
__global__ __launch_bounds__(kWide) void k_sample_row(SampleArgs a) {
  __shared__ Shared sh;
  const int at = blockIdx.x;
  const RowSource<T> src = logits_of<T>(a, at);
  HeldSource<T, N> held;
  held.load(src, 0);
  float best;
  int first;
  first_of(held, best, first);
  first_largest(sh.sum, best, first);
  const Ask q = ask_of(a, at);
  if (best == kNegInf) return write(a, at, -1, 0.f);
  if (q.greedy()) return write(a, at, first, 1.f);
  const Row row = row_of<T>(best, q.temperature, a.bits);
  u64 whole;
  Found f;
  if (!q.all() && q.listed()) {
    const int n = list_tokens(held, src, sh, limits_of(held, row, q, sh.hist, sh.digits));
    f = n <= kList ? listed_row(sh, n, row, q, true, 0, &whole)
                   : whole_row(src, src, sh, row, q, true, 0, &whole);
  } else {
    f = whole_row(held, src, sh, row, q, true, 0, &whole);
  }
  write(a, at, f.token, (float)((double)f.own / (double)whole));
}

// ------------------------------------------------------------------- slices

template <typename T>
constexpr int kPieces = kSlice / (kNarrow * RowSource<T>::E);

// What bounds it: of rows that list their tokens, or take the first, HBM (512 rows
// of 131072 fp32 logits, 268 MB: greedy 48 us, 5.5 TB/s; top_k or min_p 70, 3.8
// TB/s); of rows whose weights go by bin, those weights, 25 vector operations a
// logit, 15 of them of 64 bits (98 us; at four cycles each they are 45 us of every
// SIMD's issue, and the read 52).  A wave has 78 registers, six waves on a SIMD; at
// 64 it spills.  Tried and not kept: loads inside the loop over pieces (63 us greedy:
// conversions between them made each wait for the one before).  Without its atomics
// it is no faster.
template <typename T>
__global__ __launch_bounds__(kNarrow) void k_sample_slices(SampleArgs a) {
  __shared__ Hist hist;
  __shared__ Sums sums;
  __shared__ u64 sh_sum[kMostWaves];
  __shared__ int sh_listed;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int slice = blockIdx.x, at = a.row0 + blockIdx.y;
  const size_t rs = (size_t)blockIdx.y * a.slices + slice;
  if (slice == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.active[0] = 0;
  const RowSource<T> src = logits_of<T>(a, at);
  HeldSource<T, kPieces<T>> held;
  held.load(src, slice);
  const Ask q = ask_of(a, at);
  float best;
  int first;
  first_of(held, best, first);
  if (threadIdx.x == 0) sh_listed = 0;
  first_largest(sh_sum, best, first);
  SliceHead head{0.0, 0, best, first, 0.f, 0, 0, kBins - 1, 0, 0};
  if (best == kNegInf || q.greedy()) {
    if (threadIdx.x == 0) a.heads[rs] = head;
    return;
  }
  const Row row = row_of<T>(best, q.temperature, a.bits);
  head.base = row.base;
  head.ref = row.ref;
  const bool listed = q.listed(), all = q.all();
  if (listed) {
    const Limits l = limits_of(held, row, q, hist, sums);
    head.last = l.last;
    held.pick(src, &sh_listed, l, [&](int n, uint32_t key, int i) {
      if (n < kSliceList) a.list[rs * kSliceList + n] = make_uint2(key, (uint32_t)i);
    });
    __syncthreads();
    head.listed = sh_listed;
    if (!all && head.listed <= kSliceList) {
      if (threadIdx.x == 0) a.heads[rs] = head;
      return;
    }
  }
  head.binned = 1;
  clear_histogram(hist);
  __syncthreads();
  if (row.far) {
    held.each([&](float v, int) {
      const int b = bin_of(row, v);
      add_to_bin(hist, b, weight(row, v), q.top_k != 0 && v > kNegInf);
    });
  } else {
    add_weights(held, hist, row);
    if (q.top_k != 0)
      held.each([&](float v, int) { add_to_bin(hist, bin_of(row, v), 0, v > kNegInf); });
  }
  __syncthreads();
  u64 total = 0;
  for (int i = threadIdx.x; i < kBins; i += kNarrow) {
    u64 m = 0;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) m += hist.mass[i * kCopies + k];
    a.mass[rs * kBins + i] = m;
    total += m;
    if (q.top_k == 0) continue;  // (no one asks for numbers)
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) c += hist.count[i * kCopies + k];
    a.count[rs * kBins + i] = c;
  }
  total = running_sum(total);
  if (lane == 63) sh_sum[wave] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 0; w < kNarrow / 64; ++w) head.total += sh_sum[w];
    a.heads[rs] = head;
  }
}

// A row's slices together, lanes of a wave for them.
struct Joined {
  float largest;
  int first;
  bool whole;  // every slice has listed all that may stay of it
};
__device__ __forceinline__ Joined join_heads(const SliceHead *heads, int slices, const Ask &q) {
  u64 best = 0;
  bool more = false;
  for (int s = threadIdx.x & 63; s < slices; s += 64) {
    const SliceHead h = heads[s];
    best = max(best, (u64)key_of(h.largest) << 32 | (uint32_t)~h.first);
    more = more || h.listed > kSliceList;
  }
  best = wave_max(best);
  return {value_of((uint32_t)(best >> 32)), (int)~(uint32_t)best, q.listed() && !__any(more)};
}
// What a slice's weights are shifted by.
__device__ __forceinline__ int slice_shift(const Row &row, const SliceHead &h) {
  if (row.far) return h.largest == row.largest ? 0 : 63;
  return (int)__builtin_fmin(row.ref - h.ref, 63.0);
}

// Weights and counts by bin of all slices, as running sums: a thread a bin (of
// kMiddle), kBinsBatch slices' loads at once.  Of a slice that has listed all that may
// stay, that.
__device__ __forceinline__ void join_bins(const SampleArgs &a, int r, const Row &row, const Ask &q,
                                          Joining &sh) {
  const int t = threadIdx.x;
  const bool counts = q.top_k != 0;
  clear_histogram(sh.hist);
  if (t < a.slices) {
    const SliceHead h = a.heads[(size_t)r * a.slices + t];
    sh.base[t] = h.base;
    sh.shift[t] = h.largest > kNegInf ? slice_shift(row, h) : 0;
    // a slice without tokens is an empty list
    sh.length[t] = h.binned ? -1 : h.largest > kNegInf ? h.listed : 0;
  }
  __syncthreads();
  const size_t from = (size_t)r * a.slices * kBins + t;
#pragma unroll 1
  for (int s0 = 0; s0 < a.slices; s0 += kBinsBatch) {
    u64 m[kBinsBatch];
    uint32_t c[kBinsBatch];
#pragma unroll
    for (int j = 0; j < kBinsBatch; ++j) {
      const bool binned = s0 + j < a.slices && sh.length[s0 + j] < 0;
      m[j] = binned ? a.mass[from + (size_t)(s0 + j) * kBins] : 0;
      c[j] = binned && counts ? a.count[from + (size_t)(s0 + j) * kBins] : 0;
    }
#pragma unroll
    for (int j = 0; j < kBinsBatch; ++j) {
      if (m[j] | c[j])
        add_to_bin(sh.hist, row_bin(row, sh.base[s0 + j], t), m[j] >> uniform(sh.shift[s0 + j]), c[j]);
    }
  }
  if (q.listed()) {
    const GatherSource lists{a.list + (size_t)r * a.slices * kSliceList, sh.length, a.slices};
    lists.each([&](float v, int) { add_to_bin(sh.hist, bin_of(row, v), weight(row, v), counts); });
  }
  sum_histogram(sh.hist, sh.bins);
}

// What bounds it: latency, of the settings, the heads, the bins and the sums in
// turn, one after the other (64 rows 9 us, 512 rows of 17 slices, 36 MB, 11 us and 16
// where every row comes here).  All bins of 24 slices are in flight at once: 8
// took 11.5 and 14 us.
template <typename T>
__global__ __launch_bounds__(kMiddle) void k_sample_decide(SampleArgs a) {
  __shared__ Joining sh;
  const int r = blockIdx.x, at = a.row0 + r;
  const Ask q = ask_of(a, at);
  if (q.greedy()) return;
  const Joined joined = join_heads(a.heads + (size_t)r * a.slices, a.slices, q);
  if (joined.largest == kNegInf || joined.whole) return;
  const Row row = row_of<T>(joined.largest, q.temperature, a.bits);
  join_bins(a, r, row, q, sh);
  const u64 all = sh.bins.mass[kBins - 1];
  const Need need = need_of(sh.bins, row, q, all, all, false);
  RowState &state = a.state[r];
  for (int i = threadIdx.x; i < kBins; i += blockDim.x) {
    state.bins.mass[i] = sh.bins.mass[i];
    state.bins.count[i] = sh.bins.count[i];
  }
  if (threadIdx.x == 0) {
    state.largest = joined.largest;
    state.need = need;
    a.active[1 + atomicAdd(a.active, 1)] = r;
  }
}

// What bounds it: HBM (512 rows that all come here, 268 MB, 45 us; slices that took
// several tasks in turn had twice the registers and took 61); of 64 rows of mixed
// settings its start (9 us).
template <typename T>
__global__ __launch_bounds__(kNarrow) void k_sample_collect(SampleArgs a) {
  __shared__ int sh_n;
  const int task = blockIdx.x;
  if (task >= a.active[0] * a.slices) return;
  const int r = a.active[1 + task / a.slices], slice = task % a.slices, at = a.row0 + r;
  const size_t rs = (size_t)r * a.slices + slice;
  const RowSource<T> src = logits_of<T>(a, at);
  HeldSource<T, kPieces<T>> held;
  held.load(src, slice);
  if (threadIdx.x == 0) sh_n = 0;
  __syncthreads();
  const Needed needed(row_of<T>(a.state[r].largest, a.temperature ? a.temperature[at] : 1.f, a.bits),
                      a.state[r].need);
  held.pick(src, &sh_n, needed, [&](int n, uint32_t key, int i) {
    if (n < kSliceList) a.list[rs * kSliceList + n] = make_uint2(key, (uint32_t)i);
  });
  __syncthreads();
  if (threadIdx.x == 0) a.heads[rs].collected = sh_n;
}

// A row whose slices have listed all that may stay.
__device__ __forceinline__ void pick_listed(const SampleArgs &a, int r, Shared &sh, const Row &row,
                                            const Ask &q) {
  const int lane = threadIdx.x & 63, at = a.row0 + r;
  const SliceHead *heads = a.heads + (size_t)r * a.slices;
  u64 whole;
  // all weights, and what the slices' own first top_k leave for the row's
  // (every wave for itself; the lists' lengths all the same)
  u64 all = 0;
  uint32_t last = kBins - 1;
  for (int s = lane; s < a.slices; s += 64) {
    const SliceHead h = heads[s];
    sh.length[s] = h.listed;
    if (!(h.largest > kNegInf)) continue;
    if (q.all()) all += shifted(h.total, slice_shift(row, h));
    last = min(last, (uint32_t)row_bin(row, h.base, h.last));
  }
  all = wave_sum(all);
  last = wave_min(last);
  const GatherSource gather{a.list + (size_t)r * a.slices * kSliceList, sh.length, a.slices};
  const int n = list_tokens(gather, gather, sh, limits_of(row, q, (int)last));
  const Found f = n <= kList ? listed_row(sh, n, row, q, !q.all(), all, &whole)
                             : whole_row(gather, gather, sh, row, q, !q.all(), all, &whole);
  write(a, at, f.token, (float)((double)f.own / (double)whole));
}

// What bounds it: chains of barriers, LDS reads and loads in one workgroup (64 rows
// 17 to 20 us, 512 rows two to a compute unit 27): 2 for settings and heads, 2 to 4
// for the lists, then two questions of 4 to 9 us by top_p, or the ranks of a list by
// top_k.  Four waves a SIMD, which LDS allows.
template <typename T>
__global__ __launch_bounds__(kMiddle, 4) void k_sample_pick(SampleArgs a) {
  __shared__ Shared sh;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = blockIdx.x, at = a.row0 + r;
  const SliceHead *heads = a.heads + (size_t)r * a.slices;
  const Ask q = ask_of(a, at);
  const Joined joined = join_heads(heads, a.slices, q);
  if (joined.largest == kNegInf) return write(a, at, -1, 0.f);
  if (q.greedy()) return write(a, at, joined.first, 1.f);
  const Row row = row_of<T>(joined.largest, q.temperature, a.bits);
  if (joined.whole) return pick_listed(a, r, sh, row, q);
  const RowState &state = a.state[r];
  const Need need = state.need;
  for (int i = threadIdx.x; i < kBins; i += blockDim.x) {
    sh.bins.mass[i] = state.bins.mass[i];
    sh.bins.count[i] = state.bins.count[i];
  }
  bool more = false;
  for (int s = lane; s < a.slices; s += 64) {
    const int n = heads[s].collected;
    sh.length[s] = n;
    more = more || n > kSliceList;
  }
  const bool fits = !__any(more);
  __syncthreads();
  const u64 all = sh.bins.mass[kBins - 1];
  // the tokens in question, and of min_p's bins the weights that it leaves
  const RowSource<T> src = logits_of<T>(a, at);
  const GatherSource gather{a.list + (size_t)r * a.slices * kSliceList, sh.length, a.slices};
  const int n = fits ? list_tokens(gather, gather, sh, [](float) { return true; }) : kList + 1;
  u64 part = 0;
  if (need.m1 >= need.m0) {
    const u64 least = least_weight(row, q);
    const auto look = [&](float v, int) {
      const int b = bin_of(row, v);
      if (b < need.m0 || b > need.m1) return;
      const u64 w = weight(row, v);
      if (w >= least) part += w;
    };
    if (n <= kList) ListSource{sh, n}.each(look);
    else if (fits) gather.each(look);
    else src.each(look);
    part = running_sum(part);
    if (lane == 63) sh.sum[wave] = part;
  }
  __syncthreads();
  u64 mass_min = all;
  if (need.m1 >= need.m0) {
    mass_min = before(sh.bins, need.m0);
    for (int w = 0; w < kMiddle / 64; ++w) mass_min += sh.sum[w];
    mass_min = min(mass_min, sh.bins.mass[need.m1]);
  }
  u64 whole;
  const Found f = n <= kList ? answer(ListSource{sh, n}, sh, row, q, all, mass_min, &whole)
                  : fits     ? answer(gather, sh, row, q, all, mass_min, &whole)
                             : answer(src, sh, row, q, all, mass_min, &whole);
  write(a, at, f.token, (float)((double)f.own / (double)whole));
}

// ---------------------------------------------------------------- host side

int weight_bits(int vocab) {
  int log = 12;
  while (1 << log < vocab) ++log;
  return 63 - log;  // (the largest weighs between half of 2^bits and all of it)
}

// Slices of a row (none: a row is a workgroup's), and the workspace of the
// rows that are done at once.
struct SamplePlan {
  int pieces, slices, rows;
  size_t active, state, heads, mass, count, list, total;
};

SamplePlan sample_plan(int n_rows, int vocab, int xtype) {
  SamplePlan p{};
  p.total = 256;
  const int e = xtype == RFPX_X_BF16 ? 8 : 4;
  const int pieces = (vocab + 2 * (e - 1)) / e;  // wherever the row begins
  const int most = kRowMost / (kWide * e);
  for (p.pieces = 1; p.pieces < most && p.pieces * kWide < pieces;) p.pieces *= 2;
  if (p.pieces * kWide >= pieces) return p;
  p.rows = n_rows < kRowsAtOnce ? n_rows : kRowsAtOnce;
  p.slices = (pieces * e + kSlice - 1) / kSlice;
  const size_t rs = (size_t)p.rows * p.slices;
  p.active = 0;
  p.state = p.active + align_up(((size_t)p.rows + 1) * 4, 256);
  p.heads = p.state + align_up(p.rows * sizeof(RowState), 256);
  p.mass = p.heads + align_up(rs * sizeof(SliceHead), 256);
  p.count = p.mass + align_up(rs * kBins * 8, 256);
  p.list = p.count + align_up(rs * kBins * 4, 256);
  p.total = p.list + align_up(rs * kSliceList * 8, 256);
  if (p.total < 256) p.total = 256;
  return p;
}

template <typename T>
hipError_t launch_sample(const SamplePlan &p, SampleArgs a, uint8_t *w, hipStream_t s) {
  constexpr int most = kRowMost / (kWide * RowSource<T>::E);
  if (!p.slices) {
    void (*row)(SampleArgs) = p.pieces == 1   ? k_sample_row<T, 1>
                              : p.pieces == 2 ? k_sample_row<T, 2>
                              : p.pieces == 4 ? k_sample_row<T, 4>
                                              : k_sample_row<T, most>;
    return launch_k(row, dim3(a.n_rows), dim3(kWide), 0, s, a);
  }
  a.slices = p.slices;
  a.active = reinterpret_cast<int *>(w + p.active);
  a.state = reinterpret_cast<RowState *>(w + p.state);
  a.heads = reinterpret_cast<SliceHead *>(w + p.heads);
  a.mass = reinterpret_cast<u64 *>(w + p.mass);
  a.count = reinterpret_cast<uint32_t *>(w + p.count);
  a.list = reinterpret_cast<uint2 *>(w + p.list);
  hipError_t e = hipSuccess;
  for (a.row0 = 0; a.row0 < a.n_rows && e == hipSuccess; a.row0 += p.rows) {
    a.rows = a.n_rows - a.row0 < p.rows ? a.n_rows - a.row0 : p.rows;
    e = launch_k(k_sample_slices<T>, dim3(a.slices, a.rows), dim3(kNarrow), 0, s, a);
    if (e == hipSuccess) e = launch_k(k_sample_decide<T>, dim3(a.rows), dim3(kMiddle), 0, s, a);
    if (e == hipSuccess)
      e = launch_k(k_sample_collect<T>, dim3(a.rows * a.slices), dim3(kNarrow), 0, s, a);
    if (e == hipSuccess) e = launch_k(k_sample_pick<T>, dim3(a.rows), dim3(kMiddle), 0, s, a);
  }
  return e;
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
  return sample_plan(n_rows, vocab, xtype).total;
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
  const SamplePlan p = sample_plan(n_rows, vocab, xtype);
  if (ws_bytes < p.total)
    return fail(RFPX_E_WORKSPACE, "%s: workspace holds %zu bytes, needs %zu", fn, ws_bytes, p.total);
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
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e = xtype == RFPX_X_BF16
                           ? launch_sample<uint16_t>(p, a, static_cast<uint8_t *>(ws), s)
                           : launch_sample<uint32_t>(p, a, static_cast<uint8_t *>(ws), s);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

}  // extern "C"
