// tree.hip -- what surrounds the attention of a tree of drafted tokens:
// ancestor masks and positions, acceptance, and the move of the accepted
// columns' keys and values to where a plain sequence has them.
//
// All three are a few kilobytes of work (64 trees of up to 256 columns: 0.3 MB, 0.06
// us of HBM): what bounds them is the launch and a short chain of dependent reads
// (of deep trees the walk through their parents, which is kept in LDS).
#include "../../include/rfpx_verify.h"
#include "rfpx_attn.hpp"

namespace rfpx {
namespace {

constexpr int kThreads = 256;
constexpr int kColsMax = RFPX_TREE_COLS_MAX;

// The columns of a sequence that the call may touch: first row and number.
__device__ __forceinline__ int tree_cols(const int32_t *starts, int b, int n_rows, int *first) {
  const int s0 = starts[b];
  *first = s0;
  if (s0 < 0) return 0;
  return max(0, min(min(starts[b + 1], n_rows) - s0, kColsMax));
}

struct MaskArgs {
  const int32_t *parents, *base, *lens, *starts;
  uint32_t *masks;
  int32_t *positions;
  int n_rows, words;
};

// A workgroup a sequence, a thread a column: it climbs to its root, and since
// parents come before their children its words are done from the last to the
// first.  Two launches less than a matrix of ancestors by squaring, and no
// more reads than bits are set.  One tree of 16 columns takes 2.0 us on an MI355X,
// 64 of up to 256 columns 4.8.  Of 64 trees of 256 in 12 levels, 4.2 us, 2.4 are the
// launch and two dependent reads (one word, no climb), 0.9 the stores of eight words
// a lane (no climb 3.3), 0.9 the climb; it bounds deep trees: a chain of 256 28 us.
__global__ __launch_bounds__(kThreads) void k_tree_masks(MaskArgs a) {
  __shared__ int16_t parent[kColsMax];
  const int b = blockIdx.x;
  int s0;
  const int n = tree_cols(a.starts, b, a.n_rows, &s0);
  if (n == 0) return;
  const int base = a.base ? a.base[b] : a.lens[b] - (a.starts[b + 1] - s0);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int p = a.parents[s0 + i];
    parent[i] = (int16_t)(p >= 0 && p < i ? p : -1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    uint32_t *mask = a.masks + (size_t)(s0 + i) * a.words;
    int depth = -1, w = a.words - 1;
    uint32_t bits = 0;
    for (int j = i; j >= 0; j = parent[j]) {
      ++depth;
      if (j >> 5 >= a.words) continue;
      for (; w > j >> 5; --w) {
        mask[w] = bits;
        bits = 0;
      }
      bits |= 1u << (j & 31);
    }
    for (; w >= 0; --w) {
      mask[w] = bits;
      bits = 0;
    }
    if (a.positions) a.positions[s0 + i] = base + depth;
  }
}

struct AcceptArgs {
  const int32_t *parents, *tokens, *drawn, *lens, *starts;
  int32_t *path, *counts, *next, *lens_out;
  int n_rows, path_cols;
};

// A workgroup a sequence: every column whose token was drawn at its parent
// offers itself as the parent's next one (the smallest number wins, so the
// order of the offers is of no account), and one thread follows the chain.  One
// tree of 16 columns takes 2.2 us on an MI355X, 64 of up to 256 columns 4.0, the
// launch and dependent reads; a chain of 256 that is all confirmed 17, the walk.
__global__ __launch_bounds__(kThreads) void k_tree_accept(AcceptArgs a) {
  __shared__ int drawn[kColsMax], child[kColsMax];
  __shared__ int16_t path[kColsMax];
  __shared__ int count;
  const int b = blockIdx.x;
  int s0;
  const int n = tree_cols(a.starts, b, a.n_rows, &s0);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    drawn[i] = a.drawn[s0 + i];
    child[i] = kColsMax;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int p = a.parents[s0 + i], token = a.tokens[s0 + i];
    if (p >= 0 && p < i && token >= 0 && token == drawn[p]) atomicMin(&child[p], i);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int at = 0, k = 0, last = -1;
    while (at < n && k < a.path_cols) {
      path[k++] = (int16_t)at;
      last = at;
      at = child[at];
    }
    count = k;
    a.counts[b] = k;
    a.next[b] = last < 0 ? -1 : drawn[last];
    if (a.lens_out) a.lens_out[b] = max(0, a.lens[b] - (a.starts[b + 1] - s0) + k);
  }
  __syncthreads();
  int32_t *out = a.path + (size_t)b * a.path_cols;
  for (int i = threadIdx.x; i < a.path_cols; i += kThreads) out[i] = i < count ? path[i] : -1;
}

struct CommitArgs {
  KvView v;
  const int32_t *path, *counts;
  float *acc;
  int32_t *pos;
  int path_cols;
};

// A workgroup a sequence and kv head, sixteen lanes a move, sixteen moves at a
// time.  A slot may be where one column leaves and another arrives: entries
// ascend, so whatever the moves of one turn write lies before all that a later
// turn reads, and within a turn every read comes before the barrier and every
// write behind it.  What bounds it is a chain of three reads (lengths, path, page)
// before a token's: one tree of 16 columns 4.1 us on an MI355X, 64 trees of 64 and 8
// kv heads 4.2.
template <int NB>
__global__ __launch_bounds__(kThreads) void k_kv_commit(CommitArgs a) {
  typedef uint16_t half_t;
  constexpr int kMoves = kThreads / 16;
  const int r = threadIdx.x & 15, m = threadIdx.x >> 4;
  const int hd = blockIdx.x, b = blockIdx.y;
  const int s0 = a.v.starts[b], n = a.v.starts[b + 1] - s0;
  const int first = kv_len(a.v, b) - n;
  const int count = min(min(a.counts[b], a.path_cols), n);
  const KvGeo &g = a.v.g;
  const size_t at = ((size_t)b * a.v.hk + hd) * kv_capacity(a.v);
  const int plane = r == 0 ? g.ks : g.vs;
  for (int i0 = 0; i0 < count; i0 += kMoves) {
    const int i = i0 + m;
    int j = i < count ? a.path[(size_t)b * a.path_cols + i] : -1;
    if (j <= i || j >= n || first + i < 0) j = -1;  // (one that stays needs no move)
    const int src = first + j, dst = first + i;
    const int ts = src & (g.page_tokens - 1), td = dst & (g.page_tokens - 1);
    const uint8_t *from = nullptr;
    uint8_t *to = nullptr;
    half_t k[NB / 2], v[NB / 2], e[NB / 2];
    float weight = 0.f;
    int32_t position = 0;
    if (j >= 0) {
      from = kv_slab(a.v, b, src, hd);
      to = kv_slab(a.v, b, dst, hd);
      if (r == 2 && a.acc) weight = a.acc[at + src];
      if (r == 3 && a.pos) position = a.pos[at + src];
    }
    const bool moves = from && to;
    if (moves) {
#pragma unroll
      for (int x = 0; x < NB / 2; ++x) {
        k[x] = reinterpret_cast<const half_t *>(from + g.kc + ts * (16 * NB) + r * NB)[x];
        v[x] = *reinterpret_cast<const half_t *>(from + g.vc + v_byte(NB, ts, 2 * x, r));
        if (r < 2) e[x] = reinterpret_cast<const half_t *>(from + plane + ts * NB)[x];
      }
    }
    __syncthreads();
    if (moves) {
#pragma unroll
      for (int x = 0; x < NB / 2; ++x) {
        reinterpret_cast<half_t *>(to + g.kc + td * (16 * NB) + r * NB)[x] = k[x];
        *reinterpret_cast<half_t *>(to + g.vc + v_byte(NB, td, 2 * x, r)) = v[x];
        if (r < 2) reinterpret_cast<half_t *>(to + plane + td * NB)[x] = e[x];
      }
    }
    if (j >= 0) {
      if (r == 2 && a.acc) a.acc[at + dst] = weight;
      if (r == 3 && a.pos) a.pos[at + dst] = position;
    }
  }
}

// A batch as the calls without a cache take it, and their rows.
rfpx_status check_tree(const char *fn, const rfpx_kv_batch *b, int n_rows) {
  if (!b) return fail(RFPX_E_ARG, "%s: batch is null", fn);
  if (b->n_seqs < 1 || b->n_seqs > RFPX_SEQS_MAX)
    return fail(RFPX_E_SHAPE, "%s: n_seqs=%d: must be in [1, %d]", fn, b->n_seqs, RFPX_SEQS_MAX);
  if (b->max_cols < 0 || b->max_cols > kColsMax)
    return fail(RFPX_E_SHAPE, "%s: max_cols=%d: a tree has at most %d columns", fn, b->max_cols,
                kColsMax);
  if (n_rows < 0 || n_rows > RFPX_ROWS_MAX)
    return fail(RFPX_E_SHAPE, "%s: n_rows=%d: must be in [0, %d]", fn, n_rows, RFPX_ROWS_MAX);
  if (!b->lens || !b->starts) return fail(RFPX_E_ARG, "%s: lens or starts is null", fn);
  if ((uintptr_t)b->lens % 4 || (uintptr_t)b->starts % 4)
    return fail(RFPX_E_ALIGN, "%s: lens or starts not 4-byte aligned", fn);
  return RFPX_OK;
}

}  // namespace
}  // namespace rfpx

using namespace rfpx;

extern "C" {

rfpx_status rfpx_tree_masks(const rfpx_kv_batch *b, int n_rows, const int32_t *parents,
                            const int32_t *base, int mask_words, uint32_t *masks,
                            int32_t *positions, void *stream) {
  const char *fn = "rfpx_tree_masks";
  const rfpx_status st = check_tree(fn, b, n_rows);
  if (st) return st;
  if (mask_words < 1 || mask_words > kColsMax / 32)
    return fail(RFPX_E_SHAPE, "%s: mask_words=%d: must be in [1, %d]", fn, mask_words,
                kColsMax / 32);
  if (n_rows == 0) return RFPX_OK;
  if (!parents || !masks) return fail(RFPX_E_ARG, "%s: parents or masks is null", fn);
  if ((uintptr_t)parents % 4 || (uintptr_t)base % 4 || (uintptr_t)masks % 4 ||
      (uintptr_t)positions % 4)
    return fail(RFPX_E_ALIGN, "%s: parents, base, masks and positions must be 4-byte aligned", fn);
  MaskArgs a{};
  a.parents = parents;
  a.base = base;
  a.lens = b->lens;
  a.starts = b->starts;
  a.masks = masks;
  a.positions = positions;
  a.n_rows = n_rows;
  a.words = mask_words;
  const hipError_t e =
      launch_k(k_tree_masks, dim3(b->n_seqs), dim3(kThreads), 0, (hipStream_t)stream, a);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

rfpx_status rfpx_tree_accept(const rfpx_kv_batch *b, int n_rows, const int32_t *parents,
                             const int32_t *tokens, const int32_t *drawn, int path_cols,
                             int32_t *path, int32_t *counts, int32_t *next, int32_t *lens_out,
                             void *stream) {
  const char *fn = "rfpx_tree_accept";
  const rfpx_status st = check_tree(fn, b, n_rows);
  if (st) return st;
  if (path_cols < 1 || path_cols > kColsMax)
    return fail(RFPX_E_SHAPE, "%s: path_cols=%d: must be in [1, %d]", fn, path_cols, kColsMax);
  if (n_rows && (!parents || !tokens || !drawn))
    return fail(RFPX_E_ARG, "%s: parents, tokens or drawn is null", fn);
  if (!path || !counts || !next) return fail(RFPX_E_ARG, "%s: path, counts or next is null", fn);
  if ((uintptr_t)parents % 4 || (uintptr_t)tokens % 4 || (uintptr_t)drawn % 4 ||
      (uintptr_t)path % 4 || (uintptr_t)counts % 4 || (uintptr_t)next % 4 ||
      (uintptr_t)lens_out % 4)
    return fail(RFPX_E_ALIGN, "%s: all arrays must be 4-byte aligned", fn);
  AcceptArgs a{};
  a.parents = parents;
  a.tokens = tokens;
  a.drawn = drawn;
  a.lens = b->lens;
  a.starts = b->starts;
  a.path = path;
  a.counts = counts;
  a.next = next;
  a.lens_out = lens_out;
  a.n_rows = n_rows;
  a.path_cols = path_cols;
  const hipError_t e =
      launch_k(k_tree_accept, dim3(b->n_seqs), dim3(kThreads), 0, (hipStream_t)stream, a);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

rfpx_status rfpx_kv_commit(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int path_cols,
                           const int32_t *path, const int32_t *counts, float *acc, int32_t *pos,
                           void *stream) {
  const char *fn = "rfpx_kv_commit";
  const rfpx_status st = check_kv(fn, c, b, true);
  if (st) return st;
  if (path_cols < 1 || path_cols > kColsMax)
    return fail(RFPX_E_SHAPE, "%s: path_cols=%d: must be in [1, %d]", fn, path_cols, kColsMax);
  if (!path || !counts) return fail(RFPX_E_ARG, "%s: path or counts is null", fn);
  if ((uintptr_t)path % 4 || (uintptr_t)counts % 4 || (uintptr_t)acc % 4 || (uintptr_t)pos % 4)
    return fail(RFPX_E_ALIGN, "%s: path, counts, acc and pos must be 4-byte aligned", fn);
  CommitArgs a{};
  a.v = kv_view(c, b);
  a.path = path;
  a.counts = counts;
  a.acc = acc;
  a.pos = pos;
  a.path_cols = path_cols;
  void (*k)(CommitArgs) = c->head_dim == 64    ? k_kv_commit<2>
                          : c->head_dim == 128 ? k_kv_commit<4>
                                               : k_kv_commit<8>;
  const hipError_t e =
      launch_k(k, dim3(c->n_kv_heads, b->n_seqs), dim3(kThreads), 0, (hipStream_t)stream, a);
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

}  // extern "C"
