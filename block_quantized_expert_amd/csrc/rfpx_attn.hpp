// rfpx_attn.hpp -- what the attention sources share: the cache's layout, the
// step's batch as kernels read it, and the host checks.
//
// The 16x16x32 bf16 matrix instruction takes from lane (n = lane & 15,
// g = lane >> 4) eight k-values of its row n, and both operands may order
// their k-values alike in any way.  The layout of a slab follows from that:
//   keys    lane (n, g) of a 16-token tile reads token n's octet g of every
//           block: D/32 dwords side by side, one load;
//   values  lane (r, g) reads, for tokens 4g .. 4g+3 of a 16-token tile, byte
//           r of every block (values 32 b + 2 r and + 1): D/32 dwords, whose
//           halves belong to two neighbouring tokens, so that a mask and a
//           shift give the bf16 pairs that a sum over tokens takes.
#pragma once

#include "../../include/rfpx_attn.h"
#include "rfpx_impl.hpp"

namespace rfpx {

struct KvGeo {
  int page_tokens, page_log, head_dim, nb;
  int kc, ks, vc, vs;   // byte offsets of the four planes in a slab
  int slab;             // bytes
};

__host__ __device__ __forceinline__ KvGeo kv_geo(int head_dim, int page_tokens) {
  KvGeo g;
  g.page_tokens = page_tokens;
  g.page_log = page_tokens == 32 ? 5 : page_tokens == 64 ? 6 : page_tokens == 128 ? 7 : 8;
  g.head_dim = head_dim;
  g.nb = head_dim / 32;
  g.kc = 0;
  g.ks = page_tokens * (head_dim / 2);
  g.vc = g.ks + page_tokens * g.nb;
  g.vs = g.vc + page_tokens * (head_dim / 2);
  g.slab = g.vs + page_tokens * g.nb;
  return g;
}

// Byte of V: byte r of block b of page token t, from the start of the plane.
__device__ __forceinline__ int v_byte(int nb, int t, int b, int r) {
  return ((t >> 2) * 16 + r) * 4 * nb + (((t >> 1) & 1) * (nb >> 1) + (b >> 1)) * 4 + (t & 1) * 2 +
         (b & 1);
}

// The step as kernels see it.
struct KvView {
  uint8_t *pool;
  const int32_t *table, *lens, *starts;
  int n_seqs, pages_per_seq, n_pages, hk;
  KvGeo g;
};

#if defined(__HIPCC__)

// A uniform read of device data that no kernel of the call writes: a scalar
// load, which waits for no vector load in flight.
__device__ __forceinline__ int scalar_read(const int32_t *p) {
  return *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)p;
}
__device__ __forceinline__ int kv_capacity(const KvView &v) {
  const long long cap = (long long)v.pages_per_seq * v.g.page_tokens;
  return cap < 0x7FFFFFFF ? (int)cap : 0x7FFFFFFF;
}
__device__ __forceinline__ int kv_len(const KvView &v, int b) {
  const int len = v.lens[b], cap = kv_capacity(v);
  return len < 0 ? 0 : len < cap ? len : cap;
}
// The slab of (slot, head); null where the slot has no page in the pool.
__device__ __forceinline__ uint8_t *kv_slab(const KvView &v, int b, int slot, int head) {
  const int page = v.table[(size_t)b * v.pages_per_seq + (slot >> v.g.page_log)];
  if ((unsigned)page >= (unsigned)v.n_pages) return nullptr;
  return v.pool + ((size_t)page * v.hk + head) * v.g.slab;
}

// The sequence of a row: the last b with starts[b] <= row, by 64-way search
// (one load a level for the whole wave; row is the same in every lane).  -1
// where there is none or the row lies behind the last sequence.
__device__ __forceinline__ int kv_seq_of(const KvView &v, int row, int lane) {
  if (row < v.starts[0] || row >= v.starts[v.n_seqs]) return -1;
  int lo = 0, n = v.n_seqs;
  while (n > 1) {
    const int stride = (n + 63) / 64;
    const int i = lane * stride;
    const bool le = i < n && v.starts[lo + i] <= row;
    const int cnt = __popcll(__ballot(le));
    if (cnt == 0) return -1;
    lo += (cnt - 1) * stride;
    n = n - (cnt - 1) * stride < stride ? n - (cnt - 1) * stride : stride;
  }
  return uniform(lo);
}

// Where a row's token lies: its sequence and slot (< 0: nowhere).
__device__ __forceinline__ int kv_slot_of(const KvView &v, int row, int lane, int *seq) {
  const int b = kv_seq_of(v, row, lane);
  *seq = b;
  if (b < 0) return -1;
  const int s0 = v.starts[b], n = v.starts[b + 1] - s0;
  const int len = kv_len(v, b), slot = len - n + (row - s0);
  return slot < len ? slot : -1;
}

#endif

// ---------------------------------------------------------------- host side

inline KvView kv_view(const rfpx_kv_cache *c, const rfpx_kv_batch *b) {
  KvView v;
  v.pool = c->pool;
  v.table = b->page_table;
  v.lens = b->lens;
  v.starts = b->starts;
  v.n_seqs = b->n_seqs;
  v.pages_per_seq = b->pages_per_seq;
  v.n_pages = c->n_pages;
  v.hk = c->n_kv_heads;
  v.g = kv_geo(c->head_dim, c->page_tokens);
  return v;
}

rfpx_status check_kv(const char *fn, const rfpx_kv_cache *c, const rfpx_kv_batch *b,
                     bool pointers);
// Rows of `heads` heads at p, `stride` elements apart.
rfpx_status check_rows(const char *fn, const char *what, const void *p, long long stride, int heads,
                       int head_dim, int xtype);
inline int xtype_size(int xtype) { return xtype == RFPX_X_BF16 ? 2 : 4; }
inline bool valid_xtype(int xtype) { return xtype == RFPX_X_F32 || xtype == RFPX_X_BF16; }

}  // namespace rfpx
