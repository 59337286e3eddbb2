// evict.hip -- eviction from the FP4 cache by accumulated attention weight.
//
// A sequence of n slots is cut to the `keep` best ones of each kv head.  The
// order of slots carries no meaning, so only the kept slots behind the cut
// move, into the slots before it that go: as many of one as of the other, and
// no slot is both read and written, so that all moves run at once, in place.
//
// Two launches.  k_evict_select, a workgroup for each (sequence, kv head):
// every slot's worth becomes one whole number (32 bits, larger is better), a
// radix selection finds the number of the keep-th best (eight bits a pass,
// a histogram in LDS), and one ordered pass over the slots lists the slots
// that go and the slots that move.  k_evict_move: a wave a move.
#include "rfpx_attn.hpp"

namespace rfpx {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kMoveThreads = 256;

struct EvictArgs {
  KvView v;
  const float *acc;
  const int32_t *pos;
  float *acc_out;
  int32_t *pos_out, *lens_out;
  int32_t *head;   // [seqs][hk][2]: moves, length before
  int32_t *holes;  // [seqs][hk][list]
  int32_t *late;   // [seqs][hk][list]
  uint32_t *worth; // [seqs][hk][capacity]
  int keep, recent, list;
};

__device__ __forceinline__ uint32_t worth_of(float acc, int pos, long long edge) {
  if (pos > edge) return 0xFFFFFFFFu;
  if (acc != acc) return 0u;
  const uint32_t u = __float_as_uint(acc + 0.0f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum over the waves before this one, and over all, of a wave's count.
__device__ __forceinline__ int wave_offset(int mine, int *sh, int wave, int lane, int *total) {
  __syncthreads();
  if (lane == 0) sh[wave] = mine;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelWaves; ++w) {
    before += w < wave ? sh[w] : 0;
    all += sh[w];
  }
  *total = all;
  return before;
}

__global__ __launch_bounds__(kSelThreads) void k_evict_select(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int sh[kSelWaves];
  __shared__ int pick[2];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int hd = blockIdx.x, seq = blockIdx.y;
  const size_t cap = kv_capacity(a.v);
  const size_t bh = (size_t)seq * a.v.hk + hd;
  const float *acc = a.acc + bh * cap;
  const int32_t *pos = a.pos + bh * cap;
  uint32_t *worth = a.worth + bh * cap;
  const int len = kv_len(a.v, seq), keep = a.keep;
  const int stay = min(len, keep);
  if (acc != a.acc_out + bh * cap)
    for (int j = threadIdx.x; j < stay; j += kSelThreads) a.acc_out[bh * cap + j] = acc[j];
  if (pos != a.pos_out + bh * cap)
    for (int j = threadIdx.x; j < stay; j += kSelThreads) a.pos_out[bh * cap + j] = pos[j];
  if (len <= keep) {
    if (threadIdx.x == 0) {
      a.head[2 * bh] = 0;
      a.head[2 * bh + 1] = len;
    }
    return;
  }
  int newest = INT32_MIN;
  for (int j = threadIdx.x; j < len; j += kSelThreads) newest = max(newest, pos[j]);
#pragma unroll
  for (int off = 32; off; off >>= 1) newest = max(newest, __shfl_xor(newest, off));
  if (lane == 0) sh[wave] = newest;
  __syncthreads();
  newest = sh[0];
#pragma unroll
  for (int w = 1; w < kSelWaves; ++w) newest = max(newest, sh[w]);
  const long long edge = (long long)newest - a.recent;
  for (int j = threadIdx.x; j < len; j += kSelThreads) worth[j] = worth_of(acc[j], pos[j], edge);

  // the keep-th largest number: `want` counts down to its rank among the
  // numbers that share the bits found so far.  (A thread reads back what it
  // wrote itself: the same stride in every pass.)
  uint32_t found = 0;
  int want = keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int j0 = 0; j0 < len; j0 += kSelThreads) {
      const int j = j0 + threadIdx.x;
      const uint32_t w = j < len ? worth[j] : 0;
      const bool in = j < len && (w & above) == found;
      const int bin = (int)((w >> shift) & 255u);
      // numbers of one bin count as one addition where the wave agrees
      const uint64_t who = __ballot(in);
      if (who) {
        const int first = __shfl(bin, __ffsll((unsigned long long)who) - 1);
        const uint64_t same = __ballot(in && bin == first);
        if (lane == 0) atomicAdd(&hist[first], __popcll(same));
        if (in && bin != first) atomicAdd(&hist[bin], 1);
      }
    }
    __syncthreads();
    if (wave == 0) {
      // bins from the top: lane l holds bins 255 - 4l .. 252 - 4l
      int c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += c[i] = hist[255 - 4 * lane - i];
      int upto = sum;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(upto, off);
        if (lane >= off) upto += o;
      }
      int before = upto - sum;
      if (before < want && want <= upto) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (before < want && want <= before + c[i]) {
            pick[0] = 255 - 4 * lane - i;
            pick[1] = want - before;
          }
          before += c[i];
        }
      }
    }
    __syncthreads();
    found |= (uint32_t)pick[0] << shift;
    want = pick[1];
    __syncthreads();
  }

  // slots worth more than `found` stay, and of those worth as much the first
  // `want`.  Every wave takes a run of slots.
  __syncthreads();
  const int run = ((len + kSelWaves - 1) / kSelWaves + 63) / 64 * 64;
  const int j_first = min(len, wave * run), j_last = min(len, j_first + run);
  int equal = 0;
  for (int j0 = j_first; j0 < j_last; j0 += 64)
    equal += __popcll(__ballot(j0 + lane < j_last && worth[j0 + lane] == found));
  int total;
  const int equal_before = wave_offset(equal, sh, wave, lane, &total);
  const uint64_t below = (1ull << lane) - 1;
  int n_hole = 0, n_late = 0, at_hole = 0, at_late = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int eq = equal_before, holes = 0, late = 0;
    for (int j0 = j_first; j0 < j_last; j0 += 64) {
      const int j = j0 + lane;
      const uint32_t w = j < j_last ? worth[j] : 0;
      const uint64_t ties = __ballot(j < j_last && w == found);
      const bool stays = w > found || (w == found && eq + __popcll(ties & below) < want);
      const uint64_t h = __ballot(j < j_last && !stays && j < keep);
      const uint64_t l = __ballot(j < j_last && stays && j >= keep);
      if (pass) {
        const int hi = at_hole + holes + __popcll(h & below);
        const int li = at_late + late + __popcll(l & below);
        if ((h >> lane) & 1 && hi < a.list) a.holes[bh * a.list + hi] = j;
        if ((l >> lane) & 1 && li < a.list) a.late[bh * a.list + li] = j;
      }
      eq += __popcll(ties);
      holes += __popcll(h);
      late += __popcll(l);
    }
    if (!pass) {
      at_hole = wave_offset(holes, sh, wave, lane, &n_hole);
      at_late = wave_offset(late, sh, wave, lane, &n_late);
    }
  }
  if (threadIdx.x == 0) {
    a.head[2 * bh] = min(min(n_hole, n_late), a.list);
    a.head[2 * bh + 1] = len;
  }
}

__global__ __launch_bounds__(kMoveThreads) void k_evict_move(EvictArgs a) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int hd = blockIdx.y, seq = blockIdx.z;
  const size_t bh = (size_t)seq * a.v.hk + hd;
  const KvGeo &g = a.v.g;
  const int moves = a.head[2 * bh];
  if (blockIdx.x == 0 && hd == 0 && threadIdx.x == 0)
    a.lens_out[seq] = min(a.head[2 * bh + 1], a.keep);
  const size_t cap = kv_capacity(a.v);
  const int kd = g.head_dim / 8, vh = g.head_dim / 4;  // key dwords, value half-words
  const int items = kd + vh + 2 * g.nb + 2;
  for (int i = blockIdx.x * (kMoveThreads / 64) + wave; i < moves;
       i += gridDim.x * (kMoveThreads / 64)) {
    const int dst = uniform(a.holes[bh * a.list + i]), src = uniform(a.late[bh * a.list + i]);
    const uint8_t *from = kv_slab(a.v, seq, src, hd);
    uint8_t *to = kv_slab(a.v, seq, dst, hd);
    const int ts = src & (g.page_tokens - 1), td = dst & (g.page_tokens - 1);
    for (int it = lane; it < items; it += 64) {
      if (it >= items - 2) {
        if (it == items - 2) a.acc_out[bh * cap + dst] = a.acc[bh * cap + src];
        else a.pos_out[bh * cap + dst] = a.pos[bh * cap + src];
      } else if (!from || !to) {
      } else if (it < kd) {
        *reinterpret_cast<uint32_t *>(to + g.kc + td * (g.head_dim / 2) + 4 * it) =
            *reinterpret_cast<const uint32_t *>(from + g.kc + ts * (g.head_dim / 2) + 4 * it);
      } else if (it < kd + vh) {
        const int r = (it - kd) / (g.nb / 2), b = 2 * ((it - kd) % (g.nb / 2));
        *reinterpret_cast<uint16_t *>(to + g.vc + v_byte(g.nb, td, b, r)) =
            *reinterpret_cast<const uint16_t *>(from + g.vc + v_byte(g.nb, ts, b, r));
      } else {
        const int j = it - kd - vh;
        const int plane = j < g.nb ? g.ks : g.vs, b = j < g.nb ? j : j - g.nb;
        to[plane + td * g.nb + b] = from[plane + ts * g.nb + b];
      }
    }
  }
}

struct EvictPlan {
  size_t head, holes, late, worth, total;
  int list;
};

// A list holds at most the slots before the cut, and at most those behind it.
EvictPlan evict_plan(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int keep) {
  EvictPlan p;
  const long long cap = (long long)b->pages_per_seq * c->page_tokens;
  long long list = cap - keep < keep ? cap - keep : keep;
  if (list < 1) list = 1;
  p.list = (int)list;
  const size_t bh = (size_t)b->n_seqs * c->n_kv_heads;
  p.head = 0;
  p.holes = align_up(bh * 8, 256);
  p.late = p.holes + align_up(bh * list * 4, 256);
  p.worth = p.late + align_up(bh * list * 4, 256);
  p.total = p.worth + align_up(bh * cap * 4, 256);
  return p;
}

}  // namespace
}  // namespace rfpx

using namespace rfpx;

extern "C" {

size_t rfpx_kv_evict_workspace_bytes(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int keep) {
  if (check_kv("rfpx_kv_evict_workspace_bytes", c, b, false)) return 0;
  if (keep < 1) {
    fail(RFPX_E_SHAPE, "rfpx_kv_evict_workspace_bytes: keep=%d: must be 1 or more", keep);
    return 0;
  }
  return evict_plan(c, b, keep).total;
}

rfpx_status rfpx_kv_evict(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int keep, int recent,
                          const float *acc, const int32_t *pos, float *acc_out, int32_t *pos_out,
                          int32_t *lens_out, void *ws, size_t ws_bytes, void *stream) {
  const char *fn = "rfpx_kv_evict";
  rfpx_status st = check_kv(fn, c, b, true);
  if (st) return st;
  if (keep < 1 || recent < 0)
    return fail(RFPX_E_SHAPE, "%s: keep=%d (1 or more), recent=%d (0 or more)", fn, keep, recent);
  if (!acc || !pos || !acc_out || !pos_out || !lens_out)
    return fail(RFPX_E_ARG, "%s: acc, pos or an output is null", fn);
  if ((uintptr_t)acc % 4 || (uintptr_t)pos % 4 || (uintptr_t)acc_out % 4 ||
      (uintptr_t)pos_out % 4 || (uintptr_t)lens_out % 4)
    return fail(RFPX_E_ALIGN, "%s: acc, pos and the outputs must be 4-byte aligned", fn);
  if (!ws) return fail(RFPX_E_ARG, "%s: workspace is null", fn);
  if ((uintptr_t)ws % 256) return fail(RFPX_E_ALIGN, "%s: workspace not 256-byte aligned", fn);
  const EvictPlan p = evict_plan(c, b, keep);
  if (ws_bytes < p.total)
    return fail(RFPX_E_WORKSPACE, "%s: workspace holds %zu bytes, needs %zu", fn, ws_bytes, p.total);
  uint8_t *w = static_cast<uint8_t *>(ws);
  EvictArgs a{};
  a.v = kv_view(c, b);
  a.acc = acc;
  a.pos = pos;
  a.acc_out = acc_out;
  a.pos_out = pos_out;
  a.lens_out = lens_out;
  a.head = reinterpret_cast<int32_t *>(w + p.head);
  a.holes = reinterpret_cast<int32_t *>(w + p.holes);
  a.late = reinterpret_cast<int32_t *>(w + p.late);
  a.worth = reinterpret_cast<uint32_t *>(w + p.worth);
  a.keep = keep;
  a.recent = recent;
  a.list = p.list;
  hipStream_t s = (hipStream_t)stream;
  hipError_t e = launch_k(k_evict_select, dim3(c->n_kv_heads, b->n_seqs), dim3(kSelThreads), 0, s, a);
  if (e == hipSuccess) {
    // a wave a move, at most sixteen workgroups for each compute unit
    const long long bh = (long long)b->n_seqs * c->n_kv_heads;
    long long gx = (p.list + 3) / 4, most = (4096 + bh - 1) / bh;
    if (gx > most) gx = most;
    e = launch_k(k_evict_move, dim3((unsigned)gx, c->n_kv_heads, b->n_seqs), dim3(kMoveThreads), 0,
                 s, a);
  }
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

}  // extern "C"
