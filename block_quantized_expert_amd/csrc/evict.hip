// evict.hip -- eviction from the FP4 cache by accumulated attention weight.
//
// A sequence of n slots is cut to the `keep` best ones of each kv head.  The
// order of slots carries no meaning, so only the kept slots behind the cut
// move, into the slots before it that go: as many of one as of the other, and
// no slot is both read and written, so that all moves run at once, in place.
//
// Two launches.  k_evict_select, a workgroup for each (sequence, kv head):
// every slot's worth becomes one whole number (32 bits, larger is better; in
// registers up to 32768 slots), a radix selection finds the number of the
// keep-th best (eight bits a pass, a histogram in LDS), and one ordered pass
// over the slots lists the slots that go and the slots that move.
// k_evict_move: sixteen lanes a move.
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

__device__ __forceinline__ uint32_t worth_of(float acc, int pos, int edge, bool all_safe) {
  const uint32_t u = __float_as_uint(acc + 0.0f);  // -0 counts as 0
  const uint32_t w = acc != acc ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
  return pos > edge || all_safe ? 0xFFFFFFFFu : w;
}

// Copies of the histogram, by lane: numbers of one sequence share their upper
// bits, and additions to one address wait for each other.
constexpr int kHist = 4;

// Lanes before this one in a mask.
__device__ __forceinline__ int rank_in(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Wave w of the workgroup takes a run of slots (a multiple of 64, the same for
// every wave), 64 at a time; its numbers lie in registers (KPT > 0: at most
// 64 KPT of them) or in the workspace (KPT = 0), where a lane reads back what
// it wrote itself.  Slots behind the sequence count as numbers 0: level with
// the least at most, and behind it in order, so that they are never among the
// keep best of more than keep slots.  What bounds the kernel is the number of
// instructions of its one workgroup, and the fetching of them: 64 heads of
// 4224 slots 13.3 us, 8 heads of 32768 slots 35 us (loads a quarter, the four
// radix passes a quarter, counting and listing the rest).  Numbers in LDS with
// rolled loops measured 62 us, ballots instead of counts per lane 42 us.
template <int KPT>
__global__ __launch_bounds__(kSelThreads) void k_evict_select(EvictArgs a) {
  __shared__ __align__(16) int hist[256 * kHist];
  __shared__ __align__(16) int sh[kSelWaves][4];
  __shared__ int pick[2];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int hd = blockIdx.x, seq = blockIdx.y;
  const size_t cap = kv_capacity(a.v);
  const size_t bh = (size_t)seq * a.v.hk + hd;
  const float *acc = a.acc + bh * cap;
  const int32_t *pos = a.pos + bh * cap;
  uint32_t *worth = a.worth + bh * cap;
  const int len = uniform(kv_len(a.v, seq)), keep = a.keep;
  const int stay = min(len, keep);
  const bool copy_acc = a.acc != a.acc_out, copy_pos = a.pos != a.pos_out;
  const int groups = ((len + kSelWaves - 1) / kSelWaves + 63) / 64;  // of a wave's run
  const int j_first = wave * groups * 64;
  uint32_t w[KPT ? KPT : 1];
  // f(first slot, place in w) for every group of the wave's run
  const auto each = [&](auto &&f) {
    if constexpr (KPT > 0) {
#pragma unroll
      for (int i = 0; i < KPT; ++i)
        if (i < groups) f(j_first + 64 * i, i);
    } else {
      for (int i = 0; i < groups; ++i) f(j_first + 64 * i, 0);
    }
  };
  const auto number = [&](int j0, int i) -> uint32_t {
    if constexpr (KPT > 0) return w[i];
    else return j0 + lane < len ? worth[j0 + lane] : 0u;
  };
  int newest = INT32_MIN;
  float x[KPT ? KPT : 1];
  int p[KPT ? KPT : 1];
  if constexpr (KPT > 0) {
    // all loads in flight at once
    each([&](int j0, int i) {
      const int at = min(j0 + lane, len - 1);
      x[i] = acc[at];
      p[i] = pos[at];
    });
    each([&](int j0, int i) {
      newest = max(newest, p[i]);
      if (j0 < stay) {
        if (copy_acc && j0 + lane < stay) a.acc_out[bh * cap + j0 + lane] = x[i];
        if (copy_pos && j0 + lane < stay) a.pos_out[bh * cap + j0 + lane] = p[i];
      }
    });
  } else {
    each([&](int j0, int) {
      const int j = j0 + lane;
      if (j < len) newest = max(newest, pos[j]);
      if (copy_acc && j < stay) a.acc_out[bh * cap + j] = acc[j];
      if (copy_pos && j < stay) a.pos_out[bh * cap + j] = pos[j];
    });
  }
  if (len <= keep) {
    if (threadIdx.x == 0) {
      a.head[2 * bh] = 0;
      a.head[2 * bh + 1] = len;
    }
    return;
  }
#pragma unroll
  for (int off = 32; off; off >>= 1) newest = max(newest, __shfl_xor(newest, off));
  if (lane == 0) sh[wave][0] = newest;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kSelWaves; ++v) newest = max(newest, sh[v][0]);
  const long long wide = (long long)newest - a.recent;
  const int edge = wide < INT32_MIN ? INT32_MIN : (int)wide;
  const bool all_safe = wide < INT32_MIN;  // then INT32_MIN itself is above the edge
  each([&](int j0, int i) {
    const int j = j0 + lane;
    if constexpr (KPT > 0) w[i] = j < len ? worth_of(x[i], p[i], edge, all_safe) : 0u;
    else if (j < len) worth[j] = worth_of(acc[j], pos[j], edge, all_safe);
  });

  // the keep-th largest number: `want` counts down to its rank among the
  // numbers that share the bits found so far
  uint32_t found = 0;
  int want = keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256 * kHist; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    each([&](int j0, int i) {
      const uint32_t v = number(j0, i);
      if ((v & above) == found)
        atomicAdd(&hist[(v >> shift & 255u) * kHist + (lane & (kHist - 1))], 1);
    });
    __syncthreads();
    if (wave == 0) {
      // bins from the top: lane l holds bins 255 - 4l .. 252 - 4l
      int c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int4 v = *reinterpret_cast<const int4 *>(&hist[(255 - 4 * lane - i) * kHist]);
        sum += c[i] = v.x + v.y + v.z + v.w;
      }
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
    found |= (uint32_t)uniform(pick[0]) << shift;
    want = uniform(pick[1]);
  }

  // Slots worth more than `found` stay, and of those worth as much the first
  // `want`.  Counts of both before the cut (0) and behind it (1):
  int more0 = 0, more1 = 0, level0 = 0, level1 = 0;
  each([&](int j0, int i) {
    const uint32_t v = number(j0, i);
    if (j0 + 64 <= keep) {
      more0 += v > found;
      level0 += v == found;
    } else if (j0 >= keep) {
      more1 += v > found;
      level1 += v == found;
    } else {
      const bool first = j0 + lane < keep;
      more0 += first && v > found;
      level0 += first && v == found;
      more1 += !first && v > found;
      level1 += !first && v == found;
    }
  });
  if constexpr (KPT > 0) {  // a wave has at most 64 KPT of each: two to a word
    int m = more0 | more1 << 16, l = level0 | level1 << 16;
#pragma unroll
    for (int off = 32; off; off >>= 1) {
      m += __shfl_xor(m, off);
      l += __shfl_xor(l, off);
    }
    more0 = m & 0xFFFF;
    more1 = m >> 16;
    level0 = l & 0xFFFF;
    level1 = l >> 16;
  } else {
#pragma unroll
    for (int off = 32; off; off >>= 1) {
      more0 += __shfl_xor(more0, off);
      more1 += __shfl_xor(more1, off);
      level0 += __shfl_xor(level0, off);
      level1 += __shfl_xor(level1, off);
    }
  }
  if (lane == 0) *reinterpret_cast<int4 *>(sh[wave]) = make_int4(more0, more1, level0, level1);
  __syncthreads();
  int eq = 0, at_hole = 0, at_late = 0, n_late = 0, eq_all = 0;
#pragma unroll
  for (int v = 0; v < kSelWaves; ++v) {
    if (v == wave) {
      eq = eq_all;
      at_late = n_late;
    }
    const int4 c = *reinterpret_cast<const int4 *>(sh[v]);
    const int take0 = min(max(want - eq_all, 0), c.z);
    const int take1 = min(max(want - eq_all - c.z, 0), c.w);
    if (v < wave) at_hole += min(max(keep - v * groups * 64, 0), groups * 64) - c.x - take0;
    n_late += c.y + take1;
    eq_all += c.z + c.w;
  }
  eq = uniform(eq);
  at_hole = uniform(at_hole);
  at_late = uniform(at_late);
  int32_t *holes = a.holes + bh * a.list, *late = a.late + bh * a.list;
  each([&](int j0, int i) {
    const uint32_t v = number(j0, i);
    bool stays = v > found;
    const uint64_t ties = __ballot(v == found);
    if (ties) {
      stays = stays || (v == found && eq + rank_in(ties) < want);
      eq += __popcll(ties);
    }
    const bool first = j0 + lane < keep;
    const bool goes = first && !stays, moves = !first && stays;
    if (j0 < keep) {
      const uint64_t go = __ballot(goes);
      const int at = at_hole + rank_in(go);
      if (goes && at < a.list) holes[at] = j0 + lane;
      at_hole += __popcll(go);
    }
    if (j0 + 64 > keep) {
      const uint64_t mv = __ballot(moves);
      const int at = at_late + rank_in(mv);
      if (moves && at < a.list) late[at] = j0 + lane;
      at_late += __popcll(mv);
    }
  });
  if (threadIdx.x == 0) {
    a.head[2 * bh] = min(n_late, a.list);
    a.head[2 * bh + 1] = len;
  }
}

// Sixteen lanes a move (8 heads cut from 32768 to 8192 slots, some 6100 moves
// each: 11.3 us; a wave a move 27 us): lane r moves NB bytes of the key's
// codes and byte r of every block of the value's, two and two as they lie,
// the first four also the scales, the weight and the position.
template <int NB>
__global__ __launch_bounds__(kMoveThreads) void k_evict_move(EvictArgs a) {
  typedef uint16_t half_t;
  const int r = threadIdx.x & 15;
  const int hd = blockIdx.y, seq = blockIdx.z;
  const size_t bh = (size_t)seq * a.v.hk + hd;
  const KvGeo &g = a.v.g;
  const int moves = a.head[2 * bh];
  if (blockIdx.x == 0 && hd == 0 && threadIdx.x == 0)
    a.lens_out[seq] = min(a.head[2 * bh + 1], a.keep);
  const size_t cap = kv_capacity(a.v);
  for (int i = blockIdx.x * (kMoveThreads / 16) + (threadIdx.x >> 4); i < moves;
       i += gridDim.x * (kMoveThreads / 16)) {
    const int dst = a.holes[bh * a.list + i], src = a.late[bh * a.list + i];
    const uint8_t *from = kv_slab(a.v, seq, src, hd);
    uint8_t *to = kv_slab(a.v, seq, dst, hd);
    // (also where a page is outside the pool, whose bytes cannot move: only a
    // sequence that the caller must not hand in has such slots)
    if (r == 2) a.acc_out[bh * cap + dst] = a.acc[bh * cap + src];
    if (r == 3) a.pos_out[bh * cap + dst] = a.pos[bh * cap + src];
    if (!from || !to) continue;
    const int ts = src & (g.page_tokens - 1), td = dst & (g.page_tokens - 1);
    half_t k[NB / 2], v[NB / 2], e[NB / 2];
    const int plane = r == 0 ? g.ks : g.vs;
#pragma unroll
    for (int j = 0; j < NB / 2; ++j) {
      k[j] = reinterpret_cast<const half_t *>(from + g.kc + ts * (16 * NB) + r * NB)[j];
      v[j] = *reinterpret_cast<const half_t *>(from + g.vc + v_byte(NB, ts, 2 * j, r));
      if (r < 2) e[j] = reinterpret_cast<const half_t *>(from + plane + ts * NB)[j];
    }
#pragma unroll
    for (int j = 0; j < NB / 2; ++j) {
      reinterpret_cast<half_t *>(to + g.kc + td * (16 * NB) + r * NB)[j] = k[j];
      *reinterpret_cast<half_t *>(to + g.vc + v_byte(NB, td, 2 * j, r)) = v[j];
      if (r < 2) reinterpret_cast<half_t *>(to + plane + td * NB)[j] = e[j];
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
  // numbers in registers where the table's slots allow it
  const long long cap = (long long)b->pages_per_seq * c->page_tokens;
  void (*select)(EvictArgs) = cap <= 8 * kSelThreads    ? k_evict_select<8>
                              : cap <= 32 * kSelThreads ? k_evict_select<32>
                                                        : k_evict_select<0>;
  hipError_t e = launch_k(select, dim3(c->n_kv_heads, b->n_seqs), dim3(kSelThreads), 0, s, a);
  if (e == hipSuccess) {
    // sixteen moves a workgroup, at most sixteen workgroups a compute unit
    const long long bh = (long long)b->n_seqs * c->n_kv_heads;
    long long gx = (p.list + 15) / 16, most = (4096 + bh - 1) / bh;
    if (gx > most) gx = most;
    void (*move)(EvictArgs) = c->head_dim == 64    ? k_evict_move<2>
                              : c->head_dim == 128 ? k_evict_move<4>
                                                   : k_evict_move<8>;
    e = launch_k(move, dim3((unsigned)gx, c->n_kv_heads, b->n_seqs), dim3(kMoveThreads), 0, s, a);
  }
  return e == hipSuccess ? RFPX_OK : fail(RFPX_E_HIP, "%s: %s", fn, hipGetErrorString(e));
}

}  // extern "C"
