// evict.hip -- eviction from the FP4 cache by accumulated attention weight.
//
// A sequence of n slots is cut to the `keep` best ones of each kv head.  The
// order of slots carries no meaning, so only the kept slots behind the cut
// move, into the slots before it that go: as many of one as of the other, and
// no slot is both read and written, so that all moves run at once, in place.
//
// Two launches.  k_evict_select, a workgroup for each (sequence, kv head):
// every slot's worth becomes one whole number (32 bits, larger is better;
// in registers up to 32768 slots), a radix selection finds the number of the keep-th best (eight bits a pass,
// a histogram in LDS), and one ordered pass over the slots lists the slots
// that go and the slots that move.  k_evict_move: sixteen lanes a move.
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

// Copies of the histogram, by lane: numbers of one sequence share their upper
// bits, and additions to one address wait for each other.
constexpr int kHist = 4;

// One workgroup's slots: KPT to a thread in registers (KPT > 0), wave w
// holding a run of 64 KPT of them, slot i * 64 + lane of the run as number i;
// or (KPT = 0) as numbers in the workspace, runs of any length.
template <int KPT>
__global__ __launch_bounds__(kSelThreads) void k_evict_select(EvictArgs a) {
  __shared__ int hist[256 * kHist];
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
  const bool copy_acc = a.acc != a.acc_out, copy_pos = a.pos != a.pos_out;
  const int run = KPT ? 64 * KPT : ((len + kSelWaves - 1) / kSelWaves + 63) / 64 * 64;
  const int j_first = min(len, wave * run), j_last = min(len, j_first + run);
  uint32_t w[KPT ? KPT : 1];
  // f(slot of this lane, its place in w) for every group of the wave's run;
  // slots at or behind j_last are the lanes' own to leave out
  const auto each = [&](auto &&f) {
    if constexpr (KPT > 0) {
#pragma unroll
      for (int i = 0; i < KPT; ++i)
        if (j_first + 64 * i < j_last) f(j_first + 64 * i + lane, i);
    } else {
      for (int j0 = j_first; j0 < j_last; j0 += 64) f(j0 + lane, 0);
    }
  };
  const auto number = [&](int j, int i) {
    if constexpr (KPT > 0) return w[i];
    else return j < j_last ? worth[j] : 0u;
  };
  if (len <= keep) {
    each([&](int j, int) {
      if (j < stay && copy_acc) a.acc_out[bh * cap + j] = acc[j];
      if (j < stay && copy_pos) a.pos_out[bh * cap + j] = pos[j];
    });
    if (threadIdx.x == 0) {
      a.head[2 * bh] = 0;
      a.head[2 * bh + 1] = len;
    }
    return;
  }
  int newest = INT32_MIN;
  if constexpr (KPT > 0) {
    // all loads in flight at once
    float x[KPT];
    int p[KPT];
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const int j = min(j_first + 64 * i + lane, len - 1);
      x[i] = acc[j];
      p[i] = pos[j];
    }
#pragma unroll
    for (int i = 0; i < KPT; ++i) newest = max(newest, p[i]);
    each([&](int j, int i) {
      if (j < stay && copy_acc) a.acc_out[bh * cap + j] = x[i];
      if (j < stay && copy_pos) a.pos_out[bh * cap + j] = p[i];
    });
#pragma unroll
    for (int off = 32; off; off >>= 1) newest = max(newest, __shfl_xor(newest, off));
    if (lane == 0) sh[wave] = newest;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kSelWaves; ++v) newest = max(newest, sh[v]);
    const long long edge = (long long)newest - a.recent;
#pragma unroll
    for (int i = 0; i < KPT; ++i) w[i] = worth_of(x[i], p[i], edge);
  } else {
    each([&](int j, int) {
      if (j >= j_last) return;
      newest = max(newest, pos[j]);
      if (j < stay && copy_acc) a.acc_out[bh * cap + j] = acc[j];
      if (j < stay && copy_pos) a.pos_out[bh * cap + j] = pos[j];
    });
#pragma unroll
    for (int off = 32; off; off >>= 1) newest = max(newest, __shfl_xor(newest, off));
    if (lane == 0) sh[wave] = newest;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kSelWaves; ++v) newest = max(newest, sh[v]);
    const long long edge = (long long)newest - a.recent;
    // (a lane reads back later what it wrote itself)
    each([&](int j, int) {
      if (j < j_last) worth[j] = worth_of(acc[j], pos[j], edge);
    });
  }

  // the keep-th largest number: `want` counts down to its rank among the
  // numbers that share the bits found so far
  uint32_t found = 0;
  int want = keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256 * kHist; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    each([&](int j, int i) {
      const uint32_t v = number(j, i);
      if (j < j_last && (v & above) == found)
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
    found |= (uint32_t)pick[0] << shift;
    want = pick[1];
  }

  // slots worth more than `found` stay, and of those worth as much the first
  // `want`
  int equal = 0;
  each([&](int j, int i) { equal += __popcll(__ballot(j < j_last && number(j, i) == found)); });
  int total;
  const int equal_before = wave_offset(equal, sh, wave, lane, &total);
  const uint64_t below = (1ull << lane) - 1;
  int n_hole = 0, n_late = 0, at_hole = 0, at_late = 0;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    int eq = equal_before, holes = 0, late = 0;
    each([&](int j, int i) {
      const uint32_t v = number(j, i);
      const uint64_t ties = __ballot(j < j_last && v == found);
      const bool stays = v > found || (v == found && eq + __popcll(ties & below) < want);
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
    });
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

// Sixteen lanes a move: lane r moves NB bytes of the key's codes and byte r of
// every block of the value's, two and two as they lie, the first four also
// the scales, the weight and the position.
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
