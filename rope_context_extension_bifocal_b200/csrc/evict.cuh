// Eviction: cut each sequence's cache to `budget` slots by the attention weight its keys received.
//
// Per (sequence, kv head) of n slots, kept = min(n, budget) slots are chosen in this order: those whose
// position is protected (below `sink`, or among the newest `recent` positions), then the largest
// weights (a NaN counts as -inf), ties to the lowest slot. In place, the kept slots below `kept` stay
// where they are and the i-th kept slot from `kept` on moves into the i-th hole below it: only rows
// that must move are moved, sources and holes never overlap, so every move is independent of the
// others (slots carry their positions, attention does not need them in order). To other pages, the
// i-th kept slot moves to slot i.
//
// evict_select_kernel finds the kept-th largest key with a radix select, 11 bits a pass, over keys that it forms
// once in shared memory, then lists the rows to move. A CTA takes a segment of up to 16384 slots: its passes are
// separated by block barriers alone (a cluster's barrier costs microseconds). Longer segments are spread over a
// cluster whose CTAs add up their histograms through distributed shared memory.
// evict_move_kernel copies the rows, eight a warp in flight.
// Bound by memory: 8 bytes a slot to select (weight and position), 2 (4 D + 8) bytes a row moved; with
// few segments by the latency of the passes instead. 64 segments of up to 32768 slots cut to 4096: select 40 us (two
// CTAs a segment; with clusters of eight small CTAs it took 143 us), move 49 us (250 MB: 5.1 TB/s of 6.55). 8 segments of
// 4099 slots cut to 2048: 18 us and 7 us.
#pragma once
#include <cooperative_groups.h>

#include "common.cuh"
#include "packed.cuh"

namespace bf {

namespace ev {
constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;          // of a pass: 11 bits of the key
constexpr int COPIES = 2;           // histograms a CTA fills side by side (fewer conflicts on one bin; four took the same time)
constexpr int CTA_SLOTS = 16384;    // slots a CTA takes while a cluster of 8 suffices
constexpr int MAX_RESIDENT = 40960; // keys a CTA holds in shared memory; longer ranges are read again each pass
}  // namespace ev

struct EvictArgs {
  __nv_bfloat16* kcache;   // [rows, hkv, D]
  __nv_bfloat16* vcache;
  int* kpos;               // [hkv, rows]
  float* kweight;          // [hkv, rows]
  CacheRows src, dst;      // dst: the block table of the pages moved to (in place: src)
  const int* seq_lens;     // [B]
  const int* positions;    // [B] position of the newest token
  int* new_lens;           // [B]; may be seq_lens
  int hkv, max_len, budget, recent, sink, in_place;
  int* moves;              // [B, hkv] rows to move
  int* lens;               // [B] what new_lens becomes
  int* from;               // [B, hkv, pitch] cache rows moved, in the order of their slots (-1: a bad page)
  int* to;                 // [B, hkv, pitch] cache rows they move to
  int pitch;
  int keys_in_smem;        // keys a CTA has room for
};

__global__ void __launch_bounds__(ev::THREADS, 1) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  using namespace ev;
  namespace cg = cooperative_groups;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t* s_key = reinterpret_cast<uint32_t*>(smem);
  __shared__ int hist[COPIES][BINS];   // copy 0 becomes this CTA's sum, read by the cluster
  __shared__ int wcount[2][WARPS];
  __shared__ int cta_count[2];         // this CTA's counts, read by the cluster
  __shared__ int s_digit, s_above, s_hits;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), size = static_cast<int>(cluster.num_blocks());
  auto sync_all = [&]() {
    if (size == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const long long seg = static_cast<long long>(b) * a.hkv + h;
  pdl_launch_dependents();
  pdl_wait();
  const int n = a.seq_lens[b];
  const bool ok = n >= 0 && n <= a.max_len;  // the same for every CTA of the cluster
  const int kept = ok ? min(n, a.budget) : 0;
  if (rank == 0 && tid == 0 && h == 0) a.lens[b] = ok ? kept : n;
  if (!ok || n == 0 || (a.in_place && n <= a.budget)) {
    if (rank == 0 && tid == 0) {
      a.moves[seg] = 0;
      if (!ok) report_status(kDevIndex, 80);
    }
    return;
  }
  // this CTA's slots, and within them this warp's (whole multiples of 32)
  const int per_warp = ((n + size * WARPS - 1) / (size * WARPS) + 31) / 32 * 32;
  const int beg = min(n, rank * WARPS * per_warp), end = min(n, beg + WARPS * per_warp);
  const int wbeg = min(end, beg + warp * per_warp), wend = min(end, wbeg + per_warp);
  const long long newest = a.positions[b];
  auto row_of = [&](const CacheRows& c, int slot) -> int {
    const int page = c.page_shift >= 0 ? slot >> c.page_shift : slot / c.page_size;
    const int pg = c.block_table[static_cast<long long>(b) * c.max_pages + page];
    return pg < 0 || pg >= c.pool_pages ? -1 : pg * c.page_size + (slot - page * c.page_size);
  };
  const int* kpos = a.kpos + static_cast<long long>(h) * a.src.rows;
  const float* kweight = a.kweight + static_cast<long long>(h) * a.src.rows;
  auto key_from = [&](int pos, float w) -> uint32_t {
    if (pos < a.sink || pos > newest - a.recent) return 0xffffffffu;
    if (w != w) return 0x007fffffu;  // -inf's
    const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  };
  auto key_of = [&](int slot) -> uint32_t {
    const int r = row_of(a.src, slot);
    if (r < 0) {
      report_status(kDevIndex, 81);
      return 0u;
    }
    return key_from(kpos[r], kweight[r]);
  };
  const bool resident = end - beg <= a.keys_in_smem;
  if (resident) {
    constexpr int U = 4;  // slots a thread looks up together
    for (int s0 = beg + tid; s0 < end; s0 += U * THREADS) {
      int r[U], pos[U];
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = s0 + u * THREADS < end ? row_of(a.src, s0 + u * THREADS) : -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        pos[u] = r[u] >= 0 ? kpos[r[u]] : 0;
        w[u] = r[u] >= 0 ? kweight[r[u]] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s0 + u * THREADS < end) {
          if (r[u] < 0) report_status(kDevIndex, 81);
          s_key[s0 + u * THREADS - beg] = r[u] < 0 ? 0u : key_from(pos[u], w[u]);
        }
    }
  }
  for (int i = tid; i < COPIES * BINS; i += THREADS) (&hist[0][0])[i] = 0;
  __syncthreads();
  auto key = [&](int slot) { return resident ? s_key[slot - beg] : key_of(slot); };

  // The kept-th largest key: `cut` is it, or (when all keys that share its first bits are kept) its first bits;
  // `want` of the keys that equal it in the bits of `mask` are kept.
  uint32_t cut = 0, mask = 0;
  int want = kept;
  const bool all = kept == n;
  for (int pass = 0; !all && pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass == 2 ? 1024 : 2048;
    for (int slot = beg + tid; slot < end; slot += THREADS) {
      const uint32_t u = key(slot);
      if ((u & mask) == cut) atomicAdd(&hist[warp % COPIES][(u >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    for (int i = tid; i < BINS; i += THREADS) {
      int c = 0;
#pragma unroll
      for (int k = 0; k < COPIES; ++k) c += hist[k][i];
      hist[0][i] = c;
    }
    sync_all();
    // thread t holds bins 2047 - 2 t and 2046 - 2 t, from the top down
    int c0 = 0, c1 = 0;
    for (int r = 0; r < size; ++r) {
      const int* t = size == 1 ? hist[0] : cluster.map_shared_rank(hist[0], r);
      c0 += t[2047 - 2 * tid];
      c1 += t[2046 - 2 * tid];
    }
    int incl = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) wcount[0][warp] = incl;
    __syncthreads();
    {
      int x = wcount[0][lane];  // every warp scans the 32 sums for itself
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const int before = __shfl_sync(0xffffffffu, x, warp == 0 ? 0 : warp - 1);
      if (warp > 0) incl += before;
    }
    const int above0 = incl - c0 - c1, above1 = incl - c1;  // keys in higher bins
    if (above0 < want && above0 + c0 >= want) {
      s_digit = 2047 - 2 * tid;
      s_above = above0;
      s_hits = c0;
    } else if (above1 < want && incl >= want) {
      s_digit = 2046 - 2 * tid;
      s_above = above1;
      s_hits = c1;
    }
    sync_all();  // the digit is known, and every CTA has read the histograms
    cut |= static_cast<uint32_t>(s_digit) << shift;
    mask |= (bins - 1) << shift;
    want -= s_above;
    if (s_hits == want) break;  // every key with these bits is kept
    for (int i = tid; i < COPIES * BINS; i += THREADS) (&hist[0][0])[i] = 0;
    __syncthreads();
  }

  // Exclusive offsets of two counts over the warps of the cluster, in slot order.
  auto offsets = [&](int c0, int c1, int& o0, int& o1, int& t0) {
    sync_all();
    if (lane == 0) {
      wcount[0][warp] = c0;
      wcount[1][warp] = c1;
    }
    __syncthreads();
    if (warp < 2) {
      const int c = wcount[warp][lane];
      int x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      wcount[warp][lane] = x - c;
      if (lane == 31) cta_count[warp] = x;
    }
    sync_all();
    o0 = wcount[0][warp];
    o1 = wcount[1][warp];
    t0 = 0;
    for (int r = 0; r < size; ++r) {
      const int* t = size == 1 ? cta_count : cluster.map_shared_rank(cta_count, r);
      const int x0 = t[0], x1 = t[1];
      if (r < rank) {
        o0 += x0;
        o1 += x1;
      }
      t0 += x0;
    }
  };

  // keys equal to the cut before this warp
  int eq = 0, eq_before = 0, dummy0, dummy1;
  if (!all) {
    for (int s0 = wbeg; s0 < wend; s0 += 32) {
      const bool in = s0 + lane < wend;
      eq += __popc(__ballot_sync(0xffffffffu, in && (key(in ? s0 + lane : s0) & mask) == cut));
    }
    offsets(eq, 0, eq_before, dummy0, dummy1);
  }
  // a warp's walk over its slots: f(slot, in range?, kept?) for 32 slots at a time
  auto walk = [&](auto&& f) {
    int seen = eq_before;
    for (int s0 = wbeg; s0 < wend; s0 += 32) {
      const bool in = s0 + lane < wend;
      const uint32_t u = in ? key(s0 + lane) & mask : 0u;
      const unsigned e = __ballot_sync(0xffffffffu, in && !all && u == cut);
      const int rank_eq = seen + __popc(e & ((1u << lane) - 1u));
      const bool keep = in && (all || u > cut || (u == cut && rank_eq < want));
      seen += __popc(e);
      f(s0 + lane, in, keep);
    }
  };
  const int border = a.in_place ? kept : 0;  // sources are the kept slots from here on, holes the others before
  int n_from = 0, n_to = 0;
  walk([&](int slot, bool in, bool keep) {
    n_from += __popc(__ballot_sync(0xffffffffu, keep && slot >= border));
    n_to += __popc(__ballot_sync(0xffffffffu, in && !keep && slot < border));
  });
  int at_from, at_to, all_from;
  offsets(n_from, n_to, at_from, at_to, all_from);
  int* from = a.from + seg * a.pitch;
  int* to = a.to + seg * a.pitch;
  walk([&](int slot, bool in, bool keep) {
    const bool is_from = keep && slot >= border, is_to = in && !keep && slot < border;
    const unsigned mf = __ballot_sync(0xffffffffu, is_from), mt = __ballot_sync(0xffffffffu, is_to);
    const unsigned below = (1u << lane) - 1u;
    if (is_from) {
      const int i = at_from + __popc(mf & below);
      from[i] = row_of(a.src, slot);
      if (!a.in_place) to[i] = row_of(a.dst, i);
    }
    if (is_to) to[at_to + __popc(mt & below)] = row_of(a.src, slot);
    at_from += __popc(mf);
    at_to += __popc(mt);
  });
  if (rank == 0 && tid == 0) a.moves[seg] = all_from;
  if (size > 1) cluster.sync();  // no CTA leaves while another may read its shared memory
}

// A warp moves ROWS rows: a row's key and value are one or (D = 64) half an instruction of 16 bytes a lane, all
// of them in flight together; positions and weights go with one lane each.
template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int LPR = 2 * D / 8;        // lanes a row: K then V, 8 values each
  constexpr int RPW = 32 / LPR;         // rows an instruction
  constexpr int ROWS = 8;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
  const long long seg = static_cast<long long>(b) * a.hkv + h;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = a.lens[b];
  const int n = a.moves[seg];
  const int* from = a.from + seg * a.pitch;
  const int* to = a.to + seg * a.pitch;
  const int sub = lane / LPR, l = lane % LPR;
  __nv_bfloat16* pool = l < LPR / 2 ? a.kcache : a.vcache;
  const long long d = static_cast<long long>(h) * D + (l % (LPR / 2)) * 8, stride = static_cast<long long>(a.hkv) * D;
  const long long hs = static_cast<long long>(h) * a.src.rows;
  const int step = gridDim.x * 8 * ROWS;
  for (int i0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * ROWS; i0 < n; i0 += step) {
    // lane u < ROWS looks up row u, and carries its position; lane ROWS + u its weight
    const int i = i0 + lane % ROWS;
    int rs = i < n ? from[i] : -1, rd = i < n ? to[i] : -1;
    if (i < n && (rs < 0 || rd < 0)) {
      report_status(kDevIndex, 82);
      rs = -1;
    }
    uint32_t word = 0;
    if (rs >= 0 && lane < 2 * ROWS)
      word = lane < ROWS ? static_cast<uint32_t>(a.kpos[hs + rs]) : __float_as_uint(a.kweight[hs + rs]);
    uint4 x[ROWS / RPW];
#pragma unroll
    for (int u = 0; u < ROWS / RPW; ++u) {
      const int r = __shfl_sync(0xffffffffu, rs, u * RPW + sub);
      if (r >= 0) x[u] = *reinterpret_cast<const uint4*>(pool + r * stride + d);
    }
#pragma unroll
    for (int u = 0; u < ROWS / RPW; ++u) {
      const int r = __shfl_sync(0xffffffffu, rs, u * RPW + sub), t = __shfl_sync(0xffffffffu, rd, u * RPW + sub);
      if (r >= 0) *reinterpret_cast<uint4*>(pool + t * stride + d) = x[u];
    }
    if (rs >= 0 && lane < ROWS) a.kpos[hs + rd] = static_cast<int>(word);
    if (rs >= 0 && lane >= ROWS && lane < 2 * ROWS) a.kweight[hs + rd] = __uint_as_float(word);
  }
}

}  // namespace bf
