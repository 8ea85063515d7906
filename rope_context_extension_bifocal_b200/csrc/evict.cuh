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
// evict_select_kernel finds the kept-th largest key with a radix select, 8 bits a pass, over keys that
// it forms once in shared memory; a segment is spread over a thread-block cluster whose CTAs add up
// their histograms through distributed shared memory. evict_move_kernel copies the rows.
// Bound by memory: 8 bytes a slot to select (weight and position), 2 (4 D + 8) bytes a row moved; with
// few segments by the latency of the passes instead.
#pragma once
#include <cooperative_groups.h>

#include "common.cuh"
#include "packed.cuh"

namespace bf {

namespace ev {
constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr int COPIES = 8;           // histograms a CTA fills side by side (fewer conflicts on one bin)
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
  int* from;               // [B, hkv, pitch] source slots, ascending
  int* to;                 // [B, hkv, pitch] in place: holes, ascending
  int pitch;
  int keys_in_smem;        // keys a CTA has room for
};

__global__ void __launch_bounds__(ev::THREADS, 1) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  using namespace ev;
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t s_key[];
  __shared__ int hist[COPIES][256];
  __shared__ int total[256];           // this CTA's bins, read by the cluster
  __shared__ int wcount[2][WARPS];
  __shared__ int cta_count[2];         // this CTA's counts, read by the cluster
  __shared__ int s_digit, s_above;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), size = static_cast<int>(cluster.num_blocks());
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
  auto key_of = [&](int slot) -> uint32_t {
    const long long r = cache_row(a.src, b, slot, 0);
    if (r < 0) {
      report_status(kDevIndex, 81);
      return 0u;
    }
    const long long at = static_cast<long long>(h) * a.src.rows + r;
    const int pos = a.kpos[at];
    if (pos < a.sink || pos > newest - a.recent) return 0xffffffffu;
    const float w = a.kweight[at];
    if (w != w) return 0x007fffffu;  // -inf's
    const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  };
  const bool resident = end - beg <= a.keys_in_smem;
  if (resident)
    for (int slot = beg + tid; slot < end; slot += THREADS) s_key[slot - beg] = key_of(slot);
  __syncthreads();
  auto key = [&](int slot) { return resident ? s_key[slot - beg] : key_of(slot); };

  // The kept-th largest key `cut`, and how many keys equal to it are kept.
  uint32_t cut = 0;
  int want = kept;  // keys still to find among those that share the prefix
  if (kept < n) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < COPIES * 256; i += THREADS) (&hist[0][0])[i] = 0;
      __syncthreads();
      for (int slot = beg + tid; slot < end; slot += THREADS) {
        const uint32_t u = key(slot);
        if (shift == 24 || (u >> (shift + 8)) == (cut >> (shift + 8))) atomicAdd(&hist[warp % COPIES][(u >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid < 256) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) c += hist[i][tid];
        total[tid] = c;
      }
      cluster.sync();
      // warp 0 of every CTA finds the digit: lane l holds bins 255 - 8 l .. 248 - 8 l, from the top down
      if (warp == 0) {
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = 0;
        for (int r = 0; r < size; ++r) {
          const int* t = cluster.map_shared_rank(total, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) c[i] += t[255 - 8 * lane - i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        int above = incl - sum;  // keys in higher bins
        if (above < want && incl >= want) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (above < want && above + c[i] >= want) {
              s_digit = 255 - 8 * lane - i;
              s_above = above;
            }
            above += c[i];
          }
        }
      }
      cluster.sync();  // the digit is found everywhere before any `total` is written again
      cut |= static_cast<uint32_t>(s_digit) << shift;
      want -= s_above;
    }
  } else {
    want = 0;  // all are kept: every key is above -1
  }
  const bool all = kept == n;

  // Exclusive offsets of two counts over the warps of the cluster, in slot order.
  auto offsets = [&](int c0, int c1, int& o0, int& o1, int& t0, int& t1) {
    cluster.sync();
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
    cluster.sync();
    o0 = wcount[0][warp];
    o1 = wcount[1][warp];
    t0 = t1 = 0;
    for (int r = 0; r < size; ++r) {
      const int* t = cluster.map_shared_rank(cta_count, r);
      const int x0 = t[0], x1 = t[1];
      if (r < rank) {
        o0 += x0;
        o1 += x1;
      }
      t0 += x0;
      t1 += x1;
    }
  };

  // keys equal to the cut before this warp
  int eq = 0, eq_before, dummy0, dummy1, dummy2;
  if (!all)
    for (int s0 = wbeg; s0 < wend; s0 += 32) {
      const bool in = s0 + lane < wend;
      eq += __popc(__ballot_sync(0xffffffffu, in && key(in ? s0 + lane : s0) == cut));
    }
  offsets(eq, 0, eq_before, dummy0, dummy1, dummy2);
  // a warp's walk over its slots: f(slot, kept?) for 32 slots at a time
  auto walk = [&](auto&& f) {
    int seen = eq_before;
    for (int s0 = wbeg; s0 < wend; s0 += 32) {
      const bool in = s0 + lane < wend;
      const uint32_t u = in ? key(s0 + lane) : 0u;
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
  int at_from, at_to, all_from, all_to;
  offsets(n_from, n_to, at_from, at_to, all_from, all_to);
  int* from = a.from + seg * a.pitch;
  int* to = a.to + seg * a.pitch;
  walk([&](int slot, bool in, bool keep) {
    const bool is_from = keep && slot >= border, is_to = in && !keep && slot < border;
    const unsigned mf = __ballot_sync(0xffffffffu, is_from), mt = __ballot_sync(0xffffffffu, is_to);
    const unsigned below = (1u << lane) - 1u;
    if (is_from) from[at_from + __popc(mf & below)] = slot;
    if (is_to) to[at_to + __popc(mt & below)] = slot;
    at_from += __popc(mf);
    at_to += __popc(mt);
  });
  if (rank == 0 && tid == 0) a.moves[seg] = all_from;
  cluster.sync();  // no CTA leaves while another may read its shared memory
}

// A warp moves a row's K and V (D = 128: 16 bytes a lane; D = 64: two rows at a time), UNROLL of them in
// flight; position and weight go with the row's first lanes.
template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int LPR = 2 * D / 8;        // lanes a row: K then V, 8 values each
  constexpr int RPW = 32 / LPR;
  constexpr int UNROLL = 4;
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
  const int d = (l % (LPR / 2)) * 8;
  const int step = gridDim.x * 8 * RPW * UNROLL;
  for (int i0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * RPW * UNROLL; i0 < n; i0 += step) {
    uint4 x[UNROLL];
    long long rd[UNROLL], rs[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int i = i0 + u * RPW + sub;
      rs[u] = rd[u] = -1;
      if (i < n) {
        rs[u] = cache_row(a.src, b, from[i], 0);
        rd[u] = cache_row(a.dst, b, a.in_place ? to[i] : i, 0);
        if (rs[u] < 0 || rd[u] < 0) {
          report_status(kDevIndex, 82);
          rs[u] = -1;
        }
      }
      if (rs[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(pool + (rs[u] * a.hkv + h) * D + d);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (rs[u] < 0) continue;
      *reinterpret_cast<uint4*>(pool + (rd[u] * a.hkv + h) * D + d) = x[u];
      const long long hs = static_cast<long long>(h) * a.src.rows;
      if (l == 0) a.kpos[hs + rd[u]] = a.kpos[hs + rs[u]];
      if (l == 1) a.kweight[hs + rd[u]] = a.kweight[hs + rs[u]];
    }
  }
}

}  // namespace bf
