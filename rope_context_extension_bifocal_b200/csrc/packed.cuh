// Packed batches: sequences of different lengths laid one after another in [T, heads, D], their
// boundaries in a device array cu_seqlens [batch + 1].
//
// packed_plan_kernel turns the boundaries into a list of 128-row tiles, the ones with the most
// work first, that the attention kernels' CTAs index; rope_packed_kernel is the RoPE pass over
// the packed rows (each row's position, and the factor G of its sequence, from the boundaries).
#pragma once
#include "common.cuh"
#include "rope_prepass.cuh"

namespace bf {

// Rows of a cache: dense (row = the packed row) or paged (block_table non-null: position p of
// sequence b is row block_table[b * max_pages + p / page_size] * page_size + p % page_size).
struct CacheRows {
  const int* block_table;
  int max_pages, page_size, pool_pages;
  int rows;  // rows of the cache, and the pitch of the per-head arrays [hkv, rows]
};

// Row of position p of sequence b, or -1 when the table's entry is not a page of the pool.
__device__ __forceinline__ long long cache_row(const CacheRows& c, int b, int p, int packed_row) {
  if (!c.block_table) return packed_row;
  const int pg = c.block_table[static_cast<long long>(b) * c.max_pages + p / c.page_size];
  if (pg < 0 || pg >= c.pool_pages) return -1;
  return static_cast<long long>(pg) * c.page_size + p % c.page_size;
}

struct PlanHeader {
  int n_tiles;  // entries of the tile list; 0 when the boundaries are not valid
  int ok;
};

// One 128-row tile of a sequence: its index t within the sequence, the sequence's first row and its
// length, and (key tiles) the first row of its queries in the query forms. All a CTA needs, in one load.
struct __align__(32) PackedTile {
  int seq, t, first, n, qoff, pad[3];
};

constexpr int kPlanLevels = 1024;

struct PlanArgs {
  const int* cu;  // [batch + 1]
  int batch, total_rows, max_len;
  int obs;        // key tiles: only the last `obs` rows of a sequence are queries; 0: query tiles
  PlanHeader* head;
  PackedTile* tiles;
  int max_tiles;
  int* qoff;      // key tiles: [batch + 1] first row of each sequence's queries in the query forms
};

// Queries of a sequence of n rows, and the rows they take in the query forms: a multiple of four,
// so that a tile's log-sum-exps (4 bytes a row) start on a 16-byte boundary.
__host__ __device__ __forceinline__ int window_rows(int n, int obs) { return n < obs ? n : obs; }
__host__ __device__ __forceinline__ int window_pad(int n, int obs) { return (window_rows(n, obs) + 3) & ~3; }

// One CTA. Checks the boundaries (each in order, no sequence longer than max_len, none past the
// last row), then sorts the tiles by work with a counting sort over kPlanLevels levels: a query
// tile's work grows with its index, a key tile's with the query tiles that see it. The order
// within a level is left to the atomics: no result depends on it, only when a tile runs.
__global__ void __launch_bounds__(1024) packed_plan_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ int hist[kPlanLevels];
  __shared__ int wsum[32];
  __shared__ int carry;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  bool bad = false;
  for (int b = tid; b < a.batch; b += 1024) {
    const int s = a.cu[b], e = a.cu[b + 1];
    bad |= s < 0 || e < s || e > a.total_rows || e - s > a.max_len;
  }
  hist[tid] = 0;
  if (tid == 0) carry = 0;
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      report_status(kDevIndex, 60);
      a.head->n_tiles = 0;
      a.head->ok = 0;
    }
    return;
  }
  auto level = [&](int n, int t) {
    if (a.obs == 0) return min(t, kPlanLevels - 1);
    const int first = max(n - window_rows(n, a.obs), t * 128);
    return min((n - first + 127) / 128, kPlanLevels - 1);
  };
  // a warp per sequence, a lane per tile
  for (int b = warp; b < a.batch; b += 32) {
    const int n = a.cu[b + 1] - a.cu[b];
    for (int t = lane; t * 128LL < n; t += 32) atomicAdd(&hist[level(n, t)], 1);
  }
  __syncthreads();
  // exclusive scan from the top level down: where each level's tiles start
  {
    const int lv = kPlanLevels - 1 - tid;
    const int c = hist[lv];
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int w = wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      wsum[lane] = w;
    }
    __syncthreads();
    const int incl = x + (warp ? wsum[warp - 1] : 0);
    hist[lv] = incl - c;
    if (tid == 1023) {
      a.head->n_tiles = min(incl, a.max_tiles);
      a.head->ok = 1;
    }
  }
  __syncthreads();
  // exclusive scan of the sequences' query rows
  for (int b0 = 0; a.qoff && b0 < a.batch; b0 += 1024) {
    const int b = b0 + tid;
    const int c = b < a.batch ? window_pad(a.cu[b + 1] - a.cu[b], a.obs) : 0;
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (b < a.batch) a.qoff[b] = before + x - c;
    __syncthreads();
    if (tid == 1023) carry = before + x;
    __syncthreads();
  }
  if (a.qoff && tid == 0) a.qoff[a.batch] = carry;
  __syncthreads();  // the offsets are written: each warp reads those of its sequences
  for (int b = warp; b < a.batch; b += 32) {
    PackedTile e;
    e.seq = b;
    e.first = a.cu[b];
    e.n = a.cu[b + 1] - e.first;
    e.qoff = a.qoff ? a.qoff[b] : 0;
    e.pad[0] = e.pad[1] = e.pad[2] = 0;
    for (int t = lane; t * 128LL < e.n; t += 32) {
      e.t = t;
      const int at = atomicAdd(&hist[level(e.n, t)], 1);
      if (at < a.max_tiles) a.tiles[at] = e;
    }
  }
}

// The sequence that packed row r belongs to (the last one that starts at or before r), or -1.
__device__ __forceinline__ int sequence_of(const int* cu, int batch, int r) {
  if (r < cu[0] || r >= cu[batch]) return -1;
  int lo = 0, hi = batch;  // cu[lo] <= r < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int factor_of(int n, int w_pretrained) {
  return n <= w_pretrained ? 1 : (n - 1) / w_pretrained + 1;
}

// Whether a sequence of n rows has pairs in the long-range branch that differ from the original one.
__device__ __forceinline__ bool has_long_pairs(int n, int G, int w0) { return G > 1 && w0 < n; }

// Angles m * w for integers m, as fractions of a turn: `hi` is the first 32 bits of w / 2 pi, `lo` the rest
// times 2 pi. The integer product m * hi wraps at whole turns by itself; its top 23 bits become the
// mantissa of a float f in [1, 2), and (f - 1.5) turns, in [-1/2, 1/2), is the reduced angle: exact to 2^-23
// turns (7e-7) at any m below 2^31, for an integer multiplication, a shift and two FMAs.
struct TurnStep {
  uint32_t hi;
  float lo;
};

__device__ __forceinline__ TurnStep turn_step(double w) {
  double t = w * 0.15915494309189533576888376337251;
  t = (t - floor(t)) * 4294967296.0;
  const double hi = fmin(floor(t), 4294967295.0);
  TurnStep r;
  r.hi = static_cast<uint32_t>(hi);
  r.lo = static_cast<float>((t - hi) * (2.3283064365386962890625e-10 * 6.283185307179586476925286766559));
  return r;
}

__device__ __forceinline__ void turn_cos_sin(int m, float mf, const TurnStep& w, float& c, float& s) {
  const uint32_t ph = static_cast<uint32_t>(m) * w.hi + 0x80000100u;
  const float f = __uint_as_float(__funnelshift_r(ph, 0x7fu, 9));
  __sincosf(fmaf(f, 6.283185307179586f, fmaf(mf, w.lo, -9.42477796076938f)), &s, &c);
}

struct PackedRopeArgs {
  const void* q;
  const void* k;
  const void* v;
  const int* cu;
  const PlanHeader* head;
  int batch, total_rows, hq, hkv;
  int w0, w_pretrained, mode, window;
  __half* Qo;  // [hq, T, D]; Ql / Kl rows are written only where a sequence has a long-range branch
  __half* Ql;
  __half* Ko;  // [hkv, T, D]
  __half* Kl;
  __nv_bfloat16* Vb;      // fp32 inputs: bf16 copy of v [T, hkv, D]
  __nv_bfloat16* kcache;  // optional cache rows: keys under the original RoPE, values, positions
  __nv_bfloat16* vcache;
  int* kpos;              // [hkv, rows]
  CacheRows rows;
  double omega[64];
};

// One warp per packed row; lanes as in rope_prepass_kernel (4 groups of 8, a group per head, a lane
// 8 pairs). Memory bound: it reads q, k, v once and writes the operand forms once.
template <typename Tin, int D>
__global__ void __launch_bounds__(256) rope_packed_kernel(const __grid_constant__ PackedRopeArgs a) {
  constexpr int P = D / 2;
  constexpr int NPAIR = 8;
  constexpr int LANES_PER_ROW = P / NPAIR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x * 8 + warp;
  pdl_launch_dependents();
  pdl_wait();
  if (r >= a.total_rows || !a.head->ok) return;
  const int b = sequence_of(a.cu, a.batch, r);
  if (b < 0) return;
  const int first = a.cu[b], n = a.cu[b + 1] - first, p = r - first;
  const int G = factor_of(n, a.w_pretrained);
  const bool lng = !a.window && has_long_pairs(n, G, a.w0);
  const int grp = lane >> 3, l8 = lane & 7;
  if (l8 >= LANES_PER_ROW) return;
  const int k0 = l8 * NPAIR;
  long long crow = -1;
  if (a.kcache) {
    crow = cache_row(a.rows, b, p, r);
    if (crow < 0 && lane == 0) report_status(kDevIndex, 61);
  }

  float co[NPAIR], so[NPAIR], cl[NPAIR], sl[NPAIR];
#pragma unroll
  for (int i = 0; i < NPAIR; ++i) {
    const double w = a.omega[k0 + i];
    angle_cos_sin(static_cast<double>(p) * w, co[i], so[i]);
    if (lng) angle_cos_sin(a.mode == 0 ? static_cast<double>(p) * (w / G) : static_cast<double>(p / G) * w, cl[i], sl[i]);
  }
  const Tin* qb = static_cast<const Tin*>(a.q);
  const Tin* kb = static_cast<const Tin*>(a.k);
  const Tin* vb = static_cast<const Tin*>(a.v);
  for (int hh = grp; hh < a.hq + a.hkv; hh += 4) {
    const bool is_q = hh < a.hq;
    const int h = is_q ? hh : hh - a.hq;
    const Tin* src = (is_q ? qb + (static_cast<long long>(r) * a.hq + h) * D : kb + (static_cast<long long>(r) * a.hkv + h) * D);
    Vec8<Tin> x1, x2;
    x1.load(src + k0);
    x2.load(src + P + k0);
    float y1[8], y2[8];
    bool fin = true;
#pragma unroll
    for (int i = 0; i < NPAIR; ++i) {
      const float u = x1.get(i), w = x2.get(i);
      y1[i] = u * co[i] - w * so[i];
      y2[i] = w * co[i] + u * so[i];
      fin &= f16_ok(y1[i]) & f16_ok(y2[i]);
    }
    const long long at = (static_cast<long long>(h) * a.total_rows + r) * D;
    __half* dst_o = (is_q ? a.Qo : a.Ko) + at;
    store8_f16(dst_o + k0, y1);
    store8_f16(dst_o + P + k0, y2);
    if (!is_q && crow >= 0) {
      __nv_bfloat16* dc = a.kcache + (crow * a.hkv + h) * D;
      store8_bf16(dc + k0, y1);
      store8_bf16(dc + P + k0, y2);
      if (a.kpos && l8 == 0) a.kpos[static_cast<long long>(h) * a.rows.rows + crow] = p;
    }
    if (lng) {
#pragma unroll
      for (int i = 0; i < NPAIR; ++i) {
        const float u = x1.get(i), w = x2.get(i);
        y1[i] = u * cl[i] - w * sl[i];
        y2[i] = w * cl[i] + u * sl[i];
        fin &= f16_ok(y1[i]) & f16_ok(y2[i]);
      }
      __half* dst_l = (is_q ? a.Ql : a.Kl) + at;
      store8_f16(dst_l + k0, y1);
      store8_f16(dst_l + P + k0, y2);
    }
    if (!fin) report_status(kDevRange, 62);
  }
  if (a.Vb || crow >= 0) {
    for (int h = grp; h < a.hkv; h += 4) {
      const long long off = (static_cast<long long>(r) * a.hkv + h) * D;
      Vec8<Tin> x1, x2;
      x1.load(vb + off + k0);
      x2.load(vb + off + P + k0);
      float y1[8], y2[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y1[i] = x1.get(i);
        y2[i] = x2.get(i);
      }
      if (a.Vb) {
        store8_bf16(a.Vb + off + k0, y1);
        store8_bf16(a.Vb + off + P + k0, y2);
      }
      if (crow >= 0) {
        __nv_bfloat16* dv = a.vcache + (crow * a.hkv + h) * D;
        store8_bf16(dv + k0, y1);
        store8_bf16(dv + P + k0, y2);
      }
    }
  }
}

// What the attention kernels' packed form adds to their arguments: the tile list and boundaries.
// A CTA's tile is tiles[rank], if the list is that long.
struct PackedTiles {
  const PlanHeader* head;
  const PackedTile* tiles;
  int max_tiles;
  int total_rows;
  int w_pretrained;
};

// w0 of a sequence without a long-range branch: every pair is local (far above any distance, far
// below an overflow of the schedules' sums).
constexpr int kAllLocal = 1 << 30;

}  // namespace bf
