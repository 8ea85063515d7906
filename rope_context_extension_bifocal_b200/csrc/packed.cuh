// Packed batches: sequences of different lengths laid one after another in [T, heads, D], their
// boundaries in a device array cu_seqlens [batch + 1].
//
// plan_tiles turns the boundaries into a list of 128-row tiles, the ones with the most work first, that
// the attention kernels' CTAs index; it is one CTA's work and rides along with the pass that precedes
// them. rope_packed_kernel is the RoPE pass over the packed rows (each row's position, and the factor G of
// its sequence, from the boundaries).
#pragma once
#include "common.cuh"
#include "rope_prepass.cuh"


namespace bf {

// Rows of a cache: dense (row = the packed row) or paged (block_table non-null: position p of
// sequence b is row block_table[b * max_pages + p / page_size] * page_size + p % page_size).
struct CacheRows {
  const int* block_table;
  int max_pages, page_size, pool_pages;
  int rows;        // rows of the cache, and the pitch of the per-head arrays [hkv, rows]
  int page_shift;  // log2 of the page size, -1 when it is not a power of two (then it is divided by)
};

// Row of position p of sequence b, or -1 when the table's entry is not a page of the pool.
__device__ __forceinline__ long long cache_row(const CacheRows& c, int b, int p, int packed_row) {
  if (!c.block_table) return packed_row;
  const int page = c.page_shift >= 0 ? p >> c.page_shift : p / c.page_size;
  const int pg = c.block_table[static_cast<long long>(b) * c.max_pages + page];
  if (pg < 0 || pg >= c.pool_pages) return -1;
  return static_cast<long long>(pg) * c.page_size + (p - page * c.page_size);
}

struct PlanHeader {
  int n_tiles;  // entries of the tile list; 0 when the boundaries are not valid
};

// One 128-row tile of a sequence: its index t within the sequence, the sequence's first row and its
// length. All a CTA needs, in one load.
struct __align__(16) PackedTile {
  int seq, t, first, n;
};

constexpr int kPlanLevels = 1024;
constexpr int kPlanThreads = 256;

struct PlanArgs {
  const int* cu;  // [batch + 1]
  int batch, total_rows, max_len;
  int obs;        // key tiles: only the last `obs` rows of a sequence are queries; 0: query tiles
  PlanHeader* head;
  PackedTile* tiles;
  int max_tiles;
};

// Queries of a sequence of n rows.
__host__ __device__ __forceinline__ int window_rows(int n, int obs) { return n < obs ? n : obs; }

// Whether the boundaries are in order, no sequence longer than max_len and none past the last row. Every CTA of
// the pass that writes cache rows asks for itself (a coalesced read of the array, in L2), so that nothing at all
// is written for a batch with one bad boundary and the pass need not wait for a kernel that checks. All threads.
__device__ __forceinline__ bool boundaries_ok(const PlanArgs& a) {
  bool bad = false;
  for (int b = threadIdx.x; b < a.batch; b += kPlanThreads) {
    const int s = a.cu[b], e = a.cu[b + 1];
    bad |= s < 0 || e < s || e > a.total_rows || e - s > a.max_len;
  }
  return !__syncthreads_or(bad);
}

// The tile list, by one CTA of kPlanThreads threads: the tiles sorted by work with a counting sort over
// kPlanLevels levels. A query tile's work grows with its index, a key tile's with the queries that see it. The
// order within a level is left to the atomics: no result depends on it, only when a tile runs.
__device__ __forceinline__ void plan_tiles(const PlanArgs& a, bool ok) {
  __shared__ int hist[kPlanLevels];
  __shared__ int wsum[kPlanThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!ok) {
    if (tid == 0) {
      report_status(kDevIndex, 60);
      a.head->n_tiles = 0;
    }
    return;
  }
  constexpr int PER = kPlanLevels / kPlanThreads;
  for (int i = tid; i < kPlanLevels; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  auto level = [&](int n, int t) {
    if (a.obs == 0) return min(t, kPlanLevels - 1);
    const int first = max(n - window_rows(n, a.obs), t * 128);
    return min((n - first + 127) / 128, kPlanLevels - 1);
  };
  // a warp per sequence, a lane per tile
  for (int b = warp; b < a.batch; b += kPlanThreads / 32) {
    const int n = a.cu[b + 1] - a.cu[b];
    for (int t = lane; t * 128LL < n; t += 32) atomicAdd(&hist[level(n, t)], 1);
  }
  __syncthreads();
  // exclusive scan from the top level down: where each level's tiles start (PER levels a thread)
  {
    int c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += c[i] = hist[kPlanLevels - 1 - (tid * PER + i)];
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += wsum[w];
    if (tid == kPlanThreads - 1) a.head->n_tiles = min(x, a.max_tiles);
    x -= sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      hist[kPlanLevels - 1 - (tid * PER + i)] = x;
      x += c[i];
    }
  }
  __syncthreads();
  for (int b = warp; b < a.batch; b += kPlanThreads / 32) {
    PackedTile e;
    e.seq = b;
    e.first = a.cu[b];
    e.n = a.cu[b + 1] - e.first;
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
// times 2 pi. The integer product m * hi wraps at whole turns by itself; its top 23 bits, rounded, become the
// mantissa of a float f in [1, 2), and f - 1.5 turns, exact in fp32 and in [-1/2, 1/2), is the reduced angle, 0 for
// m = 0: within 6e-7 for m up to 2^24 (2^-24 turns of the rounding, and the roundings of the last FMA), 1e-6 up to 2^30,
// 1.4e-6 below 2^31 (m as a float), for an integer multiplication, a shift, an addition, a product and an FMA.
// With the 1.5 turns taken off inside the FMA instead, its rounding near 3 pi and that of 2 pi are not small
// against the angle: 1.3e-6, and 2.4e-7 at m = 0.
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
  __sincosf(fmaf(f - 1.5f, 6.283185307179586f, mf * w.lo), &s, &c);
}

struct PackedRopeArgs {
  const void* q;
  const void* k;
  const void* v;
  PlanArgs plan;
  int hq, hkv;
  int w0, w_pretrained, mode, window;
  __half* Qo;  // [hq, T, D]; the long-range forms are written only where they are used
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

// Eight values to fp16, and the largest magnitude among all so rounded: a value that fp16 cannot hold rounds to
// inf, a NaN stays one, and the maximum that keeps NaNs finds either with one instruction for two values.
__device__ __forceinline__ uint4 to_f16(const float (&x)[8], __half2& top) {
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[e] = pack_f16x2(x[2 * e], x[2 * e + 1]);
    top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __half2*>(&h[e])));
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}
__device__ __forceinline__ bool all_finite(__half2 top) {
  const float2 f = __half22float2(top);
  return f.x < INFINITY && f.y < INFINITY;  // false for a NaN
}

// Rows a CTA: with two, few heads leave a warp too little to keep its loads in flight (whole prefill of 3775 rows of
// 12 / 4 fp32 heads of 64: 71 us instead of 65), with eight, few rows leave SMs idle (1607 rows of 32 / 8 heads of 128:
// 48 us instead of 44); 14188 and 25012 rows take the same with either.
constexpr int kRopeRows = 4;

// What a CTA's warps need of each of its rows.
struct RopeRow {
  int b, p, G;       // sequence (-1: none), position, factor
  int lng_q, lng_k;  // whether the row's query and key are wanted in the long-range form
  int row;           // cache row, -1: none
};

// Eight pairs (x1, x2) turned by the angles of form f: cs holds {cos, sin} of pairs 8 l + 2 e, 8 l + 2 e + 1 at
// [e][l], so that the lanes of a head read consecutive 16-byte words. Products and sums are fused as the
// compiler fuses them in rope_prepass_kernel, so that both passes give the same forms bit for bit.
template <typename V, int LPR>
__device__ __forceinline__ void turn8(const V& x1, const V& x2, const float4 (&cs)[4][LPR], int l, float (&y1)[8], float (&y2)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 t = cs[e][l];
    const float u0 = x1.get(2 * e), v0 = x2.get(2 * e), u1 = x1.get(2 * e + 1), v1 = x2.get(2 * e + 1);
    y1[2 * e] = fmaf(u0, t.x, -__fmul_rn(v0, t.y));
    y2[2 * e] = fmaf(v0, t.x, __fmul_rn(u0, t.y));
    y1[2 * e + 1] = fmaf(u1, t.z, -__fmul_rn(v1, t.w));
    y2[2 * e + 1] = fmaf(v1, t.z, __fmul_rn(u1, t.w));
  }
}

// A CTA takes four rows (the first CTA makes the tile list instead): it looks them up, evaluates their angles
// once for all heads (fp64 product and reduction, see angle_cos_sin), then deals (row, four heads) units to its
// warps, eight lanes a head and eight pairs a lane. A warp keeps UNITS loads in flight, the first ones while the
// angles are formed. Memory bound: it reads q, k, v once and writes each form once: 99 us for 14188 rows of 32 / 8
// heads of 128 (480 MB: 4.8 TB/s of 6.55), 16 us for 1607 rows (latency). Token-major forms took the same time. The long-range forms that no
// pair uses are left out: of queries in the 128 rows of an attention tile that ends before w0 (no key is that
// far back), and of keys in a tile that no query of the sequence is w0 past.
template <typename Tin, int D>
__global__ void __launch_bounds__(kPlanThreads, sizeof(Tin) == 2 ? 3 : 2) rope_packed_kernel(const __grid_constant__ PackedRopeArgs a) {
  constexpr int P = D / 2;
  constexpr int LPR = P / 8;  // lanes a head
  constexpr int UNITS = 3, ROWS = kRopeRows;
  __shared__ RopeRow s_row[ROWS];
  __shared__ float4 s_cs[ROWS][2][4][LPR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 3, l8 = lane & 7, k0 = l8 * 8;
  const int r0 = static_cast<int>(blockIdx.x - 1) * ROWS;
  const int heads = a.hq + 2 * a.hkv, per_row = (heads + 3) / 4;
  const int n_units = min(ROWS, a.plan.total_rows - r0) * per_row;
  const bool want_v = a.Vb || a.vcache;
  Vec8<Tin> x1[UNITS], x2[UNITS];
  auto load = [&](int u, Vec8<Tin>& y1, Vec8<Tin>& y2) {
    const int rr = u / per_row, hh = u % per_row * 4 + grp;
    if (u >= n_units || hh >= heads || l8 >= LPR) return;
    const long long r = r0 + rr;
    const Tin* src = hh < a.hq           ? static_cast<const Tin*>(a.q) + (r * a.hq + hh) * D
                     : hh < a.hq + a.hkv ? static_cast<const Tin*>(a.k) + (r * a.hkv + hh - a.hq) * D
                                         : static_cast<const Tin*>(a.v) + (r * a.hkv + hh - a.hq - a.hkv) * D;
    if (hh >= a.hq + a.hkv && !want_v) return;
    y1.load(src + k0);
    y2.load(src + P + k0);
  };
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x > 0)
#pragma unroll
    for (int j = 0; j < UNITS; ++j) load(warp + 8 * j, x1[j], x2[j]);
  const bool ok = boundaries_ok(a.plan);
  if (blockIdx.x == 0) {
    plan_tiles(a.plan, ok);
    return;
  }
  if (!ok) return;
  if (threadIdx.x < ROWS) {
    RopeRow w;
    const int r = r0 + threadIdx.x;
    w.b = r < a.plan.total_rows ? sequence_of(a.plan.cu, a.plan.batch, r) : -1;
    w.row = -1;
    if (w.b >= 0) {
      const int first = a.plan.cu[w.b], n = a.plan.cu[w.b + 1] - first;
      w.p = r - first;
      w.G = factor_of(n, a.w_pretrained);
      const bool lng = !a.window && has_long_pairs(n, w.G, a.w0);
      w.lng_q = lng && (w.p | 127) >= a.w0;
      w.lng_k = lng && n - 1 - (w.p & ~127) >= a.w0;
      if (a.kcache) {
        const long long c = cache_row(a.rows, w.b, w.p, r);
        if (c < 0) report_status(kDevIndex, 61);
        w.row = static_cast<int>(c);
      }
    }
    s_row[threadIdx.x] = w;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ROWS * 2 * P; i += kPlanThreads) {
    const int rr = i / (2 * P), f = i / P % 2, k = i % P;
    const RopeRow w = s_row[rr];
    if (w.b < 0 || (f == 1 && !w.lng_q && !w.lng_k)) continue;
    const double om = a.omega[k];
    float c, s;
    angle_cos_sin(f == 0        ? static_cast<double>(w.p) * om
                  : a.mode == 0 ? static_cast<double>(w.p) * (om / w.G)
                                : static_cast<double>(w.p / w.G) * om,
                  c, s);
    reinterpret_cast<float2*>(&s_cs[rr][f][k % 8 / 2][k / 8])[k % 2] = make_float2(c, s);
  }
  __syncthreads();
  __half2 top = __float2half2_rn(0.f);
  for (int u0 = warp; u0 < n_units; u0 += 8 * UNITS) {
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      const int u = u0 + 8 * j;
      const int rr = min(u / per_row, ROWS - 1), hh = u % per_row * 4 + grp;
      const RopeRow w = s_row[rr];
      const bool is_q = hh < a.hq, is_v = hh >= a.hq + a.hkv;
      if (u < n_units && hh < heads && l8 < LPR && w.b >= 0 && (!is_v || want_v)) {
        const long long r = r0 + rr, crow = w.row;
        const int h = is_q ? hh : hh - a.hq - (is_v ? a.hkv : 0);
        float y1[8], y2[8];
        if (is_v) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            y1[i] = x1[j].get(i);
            y2[i] = x2[j].get(i);
          }
          if (a.Vb) {
            store8_bf16(a.Vb + (r * a.hkv + h) * D + k0, y1);
            store8_bf16(a.Vb + (r * a.hkv + h) * D + P + k0, y2);
          }
          if (crow >= 0) {
            store8_bf16(a.vcache + (crow * a.hkv + h) * D + k0, y1);
            store8_bf16(a.vcache + (crow * a.hkv + h) * D + P + k0, y2);
          }
        } else {
          const long long at = (static_cast<long long>(h) * a.plan.total_rows + r) * D;
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            if (f == 1 && !(is_q ? w.lng_q : w.lng_k)) break;
            turn8(x1[j], x2[j], s_cs[rr][f], l8, y1, y2);
            __half* dst = (is_q ? (f == 0 ? a.Qo : a.Ql) : (f == 0 ? a.Ko : a.Kl)) + at;
            *reinterpret_cast<uint4*>(dst + k0) = to_f16(y1, top);
            *reinterpret_cast<uint4*>(dst + P + k0) = to_f16(y2, top);
            if (f == 0 && !is_q && crow >= 0) {
              __nv_bfloat16* dc = a.kcache + (crow * a.hkv + h) * D;
              store8_bf16(dc + k0, y1);
              store8_bf16(dc + P + k0, y2);
              if (a.kpos && l8 == 0) a.kpos[static_cast<long long>(h) * a.rows.rows + crow] = w.p;
            }
          }
        }
      }
      load(u + 8 * UNITS, x1[j], x2[j]);
    }
  }
  if (!all_finite(top)) report_status(kDevRange, 62);
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
