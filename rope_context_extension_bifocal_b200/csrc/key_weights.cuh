// Attention weight of cached keys: for every key of a packed batch of prompts, the sum over the last
// `obs` queries of its sequence (those at or after it) and over the heads of its group of
// exp(score - lse_i), with the prefill's log-sum-exps.
//
// One CTA owns 128 keys of one kv head and streams the query tiles that see them: S^T = K Q^T, keys in
// the 128 tensor-memory lanes and QT queries in the columns. A thread so owns one key, and the column
// sum of the attention matrix is a sum along its own registers: no shuffles, no atomics, and a result
// that does not depend on the order in which CTAs run. The rows of the query forms are (query, head of the
// group) with the heads innermost, so a tile holds QT / g queries of all g heads: a window of 32 queries and
// four heads is one tile of 128 columns, not four with 32 each.
//
// Precision. A single fp16 rounding of the rotated operands moves a score by about 3e-4, and so a weight
// summed from few queries by as much, relative. Each operand is therefore split into an fp16 value and the
// fp16 rest, and S = Kh Qh + Kl Qh + Kh Ql (the term left out is 2^-22): scores exact to about 1e-6. Neither low part
// can be spared, however long the sum: a key's own rounding shifts all its scores alike (the queries that attend to it
// lean its way), and what averages out of the queries' roundings depends on how many queries carry a key's weight, one of
// each head for the last key, a few under peaked scores. Without Kh Ql all queries of 6001 tokens took 340 us, and single
// weights were 2e-4 off (1.5e-3 with queries four times the size).
//
// Keys come raw from global memory and are turned by the softmax warps themselves, once for each branch
// the tile has (the local queries first, then the long-range ones); no rotated copy of k is written. The
// query rows are turned once by weights_query_kernel and arrive by TMA.
//
// Warp roles: the first 8 or 16 warps form the key tile and then sum (groups of four warps: a visit each in turn, or a
// quarter of every visit's columns; warp w reads TMEM lanes 32 (w % 4) ..), then a TMA producer and an MMA issuer. A visit is one
// query tile under one branch. Shared memory holds the key tile (high and low part) and a ring of query tiles.
//
// Few rows (QT = 64): each key tile has a handful of visits and its time is the latency of forming it, so two
// CTAs share an SM (96 KB and 256 tensor-memory columns each). Many rows (QT = 256): one CTA, two 64 KB query slots,
// two S tiles of 256 columns, each summed by four groups; wide products, because what the issuing thread does between
// two visits is idle time of the tensor core (with 128 columns it was half of it).
// Measured, 32 / 8 heads of 128: last 32 queries of 100003 tokens 194 us (keys alone 32 us at the copy rate; the 11 us
// a key tile takes are the latency of its steps: load, turn, product, sum), all queries of 6001 tokens 462 us (the
// three products 273 us at the tensor peak; tensor pipe 70% busy).
#pragma once
#include <type_traits>

#include "common.cuh"
#include "decode.cuh"
#include "packed.cuh"
#include "prefill_tc.cuh"
#include "prefill_tc2.cuh"

namespace bf {

namespace kw {
constexpr int QROWS = 4;  // query rows a CTA of weights_query_kernel
constexpr uint32_t HALF = 16384;    // 128 rows of 64 fp16 values
constexpr int NSLOT = 2;            // query tiles in the ring
constexpr int NROW = 4;             // rows of log-sum-exps in shared memory
// S tiles in tensor memory; summing groups of four warps; groups that share a visit, each a range of its columns
template <int QT>
constexpr int buffers() { return QT == 64 ? 4 : 2; }
template <int QT>
constexpr int groups() { return QT == 64 ? 2 : 4; }
template <int QT>
constexpr int sharing() { return QT == 64 ? 1 : 4; }
template <int QT>
constexpr int threads() { return groups<QT>() * 128 + 64; }
}  // namespace kw

// A sequence's angle tables. Of pairs 8 c + 2 e and 8 c + 2 e + 1, at [form][e][c] (so that the threads of a row
// read consecutive 16-byte words): turn fractions {hi, lo, hi, lo} of a position, and {cos, cos, sin, sin} of the
// angle between rows ROW_STEP apart, in the original and the long-range form.
template <int P>
struct AngleTables {
  float4 step[2][4][P / 8], turn[2][4][P / 8];
};

struct WeightArgs {
  CUtensorMap qo_hi, qo_lo, ql_hi, ql_lo;  // [hkv][form_rows * g][D] fp16 query forms, box (64, QT, 1), 128-byte swizzle
  const void* q;
  const void* k;      // [T, hkv, D] raw
  const float* lse;   // [hq, T]
  PlanArgs plan;
  int hq, hkv;
  int window_pitch;   // queries set aside for a sequence in the forms; 0: as many as it has rows
  int w0, w_pretrained, mode, window;
  __half* forms[4];   // the forms above, as weights_query_kernel writes them: Qo high, low, Ql high, low
  float* nl;          // [hkv][nl_pitch] -lse * log2(e) of the rows of the forms
  int form_rows;      // queries of the forms (g rows each)
  void* angles;       // [batch] AngleTables of the sequences
  int row_step;       // rows between those of a thread that forms keys
  long long nl_pitch;
  float scale_log2;
  float* kweight;     // [hkv, rows]
  CacheRows rows;
  double omega[64];
};

// Values as fp16 and the fp16 rest; `top` as in to_f16.
__device__ __forceinline__ void split_f16(const float (&x)[8], uint4& hi, uint4& lo, __half2& top) {
  hi = to_f16(x, top);
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w};
  uint32_t l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
    l[e] = pack_f16x2(x[2 * e] - f.x, x[2 * e + 1] - f.y);
  }
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// The same of two values in one register pair.
__device__ __forceinline__ void split_pair(uint64_t v, uint32_t& hi, uint32_t& lo, __half2& top) {
  hi = f2_to_f16x2(v);
  const __half2 h = *reinterpret_cast<const __half2*>(&hi);
  top = __hmax2_nan(top, __habs2(h));
  const float2 f = __half22float2(h);
  lo = f2_to_f16x2(f2_sub(v, f2_pack(f.x, f.y)));
}

// Elements 2 e, 2 e + 1 of eight inputs as a register pair.
__device__ __forceinline__ uint64_t pair_of(const Vec8<__nv_bfloat16>& v, int e) { return bf16x2_to_f2((&v.u.x)[e]); }
__device__ __forceinline__ uint64_t pair_of(const Vec8<float>& v, int e) {
  const float4& f = e < 2 ? v.a : v.b;
  return e & 1 ? f2_pack(f.z, f.w) : f2_pack(f.x, f.y);
}

// First query of sequence b in the forms, a multiple of four so that a tile's log-sum-exps start on a 16-byte
// boundary: window_pitch queries a sequence, or the sequence's own rows with room for the rounding.
__device__ __forceinline__ int first_query(const WeightArgs& a, int b, int first) {
  return a.window_pitch ? b * a.window_pitch : (first + 3 * b + 3) & ~3;
}

// Query forms of the rows that count. A CTA takes QROWS of them (the first CTA makes the tile list): as in
// rope_packed_kernel it looks them up, evaluates their angles once, and deals (row, four heads) units to its warps.
template <typename Tin, int D>
__global__ void __launch_bounds__(kPlanThreads) weights_query_kernel(const __grid_constant__ WeightArgs a) {
  constexpr int P = D / 2;
  constexpr int LPR = P / 8;
  constexpr int UNITS = 2;
  struct Row {
    int w, r, p, G, lng;  // query of the forms (-1: none), packed row, position, factor, long-range form wanted
  };
  __shared__ Row s_row[kw::QROWS];
  __shared__ float4 s_cs[kw::QROWS][2][4][LPR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const bool ok = boundaries_ok(a.plan);
  if (blockIdx.x == 0) {
    plan_tiles(a.plan, ok);
    return;
  }
  if (!ok) return;
  // the CTAs share the sequences' angle tables, two of them at a time (a thread a pair and form)
  for (int b = (blockIdx.x - 1) * (kPlanThreads / (2 * P)) + threadIdx.x / (2 * P); b < a.plan.batch;
       b += (gridDim.x - 1) * (kPlanThreads / (2 * P))) {
    const int G = factor_of(a.plan.cu[b + 1] - a.plan.cu[b], a.w_pretrained);
    const int f = threadIdx.x / P % 2, k = threadIdx.x % P;
    const TurnStep t = turn_step(f == 1 && a.mode == 0 ? a.omega[k] / G : a.omega[k]);
    const int m = f == 1 && a.mode != 0 ? a.row_step / G : a.row_step;  // position aliasing: used where G divides it
    float c, s;
    turn_cos_sin(m, static_cast<float>(m), t, c, s);
    AngleTables<P>& to = static_cast<AngleTables<P>*>(a.angles)[b];
    float* step = reinterpret_cast<float*>(&to.step[f][k % 8 / 2][k / 8]) + k % 2 * 2;
    step[0] = __uint_as_float(t.hi);
    step[1] = t.lo;
    float* turn = reinterpret_cast<float*>(&to.turn[f][k % 8 / 2][k / 8]) + k % 2;
    turn[0] = c;
    turn[2] = s;
  }
  const int g = a.hq / a.hkv;
  if (threadIdx.x < kw::QROWS) {
    Row x;
    x.w = -1;
    const int u = (blockIdx.x - 1) * kw::QROWS + threadIdx.x;  // of the windows, or a packed row
    const int b = a.window_pitch ? u / a.window_pitch : u < a.plan.total_rows ? sequence_of(a.plan.cu, a.plan.batch, u) : -1;
    if (b >= 0 && b < a.plan.batch) {
      const int first = a.plan.cu[b], n = a.plan.cu[b + 1] - first, cnt = window_rows(n, a.plan.obs);
      const int i = a.window_pitch ? u % a.window_pitch : u - first - (n - cnt);
      if (i >= 0 && i < cnt) {
        x.w = first_query(a, b, first) + i;
        x.p = n - cnt + i;
        x.r = first + x.p;
        x.G = factor_of(n, a.w_pretrained);
        x.lng = !a.window && has_long_pairs(n, x.G, a.w0);
      }
    }
    s_row[threadIdx.x] = x;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kw::QROWS * 2 * P; i += kPlanThreads) {
    const int rr = i / (2 * P), f = i / P % 2, k = i % P;
    const Row x = s_row[rr];
    if (x.w < 0 || (f == 1 && !x.lng)) continue;
    const double om = a.omega[k];
    float c, s;
    angle_cos_sin(f == 0        ? static_cast<double>(x.p) * om
                  : a.mode == 0 ? static_cast<double>(x.p) * (om / x.G)
                                : static_cast<double>(x.p / x.G) * om,
                  c, s);
    reinterpret_cast<float2*>(&s_cs[rr][f][k % 8 / 2][k / 8])[k % 2] = make_float2(c, s);
  }
  __syncthreads();
  const int grp = lane >> 3, l8 = lane & 7;
  if (l8 >= LPR) return;
  const int k0 = l8 * 8, per_row = (a.hq + 3) / 4, n_units = kw::QROWS * per_row;
  __half2 top = __float2half2_rn(0.f);
  for (int u0 = warp; u0 < n_units; u0 += 8 * UNITS) {
    Vec8<Tin> x1[UNITS], x2[UNITS];
    float lse[UNITS];
    int row_of[UNITS];
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      const int u = u0 + 8 * j, rr = u / per_row, h = u % per_row * 4 + grp;
      row_of[j] = -1;
      if (u >= n_units || h >= a.hq || s_row[rr].w < 0) continue;
      row_of[j] = rr;
      const Tin* src = static_cast<const Tin*>(a.q) + (static_cast<long long>(s_row[rr].r) * a.hq + h) * D;
      x1[j].load(src + k0);
      x2[j].load(src + P + k0);
      lse[j] = l8 == 0 ? a.lse[static_cast<long long>(h) * a.plan.total_rows + s_row[rr].r] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      if (row_of[j] < 0) continue;
      const Row x = s_row[row_of[j]];
      const int h = (u0 + 8 * j) % per_row * 4 + grp, kvh = h / g;
      const long long row = static_cast<long long>(x.w) * g + h % g;  // of this kv head's rows
      if (l8 == 0) a.nl[kvh * a.nl_pitch + row] = -lse[j] * 1.44269504088896340736f;
      const long long at = (static_cast<long long>(kvh) * a.form_rows * g + row) * D;
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        if (f == 1 && !x.lng) break;
        float y1[8], y2[8];
        turn8(x1[j], x2[j], s_cs[row_of[j]][f], l8, y1, y2);
        uint4 hi, lo;
        split_f16(y1, hi, lo, top);
        *reinterpret_cast<uint4*>(a.forms[2 * f] + at + k0) = hi;
        *reinterpret_cast<uint4*>(a.forms[2 * f + 1] + at + k0) = lo;
        split_f16(y2, hi, lo, top);
        *reinterpret_cast<uint4*>(a.forms[2 * f] + at + P + k0) = hi;
        *reinterpret_cast<uint4*>(a.forms[2 * f + 1] + at + P + k0) = lo;
      }
    }
  }
  if (!all_finite(top)) report_status(kDevRange, 90);
}

// 2^x of two values on the FMA pipe: x = n + f with n the nearest integer (Cody and Waite's reduction, the
// rounding done by adding 1.5 2^23), a polynomial of degree 5 in f fitted by weighted least squares to 2^f on
// [-1/2, 1/2] (relative error 2.4e-7 in fp32), and 2^n as an exponent. x is held in [-126, 128] (a NaN stays).
__device__ __forceinline__ uint64_t exp2_fma2(uint64_t x2) {
  float x0, x1;
  f2_unpack(x2, x0, x1);
  asm("max.NaN.f32 %0, %0, 0fC2FC0000;\n\tmin.NaN.f32 %0, %0, 0f43000000;" : "+f"(x0));
  asm("max.NaN.f32 %0, %0, 0fC2FC0000;\n\tmin.NaN.f32 %0, %0, 0f43000000;" : "+f"(x1));
  x2 = f2_pack(x0, x1);
  const uint64_t magic = f2_pack(12582912.f, 12582912.f);
  const uint64_t y = f2_add(x2, magic);
  const uint64_t f = f2_sub(x2, f2_sub(y, magic));
  uint64_t p = f2_pack(1.327647129073739e-3f, 1.327647129073739e-3f);
  p = f2_fma(p, f, f2_pack(9.675540961325169e-3f, 9.675540961325169e-3f));
  p = f2_fma(p, f, f2_pack(5.550713092088699e-2f, 5.550713092088699e-2f));
  p = f2_fma(p, f, f2_pack(2.4022120237350464e-1f, 2.4022120237350464e-1f));
  p = f2_fma(p, f, f2_pack(6.931469440460205e-1f, 6.931469440460205e-1f));
  p = f2_fma(p, f, f2_pack(1.0000001192092896f, 1.0000001192092896f));
  float y0, y1;
  f2_unpack(y, y0, y1);
  const uint64_t e = f2_pack(__uint_as_float((__float_as_uint(y0) << 23) + 0x3f800000u),
                             __uint_as_float((__float_as_uint(y1) << 23) + 0x3f800000u));
  return f2_mul(p, e);
}

template <typename Tin, int D, int QT>
__global__ void __launch_bounds__(kw::threads<QT>(), QT == 64 ? 2 : 1) key_weights_kernel(const __grid_constant__ WeightArgs a) {
  using namespace kw;
  using tc::fence_after;
  using tc::fence_before;
  using tc::mma_commit;
  constexpr int P = D / 2;
  constexpr int NBUF = buffers<QT>(), NG = groups<QT>(), SHARE = sharing<QT>();
  constexpr int SUMMERS = NG * 4;                // summing warps; then the TMA and the MMA warp
  constexpr int COLS = QT / SHARE;               // columns of a visit that a group sums
  constexpr uint32_t KTILE = D / 64 * HALF;      // the key operand: 128 rows
  constexpr uint32_t QHALF = QT * 128;           // 64 dimensions of QT query rows
  constexpr uint32_t QTILE = D / 64 * QHALF;
  constexpr int KS = D / 16;                     // K-steps of a product
  constexpr uint32_t NCOL = NBUF * QT;           // tensor-memory columns
  constexpr uint32_t IDESC = (1u << 4) | (static_cast<uint32_t>(QT / 8) << 17) | (8u << 24);  // f16 x f16 -> f32, 128 x QT
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) float s_nl[NROW][QT];
  __shared__ float s_sum[NG - 1][128];
  __shared__ AngleTables<P> s_angles;
  __shared__ uint64_t q_full[NSLOT], q_empty[NSLOT], s_full[NBUF], s_free[NBUF], nl_full[NROW], nl_free[NROW], k_ready, k_free, drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int idx = static_cast<int>(blockIdx.x);
  // heaviest tiles first over all heads (a head after the other, whose query forms share L2, takes 501 us
  // instead of 462 at 6001 tokens, 4.01 ms instead of 4.12 at 20000)
  const int kvh = idx % a.hkv, rank = idx / a.hkv;
  const PackedTile tile = a.plan.tiles[rank];
  if (rank >= a.plan.head->n_tiles) return;
  const int g = a.hq / a.hkv;
  const int L = tile.n;
  const int cnt = window_rows(L, a.plan.obs), start = L - cnt;  // queries start .. L - 1
  const int j0 = tile.t * 128;
  const int G = factor_of(L, a.w_pretrained);
  const bool lng_pairs = !a.window && has_long_pairs(L, G, a.w0);
  const int w0 = (a.window || lng_pairs) ? a.w0 : kAllLocal;
  const int rows = cnt * g;              // (query, head) rows
  const int qrow = first_query(a, tile.seq, tile.first) * g;  // their first row in the forms
  // Query tile t holds rows QT t .. QT t + QT - 1: queries start + QT t / g .. start + (QT t + QT - 1) / g. Tiles
  // [t_first, t_oe) have local pairs with these keys, tiles [t_lb, n_t) long-range ones; a tile in both is
  // visited under either branch.
  const int n_t = (rows + QT - 1) / QT;
  const int t_first = j0 > start ? static_cast<int>(static_cast<long long>(j0 - start) * g / QT) : 0;
  auto clamp_t = [&](long long x) { return static_cast<int>(min(static_cast<long long>(n_t), max(static_cast<long long>(t_first), x))); };
  const long long x_loc = (static_cast<long long>(w0) + j0 + 127 - start) * g, x_far = (static_cast<long long>(w0) + j0 - start) * g;
  const int t_oe = w0 > 0 ? clamp_t(x_loc > 0 ? (x_loc + QT - 1) / QT : 0) : t_first;
  const int t_lb = lng_pairs ? clamp_t(x_far > 0 ? x_far / QT : 0) : n_t;
  const int n_o = t_oe - t_first, n_l = n_t - t_lb, nv = n_o + n_l;

  // The keys' loads go out first: with 16-bit inputs a thread's rows fit its registers until they are used.
  constexpr int CPR = P / 8;             // threads a row of the key tile, 8 pairs each
  constexpr int ROW_STEP = SUMMERS * 32 / CPR;        // rows between a thread's
  constexpr int RPT = 128 / ROW_STEP;    // rows a thread
  constexpr int RB = sizeof(Tin) == 2 || RPT == 1 ? RPT : RPT / 2;  // of them loaded together
  const int c8 = threadIdx.x % CPR, k0 = c8 * 8, row0 = threadIdx.x / CPR;
  Vec8<Tin> x1[RB], x2[RB];
  auto load_keys = [&](int i0) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int row = row0 + (i0 + i) * ROW_STEP;
      const Tin* src = static_cast<const Tin*>(a.k) + (static_cast<long long>(tile.first + min(j0 + row, L - 1)) * a.hkv + kvh) * D;
      x1[i].load(src + k0);
      x2[i].load(src + P + k0);
    }
  };
  if (warp < SUMMERS && nv > 0) load_keys(0);

  const uint32_t base = smem_u32(smem);
  const uint32_t k_hi = base, k_lo = base + KTILE, ring = base + 2 * KTILE;
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4 * SHARE);
    }
    for (int i = 0; i < NROW; ++i) {
      mbar_init(&nl_full[i], 1);
      mbar_init(&nl_free[i], 4 * SHARE);
    }
    mbar_init(&k_ready, SUMMERS);
    mbar_init(&k_free, 1);
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (threadIdx.x < sizeof(AngleTables<P>) / 16)
    reinterpret_cast<float4*>(&s_angles)[threadIdx.x] =
        reinterpret_cast<const float4*>(static_cast<const AngleTables<P>*>(a.angles) + tile.seq)[threadIdx.x];
  if (warp == SUMMERS + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(NCOL));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base_sh;
  auto tile_of = [&](int v) { return v >= n_o ? t_lb + v - n_o : t_first + v; };

  if (warp == SUMMERS) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t used = 0, par = 0, nl_used = 0, nl_par = 0;
      for (int v = 0; v < nv; ++v) {
        const int t = tile_of(v), buf = v % NROW;
        const bool lng = v >= n_o;
        // a log-sum-exp row is free once its last visit has been summed
        if (v >= NROW && !mbar_wait_suspend(&nl_free[buf], (v / NROW - 1) & 1, 100, &s_abort)) break;
        mbar_arrive_expect_tx(&nl_full[buf], QT * 4);
        asm volatile(
            "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                smem_u32(&s_nl[buf][0])),
            "l"(a.nl + kvh * a.nl_pitch + qrow + t * QT), "r"(QT * 4), "r"(smem_u32(&nl_full[buf]))
            : "memory");
        nl_used |= 1u << buf;
        nl_par ^= 1u << buf;
        bool ok = true;
        for (int x = 0; x < 2; ++x) {
          const int n = 2 * v + x, slot = n % NSLOT;
          if (n >= NSLOT && !mbar_wait_suspend(&q_empty[slot], (n / NSLOT - 1) & 1, 101, &s_abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&q_full[slot], QTILE);
          const CUtensorMap* m = lng ? (x == 0 ? &a.ql_hi : &a.ql_lo) : (x == 0 ? &a.qo_hi : &a.qo_lo);
#pragma unroll
          for (int hf = 0; hf < D / 64; ++hf)
            tma_load_3d(smem + (ring - base) + slot * QTILE + hf * QHALF, m, &q_full[slot], 64 * hf, qrow + t * QT, kvh);
          used |= 1u << slot;
          par ^= 1u << slot;
        }
        if (!ok) break;
      }
      // every copy issued has landed before the CTA may exit
      for (int i = 0; i < NSLOT; ++i)
        if (used & (1u << i)) mbar_wait_sleepy(&q_full[i], ((par >> i) & 1u) ^ 1u, 102);
      for (int i = 0; i < NROW; ++i)
        if (nl_used & (1u << i)) mbar_wait_sleepy(&nl_full[i], ((nl_par >> i) & 1u) ^ 1u, 103);
    }
  } else if (warp == SUMMERS + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && nv > 0) {
      const uint64_t dkh = tc::k_desc(k_hi, 0), dkl = tc::k_desc(k_lo, 0), dq0 = tc::k_desc(ring, 0);
      auto product = [&](uint32_t d, uint64_t da, uint64_t db, bool acc) {
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
          tc2::mma_ss(d, da + (((kk >> 2) * HALF + (kk & 3) * 32) >> 4), db + (((kk >> 2) * QHALF + (kk & 3) * 32) >> 4),
                      IDESC, acc || kk > 0);
      };
      // Everything between two visits' products is time the tensor core idles (an MMA is issued only once the one
      // before it has been taken), so the loop keeps its ring positions and phases instead of dividing.
      int buf = 0, slot = 0;
      uint32_t buf_ph = 1, slot_ph = 0;  // phase of a buffer's last release, of a slot's fill
      for (int v = 0; v < nv; ++v) {
        if (v == 0 && !mbar_wait_abortable(&k_ready, 0, 110, &s_abort)) break;
        if (v == n_o && n_o > 0 && !mbar_wait_abortable(&k_ready, 1, 111, &s_abort)) break;
        if (v >= NBUF && !mbar_wait_abortable(&s_free[buf], buf_ph, 112, &s_abort)) break;
        if (!mbar_wait_abortable(&q_full[slot], slot_ph, 113, &s_abort)) break;
        fence_after();
        const uint32_t d = tmem + buf * QT;
        const uint64_t bh = dq0 + static_cast<uint64_t>(slot * (QTILE >> 4));
        product(d, dkh, bh, false);
        product(d, dkl, bh, true);
        mma_commit(&q_empty[slot]);
        if (++slot == NSLOT) slot = 0, slot_ph ^= 1u;
        if (!mbar_wait_abortable(&q_full[slot], slot_ph, 114, &s_abort)) break;
        fence_after();
        product(d, dkh, dq0 + static_cast<uint64_t>(slot * (QTILE >> 4)), true);
        mma_commit(&q_empty[slot]);
        if (++slot == NSLOT) slot = 0, slot_ph ^= 1u;
        mma_commit(&s_full[buf]);
        if (v == n_o - 1 && n_l > 0) mma_commit(&k_free);
        if (++buf == NBUF) buf = 0, buf_ph ^= 1u;
      }
      mma_commit(&drain);
      mbar_wait(&drain, 0, 115);
    }
  } else {
    // ------------------------------------------------------------ key tile, then sums
    const int group = warp >> 2, quad = warp & 3;
    const int col0 = group % SHARE * COLS;
    const int r = quad * 32 + lane;
    // The key tile under one branch, split in two: a thread has 8 pairs of every ROW_STEP-th row; rows past the
    // sequence are zero. A row's angles follow from those of the row ROW_STEP before by one rotation (a product of
    // complex numbers on packed pairs) where the angle is linear in that step: always but for position aliasing
    // with a G that does not divide it.
    auto form_keys = [&](bool lng, bool loaded) {
      __half2 top = __float2half2_rn(0.f);
      const int d2 = P + k0, f = lng ? 1 : 0;
      const bool alias = lng && a.mode != 0;
      const bool linear = !alias || ROW_STEP % G == 0;
      uint64_t c2[4], s2[4];
#pragma unroll 1
      for (int i0 = 0; i0 < RPT; i0 += RB) {
        if (i0 > 0 || !loaded) load_keys(i0);
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const int row = row0 + (i0 + i) * ROW_STEP, j = j0 + row;
          if (i0 + i == 0 || !linear) {
            const int m = alias ? j / G : j;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 t = s_angles.step[f][e][c8];
              float c[2], s[2];
              turn_cos_sin(m, static_cast<float>(m), TurnStep{__float_as_uint(t.x), t.y}, c[0], s[0]);
              turn_cos_sin(m, static_cast<float>(m), TurnStep{__float_as_uint(t.z), t.w}, c[1], s[1]);
              c2[e] = f2_pack(c[0], c[1]);
              s2[e] = f2_pack(s[0], s[1]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 t = s_angles.turn[f][e][c8];
              const uint64_t tc = f2_pack(t.x, t.y), ts = f2_pack(t.z, t.w);
              const uint64_t nc = f2_sub(f2_mul(c2[e], tc), f2_mul(s2[e], ts));
              s2[e] = f2_fma(s2[e], tc, f2_mul(c2[e], ts));
              c2[e] = nc;
            }
          }
          uint32_t h1[4], l1[4], h2[4], l2[4];
          if (j >= L) {  // its angles stay as they are for the next row
#pragma unroll
            for (int e = 0; e < 4; ++e) h1[e] = l1[e] = h2[e] = l2[e] = 0u;
          } else
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t u = pair_of(x1[i], e), v = pair_of(x2[i], e);
            split_pair(f2_sub(f2_mul(u, c2[e]), f2_mul(v, s2[e])), h1[e], l1[e], top);
            split_pair(f2_fma(v, c2[e], f2_mul(u, s2[e])), h2[e], l2[e], top);
          }
          // element d of a row: half d / 64, 16-byte chunk (d % 64) / 8 of its 128 bytes, swizzled
          const uint32_t o1 = (k0 / 64) * HALF + sw128(row, (k0 % 64) / 8), o2 = (d2 / 64) * HALF + sw128(row, (d2 % 64) / 8);
          *reinterpret_cast<uint4*>(smem + o1) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
          *reinterpret_cast<uint4*>(smem + o2) = make_uint4(h2[0], h2[1], h2[2], h2[3]);
          *reinterpret_cast<uint4*>(smem + KTILE + o1) = make_uint4(l1[0], l1[1], l1[2], l1[3]);
          *reinterpret_cast<uint4*>(smem + KTILE + o2) = make_uint4(l2[0], l2[1], l2[2], l2[3]);
        }
      }
      if (!all_finite(top)) report_status(kDevRange, 91);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_ready);
    };
    // where this thread's key goes, looked up while the products run
    long long at = -1;
    const bool mine = group == 0 && j0 + r < L;
    bool ok = true;
    if (nv > 0) form_keys(n_o == 0, true);
    if (mine) {
      at = cache_row(a.rows, tile.seq, j0 + r, tile.first + j0 + r);
      if (at < 0) report_status(kDevIndex, 92);
    }
    bool switched = n_o == 0 || n_l == 0;  // one branch only
    auto to_long = [&]() {
      // every product with the local form has been computed before it is overwritten
      ok = ok && __all_sync(0xffffffffu, mbar_wait_suspend(&k_free, 0, 120, &s_abort));
      if (ok) form_keys(true, false);
      switched = true;
    };
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float sc = a.scale_log2;
    // Query i sees key j under the local branch from i = j on, under the long-range one from i = j + w0 on: as rows
    // (i - start) g, for this thread's key and for the tile's last and first.
    auto row_of = [&](long long i) { return static_cast<int>(min(max((i - start) * g, 0LL), 0x7fffffffLL)); };
    const int own_seen = row_of(j0 + r), own_far = row_of(static_cast<long long>(j0) + r + w0);
    const int all_seen = row_of(j0 + 127), all_far = row_of(static_cast<long long>(j0) + 127 + w0);
    const int all_near = row_of(static_cast<long long>(j0) + w0);
    float sum = 0.f;
    for (int v = group / SHARE; v < nv && ok; v += NG / SHARE) {
      if (v >= n_o && !switched) to_long();
      if (!ok) break;
      const int t = tile_of(v), buf = v % NBUF, nlr = v % NROW;
      const bool lng = v >= n_o;
      if (!__all_sync(0xffffffffu, mbar_wait_suspend(&nl_full[nlr], (v / NROW) & 1, 121, &s_abort) &&
                                       mbar_wait_suspend(&s_full[buf], (v / NBUF) & 1, 122, &s_abort))) {
        ok = false;
        break;
      }
      fence_after();
      const int r0 = t * QT + col0;  // this group's columns of the visit: rows r0 ..
      // the thread's scores into registers at once: the tensor core gets the S tile back before they are summed
      float s[COLS];
#pragma unroll
      for (int c0 = 0; c0 < COLS; c0 += 32) tc::tmem_ld32(lane_addr + buf * QT + col0 + c0, s + c0);
#pragma unroll
      for (int c0 = 0; c0 < COLS; c0 += 32) tc::wait_ld32(s + c0);
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free[buf]);
      const bool whole = r0 + COLS <= rows && (lng ? r0 >= all_far : r0 >= all_seen && r0 + COLS <= all_near);
      int c_lo = 0, c_hi = COLS;
      if (!whole) {
        c_lo = max((lng ? own_far : own_seen) - r0, 0);
        c_hi = min(COLS, (lng ? rows : min(rows, own_far)) - r0);
      }
      auto add_up = [&](auto masked) {
        const uint64_t sc2 = f2_pack(sc, sc);
        const uint32_t span = c_hi > c_lo ? c_hi - c_lo : 0;
        uint64_t acc[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u] = f2_pack(0.f, 0.f);
        const ulonglong2* nl2 = reinterpret_cast<const ulonglong2*>(&s_nl[nlr][col0]);
#pragma unroll
        for (int c = 0; c < COLS; c += 4) {
          const ulonglong2 nl = nl2[c / 4];
          float p[4];
          f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), sc2, nl.x), p[0], p[1]);
          const uint64_t x23 = f2_fma(f2_pack(s[c + 2], s[c + 3]), sc2, nl.y);
          if (!decltype(masked)::value && c % 16 == 4) {
            // an eighth of the powers on the FMA pipe, about where the ex2 unit and the issue slots are equally busy
            acc[(c / 2) & 3] = f2_add(acc[(c / 2) & 3], f2_pack(fast_exp2(p[0]), fast_exp2(p[1])));
            acc[(c / 2 + 1) & 3] = f2_add(acc[(c / 2 + 1) & 3], exp2_fma2(x23));
            continue;
          }
          f2_unpack(x23, p[2], p[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = fast_exp2(p[e]);
            if (decltype(masked)::value) p[e] = static_cast<uint32_t>(c + e - c_lo) < span ? p[e] : 0.f;
          }
          acc[(c / 2) & 3] = f2_add(acc[(c / 2) & 3], f2_pack(p[0], p[1]));
          acc[(c / 2 + 1) & 3] = f2_add(acc[(c / 2 + 1) & 3], f2_pack(p[2], p[3]));
        }
        float lo, hi;
        f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), lo, hi);
        return lo + hi;
      };
      const float part = whole ? add_up(std::false_type()) : add_up(std::true_type());
      __syncwarp();
      if (lane == 0) mbar_arrive(&nl_free[nlr]);
      sum += part;
    }
    if (!switched && ok) to_long();
    // the groups' sums, in a fixed order
    if (group > 0) s_sum[group - 1][r] = sum;
    asm volatile("bar.sync 1, %0;" ::"n"(SUMMERS * 32) : "memory");
    if (mine && at >= 0 && !*reinterpret_cast<volatile int*>(&s_abort)) {
#pragma unroll
      for (int i = 0; i < NG - 1; ++i) sum += s_sum[i][r];
      a.kweight[static_cast<long long>(kvh) * a.rows.rows + at] = sum;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == SUMMERS + 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(NCOL));
}

template <int D, int QT>
constexpr int key_weights_smem_bytes() {
  return (D / 64) * (2 * static_cast<int>(kw::HALF) + kw::NSLOT * QT * 128);
}

}  // namespace bf
