// Attention weight of cached keys: for every key of a packed batch of prompts, the sum over the last
// `obs` queries of its sequence (those at or after it) and over the heads of its group of
// exp(score - lse_i), with the prefill's log-sum-exps.
//
// One CTA owns 128 keys of one kv head and streams the query tiles that see them: S^T = K Q^T, keys in
// the 128 tensor-memory lanes and 128 queries in the columns. A thread so owns one key, and the column
// sum of the attention matrix is a sum along its own registers: no shuffles, no atomics, and a result
// that does not depend on the order in which CTAs run.
//
// Precision. A single fp16 rounding of the rotated operands moves a score by about 3e-4, and so a weight
// summed from few queries by as much, relative. Each operand is therefore split into an fp16 value and the
// fp16 rest, and S = Kh Qh + Kl Qh + Kh Ql (the term left out is 2^-22): scores exact to about 1e-6.
//
// Keys come raw from global memory and are turned by the softmax warps themselves, once for each branch
// the tile has (the local queries first, then the long-range ones); no rotated copy of k is written. The
// query rows are turned once by weights_query_kernel and arrive by TMA.
//
// Warp roles: warps 0..7 form the key tile and then sum (two groups of four warps, one visit each in
// turn; warp w reads TMEM lanes 32 (w % 4) ..), warp 8 = TMA producer, warp 9 = MMA issuer. A visit is one
// query tile of one head under one branch. Tensor memory holds four S tiles, shared memory the key tile
// (high and low part) and a ring of four query tiles.
#pragma once
#include "common.cuh"
#include "decode.cuh"
#include "packed.cuh"
#include "prefill_tc.cuh"
#include "prefill_tc2.cuh"

namespace bf {

namespace kw {
constexpr int NBUF = 4;   // S tiles in tensor memory, and log-sum-exp rows in shared memory
constexpr int NSLOT = 4;  // query tiles in the ring (two visits: a high and a low part each)
constexpr int NTHREADS = 320;
constexpr uint32_t HALF = 16384;  // 128 rows of 64 fp16 values
}  // namespace kw

struct WeightArgs {
  CUtensorMap qo_hi, qo_lo, ql_hi, ql_lo;  // [hq][Wp][D] fp16 query forms, box (64, 128, 1), 128-byte swizzle
  const void* q;
  const void* k;      // [T, hkv, D] raw
  const float* lse;   // [hq, T]
  const int* cu;
  const PlanHeader* head;
  const int2* tiles;
  const int* qoff;    // [batch + 1] first row of a sequence's queries in the forms
  int batch, total_rows, hq, hkv, max_tiles;
  int obs, w0, w_pretrained, mode, window;
  __half* forms[4];   // the forms above, as weights_query_kernel writes them: Qo high, low, Ql high, low
  float* nl;          // [hq][nl_pitch] -lse * log2(e) of the queries in the forms
  int form_rows, nl_pitch;
  float scale_log2;
  float* kweight;     // [hkv, rows]
  CacheRows rows;
  double omega[64];
};

__device__ __forceinline__ void split_f16(const float (&x)[8], uint4& hi, uint4& lo, bool& fin) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    fin &= f16_ok(x[2 * e]) & f16_ok(x[2 * e + 1]);
    h[e] = pack_f16x2(x[2 * e], x[2 * e + 1]);
    const __half2 v = *reinterpret_cast<const __half2*>(&h[e]);
    const float2 f = __half22float2(v);
    l[e] = pack_f16x2(x[2 * e] - f.x, x[2 * e + 1] - f.y);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// The angles of pairs k0 .. k0 + 7 at position p: original, or long-range with factor G.
__device__ __forceinline__ void angles8(const double* omega, int k0, int p, int G, int mode, bool lng, float (&c)[8],
                                        float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double w = omega[k0 + i];
    angle_cos_sin(!lng ? static_cast<double>(p) * w
                       : mode == 0 ? static_cast<double>(p) * (w / G) : static_cast<double>(p / G) * w,
                  c[i], s[i]);
  }
}

// Query forms of the rows that count: one warp per row of the forms, lanes as in rope_packed_kernel.
template <typename Tin, int D>
__global__ void __launch_bounds__(256) weights_query_kernel(const __grid_constant__ WeightArgs a) {
  constexpr int P = D / 2;
  constexpr int LANES_PER_ROW = P / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int w = blockIdx.x * 8 + warp;
  if (!a.head->ok || w >= a.qoff[a.batch]) return;
  int b = sequence_of(a.qoff, a.batch, w);
  if (b < 0) return;
  const int first = a.cu[b], n = a.cu[b + 1] - first, cnt = window_rows(n, a.obs);
  const int i = w - a.qoff[b];
  if (i >= cnt) return;  // padding up to a multiple of four
  const int p = n - cnt + i, r = first + p;
  const int G = factor_of(n, a.w_pretrained);
  const bool lng = !a.window && has_long_pairs(n, G, a.w0);
  for (int h = lane; h < a.hq; h += 32)
    a.nl[static_cast<long long>(h) * a.nl_pitch + w] =
        -a.lse[static_cast<long long>(h) * a.total_rows + r] * 1.44269504088896340736f;
  const int grp = lane >> 3, l8 = lane & 7;
  if (l8 >= LANES_PER_ROW) return;
  const int k0 = l8 * 8;
  bool fin = true;
  for (int f = 0; f < (lng ? 2 : 1); ++f) {
    float c[8], s[8];
    angles8(a.omega, k0, p, G, a.mode, f == 1, c, s);
    for (int h = grp; h < a.hq; h += 4) {
      const Tin* src = static_cast<const Tin*>(a.q) + (static_cast<long long>(r) * a.hq + h) * D;
      Vec8<Tin> x1, x2;
      x1.load(src + k0);
      x2.load(src + P + k0);
      float y1[8], y2[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = x1.get(e), v = x2.get(e);
        y1[e] = u * c[e] - v * s[e];
        y2[e] = v * c[e] + u * s[e];
      }
      const long long at = (static_cast<long long>(h) * a.form_rows + w) * D;
      uint4 hi, lo;
      split_f16(y1, hi, lo, fin);
      *reinterpret_cast<uint4*>(a.forms[2 * f] + at + k0) = hi;
      *reinterpret_cast<uint4*>(a.forms[2 * f + 1] + at + k0) = lo;
      split_f16(y2, hi, lo, fin);
      *reinterpret_cast<uint4*>(a.forms[2 * f] + at + P + k0) = hi;
      *reinterpret_cast<uint4*>(a.forms[2 * f + 1] + at + P + k0) = lo;
    }
  }
  if (!fin) report_status(kDevRange, 90);
}

template <typename Tin, int D>
__global__ void __launch_bounds__(kw::NTHREADS, 1) key_weights_kernel(const __grid_constant__ WeightArgs a) {
  using namespace kw;
  using tc::fence_after;
  using tc::fence_before;
  using tc::mma_commit;
  constexpr int P = D / 2;
  constexpr uint32_t TILE = D / 64 * HALF;  // one 128-row operand tile
  constexpr int KS = D / 16;                // K-steps of a product
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) float s_nl[NBUF][128];
  __shared__ float s_sum[128];
  __shared__ uint64_t q_full[NSLOT], q_empty[NSLOT], s_full[NBUF], s_free[NBUF], nl_full[NBUF], k_ready, k_free, drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int kvh = static_cast<int>(blockIdx.x) / a.max_tiles, rank = static_cast<int>(blockIdx.x) % a.max_tiles;
  if (rank >= a.head->n_tiles) return;
  const int2 tile = a.tiles[rank];
  const int g = a.hq / a.hkv;
  const int first = a.cu[tile.x], L = a.cu[tile.x + 1] - first;
  const int cnt = window_rows(L, a.obs), start = L - cnt;  // queries start .. L - 1
  const int j0 = tile.y * 128;
  const int G = factor_of(L, a.w_pretrained);
  const bool lng_pairs = !a.window && has_long_pairs(L, G, a.w0);
  const int w0 = (a.window || lng_pairs) ? a.w0 : kAllLocal;
  const int qrow = a.qoff[tile.x];
  // Query tile t holds queries start + 128 t .. + 127. Tiles [t_first, t_oe) have local pairs with these
  // keys, tiles [t_lb, n_t) long-range ones; a tile in both is visited under either branch.
  const int n_t = (cnt + 127) / 128;
  const int t_first = j0 > start ? (j0 - start) / 128 : 0;
  auto tiles_below = [&](long long x) { return static_cast<int>(min(static_cast<long long>(n_t), max(static_cast<long long>(t_first), x > 0 ? (x + 127) / 128 : 0))); };
  const int t_oe = w0 > 0 ? tiles_below(static_cast<long long>(w0) + j0 + 127 - start) : t_first;
  const int t_lb = lng_pairs ? tiles_below(static_cast<long long>(w0) + j0 - 127 - start) : n_t;
  const int n_o = (t_oe - t_first) * g, n_l = (n_t - t_lb) * g, nv = n_o + n_l;

  const uint32_t base = smem_u32(smem);
  const uint32_t k_hi = base, k_lo = base + TILE, ring = base + 2 * TILE;
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&nl_full[i], 1);
    }
    mbar_init(&k_ready, 8);
    mbar_init(&k_free, 1);
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base_sh;
  // tile and head (within the group) of visit v
  auto visit = [&](int v, int& t, int& hg, bool& lng) {
    lng = v >= n_o;
    const int u = lng ? v - n_o : v;
    t = (lng ? t_lb : t_first) + u / g;
    hg = u % g;
  };

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t used = 0, par = 0, nl_used = 0, nl_par = 0;
      for (int v = 0; v < nv; ++v) {
        int t, hg;
        bool lng;
        visit(v, t, hg, lng);
        const int h = kvh * g + hg, buf = v % NBUF;
        // the buffer's log-sum-exp row is free once its last visit has been summed
        if (v >= NBUF && !mbar_wait_abortable(&s_free[buf], (v / NBUF - 1) & 1, 100, &s_abort)) break;
        mbar_arrive_expect_tx(&nl_full[buf], 512);
        asm volatile(
            "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                smem_u32(&s_nl[buf][0])),
            "l"(a.nl + static_cast<long long>(h) * a.nl_pitch + qrow + t * 128), "r"(512), "r"(smem_u32(&nl_full[buf]))
            : "memory");
        nl_used |= 1u << buf;
        nl_par ^= 1u << buf;
        bool ok = true;
        for (int x = 0; x < 2 && ok; ++x) {
          const int n = 2 * v + x, slot = n % NSLOT;
          if (n >= NSLOT && !mbar_wait_abortable(&q_empty[slot], (n / NSLOT - 1) & 1, 101, &s_abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&q_full[slot], TILE);
          const CUtensorMap* m = lng ? (x == 0 ? &a.ql_hi : &a.ql_lo) : (x == 0 ? &a.qo_hi : &a.qo_lo);
#pragma unroll
          for (int hf = 0; hf < D / 64; ++hf)
            tma_load_3d(smem + (ring - base) + slot * TILE + hf * HALF, m, &q_full[slot], 64 * hf, qrow + t * 128, h);
          used |= 1u << slot;
          par ^= 1u << slot;
        }
        if (!ok) break;
      }
      // every copy issued has landed before the CTA may exit
      for (int i = 0; i < NSLOT; ++i)
        if (used & (1u << i)) mbar_wait_sleepy(&q_full[i], ((par >> i) & 1u) ^ 1u, 102);
      for (int i = 0; i < NBUF; ++i)
        if (nl_used & (1u << i)) mbar_wait_sleepy(&nl_full[i], ((nl_par >> i) & 1u) ^ 1u, 103);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && nv > 0) {
      const uint64_t dkh = tc::k_desc(k_hi, 0), dkl = tc::k_desc(k_lo, 0), dq0 = tc::k_desc(ring, 0);
      auto product = [&](uint32_t d, uint64_t da, uint64_t db, bool acc) {
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          const uint64_t step = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
          tc2::mma_ss(d, da + step, db + step, tc::IDESC_QK, acc || kk > 0);
        }
      };
      for (int v = 0; v < nv; ++v) {
        const int buf = v % NBUF, hi = (2 * v) % NSLOT, lo = (2 * v + 1) % NSLOT;
        if (v == 0 && !mbar_wait_abortable(&k_ready, 0, 110, &s_abort)) break;
        if (v == n_o && n_o > 0 && !mbar_wait_abortable(&k_ready, 1, 111, &s_abort)) break;
        if (v >= NBUF && !mbar_wait_abortable(&s_free[buf], (v / NBUF - 1) & 1, 112, &s_abort)) break;
        if (!mbar_wait_abortable(&q_full[hi], ((2 * v) / NSLOT) & 1, 113, &s_abort)) break;
        fence_after();
        const uint32_t d = tmem + buf * 128;
        const uint64_t bh = dq0 + static_cast<uint64_t>(hi * (TILE >> 4)), bl = dq0 + static_cast<uint64_t>(lo * (TILE >> 4));
        product(d, dkh, bh, false);
        product(d, dkl, bh, true);
        mma_commit(&q_empty[hi]);
        if (!mbar_wait_abortable(&q_full[lo], ((2 * v + 1) / NSLOT) & 1, 114, &s_abort)) break;
        fence_after();
        product(d, dkh, bl, true);
        mma_commit(&q_empty[lo]);
        mma_commit(&s_full[buf]);
        if (v == n_o - 1 && n_l > 0) mma_commit(&k_free);
      }
      mma_commit(&drain);
      mbar_wait(&drain, 0, 115);
    }
  } else {
    // ------------------------------------------------------------ key tile, then sums
    const int group = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    // The key tile under one branch, split in two: thread item = (row, 8 pairs); rows past the sequence are zero.
    auto form_keys = [&](bool lng) {
      bool fin = true;
      constexpr int CPR = P / 8;  // items a row
#pragma unroll 1
      for (int it = threadIdx.x; it < 128 * CPR; it += 256) {
        const int row = it / CPR, c8 = it % CPR, k0 = c8 * 8;
        float y1[8], y2[8];
        if (j0 + row < L) {
          const Tin* src = static_cast<const Tin*>(a.k) + (static_cast<long long>(first + j0 + row) * a.hkv + kvh) * D;
          Vec8<Tin> x1, x2;
          x1.load(src + k0);
          x2.load(src + P + k0);
          float c[8], s[8];
          angles8(a.omega, k0, j0 + row, G, a.mode, lng, c, s);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = x1.get(e), v = x2.get(e);
            y1[e] = u * c[e] - v * s[e];
            y2[e] = v * c[e] + u * s[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y1[e] = y2[e] = 0.f;
        }
        // element d of a row: half d / 64, 16-byte chunk (d % 64) / 8 of its 128 bytes, swizzled
        const int d2 = P + k0;
        const uint32_t o1 = (k0 / 64) * HALF + sw128(row, (k0 % 64) / 8), o2 = (d2 / 64) * HALF + sw128(row, (d2 % 64) / 8);
        uint4 hi, lo;
        split_f16(y1, hi, lo, fin);
        *reinterpret_cast<uint4*>(smem + o1) = hi;
        *reinterpret_cast<uint4*>(smem + TILE + o1) = lo;
        split_f16(y2, hi, lo, fin);
        *reinterpret_cast<uint4*>(smem + o2) = hi;
        *reinterpret_cast<uint4*>(smem + TILE + o2) = lo;
      }
      if (!fin) report_status(kDevRange, 91);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_ready);
    };
    bool ok = true;
    if (nv > 0) form_keys(n_o == 0);
    bool switched = n_o == 0 || n_l == 0;  // one branch only
    auto to_long = [&]() {
      // every product with the local form has been computed before it is overwritten
      ok = ok && __all_sync(0xffffffffu, mbar_wait_abortable(&k_free, 0, 120, &s_abort));
      if (ok) form_keys(true);
      switched = true;
    };
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float sc = a.scale_log2;
    float sum = 0.f;
    for (int v = group; v < nv && ok; v += 2) {
      if (v >= n_o && !switched) to_long();
      if (!ok) break;
      int t, hg;
      bool lng;
      visit(v, t, hg, lng);
      const int buf = v % NBUF;
      if (!__all_sync(0xffffffffu, mbar_wait_abortable(&nl_full[buf], (v / NBUF) & 1, 121, &s_abort) &&
                                       mbar_wait_abortable(&s_full[buf], (v / NBUF) & 1, 122, &s_abort))) {
        ok = false;
        break;
      }
      fence_after();
      const int i0 = start + t * 128;
      const int dmin = i0 - (j0 + 127), dmax = i0 + 127 - j0;
      const int valid = min(128, cnt - t * 128);
      const bool masked = dmin < 0 || valid < 128 || (lng ? dmin < w0 : dmax >= w0);
      const int lo = lng ? max(w0, 0) : 0, hi = lng ? 0x7fffffff : w0;
      const int d0 = i0 - j0 - r;  // i - j of column 0
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 32) {
        float s[32];
        tc::tmem_ld32(lane_addr + buf * 128 + c0, s);
        tc::wait_ld();
        const float4* nl4 = reinterpret_cast<const float4*>(&s_nl[buf][c0]);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 nl = nl4[c / 4];
          float p[4] = {fast_exp2(fmaf(s[c], sc, nl.x)), fast_exp2(fmaf(s[c + 1], sc, nl.y)),
                        fast_exp2(fmaf(s[c + 2], sc, nl.z)), fast_exp2(fmaf(s[c + 3], sc, nl.w))};
          if (masked) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int cc = c0 + c + e, d = d0 + cc;
              p[e] = (cc < valid && d >= lo && d < hi) ? p[e] : 0.f;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) part[e] += p[e];
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free[buf]);
      sum += (part[0] + part[1]) + (part[2] + part[3]);
    }
    if (!switched && ok) to_long();
    // the two groups' sums, in a fixed order
    if (group == 1) s_sum[r] = sum;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (group == 0 && j0 + r < L && !*reinterpret_cast<volatile int*>(&s_abort)) {
      const long long at = cache_row(a.rows, tile.x, j0 + r, first + j0 + r);
      if (at < 0)
        report_status(kDevIndex, 92);
      else
        a.kweight[static_cast<long long>(kvh) * a.rows.rows + at] = sum + s_sum[r];
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

template <int D>
constexpr int key_weights_smem_bytes() {
  return (2 + kw::NSLOT) * (D / 64) * static_cast<int>(kw::HALF);
}

}  // namespace bf
