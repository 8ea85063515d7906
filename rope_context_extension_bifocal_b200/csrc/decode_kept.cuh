// Decode over kept slots: a paged cache whose slots no longer are positions.
//
// After an eviction slot s of a kv head holds the key of some position kpos[head, row], another one
// in every head. A step appends the new token at slot n - 1 and attends to all n slots, each key
// under the branch its own position asks for; with kweight it then adds to every slot the attention
// weight its key received, summed over the head's group.
//
// One rotation for both branches. The cache holds R_o(j) k. With q' = R_l(i) q, the long-range score
// is <q', C(j) R_o(j) k> with C(p) = R_l(p) R_o(p)^-1, and the local one
//   <R_o(i) q, R_o(j) k> = <R_l(i) R_o(i)^-1 R_o(i) q, C(i) R_o(j) k> = <q', C(i) R_o(j) k>,
// so every key is turned by C(its position, or the query's when it is local): one form of the query,
// no branch per key, and keys of both kinds may lie in any order. C(p) turns pair k by m(p) c_k,
// with m = p, c_k = w_k (1/G - 1) under frequency interpolation and m = p - floor(p / G), c_k = -w_k
// under position aliasing (angles as in turn_cos_sin).
//
// What bounds it: 4 D bytes of K and V a slot and kv head from HBM, and, next to that, instructions
// (about 80 of a warp a slot and kv head for four query heads at D = 128; a fifth of them are sines and
// cosines, which no table can share since every head has positions of its own). QK^T and PV run on
// packed fp32 FMAs: with at most 8 query rows they cost less than the conversions and the split
// operands that the tensor cores would need to keep scores, and so weights, exact to fp32.
// Measured: 16 sequences of 640 to 8192 slots, 32 / 8 heads of 128 with weights (314 MB): 103 us (3.0 TB/s of 6.55, 61%
// of the issue slots busy) and 14 us for the merge, 112 us the call, where the launches overlap; the same rows held in registers instead of a ring in
// shared memory (8 warps an SM instead of 16) took 190 us.
//
// Work split: a CTA takes a range of slots of one (sequence, kv head), a warp every fourth block of 32 of
// it; D / 8 lanes share a key (4 pairs each). A second kernel merges the ranges and adds the weights.
// Padded to 1, 2, 4 or 8 query heads a kv head (GP).
#pragma once
#include "common.cuh"
#include "packed.cuh"

namespace bf {

namespace kept {
constexpr int WARPS = 4;
constexpr int NK = 4;       // keys a lane group holds at a time
constexpr int STAGES = 3;   // stages of a warp's ring: two on their way while one is used
constexpr int STAGE_BYTES = 4096;
constexpr int MAX_G = 8;    // query heads per kv head (max)
}  // namespace kept

struct KeptArgs {
  CUtensorMap k_map, v_map;    // cache rows [rows][hkv][D], box (D, 1, a stage's slots); with boxes
  int boxes;                   // pages hold whole stages
  const __nv_bfloat16* q;      // [B, hq, D] raw
  const __nv_bfloat16* k_new;  // [B, hkv, D] raw
  const __nv_bfloat16* v_new;
  __nv_bfloat16* kcache;       // [rows, hkv, D]
  __nv_bfloat16* vcache;
  int* kpos;                   // [hkv, rows]
  float* kweight;              // [hkv, rows] or null
  CacheRows rows;
  const int* seq_lens;         // [B] slots with the new token's
  const int* positions;        // [B] position of the new token
  int hq, hkv, w0, w_pretrained, mode, window, max_len;
  int split_len, n_split;
  float scale_log2;
  float* part_o;               // [B, hq, n_split, D] unnormalised
  float* part_ml;              // [B, hq, n_split, 2]: max (log2 domain), sum
  float* scores;               // [B, hq, pitch] log2-domain scores (with kweight)
  int pitch;
  __nv_bfloat16* out;          // [B, hq, D]
  float* lse;                  // [B, hq] or null
  double omega[64];
};

// What a sequence's CTAs agree on.
struct KeptSeq {
  int n, now, G;
  bool ok, rot;
};

__device__ __forceinline__ KeptSeq kept_seq(const KeptArgs& a, int b) {
  KeptSeq s;
  s.n = a.seq_lens[b];
  s.now = a.positions[b];
  s.ok = s.n >= 1 && s.n <= a.max_len && s.now >= 0 && s.now < 0x7fffffff;
  s.G = s.ok ? factor_of(s.now + 1, a.w_pretrained) : 1;
  s.rot = !a.window && s.G > 1 && a.w0 <= s.now;  // some position 0 .. now is in the long-range branch
  return s;
}

__device__ __forceinline__ int far_multiple(int p, int G, int mode) { return mode == 0 ? p : p - p / G; }

// Shared memory of a CTA: the warps' stages; reused for the merge at the end.
template <int D, int GP>
constexpr int kept_smem_bytes() {
  return kept::WARPS * kept::STAGES * kept::STAGE_BYTES > kept::WARPS * GP * D * 4 ? kept::WARPS * kept::STAGES * kept::STAGE_BYTES
                                                                                 : kept::WARPS * GP * D * 4;
}

// Four CTAs on an SM for up to four heads (128 registers a thread), two for eight (their queries and
// accumulators alone are 128).
template <int D, int GP>
__global__ void __launch_bounds__(kept::WARPS * 32, GP <= 4 ? 4 : 2) decode_kept_kernel(const __grid_constant__ KeptArgs a) {
  using namespace kept;
  constexpr int P = D / 2;
  constexpr int LPK = D / 8;        // lanes a key
  constexpr int KPW = 32 / LPK;     // keys side by side in a warp
  constexpr int CH = NK * KPW;      // keys of a warp's stage
  constexpr int SUB = 32 / CH;      // stages of a block of 32 slots
  constexpr int NV = NK * GP;       // scores a lane group reduces
  constexpr int OWN = NV > LPK ? NV / LPK : 1;  // of which a lane keeps this many
  static_assert(CH * D * 4 == STAGE_BYTES, "a stage holds the keys and values of CH slots");
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) float2 sp[WARPS][KPW][NV];  // probabilities, twice each (packed operands)
  __shared__ uint64_t s_full[WARPS * STAGES];          // a warp's stages have landed
  __shared__ float sm[WARPS][GP], sl[WARPS][GP];

  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ll = lane % LPK, kg = lane / LPK;
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int g = a.hq / a.hkv;
  pdl_wait();
  const KeptSeq seq = kept_seq(a, b);
  if (!seq.ok) {
    if (threadIdx.x == 0) report_status(kDevIndex, 70);
    return;
  }
  const int s_beg = split * a.split_len, s_end = min(seq.n, s_beg + a.split_len);
  if (s_beg >= s_end) return;

  // Row and position of this lane's slot of a block of 32 (row -1: past the range, or a bad page)
  const int* trow = a.rows.block_table + static_cast<long long>(b) * a.rows.max_pages;
  const int* kpos = a.kpos + static_cast<long long>(kvh) * a.rows.rows;
  auto lookup = [&](int base, int& row, int& pos) {
    const int slot = base + lane;
    row = -1;
    pos = seq.now;
    if (slot < s_end) {
      const int page = a.rows.page_shift >= 0 ? slot >> a.rows.page_shift : slot / a.rows.page_size;
      const int pg = trow[page];
      if (pg < 0 || pg >= a.rows.pool_pages) {
        report_status(kDevIndex, 71);
      } else {
        row = pg * a.rows.page_size + (slot - page * a.rows.page_size);
        if (slot != seq.n - 1) pos = kpos[row];
      }
    }
  };
  // One stage: the K and V rows of slots CH sub .. of the block whose rows are `row`, as one box each where pages
  // hold whole stages (two instructions of one lane), else row by row (a lane each). Rows that are no slot of the
  // range are whatever is there; they are zeroed when the stage is used.
  uint8_t* stages = smem + warp * STAGES * STAGE_BYTES;
  uint64_t* full = s_full + warp * STAGES;
  auto fill = [&](int stage, int row, int sub) {
    uint8_t* dst = stages + stage * STAGE_BYTES;
    if (a.boxes) {
      const int r = __shfl_sync(0xffffffffu, row, sub * CH);
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[stage], STAGE_BYTES);
        tma_load_3d(dst, &a.k_map, &full[stage], 0, kvh, max(r, 0));
        tma_load_3d(dst + STAGE_BYTES / 2, &a.v_map, &full[stage], 0, kvh, max(r, 0));
      }
    } else {
      const int r = __shfl_sync(0xffffffffu, row, sub * CH + lane % CH);
      if (lane == 0) mbar_arrive_expect_tx(&full[stage], STAGE_BYTES);
      __syncwarp();
      if (lane < 2 * CH) {
        const __nv_bfloat16* src = (lane < CH ? a.kcache : a.vcache) + (static_cast<long long>(max(r, 0)) * a.hkv + kvh) * D;
        asm volatile(
            "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                smem_u32(dst + lane * (2 * D))),
            "l"(src), "r"(2 * D), "r"(smem_u32(&full[stage]))
            : "memory");
      }
    }
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < WARPS * STAGES; ++i) mbar_init(&s_full[i], 1);
    fence_barrier_init();
  }
  __syncthreads();

  int row, pos, nrow, npos;
  int base = s_beg + warp * 32;
  lookup(base, row, pos);
  lookup(base + WARPS * 32, nrow, npos);
  // two stages ahead of the one in use; a stage past the range is not filled
  uint32_t used = 0, par = 0;  // per stage: filled at all, parity of its fills
  auto fill_ahead = [&](int stage, int at, int r, int sub) {
    if (at >= s_end) return;
    fill(stage, r, sub);
    used |= 1u << stage;
    par ^= 1u << stage;
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    if (i < SUB)
      fill_ahead(i, base + i * CH, row, i);
    else
      fill_ahead(i, base + WARPS * 32 + (i - SUB) * CH, nrow, i - SUB);
  }

  // the query heads' rows under R_l(now) (R_o when nothing is long-range), in the log2 domain, and
  // the turn fractions of the correction: this lane's pairs 4 ll .. 4 ll + 3
  uint64_t q2[GP][4];  // packed pairs: x of pairs (0,1), (2,3); y of pairs (0,1), (2,3)
  TurnStep corr[4];
  {
    float c[4], s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double w = a.omega[4 * ll + e];
      const double ang = !seq.rot ? static_cast<double>(seq.now) * w
                         : a.mode == 0 ? static_cast<double>(seq.now) * (w / seq.G)
                                       : static_cast<double>(seq.now / seq.G) * w;
      angle_cos_sin(ang, c[e], s[e]);
      corr[e] = turn_step(a.mode == 0 ? w / seq.G - w : -w);
    }
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
      if (h < g) {
        const __nv_bfloat16* qr = a.q + (static_cast<long long>(b) * a.hq + kvh * g + h) * D + 4 * ll;
        const uint2 u = *reinterpret_cast<const uint2*>(qr), w = *reinterpret_cast<const uint2*>(qr + P);
        const float2 u0 = unpack_bf16x2(u.x), u1 = unpack_bf16x2(u.y), w0 = unpack_bf16x2(w.x), w1 = unpack_bf16x2(w.y);
        const float xr[4] = {u0.x, u0.y, u1.x, u1.y}, yr[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = (xr[e] * c[e] - yr[e] * s[e]) * a.scale_log2;
          y[e] = (yr[e] * c[e] + xr[e] * s[e]) * a.scale_log2;
        }
      }
      q2[h][0] = f2_pack(x[0], x[1]);
      q2[h][1] = f2_pack(x[2], x[3]);
      q2[h][2] = f2_pack(y[0], y[1]);
      q2[h][3] = f2_pack(y[2], y[3]);
    }
  }
  const int m_now = far_multiple(seq.now, seq.G, a.mode);

  uint64_t o2[GP][4];
#pragma unroll
  for (int h = 0; h < GP; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) o2[h][e] = f2_pack(0.f, 0.f);
  // Score idx = n * GP + h of a lane group ends, after the reduction, with lane idx * LPK / NV of it:
  // a lane keeps OWN scores from own0 on (or shares one with the LPK / NV - 1 lanes after it).
  const int own0 = ll * NV / LPK;
  const bool first_copy = NV >= LPK || ll % (LPK / NV > 0 ? LPK / NV : 1) == 0;
  float m_own[OWN], l_own[OWN];  // running maximum (of the whole warp) and own sum, per own score's head
#pragma unroll
  for (int u = 0; u < OWN; ++u) m_own[u] = -INFINITY, l_own[u] = 0.f;
  // lane bits that select the head of a score; the others select the key or a copy
  auto head_bit = [](int mask) { return mask < LPK && mask * NV / LPK >= 1 && mask * NV / LPK < GP; };
  float* score_at = a.scores ? a.scores + (static_cast<long long>(b) * a.hq + kvh * g) * a.pitch : nullptr;

  int stage = 0;
  uint32_t phase = 0;  // parity of the next wait on each stage
  bool ok = true;
  for (; base < s_end && ok; base += WARPS * 32) {
    const bool is_local = seq.now - pos < a.w0;
    const int mult = is_local ? m_now : far_multiple(pos, seq.G, a.mode);
    const unsigned local_mask = __ballot_sync(0xffffffffu, is_local), row_mask = __ballot_sync(0xffffffffu, row >= 0);
#pragma unroll 1
    for (int sub = 0; sub < SUB; ++sub) {
      const int sbase = base + sub * CH;
      if (sbase >= s_end) break;  // warp-uniform: the rest of the last block
      // two stages on: this block's, or the next one's first
      {
        const int ahead = sub + STAGES - 1, to = stage == 0 ? STAGES - 1 : stage - 1;
        if (ahead < SUB)
          fill_ahead(to, base + ahead * CH, row, ahead);
        else
          fill_ahead(to, base + WARPS * 32 + (ahead - SUB) * CH, nrow, ahead - SUB);
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], (phase >> stage) & 1u, 72));
      if (!ok) break;
      phase ^= 1u << stage;
      uint8_t* st = stages + stage * STAGE_BYTES;
      const unsigned rows_here = (row_mask >> (sub * CH)) & ((1u << CH) - 1u);
      const bool append = sbase + CH >= seq.n;
      if (rows_here != (1u << CH) - 1u || append) {
        // Rare: rows past the range or of a bad page are zeroed, and the new token's row is written (unless its
        // page is bad): its key rotated and rounded to the cache's bf16, so that this step uses it as every later one will.
        for (int i = 0; i < CH; ++i)
          if (!((rows_here >> i) & 1u) && lane < 2 * LPK)
            *reinterpret_cast<uint4*>(st + (lane < LPK ? 0 : STAGE_BYTES / 2) + i * (2 * D) + (lane % LPK) * 16) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
        const int i = seq.n - 1 - sbase, new_row = __shfl_sync(0xffffffffu, row, (sub * CH + i) & 31);
        if (i >= 0 && i < CH && new_row >= 0 && lane < LPK) {
          const long long src = (static_cast<long long>(b) * a.hkv + kvh) * D;
          const uint2 u = *reinterpret_cast<const uint2*>(a.k_new + src + 4 * ll);
          const uint2 w = *reinterpret_cast<const uint2*>(a.k_new + src + P + 4 * ll);
          const float2 u0 = unpack_bf16x2(u.x), u1 = unpack_bf16x2(u.y), w0 = unpack_bf16x2(w.x), w1 = unpack_bf16x2(w.y);
          const float xr[4] = {u0.x, u0.y, u1.x, u1.y}, yr[4] = {w0.x, w0.y, w1.x, w1.y};
          float x[4], y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float c, s;
            angle_cos_sin(static_cast<double>(seq.now) * a.omega[4 * ll + e], c, s);
            x[e] = xr[e] * c - yr[e] * s;
            y[e] = yr[e] * c + xr[e] * s;
          }
          const uint2 kx = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
          const uint2 ky = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
          const uint4 v = *reinterpret_cast<const uint4*>(a.v_new + src + 8 * ll);
          *reinterpret_cast<uint2*>(st + i * (2 * D) + ll * 8) = kx;
          *reinterpret_cast<uint2*>(st + i * (2 * D) + D + ll * 8) = ky;
          *reinterpret_cast<uint4*>(st + STAGE_BYTES / 2 + i * (2 * D) + ll * 16) = v;
          const long long at = (static_cast<long long>(new_row) * a.hkv + kvh) * D;
          *reinterpret_cast<uint2*>(a.kcache + at + 4 * ll) = kx;
          *reinterpret_cast<uint2*>(a.kcache + at + P + 4 * ll) = ky;
          *reinterpret_cast<uint4*>(a.vcache + at + 8 * ll) = v;
          if (ll == 0) a.kpos[static_cast<long long>(kvh) * a.rows.rows + new_row] = seq.now;
        }
        fence_proxy_async_smem();  // before the copy that will overwrite the stage
        __syncwarp();
      }
      // scores: this lane's share of each (key, head), then the sum over the key's lanes
      float val[NV];
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        const int i = n * KPW + kg;
        const uint2 kx = *reinterpret_cast<const uint2*>(st + i * (2 * D) + ll * 8);
        const uint2 ky = *reinterpret_cast<const uint2*>(st + i * (2 * D) + D + ll * 8);
        uint64_t x0 = bf16x2_to_f2(kx.x), x1 = bf16x2_to_f2(kx.y), y0 = bf16x2_to_f2(ky.x), y1 = bf16x2_to_f2(ky.y);
        if (seq.rot) {
          const int m = __shfl_sync(0xffffffffu, mult, sub * CH + i);
          const float mf = static_cast<float>(m);
          float c[4], s[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) turn_cos_sin(m, mf, corr[e], c[e], s[e]);
          const uint64_t c0 = f2_pack(c[0], c[1]), c1 = f2_pack(c[2], c[3]), s0 = f2_pack(s[0], s[1]), s1 = f2_pack(s[2], s[3]);
          const uint64_t rx0 = f2_sub(f2_mul(x0, c0), f2_mul(y0, s0)), rx1 = f2_sub(f2_mul(x1, c1), f2_mul(y1, s1));
          y0 = f2_fma(x0, s0, f2_mul(y0, c0));
          y1 = f2_fma(x1, s1, f2_mul(y1, c1));
          x0 = rx0;
          x1 = rx1;
        }
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const uint64_t t = f2_fma(q2[h][0], x0, f2_fma(q2[h][1], x1, f2_fma(q2[h][2], y0, f2_mul(q2[h][3], y1))));
          float lo, hi;
          f2_unpack(t, lo, hi);
          val[n * GP + h] = lo + hi;
        }
      }
      // reduce over the LPK lanes: each halving step hands half of the values to the partner lane
      {
        int cnt = NV;
#pragma unroll
        for (int mask = LPK / 2; mask > 0; mask >>= 1) {
          if (cnt > 1) {
            const bool up = ll & mask;
#pragma unroll
            for (int i = 0; i < NV / 2; ++i)
              if (i < cnt / 2) {
                const float send = up ? val[i] : val[i + cnt / 2], keep = up ? val[i + cnt / 2] : val[i];
                val[i] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
              }
            cnt >>= 1;
          } else {
            val[0] += __shfl_xor_sync(0xffffffffu, val[0], mask);
          }
        }
      }
      // this lane's own scores: key n = idx / GP, head idx % GP
      bool grew = false;
      float alpha[OWN];
#pragma unroll
      for (int u = 0; u < OWN; ++u) {
        const int n = (own0 + u) / GP, h = (own0 + u) % GP, slot = sbase + n * KPW + kg;
        const bool near = (local_mask >> (sub * CH + n * KPW + kg)) & 1u;
        if (slot >= s_end || (a.window && !near)) val[u] = -INFINITY;
        if (score_at && slot < s_end && h < g && first_copy) score_at[static_cast<long long>(h) * a.pitch + slot] = val[u];
        float mx = val[u];
#pragma unroll
        for (int mask = 1; mask < 32; mask <<= 1)
          if (!head_bit(mask)) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, mask));
        const float m_new = fmaxf(m_own[u], mx);
        alpha[u] = m_new == -INFINITY ? 1.f : fast_exp2(m_own[u] - m_new);
        grew |= m_new > m_own[u];
        m_own[u] = m_new;
        const float p = val[u] == -INFINITY ? 0.f : fast_exp2(val[u] - m_new);
        l_own[u] = l_own[u] * alpha[u] + p;
        if (first_copy) sp[warp][kg][own0 + u] = make_float2(p, p);
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float f = __shfl_sync(0xffffffffu, alpha[h % OWN], h * LPK / NV);
          const uint64_t f2 = f2_pack(f, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) o2[h][e] = f2_mul(o2[h][e], f2);
        }
      }
      __syncwarp();
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        const uint4 v = *reinterpret_cast<const uint4*>(st + STAGE_BYTES / 2 + (n * KPW + kg) * (2 * D) + ll * 16);
        const uint64_t v0 = bf16x2_to_f2(v.x), v1 = bf16x2_to_f2(v.y), v2 = bf16x2_to_f2(v.z), v3 = bf16x2_to_f2(v.w);
        uint64_t pp[GP];
        if (GP == 1)
          pp[0] = *reinterpret_cast<const uint64_t*>(&sp[warp][kg][n]);
        else
#pragma unroll
          for (int h = 0; h < GP; h += 2) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(&sp[warp][kg][n * GP + h]);
            pp[h] = t.x;
            pp[h + 1 < GP ? h + 1 : h] = t.y;
          }
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const uint64_t p2 = pp[h];
          o2[h][0] = f2_fma(p2, v0, o2[h][0]);
          o2[h][1] = f2_fma(p2, v1, o2[h][1]);
          o2[h][2] = f2_fma(p2, v2, o2[h][2]);
          o2[h][3] = f2_fma(p2, v3, o2[h][3]);
        }
      }
      __syncwarp();  // sp and the stage are free again
      stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
    row = nrow;
    pos = npos;
    lookup(base + 2 * WARPS * 32, nrow, npos);
  }
  // every copy issued has landed (only an expired wait leaves any), and every warp is done with its stages: the
  // merge reuses them
  if (!ok)
    for (int i = 0; i < STAGES; ++i)
      if (used & (1u << i)) mbar_wait(&full[i], ((par >> i) & 1u) ^ 1u, 73);
  __syncthreads();
  float (*so)[GP][D] = reinterpret_cast<float(*)[GP][D]>(smem);

  // merge: lane groups by shuffles, warps through shared memory in a fixed order
#pragma unroll
  for (int u = 0; u < OWN; ++u) {
    float l = first_copy ? l_own[u] : 0.f;
#pragma unroll
    for (int mask = 1; mask < 32; mask <<= 1)
      if (!head_bit(mask)) l += __shfl_xor_sync(0xffffffffu, l, mask);
    if (own0 + u < GP && kg == 0 && first_copy) {
      sm[warp][own0 + u] = m_own[u];
      sl[warp][own0 + u] = l;
    }
  }
#pragma unroll
  for (int h = 0; h < GP; ++h) {
    float o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) f2_unpack(o2[h][e], o[2 * e], o[2 * e + 1]);
#pragma unroll
    for (int mask = LPK; mask < 32; mask <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], mask);
    if (kg == 0) {
      *reinterpret_cast<float4*>(&so[warp][h][8 * ll]) = make_float4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<float4*>(&so[warp][h][8 * ll + 4]) = make_float4(o[4], o[5], o[6], o[7]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < g * D; i += WARPS * 32) {
    const int h = i / D, d = i % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm[w][h]);
    float acc = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = sm[w][h] == -INFINITY ? 0.f : fast_exp2(sm[w][h] - M);
      acc += so[w][h][d] * f;
      l += sl[w][h] * f;
    }
    const long long part = (static_cast<long long>(b) * a.hq + kvh * g + h) * a.n_split + split;
    a.part_o[part * D + d] = acc;
    if (d == 0) {
      a.part_ml[part * 2] = M;
      a.part_ml[part * 2 + 1] = l;
    }
  }
}

// Merges the ranges' partial results and adds the weights. CTA (x, kv head, sequence): every CTA forms
// the log-sum-exps of the head's group from the partial maxima and sums (a few hundred bytes), writes out and lse
// of the query heads x, x + gridDim.x, .., and the weights of the SLOTS slots from x SLOTS on.
constexpr int KEPT_FINISH_THREADS = 256, KEPT_FINISH_SLOTS = 1024;

template <int D>
__global__ void __launch_bounds__(KEPT_FINISH_THREADS) decode_kept_finish_kernel(const __grid_constant__ KeptArgs a) {
  __shared__ float s_lse2[kept::MAX_G];
  pdl_launch_dependents();
  pdl_wait();
  const int kvh = blockIdx.y, b = blockIdx.z, g = a.hq / a.hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const KeptSeq seq = kept_seq(a, b);
  const long long head0 = static_cast<long long>(b) * a.hq + kvh * g;
  if (!seq.ok) {
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < g * D; i += KEPT_FINISH_THREADS) {
        a.out[head0 * D + i] = __float2bfloat16(__int_as_float(0x7fc00000));
        if (a.lse && i % D == 0) a.lse[head0 + i / D] = __int_as_float(0x7fc00000);
      }
    return;
  }
  const int beg = blockIdx.x * KEPT_FINISH_SLOTS;
  if (blockIdx.x >= g && beg >= seq.n) return;
  const int n_split = (seq.n + a.split_len - 1) / a.split_len;
  if (warp < g) {
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + (head0 + warp) * a.n_split;
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < n_split; i += 32) {
      const float2 x = ml[i];
      const float M = fmaxf(m, x.x);
      if (M > -INFINITY) l = l * fast_exp2(m - M) + x.y * fast_exp2(x.x - M);
      m = M;
    }
#pragma unroll
    for (int mask = 16; mask > 0; mask >>= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m, mask), lo = __shfl_xor_sync(0xffffffffu, l, mask);
      const float M = fmaxf(m, mo);
      if (M > -INFINITY) l = l * fast_exp2(m - M) + lo * fast_exp2(mo - M);
      m = M;
    }
    if (lane == 0) s_lse2[warp] = m + log2f(l);
  }
  __syncthreads();
  // out: the CTAs of a (sequence, kv head) take its query heads in turn; four values a thread, the ranges dealt to
  // the thread groups that share them, summed in a fixed order
  constexpr int Q = D / 4;                         // threads a row
  constexpr int SLICES = KEPT_FINISH_THREADS / Q;  // ranges in flight
  __shared__ float4 s_part[KEPT_FINISH_THREADS];
  const int sl = threadIdx.x / Q, d4 = threadIdx.x % Q;
  for (int h = blockIdx.x; h < g; h += gridDim.x) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + (head0 + h) * a.n_split;
    const float4* src = reinterpret_cast<const float4*>(a.part_o + (head0 + h) * a.n_split * D) + d4;
#pragma unroll 4
    for (int sp = sl; sp < n_split; sp += SLICES) {
      const float4 x = src[static_cast<long long>(sp) * Q];
      const float f = fast_exp2(ml[sp].x - s_lse2[h]);
      acc.x += x.x * f;
      acc.y += x.y * f;
      acc.z += x.z * f;
      acc.w += x.w * f;
    }
    s_part[threadIdx.x] = acc;
    __syncthreads();
    if (sl == 0) {
      for (int i = 1; i < SLICES; ++i) {
        const float4 x = s_part[i * Q + d4];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      *reinterpret_cast<uint2*>(a.out + (head0 + h) * D + 4 * d4) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
      if (a.lse && d4 == 0) a.lse[head0 + h] = s_lse2[h] * 0.69314718055994530942f;
    }
    __syncthreads();
  }
  if (!a.kweight) return;
  // four slots a thread in flight
  const int end = min(seq.n, beg + KEPT_FINISH_SLOTS);
  const float* sc = a.scores + head0 * a.pitch;
  constexpr int U = KEPT_FINISH_SLOTS / KEPT_FINISH_THREADS;
  float w[U], old[U];
  long long at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int slot = beg + u * KEPT_FINISH_THREADS + threadIdx.x;
    at[u] = -1;
    w[u] = old[u] = 0.f;
    if (slot < end) {
      const long long r = cache_row(a.rows, b, slot, 0);
      if (r >= 0) at[u] = static_cast<long long>(kvh) * a.rows.rows + r;
    }
    if (at[u] >= 0 && slot != seq.n - 1) old[u] = a.kweight[at[u]];  // the new token's slot starts at zero
  }
  for (int h = 0; h < g; ++h)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int slot = beg + u * KEPT_FINISH_THREADS + threadIdx.x;
      if (slot < end) w[u] += fast_exp2(sc[static_cast<long long>(h) * a.pitch + slot] - s_lse2[h]);
    }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (at[u] >= 0) a.kweight[at[u]] = old[u] + w[u];
}

}  // namespace bf
