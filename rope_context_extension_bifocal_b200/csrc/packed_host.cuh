// Host side of the packed-prompt and cache-eviction operators: validation, workspace layout and
// launches. Included by bifocal_lib.cu (same translation unit as the other entry points).
#pragma once

namespace {

// ------------------------------------------------------------------ shared by the operators
// Cache rows of a call: dense (block_table null: cache row = packed row) or paged.
bf_status_t make_cache_rows(int64_t cache_rows, int32_t page_size, const int32_t* block_table, int32_t max_pages,
                            bf::CacheRows* r) {
  std::memset(r, 0, sizeof(*r));
  if (cache_rows < 1 || cache_rows > 0x7fffffffLL) return BF_ERR_INVALID;
  r->rows = static_cast<int>(cache_rows);
  if (!block_table) return BF_OK;
  if (!aligned(block_table, 4) || max_pages < 1 || page_size < 1 || cache_rows % page_size) return BF_ERR_INVALID;
  r->block_table = block_table;
  r->max_pages = max_pages;
  r->page_size = page_size;
  r->pool_pages = static_cast<int>(cache_rows / page_size);
  r->page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page_size == 1 << i) r->page_shift = i;
  return BF_OK;
}

int64_t packed_max_tiles(int64_t total_rows, int64_t batch) {
  return total_rows / 128 + std::min(batch, total_rows);
}

bf_status_t check_packed(int32_t dtype, int32_t batch, int32_t total_rows, int32_t max_len, const bf_params_t* p) {
  const bf_status_t s = check_params(p, true);
  if (s != BF_OK) return s;
  if (batch < 1 || total_rows < 1 || max_len < 1) return BF_ERR_INVALID;
  if (dtype != BF_DTYPE_BF16 && dtype != BF_DTYPE_FP32) return BF_ERR_UNSUPPORTED;
  if ((p->flags & BF_FLAG_WINDOW) && p->w0 < 1) return BF_ERR_INVALID;
  if (p->flags & BF_FLAG_MMA_SYNC) return BF_ERR_UNSUPPORTED;
  return BF_OK;
}

bf::PlanArgs make_plan(const int32_t* cu, int batch, int total_rows, int max_len, int obs, uint8_t* ws, size_t tiles,
                       int max_tiles) {
  bf::PlanArgs a{};
  a.cu = cu;
  a.batch = batch;
  a.total_rows = total_rows;
  a.max_len = max_len;
  a.obs = obs;
  a.head = reinterpret_cast<bf::PlanHeader*>(ws);
  a.tiles = reinterpret_cast<bf::PackedTile*>(ws + tiles);
  a.max_tiles = max_tiles;
  return a;
}

// ------------------------------------------------------------------ packed prefill
struct PackedLayout {
  size_t tiles, qo, ql, ko, kl, vb, total;
  int64_t max_tiles;
};

PackedLayout packed_layout(int dtype, int batch, int T, const bf_params_t* p) {
  PackedLayout w{};
  w.max_tiles = packed_max_tiles(T, batch);
  const size_t qbytes = align256(static_cast<size_t>(T) * p->hq * p->head_dim * 2);
  const size_t kbytes = align256(static_cast<size_t>(T) * p->hkv * p->head_dim * 2);
  w.tiles = 256;
  w.qo = w.tiles + align256(static_cast<size_t>(w.max_tiles) * sizeof(bf::PackedTile));
  w.ql = w.qo + qbytes;
  w.ko = w.ql + qbytes;
  w.kl = w.ko + kbytes;
  w.vb = w.kl + kbytes;
  w.total = w.vb + (dtype == BF_DTYPE_FP32 ? kbytes : 0);
  return w;
}

// Operand forms [heads][rows][D] fp16, box (64, box_rows, 1), 128B swizzle.
bool make_form_map(CUtensorMap* map, const void* base, int64_t rows, int heads, int D, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(heads)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(rows) * D * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Values [rows][hkv][D] bf16, box (64, 1, 128), 128B swizzle.
bool make_value_map(CUtensorMap* map, const void* base, int64_t rows, int hkv, int D) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(hkv), static_cast<cuuint64_t>(rows), 1};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(hkv) * D * 2,
                           static_cast<cuuint64_t>(rows) * hkv * D * 2};
  cuuint32_t box[4] = {64, 1, 128, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <typename Args>
cudaError_t launch_packed(void (*kern)(const Args), int64_t ctas, int threads, int smem, const Args& args, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(threads), smem, st, args);
}

// The ping-pong kernel (even groups) and the single-tile kernel (odd ones), for either head size.
template <int D>
cudaError_t launch_packed_tc2(bool window, bool bif, const bf::Tc2Args& a, int64_t ctas, cudaStream_t st) {
  using namespace bf::tc2;
  auto kern = window ? bf::attn_tc2_kernel<KIND_WINDOW, false, true, D>
              : bif  ? bf::attn_tc2_kernel<KIND_BIFOCAL, false, true, D>
                     : bf::attn_tc2_kernel<KIND_PLAIN, false, true, D>;
  return launch_packed(kern, ctas, NTHREADS2, bf::attn_tc2_smem_bytes(), a, st);
}
template <int D>
cudaError_t launch_packed_tc(bool bif, const bf::TcArgs& a, int64_t ctas, cudaStream_t st) {
  auto kern = bif ? bf::attn_tc_kernel<true, true, D> : bf::attn_tc_kernel<false, true, D>;
  return launch_packed(kern, ctas, bf::tc::NTHREADS, bf::attn_tc_smem_bytes(), a, st);
}

template <typename Tin, int D>
cudaError_t launch_rope_packed(const bf::PackedRopeArgs& a, cudaStream_t st) {
  constexpr int rows = bf::kRopeRows;
  return launch_pdl(bf::rope_packed_kernel<Tin, D>,
                    dim3(static_cast<unsigned>((static_cast<int64_t>(a.plan.total_rows) + rows - 1) / rows + 1)),
                    dim3(bf::kPlanThreads), 0, st, a);
}

bf_status_t prefill_packed_impl(const void* q, const void* k, const void* v, int32_t dtype, int32_t total_rows,
                                int32_t batch, const int32_t* cu_seqlens, int32_t max_len, const bf_params_t* p,
                                void* out, float* lse, void* kcache, void* vcache, int32_t* kpos, int64_t cache_rows,
                                int32_t page_size, const int32_t* block_table, int32_t max_pages, void* workspace,
                                size_t ws_bytes, void* stream) {
  bf_status_t s = check_packed(dtype, batch, total_rows, max_len, p);
  if (s != BF_OK) return s;
  if (!q || !k || !v || !cu_seqlens || !out) return BF_ERR_INVALID;
  const size_t align_in = dtype == BF_DTYPE_FP32 ? 32 : 16;
  if (!aligned(q, align_in) || !aligned(k, align_in) || !aligned(v, align_in) || !aligned(out, 16) ||
      !aligned(cu_seqlens, 4) || (lse && !aligned(lse, 4)))
    return BF_ERR_INVALID;
  const bool window = (p->flags & BF_FLAG_WINDOW) != 0;
  // Even groups: two heads of a group a CTA, in the ping-pong kernel (whole call, 32 / 8 heads of 128: 64 prompts of 128
  // rows 126 us, with the single-tile kernel 161; 4 of 1000 rows 97 and 110; one of 1000, too few CTAs for the GPU, 33
  // and 31)
  const bool even = (p->hq / p->hkv) % 2 == 0;
  if (window && !even) return BF_ERR_UNSUPPORTED;
  bf::CacheRows rows{};
  if (kcache || vcache || kpos) {
    if (!kcache || !vcache || !aligned(kcache, 16) || !aligned(vcache, 16) || (kpos && !aligned(kpos, 4)))
      return BF_ERR_INVALID;
    s = make_cache_rows(cache_rows, page_size, block_table, max_pages, &rows);
    if (s != BF_OK) return s;
    if (block_table ? static_cast<int64_t>(max_pages) * page_size < max_len : cache_rows < total_rows)
      return BF_ERR_INVALID;
  }
  const PackedLayout lay = packed_layout(dtype, batch, total_rows, p);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < lay.total) return BF_ERR_WORKSPACE;
  const int64_t per_tile = even ? p->hq / 2 : p->hq;
  if (lay.max_tiles * per_tile > 0x7fffffffLL || p->hq > 65535) return BF_ERR_UNSUPPORTED;
  const int max_tiles = static_cast<int>(lay.max_tiles);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int D = p->head_dim;

  // 1. the RoPE pass: operand forms and cache rows; its first CTA makes the tile list
  const Rope rope = make_rope(p->rope_theta, D, 1);
  bf::PackedRopeArgs pa{};
  pa.q = q;
  pa.k = k;
  pa.v = v;
  pa.plan = make_plan(cu_seqlens, batch, total_rows, max_len, 0, ws, lay.tiles, max_tiles);
  pa.hq = p->hq;
  pa.hkv = p->hkv;
  pa.w0 = p->w0;
  pa.w_pretrained = p->w_pretrained;
  pa.mode = p->mode;
  pa.window = window ? 1 : 0;
  pa.Qo = reinterpret_cast<__half*>(ws + lay.qo);
  pa.Ql = reinterpret_cast<__half*>(ws + lay.ql);
  pa.Ko = reinterpret_cast<__half*>(ws + lay.ko);
  pa.Kl = reinterpret_cast<__half*>(ws + lay.kl);
  pa.Vb = dtype == BF_DTYPE_FP32 ? reinterpret_cast<bf16*>(ws + lay.vb) : nullptr;
  pa.kcache = static_cast<bf16*>(kcache);
  pa.vcache = static_cast<bf16*>(vcache);
  pa.kpos = kpos;
  pa.rows = rows;
  std::memcpy(pa.omega, rope.omega, sizeof(pa.omega));
  cudaError_t e;
  if (dtype == BF_DTYPE_BF16)
    e = D == 128 ? launch_rope_packed<bf16, 128>(pa, st) : launch_rope_packed<bf16, 64>(pa, st);
  else
    e = D == 128 ? launch_rope_packed<float, 128>(pa, st) : launch_rope_packed<float, 64>(pa, st);
  if (e != cudaSuccess) return BF_ERR_CUDA;

  // 2. attention. The two-branch kernel only when some sequence may be longer than both the
  // pretrained window and w0; one without long-range pairs runs it with every pair local
  const void* vsrc = dtype == BF_DTYPE_FP32 ? static_cast<const void*>(ws + lay.vb) : v;
  const bool bif = !window && factor(max_len, p->w_pretrained) > 1 && p->w0 < max_len;
  bf::PackedTiles pt{};
  pt.head = pa.plan.head;
  pt.tiles = pa.plan.tiles;
  pt.max_tiles = max_tiles;
  pt.total_rows = total_rows;
  pt.w_pretrained = p->w_pretrained;
  CUtensorMap ko, kl, vm;
  if (!make_form_map(&ko, pa.Ko, total_rows, p->hkv, D, 128) || !make_form_map(&kl, pa.Kl, total_rows, p->hkv, D, 128) ||
      !make_value_map(&vm, vsrc, total_rows, p->hkv, D))
    return BF_ERR_CUDA;
  const int64_t ctas = max_tiles * per_tile;
  if (even) {
    bf::Tc2Args ta;
    std::memset(&ta, 0, sizeof(ta));
    if (!make_form_map(&ta.qo_map, pa.Qo, total_rows, p->hq, D, 128) ||
        !make_form_map(&ta.ql_map, pa.Ql, total_rows, p->hq, D, 128))
      return BF_ERR_CUDA;
    ta.ko_map = ko;
    ta.kl_map = kl;
    ta.v_map = vm;
    ta.out = static_cast<bf16*>(out);
    ta.lse = lse;
    ta.hq = p->hq;
    ta.hkv = p->hkv;
    ta.batch = 1;
    ta.w0 = p->w0;
    ta.scale_log2 = scale_log2(p);
    ta.packed = pt;
    e = D == 128 ? launch_packed_tc2<128>(window, bif, ta, ctas, st) : launch_packed_tc2<64>(window, bif, ta, ctas, st);
  } else {
    bf::TcArgs ta;
    std::memset(&ta, 0, sizeof(ta));
    ta.ko_map = ko;
    ta.kl_map = kl;
    ta.v_map = vm;
    ta.Qo = pa.Qo;
    ta.Ql = pa.Ql;
    ta.out = static_cast<bf16*>(out);
    ta.lse = lse;
    ta.hq = p->hq;
    ta.hkv = p->hkv;
    ta.w0 = p->w0;
    ta.scale_log2 = scale_log2(p);
    ta.packed = pt;
    e = D == 128 ? launch_packed_tc<128>(bif, ta, ctas, st) : launch_packed_tc<64>(bif, ta, ctas, st);
  }
  return e == cudaSuccess ? BF_OK : BF_ERR_CUDA;
}

// ------------------------------------------------------------------ decode over kept slots
struct KeptLayout {
  size_t part_o, part_ml, scores, total;
  int n_split, split_len, pitch;
};

// Ranges of slots: about 1024 CTAs in all, by the host's bound of the lengths (four of 128 threads are resident on an SM,
// two with more than four heads a kv head), as long as a range keeps 64 slots, and never more than 512 slots in one, so
// that a batch of unequal lengths fills the GPU evenly (75.6K slots of
// 16 sequences: 112 us; ranges of up to 1024 slots 119 us, of 256 112.5 us, which costs two caches of 104K slots in all 5%).
KeptLayout kept_layout(int batch, int max_len, bool accumulate, const bf_params_t* p) {
  KeptLayout w{};
  const int64_t segs = static_cast<int64_t>(batch) * p->hkv;
  int64_t n = std::max<int64_t>((1024 + segs - 1) / segs, (static_cast<int64_t>(max_len) + 511) / 512);
  n = std::min<int64_t>(n, (static_cast<int64_t>(max_len) + 63) / 64);
  int64_t len = (max_len + n - 1) / n;
  len = (len + 63) / 64 * 64;
  w.split_len = static_cast<int>(len);
  w.n_split = static_cast<int>((max_len + len - 1) / len);
  w.pitch = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(max_len) + 7) / 8 * 8, 0x7fffffff));
  const size_t rows = static_cast<size_t>(batch) * p->hq;
  w.part_ml = align256(rows * w.n_split * p->head_dim * 4);
  w.scores = w.part_ml + align256(rows * w.n_split * 2 * 4);
  w.total = w.scores + (accumulate ? align256(rows * w.pitch * 4) : 0);
  return w;
}

bf_status_t check_kept(int32_t batch, int32_t max_len, const bf_params_t* p) {
  const bf_status_t s = check_params(p, true);
  if (s != BF_OK) return s;
  if (batch < 1 || max_len < 1) return BF_ERR_INVALID;
  if ((p->flags & BF_FLAG_WINDOW) && p->w0 < 1) return BF_ERR_INVALID;
  if (p->hq / p->hkv > bf::kept::MAX_G || batch > 65535 || p->hkv > 65535) return BF_ERR_UNSUPPORTED;
  return BF_OK;
}

// Cache rows [rows][hkv][D] bf16, a box of one stage's slots of one head.
bool make_slot_map(CUtensorMap* map, const void* base, int64_t rows, int hkv, int D) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(hkv), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(hkv) * D * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(D), 1, static_cast<cuuint32_t>(bf::kept::STAGE_BYTES / (4 * D))};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int GP>
cudaError_t launch_kept_g(const bf::KeptArgs& a, int batch, cudaStream_t st) {
  constexpr int smem = bf::kept_smem_bytes<D, GP>();
  auto kern = bf::decode_kept_kernel<D, GP>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.n_split, a.hkv, batch), dim3(bf::kept::WARPS * 32), smem, st, a);
}

template <int D>
cudaError_t launch_kept(const bf::KeptArgs& a, int batch, cudaStream_t st) {
  const int g = a.hq / a.hkv;
  const cudaError_t e = g == 1   ? launch_kept_g<D, 1>(a, batch, st)
                        : g == 2 ? launch_kept_g<D, 2>(a, batch, st)
                        : g <= 4 ? launch_kept_g<D, 4>(a, batch, st)
                                 : launch_kept_g<D, 8>(a, batch, st);
  if (e != cudaSuccess) return e;
  // a CTA a query head, and one every KEPT_FINISH_SLOTS slots whose weights are added
  const int64_t chunks = std::max<int64_t>(g, a.kweight ? (static_cast<int64_t>(a.max_len) + bf::KEPT_FINISH_SLOTS - 1) / bf::KEPT_FINISH_SLOTS : 1);
  return launch_pdl(bf::decode_kept_finish_kernel<D>, dim3(static_cast<unsigned>(chunks), a.hkv, batch),
                    dim3(bf::KEPT_FINISH_THREADS), 0, st, a);
}

bf_status_t decode_kept_impl(const void* q, const void* k_new, const void* v_new, void* kcache, void* vcache,
                             int32_t* kpos, float* kweight, int64_t cache_rows, int32_t page_size,
                             const int32_t* block_table, int32_t max_pages, const int32_t* seq_lens,
                             const int32_t* positions, int32_t max_len, int32_t batch, const bf_params_t* p, void* out,
                             float* lse, void* workspace, size_t ws_bytes, void* stream) {
  bf_status_t s = check_kept(batch, max_len, p);
  if (s != BF_OK) return s;
  if (!q || !k_new || !v_new || !kcache || !vcache || !kpos || !block_table || !seq_lens || !positions || !out)
    return BF_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(kcache, 16) || !aligned(vcache, 16) ||
      !aligned(kpos, 4) || !aligned(seq_lens, 4) || !aligned(positions, 4) || !aligned(out, 16) ||
      (kweight && !aligned(kweight, 4)) || (lse && !aligned(lse, 4)))
    return BF_ERR_INVALID;
  bf::KeptArgs a;
  std::memset(&a, 0, sizeof(a));
  s = make_cache_rows(cache_rows, page_size, block_table, max_pages, &a.rows);
  if (s != BF_OK) return s;
  if (static_cast<int64_t>(max_pages) * page_size < max_len) return BF_ERR_INVALID;
  const KeptLayout lay = kept_layout(batch, max_len, kweight != nullptr, p);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < lay.total) return BF_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const Rope rope = make_rope(p->rope_theta, p->head_dim, 1);
  // A stage's slots share a page, and are one box of the pool, where pages hold whole stages; other page sizes are
  // copied row by row (75.6K slots: 112 us with pages of 64, 133 us with pages of 12).
  a.boxes = page_size % (bf::kept::STAGE_BYTES / (4 * p->head_dim)) == 0 ? 1 : 0;
  if (a.boxes && (!make_slot_map(&a.k_map, kcache, cache_rows, p->hkv, p->head_dim) ||
                  !make_slot_map(&a.v_map, vcache, cache_rows, p->hkv, p->head_dim)))
    return BF_ERR_CUDA;
  a.q = static_cast<const bf16*>(q);
  a.k_new = static_cast<const bf16*>(k_new);
  a.v_new = static_cast<const bf16*>(v_new);
  a.kcache = static_cast<bf16*>(kcache);
  a.vcache = static_cast<bf16*>(vcache);
  a.kpos = kpos;
  a.kweight = kweight;
  a.seq_lens = seq_lens;
  a.positions = positions;
  a.hq = p->hq;
  a.hkv = p->hkv;
  a.w0 = p->w0;
  a.w_pretrained = p->w_pretrained;
  a.mode = p->mode;
  a.window = (p->flags & BF_FLAG_WINDOW) ? 1 : 0;
  a.max_len = max_len;
  a.split_len = lay.split_len;
  a.n_split = lay.n_split;
  a.scale_log2 = scale_log2(p);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(ws + lay.part_ml);
  a.scores = kweight ? reinterpret_cast<float*>(ws + lay.scores) : nullptr;
  a.pitch = lay.pitch;
  a.out = static_cast<bf16*>(out);
  a.lse = lse;
  std::memcpy(a.omega, rope.omega, sizeof(a.omega));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->head_dim == 128 ? launch_kept<128>(a, batch, st) : launch_kept<64>(a, batch, st);
  return e == cudaSuccess ? BF_OK : BF_ERR_CUDA;
}

// ------------------------------------------------------------------ eviction
struct EvictLayout {
  size_t lens, from, to, total;
  int pitch;
};

EvictLayout evict_layout(int batch, int hkv, int max_len, int budget) {
  EvictLayout w{};
  const size_t segs = static_cast<size_t>(batch) * hkv;
  w.pitch = std::min(max_len, budget);
  const size_t list = align256(segs * w.pitch * 4);
  w.lens = align256(segs * 4);
  w.from = w.lens + align256(static_cast<size_t>(batch) * 4);
  w.to = w.from + list;
  w.total = w.to + list;
  return w;
}

bf_status_t check_evict(int32_t batch, int32_t hkv, int32_t head_dim, int32_t max_len, int32_t budget) {
  if (batch < 1 || hkv < 1 || max_len < 1 || budget < 1) return BF_ERR_INVALID;
  if ((head_dim != 64 && head_dim != 128) || batch > 65535 || hkv > 65535) return BF_ERR_UNSUPPORTED;
  return BF_OK;
}

bf_status_t cache_evict_impl(void* kcache, void* vcache, int32_t* kpos, float* kweight, int64_t cache_rows,
                             int32_t page_size, const int32_t* block_table, int32_t max_pages,
                             const int32_t* dst_block_table, int32_t dst_max_pages, const int32_t* seq_lens,
                             const int32_t* positions, int32_t* new_lens, int32_t batch, int32_t hkv, int32_t head_dim,
                             int32_t max_len, int32_t budget, int32_t recent, int32_t sink, void* workspace,
                             size_t ws_bytes, void* stream) {
  bf_status_t s = check_evict(batch, hkv, head_dim, max_len, budget);
  if (s != BF_OK) return s;
  if (!kcache || !vcache || !kpos || !kweight || !block_table || !seq_lens || !positions || !new_lens)
    return BF_ERR_INVALID;
  if (recent < 0 || sink < 0 || static_cast<int64_t>(recent) + sink > budget) return BF_ERR_INVALID;
  if (!aligned(kcache, 16) || !aligned(vcache, 16) || !aligned(kpos, 4) || !aligned(kweight, 4) ||
      !aligned(seq_lens, 4) || !aligned(positions, 4) || !aligned(new_lens, 4))
    return BF_ERR_INVALID;
  bf::EvictArgs a{};
  s = make_cache_rows(cache_rows, page_size, block_table, max_pages, &a.src);
  if (s != BF_OK) return s;
  if (static_cast<int64_t>(max_pages) * page_size < max_len) return BF_ERR_INVALID;
  a.in_place = dst_block_table ? 0 : 1;
  a.dst = a.src;
  const EvictLayout lay = evict_layout(batch, hkv, max_len, budget);
  if (dst_block_table) {
    s = make_cache_rows(cache_rows, page_size, dst_block_table, dst_max_pages, &a.dst);
    if (s != BF_OK) return s;
    if (static_cast<int64_t>(dst_max_pages) * page_size < lay.pitch) return BF_ERR_INVALID;
  }
  if (!workspace || !aligned(workspace, 256) || ws_bytes < lay.total) return BF_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.kcache = static_cast<bf16*>(kcache);
  a.vcache = static_cast<bf16*>(vcache);
  a.kpos = kpos;
  a.kweight = kweight;
  a.seq_lens = seq_lens;
  a.positions = positions;
  a.new_lens = new_lens;
  a.hkv = hkv;
  a.max_len = max_len;
  a.budget = budget;
  a.recent = recent;
  a.sink = sink;
  a.moves = reinterpret_cast<int*>(ws);
  a.lens = reinterpret_cast<int*>(ws + lay.lens);
  a.from = reinterpret_cast<int*>(ws + lay.from);
  a.to = reinterpret_cast<int*>(ws + lay.to);
  a.pitch = lay.pitch;
  // a CTA for every CTA_SLOTS slots, in clusters of up to 8 (a cluster's barrier costs more than a CTA's passes over
  // 16384 keys: 150K slots in 64 segments took 143 us with a CTA for 4096 slots, 40 us so)
  int size = 1;
  while (size < 8 && static_cast<int64_t>(size) * bf::ev::CTA_SLOTS < max_len) size *= 2;
  // the slots of a CTA as the kernel divides them
  const int64_t per_cta = ((static_cast<int64_t>(max_len) + size * bf::ev::WARPS - 1) / (size * bf::ev::WARPS) + 31) / 32 *
                          32 * bf::ev::WARPS;
  a.keys_in_smem = static_cast<int>(std::min<int64_t>(per_cta, bf::ev::MAX_RESIDENT));
  const int smem = a.keys_in_smem * 4;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaFuncSetAttribute(bf::evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       bf::ev::MAX_RESIDENT * 4);
  if (e != cudaSuccess) return BF_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size, hkv, batch);
  cfg.blockDim = dim3(bf::ev::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = size;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, bf::evict_select_kernel, a);
  if (e != cudaSuccess) return BF_ERR_CUDA;
  // rows to move: eight a warp, 64 a CTA; at most about 16384 CTAs, which then take several turns
  const int64_t segs = static_cast<int64_t>(batch) * hkv;
  const int64_t x = std::max<int64_t>(1, std::min<int64_t>((lay.pitch + 63) / 64, (16384 + segs - 1) / segs));
  const dim3 grid(static_cast<unsigned>(x), hkv, batch);
  e = head_dim == 128 ? launch_pdl(bf::evict_move_kernel<128>, grid, dim3(256), 0, st, a)
                      : launch_pdl(bf::evict_move_kernel<64>, grid, dim3(256), 0, st, a);
  return e == cudaSuccess ? BF_OK : BF_ERR_CUDA;
}

// ------------------------------------------------------------------ attention weight of keys
struct WeightLayout {
  size_t tiles, angles, forms, form_bytes, nl, total;
  int64_t max_tiles, rows;  // rows: queries of the forms
  int window_pitch;         // of them a sequence, 0: as many as it has rows
};

WeightLayout weight_layout(int batch, int T, int obs, const bf_params_t* p) {
  WeightLayout w{};
  w.max_tiles = packed_max_tiles(T, batch);
  // a window of obs queries a sequence, or (when that is more) the rows of the sequences themselves
  const int64_t pitch = (static_cast<int64_t>(obs) + 3) / 4 * 4, packed = (static_cast<int64_t>(T) + 3LL * batch + 7) / 4 * 4;
  w.window_pitch = pitch * batch <= packed ? static_cast<int>(pitch) : 0;
  w.rows = w.window_pitch ? pitch * batch : packed;
  w.tiles = 256;
  w.angles = w.tiles + align256(static_cast<size_t>(w.max_tiles) * sizeof(bf::PackedTile));
  w.forms = w.angles + align256(static_cast<size_t>(batch) * (p->head_dim == 128 ? sizeof(bf::AngleTables<64>) : sizeof(bf::AngleTables<32>)));
  w.form_bytes = align256(static_cast<size_t>(w.rows) * p->hq * p->head_dim * 2);
  w.nl = w.forms + 4 * w.form_bytes;
  w.total = w.nl + align256((static_cast<size_t>(w.rows) * (p->hq / p->hkv) + 256) * p->hkv * 4);
  return w;
}

template <typename Tin, int D, int QT>
cudaError_t launch_weights_qt(const bf::WeightArgs& a, cudaStream_t st) {
  constexpr int smem = bf::key_weights_smem_bytes<D, QT>();
  auto kern = bf::key_weights_kernel<Tin, D, QT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(a.plan.max_tiles) * a.hkv), dim3(bf::kw::threads<QT>()), smem, st, a);
}

template <typename Tin, int D>
cudaError_t launch_weights(const bf::WeightArgs& a, int qt, cudaStream_t st) {
  const int64_t units = a.window_pitch ? a.form_rows : a.plan.total_rows;
  const cudaError_t e = launch_pdl(bf::weights_query_kernel<Tin, D>,
                                   dim3(static_cast<unsigned>((units + bf::kw::QROWS - 1) / bf::kw::QROWS + 1)),
                                   dim3(bf::kPlanThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  return qt == 64 ? launch_weights_qt<Tin, D, 64>(a, st) : launch_weights_qt<Tin, D, 256>(a, st);
}

bf_status_t key_weights_impl(const void* q, const void* k, int32_t dtype, const float* lse, int32_t total_rows,
                             int32_t batch, const int32_t* cu_seqlens, int32_t max_len, int32_t obs,
                             const bf_params_t* p, float* kweight, int64_t cache_rows, int32_t page_size,
                             const int32_t* block_table, int32_t max_pages, void* workspace, size_t ws_bytes,
                             void* stream) {
  bf_status_t s = check_packed(dtype, batch, total_rows, max_len, p);
  if (s != BF_OK) return s;
  if (!q || !k || !lse || !cu_seqlens || !kweight || obs < 1) return BF_ERR_INVALID;
  const size_t align_in = dtype == BF_DTYPE_FP32 ? 32 : 16;
  if (!aligned(q, align_in) || !aligned(k, align_in) || !aligned(lse, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(kweight, 4))
    return BF_ERR_INVALID;
  bf::WeightArgs a;
  std::memset(&a, 0, sizeof(a));
  s = make_cache_rows(cache_rows, page_size, block_table, max_pages, &a.rows);
  if (s != BF_OK) return s;
  if (block_table ? static_cast<int64_t>(max_pages) * page_size < max_len : cache_rows < total_rows)
    return BF_ERR_INVALID;
  obs = std::min(obs, max_len);
  const WeightLayout lay = weight_layout(batch, total_rows, obs, p);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < lay.total) return BF_ERR_WORKSPACE;
  const int g = p->hq / p->hkv;
  if (lay.max_tiles * p->hkv > 0x7fffffffLL || lay.rows * g > 0x7ffffe00LL || p->hq > 65535)
    return BF_ERR_UNSUPPORTED;
  // Few rows a key tile: 64-row query tiles, two CTAs an SM. Of 27461 tokens, 4 heads a kv head: 256 rows 89 us (with
  // 256-row tiles 108), 512 rows 129 us (132), 1024 rows 215 us with 64-row tiles and 199 with 256-row ones.
  const int qt = static_cast<int64_t>(obs) * g <= 512 ? 64 : 256;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int D = p->head_dim;
  CUtensorMap* maps[4] = {&a.qo_hi, &a.qo_lo, &a.ql_hi, &a.ql_lo};
  for (int i = 0; i < 4; ++i) {
    a.forms[i] = reinterpret_cast<__half*>(ws + lay.forms + i * lay.form_bytes);
    if (!make_form_map(maps[i], a.forms[i], lay.rows * g, p->hkv, D, qt)) return BF_ERR_CUDA;
  }
  const Rope rope = make_rope(p->rope_theta, D, 1);
  a.q = q;
  a.k = k;
  a.lse = lse;
  a.plan = make_plan(cu_seqlens, batch, total_rows, max_len, obs, ws, lay.tiles, static_cast<int>(lay.max_tiles));
  a.window_pitch = lay.window_pitch;
  a.hq = p->hq;
  a.hkv = p->hkv;
  a.w0 = p->w0;
  a.w_pretrained = p->w_pretrained;
  a.mode = p->mode;
  a.window = (p->flags & BF_FLAG_WINDOW) ? 1 : 0;
  a.angles = ws + lay.angles;
  a.row_step = (qt == 64 ? bf::kw::groups<64>() : bf::kw::groups<256>()) * 128 / (D / 16);
  a.nl = reinterpret_cast<float*>(ws + lay.nl);
  a.form_rows = static_cast<int>(lay.rows);
  a.nl_pitch = lay.rows * g + 256;
  a.scale_log2 = scale_log2(p);
  a.kweight = kweight;
  std::memcpy(a.omega, rope.omega, sizeof(a.omega));
  cudaError_t e;
  if (dtype == BF_DTYPE_BF16)
    e = D == 128 ? launch_weights<bf16, 128>(a, qt, st) : launch_weights<bf16, 64>(a, qt, st);
  else
    e = D == 128 ? launch_weights<float, 128>(a, qt, st) : launch_weights<float, 64>(a, qt, st);
  return e == cudaSuccess ? BF_OK : BF_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t bifocal_prefill_packed_workspace_size(int32_t dtype, int32_t batch, int32_t total_rows, const bf_params_t* p) {
  if (check_packed(dtype, batch, total_rows, 1, p) != BF_OK) return 0;
  return packed_layout(dtype, batch, total_rows, p).total;
}

bf_status_t bifocal_prefill_packed(const void* q, const void* k, const void* v, int32_t dtype, int32_t total_rows,
                                   int32_t batch, const int32_t* cu_seqlens, int32_t max_len, const bf_params_t* p,
                                   void* out, float* lse, void* kcache, void* vcache, int32_t* kpos,
                                   int64_t cache_rows, int32_t page_size, const int32_t* block_table,
                                   int32_t max_pages, void* workspace, size_t ws_bytes, void* stream) {
  return prefill_packed_impl(q, k, v, dtype, total_rows, batch, cu_seqlens, max_len, p, out, lse, kcache, vcache, kpos,
                             cache_rows, page_size, block_table, max_pages, workspace, ws_bytes, stream);
}

size_t bifocal_decode_kept_workspace_size(int32_t batch, int32_t max_len, int32_t accumulate, const bf_params_t* p) {
  if (check_kept(batch, max_len, p) != BF_OK) return 0;
  return kept_layout(batch, max_len, accumulate != 0, p).total;
}

bf_status_t bifocal_decode_kept(const void* q, const void* k_new, const void* v_new, void* kcache, void* vcache,
                                int32_t* kpos, float* kweight, int64_t cache_rows, int32_t page_size,
                                const int32_t* block_table, int32_t max_pages, const int32_t* seq_lens,
                                const int32_t* positions, int32_t max_len, int32_t batch, const bf_params_t* p,
                                void* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  return decode_kept_impl(q, k_new, v_new, kcache, vcache, kpos, kweight, cache_rows, page_size, block_table, max_pages,
                          seq_lens, positions, max_len, batch, p, out, lse, workspace, ws_bytes, stream);
}

size_t bifocal_cache_evict_workspace_size(int32_t batch, int32_t hkv, int32_t max_len, int32_t budget) {
  if (check_evict(batch, hkv, 64, max_len, budget) != BF_OK) return 0;
  return evict_layout(batch, hkv, max_len, budget).total;
}

bf_status_t bifocal_cache_evict(void* kcache, void* vcache, int32_t* kpos, float* kweight, int64_t cache_rows,
                                int32_t page_size, const int32_t* block_table, int32_t max_pages,
                                const int32_t* dst_block_table, int32_t dst_max_pages, const int32_t* seq_lens,
                                const int32_t* positions, int32_t* new_lens, int32_t batch, int32_t hkv,
                                int32_t head_dim, int32_t max_len, int32_t budget, int32_t recent, int32_t sink,
                                void* workspace, size_t ws_bytes, void* stream) {
  return cache_evict_impl(kcache, vcache, kpos, kweight, cache_rows, page_size, block_table, max_pages, dst_block_table,
                          dst_max_pages, seq_lens, positions, new_lens, batch, hkv, head_dim, max_len, budget, recent,
                          sink, workspace, ws_bytes, stream);
}

size_t bifocal_key_weights_workspace_size(int32_t batch, int32_t total_rows, int32_t max_len, int32_t obs,
                                          const bf_params_t* p) {
  if (check_packed(BF_DTYPE_BF16, batch, total_rows, max_len, p) != BF_OK || obs < 1) return 0;
  return weight_layout(batch, total_rows, std::min(obs, max_len), p).total;
}

bf_status_t bifocal_key_weights(const void* q, const void* k, int32_t dtype, const float* lse, int32_t total_rows,
                                int32_t batch, const int32_t* cu_seqlens, int32_t max_len, int32_t obs,
                                const bf_params_t* p, float* kweight, int64_t cache_rows, int32_t page_size,
                                const int32_t* block_table, int32_t max_pages, void* workspace, size_t ws_bytes,
                                void* stream) {
  return key_weights_impl(q, k, dtype, lse, total_rows, batch, cu_seqlens, max_len, obs, p, kweight, cache_rows, page_size,
                          block_table, max_pages, workspace, ws_bytes, stream);
}

}  // extern "C"
