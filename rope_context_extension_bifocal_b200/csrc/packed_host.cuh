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

cudaError_t launch_plan(const int32_t* cu, int batch, int total_rows, int max_len, int obs, bf::PlanHeader* head,
                        int2* tiles, int max_tiles, int* qoff, cudaStream_t st) {
  bf::PlanArgs a{};
  a.cu = cu;
  a.batch = batch;
  a.total_rows = total_rows;
  a.max_len = max_len;
  a.obs = obs;
  a.head = head;
  a.tiles = tiles;
  a.max_tiles = max_tiles;
  a.qoff = qoff;
  return launch_pdl(bf::packed_plan_kernel, dim3(1), dim3(1024), 0, st, a);
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
  w.qo = w.tiles + align256(static_cast<size_t>(w.max_tiles) * sizeof(int2));
  w.ql = w.qo + qbytes;
  w.ko = w.ql + qbytes;
  w.kl = w.ko + kbytes;
  w.vb = w.kl + kbytes;
  w.total = w.vb + (dtype == BF_DTYPE_FP32 ? kbytes : 0);
  return w;
}

template <int D, bool BIF>
cudaError_t launch_packed_mma(const bf::AttnArgs& a, int max_tiles, cudaStream_t st) {
  constexpr int smem = bf::attn_mma_smem_bytes<D, BIF>();
  auto kern = bf::attn_mma_kernel<D, BIF, true>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3(max_tiles, a.hq), bf::mma_cfg::WARPS * 32, smem, st>>>(a);
  return cudaGetLastError();
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
  const bool tc2 = tc2_path(p);
  if (window && !tc2) return BF_ERR_UNSUPPORTED;
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
  const int64_t per_tile = tc2 ? p->hq / 2 : p->hq;
  if (lay.max_tiles * per_tile > 0x7fffffffLL || p->hq > 65535) return BF_ERR_UNSUPPORTED;
  const int max_tiles = static_cast<int>(lay.max_tiles);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int D = p->head_dim;
  auto* head = reinterpret_cast<bf::PlanHeader*>(ws);
  auto* tiles = reinterpret_cast<int2*>(ws + lay.tiles);

  // 1. the tile list
  if (launch_plan(cu_seqlens, batch, total_rows, max_len, 0, head, tiles, max_tiles, nullptr, st) != cudaSuccess)
    return BF_ERR_CUDA;

  // 2. the RoPE pass: operand forms and cache rows
  const Rope rope = make_rope(p->rope_theta, D, 1);
  bf::PackedRopeArgs pa{};
  pa.q = q;
  pa.k = k;
  pa.v = v;
  pa.cu = cu_seqlens;
  pa.head = head;
  pa.batch = batch;
  pa.total_rows = total_rows;
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
  const dim3 pgrid(static_cast<unsigned>((static_cast<int64_t>(total_rows) + 7) / 8));
  cudaError_t e;
  if (dtype == BF_DTYPE_BF16)
    e = D == 128 ? launch_pdl(bf::rope_packed_kernel<bf16, 128>, pgrid, dim3(256), 0, st, pa)
                 : launch_pdl(bf::rope_packed_kernel<bf16, 64>, pgrid, dim3(256), 0, st, pa);
  else
    e = D == 128 ? launch_pdl(bf::rope_packed_kernel<float, 128>, pgrid, dim3(256), 0, st, pa)
                 : launch_pdl(bf::rope_packed_kernel<float, 64>, pgrid, dim3(256), 0, st, pa);
  if (e != cudaSuccess) return BF_ERR_CUDA;

  // 3. attention. The two-branch kernel only when some sequence may be longer than both the
  // pretrained window and w0; one without long-range pairs runs it with every pair local
  const void* vsrc = dtype == BF_DTYPE_FP32 ? static_cast<const void*>(ws + lay.vb) : v;
  const bool bif = !window && factor(max_len, p->w_pretrained) > 1 && p->w0 < max_len;
  bf::PackedTiles pt{};
  pt.head = head;
  pt.tiles = tiles;
  pt.cu = cu_seqlens;
  pt.max_tiles = max_tiles;
  pt.total_rows = total_rows;
  pt.w_pretrained = p->w_pretrained;
  if (tc2) {
    bf::Tc2Args ta;
    std::memset(&ta, 0, sizeof(ta));
    if (!make_k_map(&ta.qo_map, pa.Qo, total_rows, p->hq) || !make_k_map(&ta.ql_map, pa.Ql, total_rows, p->hq) ||
        !make_k_map(&ta.ko_map, pa.Ko, total_rows, p->hkv) || !make_k_map(&ta.kl_map, pa.Kl, total_rows, p->hkv) ||
        !make_v_map(&ta.v_map, vsrc, total_rows, p->hkv, 1))
      return BF_ERR_CUDA;
    ta.out = static_cast<bf16*>(out);
    ta.lse = lse;
    ta.hq = p->hq;
    ta.hkv = p->hkv;
    ta.batch = 1;
    ta.w0 = p->w0;
    ta.scale_log2 = scale_log2(p);
    ta.packed = pt;
    constexpr int smem = bf::attn_tc2_smem_bytes();
    auto kern = window ? bf::attn_tc2_kernel<bf::tc2::KIND_WINDOW, false, true>
                : bif  ? bf::attn_tc2_kernel<bf::tc2::KIND_BIFOCAL, false, true>
                       : bf::attn_tc2_kernel<bf::tc2::KIND_PLAIN, false, true>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) {
      kern<<<static_cast<unsigned>(max_tiles * per_tile), bf::tc2::NTHREADS2, smem, st>>>(ta);
      e = cudaGetLastError();
    }
  } else if (D == 128) {
    bf::TcArgs ta;
    std::memset(&ta, 0, sizeof(ta));
    if (!make_k_map(&ta.ko_map, pa.Ko, total_rows, p->hkv) || !make_k_map(&ta.kl_map, pa.Kl, total_rows, p->hkv) ||
        !make_v_map(&ta.v_map, vsrc, total_rows, p->hkv, 1))
      return BF_ERR_CUDA;
    ta.Qo = pa.Qo;
    ta.Ql = pa.Ql;
    ta.out = static_cast<bf16*>(out);
    ta.lse = lse;
    ta.hq = p->hq;
    ta.hkv = p->hkv;
    ta.w0 = p->w0;
    ta.scale_log2 = scale_log2(p);
    ta.packed = pt;
    constexpr int smem = bf::attn_tc_smem_bytes();
    auto kern = bif ? bf::attn_tc_kernel<true, true> : bf::attn_tc_kernel<false, true>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) {
      kern<<<static_cast<unsigned>(max_tiles * per_tile), bf::tc::NTHREADS, smem, st>>>(ta);
      e = cudaGetLastError();
    }
  } else {
    bf::AttnArgs aa{};
    aa.Qo = pa.Qo;
    aa.Ql = pa.Ql;
    aa.Ko = pa.Ko;
    aa.Kl = pa.Kl;
    aa.V = static_cast<const bf16*>(vsrc);
    aa.v_row_stride = static_cast<long long>(p->hkv) * D;
    aa.out = static_cast<bf16*>(out);
    aa.lse = lse;
    aa.hq = p->hq;
    aa.hkv = p->hkv;
    aa.w0 = p->w0;
    aa.scale_log2 = scale_log2(p);
    aa.packed = pt;
    e = bif ? launch_packed_mma<64, true>(aa, max_tiles, st) : launch_packed_mma<64, false>(aa, max_tiles, st);
  }
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

}  // extern "C"
