// fd_int4_api.cuh — host side of the 4-bit cache and of the page bookkeeping:
// argument checks and launches.  Part of fd_api.cu, whose helpers it uses; see
// include/fd.h for the contract of every entry point.
#pragma once

namespace {

// The cache that p describes, checked.
fd_status int4_cache(const fd_problem* p, const void* k4, const void* v4, const void* params,
                     fd::Int4Cache* c) {
  if (!p || !k4 || !v4 || !params) return FD_ERR_INVALID_ARGUMENT;
  const fd_status st = check_shape(p->B, p->Hq, p->Hkv, p->D, p->max_len, p->block_size);
  if (st != FD_OK) return st;
  if (p->kv_layout != FD_LAYOUT_HND && p->kv_layout != FD_LAYOUT_NHD) return FD_ERR_INVALID_ARGUMENT;
  if (p->kv_dtype != FD_KV_INT4) return FD_ERR_INVALID_ARGUMENT;
  if (p->max_len > 0x7fffff00) return FD_ERR_INVALID_ARGUMENT;   // lengths are rounded up in int32
  if (p->block_size != 0) {
    if (p->num_blocks < 1 || p->max_blocks_per_seq < 1) return FD_ERR_INVALID_ARGUMENT;
    if (static_cast<long long>(p->max_blocks_per_seq) * p->block_size < p->max_len)
      return FD_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(k4, 16) || !aligned(v4, 16) || !aligned(params, 16)) return FD_ERR_INVALID_ARGUMENT;
  c->k4 = static_cast<uint8_t*>(const_cast<void*>(k4));
  c->v4 = static_cast<uint8_t*>(const_cast<void*>(v4));
  c->params = static_cast<uint8_t*>(const_cast<void*>(params));
  c->planes = p->block_size ? p->num_blocks : p->B;
  c->rows = p->block_size ? p->block_size : p->max_len;
  c->Hkv = p->Hkv;
  c->nhd = p->kv_layout == FD_LAYOUT_NHD;
  return FD_OK;
}

fd_status this_device(int* dev) {
  if (current_device(dev) != FD_OK) return FD_ERR_CUDA;
  return device_is_sm100(*dev);
}

// Launches that may start while the previous kernel of the stream ends (every
// kernel waits for it before its first read).
template <class Kernel, class... Args>
fd_status launch_clusters(Kernel kernel, dim3 grid, int cluster, int threads, size_t smem, fd_stream_t stream,
                          const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}
template <class Kernel, class... Args>
fd_status launch_chained(Kernel kernel, dim3 grid, int threads, size_t smem, fd_stream_t stream,
                         const Args&... args) {
  return launch_clusters(kernel, grid, 1, threads, smem, stream, args...);
}

// Tensor maps of a 4-bit cache, {byte, head, row, plane}: the codes of K and of
// V (a box row is a whole code row, swizzled over its own width) and the
// records (16 bytes a box row).  Coordinates outside the cache read zeros.
struct Int4Maps {
  CUtensorMap k, v, p;
};

fd_status make_int4_map(CUtensorMap* tm, const void* base, int row_bytes, const fd::Int4Cache& c,
                        int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  if (encoder(&enc) != FD_OK) return FD_ERR_CUDA;
  const cuuint64_t rb = static_cast<cuuint64_t>(row_bytes), rows = static_cast<cuuint64_t>(std::max(c.rows, 1));
  cuuint64_t dims[4] = {rb, static_cast<cuuint64_t>(c.Hkv), rows, static_cast<cuuint64_t>(c.planes)};
  cuuint64_t strides[3] = {c.nhd ? rb : rows * rb, c.nhd ? c.Hkv * rb : rb, c.Hkv * rows * rb};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(row_bytes), 1, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle swizzle = row_bytes == 64   ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : row_bytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                       : CU_TENSOR_MAP_SWIZZLE_NONE;
  // Fetching 256 bytes at a time pays where a head's rows are neighbours.  Token-
  // major it fetched other heads' rows (8 x 40,000 tokens in pages of 16: 57.7 us;
  // 50.2 us without, and without evict-first).
  const CUtensorMapL2promotion promotion =
      c.nhd ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides,
                         box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                         promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FD_OK : FD_ERR_CUDA;
}

// The maps depend only on addresses, shape and device: each host thread keeps
// the last few it encoded, as cached_cache_map does.
fd_status cached_int4_maps(Int4Maps* m, const fd::Int4Cache& c, int D, int box_rows, int dev) {
  struct Entry {
    fd::Int4Cache c;
    int D, box_rows, dev;
    Int4Maps maps;
  };
  constexpr int kEntries = 8;
  thread_local Entry entries[kEntries] = {};
  thread_local int next = 0;
  for (const Entry& e : entries) {
    if (e.D == D && e.box_rows == box_rows && e.dev == dev && e.c.k4 == c.k4 && e.c.v4 == c.v4 &&
        e.c.params == c.params && e.c.planes == c.planes && e.c.rows == c.rows && e.c.Hkv == c.Hkv &&
        e.c.nhd == c.nhd) {
      *m = e.maps;
      return FD_OK;
    }
  }
  if (make_int4_map(&m->k, c.k4, D / 2, c, box_rows) != FD_OK ||
      make_int4_map(&m->v, c.v4, D / 2, c, box_rows) != FD_OK ||
      make_int4_map(&m->p, c.params, 16, c, box_rows) != FD_OK)
    return FD_ERR_CUDA;
  entries[next] = Entry{c, D, box_rows, dev, *m};
  next = (next + 1) % kEntries;
  return FD_OK;
}

template <int D, int NB, class SH>
fd_status launch_split_int4(const Int4Maps& m, const fd::Int4DecodeArgs& a, dim3 grid, int dev,
                            fd_stream_t s) {
  using L = fd::Int4Smem<D, NB, SH>;
  auto kern = fd::fd_split_int4_kernel<D, NB, SH>;
  static std::atomic<unsigned long long> attr_ctx[kMaxDevices];   // as launch_split's
  const unsigned long long ctx = current_context_id();
  if (ctx == 0 || attr_ctx[dev].load() != ctx) {
    // The warps' shares of the registers have to be there when it starts.
    cudaFuncAttributes built;
    if (cudaFuncGetAttributes(&built, kern) != cudaSuccess || built.numRegs < fd::kInt4StartRegs)
      return FD_ERR_CUDA;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             L::kDynamicBytes) != cudaSuccess)
      return FD_ERR_CUDA;
    attr_ctx[dev].store(ctx);
  }
  return launch_clusters(kern, grid, a.cluster, (SH::WARPS + fd::kInt4CopyWarps) * 32, L::kDynamicBytes, s,
                         m.k, m.v, m.p, a);
}

// Rows of many parts (on average) are merged by four warps per query head, which
// ask for 64 of them at once; otherwise by one, with more of them resident.
template <int D, int U>
fd_status launch_combine_int4(const fd::Int4DecodeArgs& d, int rows, fd_stream_t s) {
  const int cand = std::min(rows, d.ctas);
  const bool many = d.ctas > 10 * cand;
  const long long warps = static_cast<long long>(cand) * d.heads * d.a.G * (many ? fd::kInt4CombineWarps : 1);
  const dim3 grid(static_cast<unsigned>((warps + fd::kInt4CombineWarps - 1) / fd::kInt4CombineWarps));
  const int threads = fd::kInt4CombineWarps * 32;
  return many ? launch_chained(fd::fd_combine_int4_kernel<D, U, fd::kInt4CombineWarps, 16>, grid, threads, 0, s, d)
              : launch_chained(fd::fd_combine_int4_kernel<D, U, 1, 8>, grid, threads, 0, s, d);
}

// Do two arrays of int32 share memory?
bool overlap(const void* x, size_t nx, const void* y, size_t ny) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b + 4 * ny && b < a + 4 * nx;
}

fd_status check_pages(int B, int block_size, int max_blocks_per_seq, int num_pages) {
  if (B < 1 || B > 65535 || max_blocks_per_seq < 1 || num_pages < 1 || block_size < 1)
    return FD_ERR_INVALID_ARGUMENT;
  if (!is_pow2(block_size) || block_size < 8 || block_size > 256) return FD_ERR_UNSUPPORTED;
  return FD_OK;
}

// One launch expands and writes the state.  When the new state lies over the
// old one and several CTAs read the old, a second launch writes the state.
template <class Kernel>
fd_status launch_pages(Kernel kernel, fd::PageArgs a, long long items, fd_stream_t s) {
  int dev = 0;
  const fd_status st = this_device(&dev);
  if (st != FD_OK) return st;
  int sms = 0;
  if (device_sms(dev, &sms) != FD_OK) return FD_ERR_CUDA;
  const long long per = std::max<long long>(fd::kPageThreads, (items + 2LL * sms - 1) / (2LL * sms));
  const int grid = static_cast<int>(std::max<long long>(1, (items + per - 1) / per));
  const bool in_place = overlap(a.seqlens, a.B, a.seqlens_out, a.B) ||
                        overlap(a.free_count, 1, a.free_count_out, 1);
  a.items_per_cta = static_cast<int>(per);
  a.write_items = true;
  a.write_state = grid == 1 || !in_place;
  fd_status r = launch_chained(kernel, dim3(static_cast<unsigned>(grid)), fd::kPageThreads, 0, s, a);
  if (r == FD_OK && !a.write_state) {
    a.write_items = false;
    a.write_state = true;
    r = launch_chained(kernel, dim3(1), fd::kPageThreads, 0, s, a);
  }
  return r;
}

}  // namespace

extern "C" {

fd_status fd_append_int4(const fd_problem* p, int n_tokens, const void* k_new, int64_t k_stride,
                         const void* v_new, int64_t v_stride, const int64_t* slots, void* k4,
                         void* v4, void* params, fd_stream_t stream) {
  fd::AppendArgs a{};
  const fd_status st = int4_cache(p, k4, v4, params, &a.c);
  if (st != FD_OK) return st;
  if (n_tokens < 0 || !k_new || !v_new || !slots) return FD_ERR_INVALID_ARGUMENT;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(slots, 8)) return FD_ERR_INVALID_ARGUMENT;
  // Tokens start 16 bytes aligned and do not overlap.
  const int64_t row = static_cast<int64_t>(p->Hkv) * p->D;
  if (k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride < row || v_stride < row)
    return FD_ERR_INVALID_ARGUMENT;
  const long long rows = static_cast<long long>(n_tokens) * p->Hkv;
  if (rows > 0x7fffffffLL) return FD_ERR_INVALID_ARGUMENT;
  if (n_tokens == 0 || a.c.rows == 0) return FD_OK;
  int dev = 0;
  const fd_status arch = this_device(&dev);
  if (arch != FD_OK) return arch;
  a.k = static_cast<const __nv_bfloat16*>(k_new);
  a.v = static_cast<const __nv_bfloat16*>(v_new);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.n_rows = static_cast<uint32_t>(rows);
  while ((1 << a.head_shift) < p->Hkv) ++a.head_shift;     // Granlund and Montgomery's division
  a.head_mul = static_cast<uint32_t>(((1ull << (31 + a.head_shift)) + p->Hkv - 1) / p->Hkv);
  a.log2_rows = p->block_size ? ilog2(p->block_size) : -1;
  const long long per = 256 / (p->D / 16);
  const dim3 g(static_cast<unsigned>((rows + per - 1) / per));
  return p->D == 128 ? launch_chained(fd::fd_append_int4_kernel<128>, g, 256, 0, stream, a)
                     : launch_chained(fd::fd_append_int4_kernel<64>, g, 256, 0, stream, a);
}

fd_status fd_expand_int4(const fd_problem* p, const void* k4, const void* v4, const void* params,
                         const int32_t* seqlens, const int32_t* block_table, void* k_out,
                         void* v_out, fd_stream_t stream) {
  fd::ExpandArgs a{};
  const fd_status st = int4_cache(p, k4, v4, params, &a.c);
  if (st != FD_OK) return st;
  if (!k_out || !v_out || (p->block_size != 0) != (block_table != nullptr)) return FD_ERR_INVALID_ARGUMENT;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(seqlens, 4) || !aligned(block_table, 4))
    return FD_ERR_INVALID_ARGUMENT;
  if (p->max_len == 0) return FD_OK;
  int dev = 0;
  const fd_status arch = this_device(&dev);
  if (arch != FD_OK) return arch;
  a.seqlens = seqlens;
  a.block_table = block_table;
  a.log2_block_size = p->block_size ? ilog2(p->block_size) : 0;
  a.max_blocks = p->max_blocks_per_seq;
  a.max_len = p->max_len;
  a.k = static_cast<__nv_bfloat16*>(k_out);
  a.v = static_cast<__nv_bfloat16*>(v_out);
  const dim3 grid(static_cast<unsigned>((p->max_len + fd::kExpandTokens - 1LL) / fd::kExpandTokens),
                  static_cast<unsigned>(p->Hkv), static_cast<unsigned>(p->B));
  return p->D == 128 ? launch_chained(fd::fd_expand_int4_kernel<128>, grid, 256, 0, stream, a)
                     : launch_chained(fd::fd_expand_int4_kernel<64>, grid, 256, 0, stream, a);
}

fd_status fd_decode_int4(const fd_problem* p, const void* q, const void* k4, const void* v4,
                         const void* params, const int32_t* seqlens, const int32_t* block_table,
                         float scale, int num_splits, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, fd_stream_t stream) {
  fd::Int4DecodeArgs d{};
  fd::Int4Cache c;
  const fd_status st = int4_cache(p, k4, v4, params, &c);
  if (st != FD_OK) return st;
  if (!q || !out || (p->block_size != 0) != (block_table != nullptr)) return FD_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FD_ERR_INVALID_ARGUMENT;
  if (num_splits < 1 || num_splits > kMaxSplits) return FD_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16) ||
      !aligned(seqlens, 4) || !aligned(block_table, 4))
    return FD_ERR_INVALID_ARGUMENT;
  fd::SplitArgs& a = d.a;
  const size_t need = fd_workspace_bytes(p->B, p->Hq, p->D, num_splits);
  if (num_splits > 1 && (!workspace || workspace_bytes < need)) return FD_ERR_WORKSPACE;
  int dev = 0;
  const fd_status arch = this_device(&dev);
  if (arch != FD_OK) return arch;
  Int4Maps maps;
  using ShapeN = fd::Int4Shape<8, 1, 64, 2>;
  using ShapeW = fd::Int4Shape<8, 1, 32, 3>;
  const int unit = p->Hq / p->Hkv <= 8 ? ShapeN::UNIT : ShapeW::UNIT;
  const int box_rows = p->block_size ? std::min(p->block_size, unit) : unit;
  if (cached_int4_maps(&maps, c, p->D, box_rows, dev) != FD_OK) return FD_ERR_CUDA;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.seqlens = seqlens;
  a.block_table = block_table;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.G = p->Hq / p->Hkv;
  a.max_len = p->max_len;
  a.block_size = p->block_size;
  a.log2_block_size = p->block_size ? ilog2(p->block_size) : 0;
  a.max_blocks_per_seq = p->max_blocks_per_seq;
  d.scale_m = static_cast<float>(std::frexp(static_cast<double>(scale) * 1.4426950408889634074f, &d.scale_e));
  d.B = p->B;
  int sms = 0;
  if (device_sms(dev, &sms) != FD_OK) return FD_ERR_CUDA;
  sms = std::min(sms, fd::kInt4MaxCtas);
  const long long rows = static_cast<long long>(p->B) * p->Hkv;
  if (rows * ((p->max_len + unit - 1LL) / unit + 1) > 0x7fffffffLL) return FD_ERR_INVALID_ARGUMENT;
  d.by_row = num_splits == 1;
  d.evict_first = !c.nhd;
  d.heads = !d.by_row && int4_heads(sms, p->B, p->Hkv, num_splits) ? 8 : 1;
  d.groups = p->Hkv / d.heads;
  if (!d.by_row) {
    d.ctas = d.heads > 1 ? sms : int4_ctas(sms, rows, num_splits);
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = a.part_o + static_cast<size_t>(2) * d.ctas * d.heads * a.G * p->D;
  }
  d.cluster = d.by_row ? int4_cluster(sms, rows, p->max_len) : 1;
  const dim3 grid = d.by_row ? dim3(static_cast<unsigned>(p->Hkv * d.cluster), static_cast<unsigned>(p->B))
                             : dim3(static_cast<unsigned>(d.ctas));
  fd_status r;
  if (p->D == 128)
    r = a.G <= 8 ? launch_split_int4<128, 1, ShapeN>(maps, d, grid, dev, stream)
                 : launch_split_int4<128, 2, ShapeW>(maps, d, grid, dev, stream);
  else
    r = a.G <= 8 ? launch_split_int4<64, 1, ShapeN>(maps, d, grid, dev, stream)
                 : launch_split_int4<64, 2, ShapeW>(maps, d, grid, dev, stream);
  if (r == FD_OK && !d.by_row && d.ctas > 1) {
    const int cut_rows = static_cast<int>(rows / d.heads);
    if (p->D == 128)
      r = unit == 64 ? launch_combine_int4<128, 64>(d, cut_rows, stream)
                     : launch_combine_int4<128, 32>(d, cut_rows, stream);
    else
      r = unit == 64 ? launch_combine_int4<64, 64>(d, cut_rows, stream)
                     : launch_combine_int4<64, 32>(d, cut_rows, stream);
  }
  return r;
}

fd_status fd_alloc_pages(int B, int block_size, int max_blocks_per_seq, int max_tokens,
                         int num_pages, const int32_t* seqlens, const int32_t* new_lens,
                         const int32_t* free_pages, const int32_t* free_count,
                         int32_t* block_table, int32_t* seqlens_out, int32_t* cu_new,
                         int64_t* slots, int32_t* positions, int32_t* free_count_out,
                         fd_stream_t stream) {
  const fd_status st = check_pages(B, block_size, max_blocks_per_seq, num_pages);
  if (st != FD_OK) return st;
  if (max_tokens < 0 || !seqlens || !new_lens || !free_pages || !free_count || !block_table ||
      !seqlens_out || !cu_new || (!slots && max_tokens > 0) || !free_count_out)
    return FD_ERR_INVALID_ARGUMENT;
  if (!aligned(seqlens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) ||
      !aligned(free_count, 4) || !aligned(block_table, 4) || !aligned(seqlens_out, 4) ||
      !aligned(cu_new, 4) || !aligned(slots, 8) || !aligned(positions, 4) ||
      !aligned(free_count_out, 4))
    return FD_ERR_INVALID_ARGUMENT;
  fd::PageArgs a{};
  a.B = B;
  a.log2_block_size = ilog2(block_size);
  a.max_blocks = max_blocks_per_seq;
  a.num_pages = num_pages;
  a.max_items = max_tokens;
  a.seqlens = seqlens;
  a.new_lens = new_lens;
  a.free_pages = const_cast<int32_t*>(free_pages);
  a.free_count = free_count;
  a.block_table = block_table;
  a.seqlens_out = seqlens_out;
  a.cu_new = cu_new;
  a.slots = slots;
  a.positions = positions;
  a.free_count_out = free_count_out;
  return launch_pages(fd::fd_alloc_pages_kernel, a, max_tokens, stream);
}

fd_status fd_release_pages(int B, int block_size, int max_blocks_per_seq, int num_pages,
                           const int32_t* seqlens, const uint8_t* done,
                           const int32_t* block_table, int32_t* free_pages,
                           const int32_t* free_count, int32_t* seqlens_out,
                           int32_t* free_count_out, fd_stream_t stream) {
  const fd_status st = check_pages(B, block_size, max_blocks_per_seq, num_pages);
  if (st != FD_OK) return st;
  if (!seqlens || !done || !block_table || !free_pages || !free_count || !seqlens_out ||
      !free_count_out)
    return FD_ERR_INVALID_ARGUMENT;
  if (!aligned(seqlens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
      !aligned(free_count, 4) || !aligned(seqlens_out, 4) || !aligned(free_count_out, 4))
    return FD_ERR_INVALID_ARGUMENT;
  fd::PageArgs a{};
  a.B = B;
  a.log2_block_size = ilog2(block_size);
  a.max_blocks = max_blocks_per_seq;
  a.num_pages = num_pages;
  a.seqlens = seqlens;
  a.done = done;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.block_table = const_cast<int32_t*>(block_table);
  a.seqlens_out = seqlens_out;
  a.free_count_out = free_count_out;
  const long long most = std::min<long long>(num_pages, static_cast<long long>(B) * max_blocks_per_seq);
  return launch_pages(fd::fd_release_pages_kernel, a, most, stream);
}

}  // extern "C"
