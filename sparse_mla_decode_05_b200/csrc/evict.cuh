// Eviction: which cache positions a sequence keeps, by the attention weight
// they accumulated, and the compaction of its paged caches to them.  Included
// by sparse_mla.cu after indexer.cuh (same translation unit).

namespace smla {

constexpr int kEvThreads = 1024;       // selection: one CTA per sequence
constexpr int kEvPer = 8;              // keys per thread in registers

static_assert(sizeof(smla_evict_shape) == 48 && offsetof(smla_evict_shape, num_kv_rows) == 32, "smla_evict_shape layout");

struct SelectParams {
  const float* acc;
  const int32_t* ctx_len;
  int32_t* kept;         // [B, budget]
  int32_t* new_len;      // [B]
  float* acc_out;        // [B, max_ctx], may be acc
  int max_ctx, budget, sinks, recent;
};

// Order of keeping: protected positions above all others, a NaN weight below.
__device__ __forceinline__ uint32_t evict_key(float w, int i, int sinks, int tail) {
  if (i < sinks || i >= tail) return 0xFFFFFFFFu;
  return w == w ? order_key(w) : 0u;
}

// One CTA per sequence.  Radix select of the budget-th largest key (four
// digits of eight bits), then the positions above it and the lowest ones
// equal to it, compacted in ascending order with their weights.  The
// compaction walks the positions upwards and writes at or below where it
// reads, so acc_out may be acc.
__global__ void __launch_bounds__(kEvThreads, 1) smla_evict_select_kernel(const SelectParams p) {
  __shared__ uint32_t hist[256];
  __shared__ int sums[65];
  __shared__ uint32_t s_digit;
  __shared__ int s_need;
  grid_dep_wait();
  const int b = blockIdx.x, t = threadIdx.x, lane = t & 31;
  int n = p.ctx_len[b];
  if (n < 0 || n > p.max_ctx) {
    if (t == 0) atomicOr(&g_error_word, 4u);
    n = n < 0 ? 0 : p.max_ctx;
  }
  const float* acc = p.acc + (size_t)b * p.max_ctx;
  float* out = p.acc_out + (size_t)b * p.max_ctx;
  int32_t* kept = p.kept + (size_t)b * p.budget;
  __syncthreads();       // ctx_len read by all before new_len (which may be it) is written
  if (n <= p.budget) {
    for (int i = t; i < p.budget; i += kEvThreads) kept[i] = i < n ? i : -1;
    if (out != acc)
      for (int i = t; i < n; i += kEvThreads) out[i] = acc[i];
    if (t == 0) p.new_len[b] = n;
    return;
  }
  const int tail = n - p.recent;
  uint32_t prefix = 0, mask = 0;
  int need = p.budget;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    if (t < 256) hist[t] = 0;
    __syncthreads();
#pragma unroll 1
    for (int base = 0; base < n; base += kEvThreads) {
      const int i = base + t;
      const uint32_t key = i < n ? evict_key(acc[i], i, p.sinks, tail) : 0u;
      const bool in = i < n && (key & mask) == prefix;
      const uint32_t digit = (key >> shift) & 255u;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (in) {
        const unsigned same = __match_any_sync(act, digit);
        if (lane == __ffs(same) - 1) atomicAdd(&hist[digit], (uint32_t)__popc(same));
      }
    }
    __syncthreads();
    if (t < 32) radix_pick(hist, need, &s_digit, &s_need);
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= 255u << shift;
    need = s_need;
    __syncthreads();
  }
  int written = 0, ties = 0;
#pragma unroll 1
  for (int base = 0; base < n; base += kEvThreads) {
    const int i = base + t;
    const float w = i < n ? acc[i] : 0.f;
    const uint32_t key = i < n ? evict_key(w, i, p.sinks, tail) : 0u;
    const bool gt = i < n && key > prefix, eq = i < n && key == prefix;
    int eq_total, sel_total;
    const int eq_rank = block_prefix_count(eq, sums, &eq_total);
    const bool sel = gt || (eq && ties + eq_rank < need);
    const int pos = block_prefix_count(sel, sums, &sel_total);
    if (sel && written + pos < p.budget) {
      kept[written + pos] = i;
      out[written + pos] = w;
    }
    written += sel_total;
    ties += eq_total;
  }
  __syncthreads();
  for (int i = p.budget + t; i < n; i += kEvThreads) out[i] = 0.f;
  if (t == 0) p.new_len[b] = p.budget;
}

// ------------------------------------------------------------ compaction
// A cache as planes: each a run of bytes per row, 64 rows to a page.
struct EvictPlane {
  uint8_t* base;
  long long page_stride;     // bytes from page to page
  int row_stride, width;     // bytes from row to row in a page; bytes moved per row
  int unit;                  // bytes per thread and row: 16, 8 or 4
  int cta0;                  // first CTA (blockIdx.x) of the plane
  int rows_limit;            // rows in the plane
};
struct CompactParams {
  EvictPlane plane[3];
  int planes;
  const int32_t* kept;
  const int32_t* new_len;
  const int32_t* from;       // page table of the source
  const int32_t* to;         // of the destination (the same: in place)
  int budget, pages_from, pages_to;
};

constexpr int kCpThreads = 256;
constexpr int kCpSlice = 128;          // bytes of a row per CTA (16-byte units)
constexpr int kCpBatch = 8;            // rows a thread has in flight

template <int kUnit> struct UnitOf;
template <> struct UnitOf<16> { using T = uint4; };
template <> struct UnitOf<8> { using T = uint2; };
template <> struct UnitOf<4> { using T = uint32_t; };

// address of a row of a plane, null where the page lies outside the pool
__device__ __forceinline__ uint8_t* evict_row(const EvictPlane& pl, const int32_t* pages, int npages, int pos) {
  if ((pos >> 6) >= npages) return nullptr;
  const int page = __ldg(pages + (pos >> 6));
  if (page < 0 || (long long)page * 64 + (pos & 63) >= pl.rows_limit) return nullptr;
  return pl.base + page * pl.page_stride + (pos & 63) * (long long)pl.row_stride;
}

// Moves row kept[i] to row i for every kept position of a sequence, for the
// byte columns [slice, slice + lanes x unit) of a plane.  In place this is
// safe without any exchange between CTAs: columns are independent, kept[i] >=
// i, and a CTA walks i upwards in blocks of R rows, writing a block only after
// the whole block is read.  Writing rows [i, i + R) destroys only sources
// that rows up to i + R - 1 needed, all read by then.
template <int kUnit>
__device__ __forceinline__ void compact_slice(const CompactParams& p, const EvictPlane& pl, int slice, int lanes) {
  using U = typename UnitOf<kUnit>::T;
  const int b = blockIdx.y, t = threadIdx.x;
  const int n = min(p.new_len[b], p.budget);
  const int32_t* kept = p.kept + (size_t)b * p.budget;
  const int32_t* from = p.from + (size_t)b * p.pages_from;
  const int32_t* to = p.to + (size_t)b * p.pages_to;
  const int rows = kCpThreads / lanes;              // rows per step
  const int col = slice + (t % lanes) * kUnit, r0 = t / lanes;
  const bool live = r0 < rows && col < pl.width;
  const bool in_place = p.from == p.to;
  bool outside = false;
  for (int base = 0; base < n; base += rows * kCpBatch) {
    U v[kCpBatch];
    uint8_t* dst[kCpBatch];
#pragma unroll
    for (int k = 0; k < kCpBatch; ++k) {
      const int i = base + k * rows + r0;
      dst[k] = nullptr;
      if (!live || i >= n) continue;
      const int old = __ldg(kept + i);
      if (old < 0 || (in_place && old == i)) continue;
      const uint8_t* src = evict_row(pl, from, p.pages_from, old);
      uint8_t* d = evict_row(pl, to, p.pages_to, i);
      if (!src || !d) {
        outside = true;
        continue;
      }
      v[k] = *reinterpret_cast<const U*>(src + col);
      dst[k] = d + col;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kCpBatch; ++k)
      if (dst[k]) *reinterpret_cast<U*>(dst[k]) = v[k];
  }
  if (outside) atomicOr(&g_error_word, 4u);
}

__global__ void __launch_bounds__(kCpThreads) smla_evict_compact_kernel(const __grid_constant__ CompactParams p) {
  grid_dep_wait();
  int k = p.planes - 1;
  while ((int)blockIdx.x < p.plane[k].cta0) --k;
  const EvictPlane& pl = p.plane[k];
  const int slice = ((int)blockIdx.x - pl.cta0) * kCpSlice;
  if (pl.unit == 16) compact_slice<16>(p, pl, slice, kCpSlice / 16);
  else if (pl.unit == 8) compact_slice<8>(p, pl, slice, 1);
  else compact_slice<4>(p, pl, slice, 1);
}

// ------------------------------------------------------------------ host
static smla_status validate_evict_shape(const smla_evict_shape* s) {
  if (!s) return SMLA_ERR_INVALID_ARG;
  if (s->batch < 1 || s->batch > 65535 || s->max_ctx < 1 || s->max_ctx > (1 << 20)) return SMLA_ERR_INVALID_ARG;
  if (s->budget < 1 || s->budget > s->max_ctx || s->sinks < 0 || s->recent < 0) return SMLA_ERR_INVALID_ARG;
  if ((long long)s->sinks + s->recent > s->budget) return SMLA_ERR_INVALID_ARG;
  if (s->kv_dtype != SMLA_KV_BF16 && s->kv_dtype != SMLA_KV_FP8_E4M3_ROWSCALE && s->kv_dtype != SMLA_KV_DSV4_PAGED)
    return SMLA_ERR_UNSUPPORTED;
  if (s->num_kv_rows < 64 || s->num_kv_rows > 0x7FFFFFFFLL || s->num_kv_rows % 64) return SMLA_ERR_INVALID_ARG;
  if (s->num_key_rows < 0 || s->num_key_rows > 0x7FFFFFFFLL || s->num_key_rows % 64) return SMLA_ERR_INVALID_ARG;
  if (s->pages_per_seq < 1 || (long long)s->pages_per_seq * 64 < s->max_ctx) return SMLA_ERR_INVALID_ARG;
  if (s->new_pages_per_seq < 0) return SMLA_ERR_INVALID_ARG;
  return SMLA_OK;
}

static smla_status check_select(const smla_evict_shape* s, const float* acc, const int32_t* ctx_len, int32_t* kept,
                                int32_t* new_len, float* acc_out) {
  const smla_status st = validate_evict_shape(s);
  if (st != SMLA_OK) return st;
  if (!acc || !ctx_len || !kept || !new_len || !acc_out) return SMLA_ERR_INVALID_ARG;
  if (!aligned(acc, 4) || !aligned(ctx_len, 4) || !aligned(kept, 4) || !aligned(new_len, 4) || !aligned(acc_out, 4))
    return SMLA_ERR_INVALID_ARG;
  return SMLA_OK;
}
static smla_status run_select(const smla_evict_shape* s, const float* acc, const int32_t* ctx_len, int32_t* kept,
                              int32_t* new_len, float* acc_out, cudaStream_t stream) {
  SelectParams p = {acc, ctx_len, kept, new_len, acc_out, s->max_ctx, s->budget, s->sinks, s->recent};
  void* args[] = {&p};
  const cudaError_t e = launch_pdl((const void*)smla_evict_select_kernel, dim3((unsigned)s->batch), dim3(kEvThreads), 0,
                                   stream, args);
  return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

static smla_status check_compact(const smla_evict_shape* s, const int32_t* kept, const int32_t* new_len,
                                 const int32_t* page_table, const int32_t* new_page_table, const void* kv,
                                 const float* kv_row_scale, const void* k_cache) {
  const smla_status st = validate_evict_shape(s);
  if (st != SMLA_OK) return st;
  if (!kept || !new_len || !page_table || !kv) return SMLA_ERR_INVALID_ARG;
  if (!aligned(kept, 4) || !aligned(new_len, 4) || !aligned(page_table, 4) || !aligned(new_page_table, 4) ||
      !aligned(kv, 16) || !aligned(kv_row_scale, 4) || !aligned(k_cache, 16))
    return SMLA_ERR_INVALID_ARG;
  if ((s->kv_dtype == SMLA_KV_FP8_E4M3_ROWSCALE) != (kv_row_scale != nullptr)) return SMLA_ERR_INVALID_ARG;
  if ((s->num_key_rows > 0) != (k_cache != nullptr)) return SMLA_ERR_INVALID_ARG;
  if (new_page_table && new_page_table != page_table && (long long)s->new_pages_per_seq * 64 < s->budget)
    return SMLA_ERR_INVALID_ARG;
  return SMLA_OK;
}
static smla_status run_compact(const smla_evict_shape* s, const int32_t* kept, const int32_t* new_len,
                               const int32_t* page_table, const int32_t* new_page_table, void* kv, float* kv_row_scale,
                               void* k_cache, cudaStream_t stream) {
  CompactParams p;
  memset(&p, 0, sizeof(p));
  int ctas = 0;
  auto plane = [&](void* base, long long page_stride, int row_stride, int width, int unit, long long rows) {
    EvictPlane& pl = p.plane[p.planes++];
    pl = {static_cast<uint8_t*>(base), page_stride, row_stride, width, unit, ctas, (int)rows};
    ctas += unit == 16 ? (width + kCpSlice - 1) / kCpSlice : 1;
  };
  if (s->kv_dtype == SMLA_KV_BF16) {
    plane(kv, 64ll * kRowBytesBf16, kRowBytesBf16, kRowBytesBf16, 16, s->num_kv_rows);
  } else if (s->kv_dtype == SMLA_KV_FP8_E4M3_ROWSCALE) {
    plane(kv, 64ll * kRowBytesFp8, kRowBytesFp8, kRowBytesFp8, 16, s->num_kv_rows);
    plane(kv_row_scale, 64 * 4, 4, 4, 4, s->num_kv_rows);
  } else {
    plane(kv, kDsv4Page, kDsv4Slot, kDsv4Slot, 16, s->num_kv_rows);
    plane(static_cast<uint8_t*>(kv) + kDsv4ScaleOff, kDsv4Page, 8, 8, 8, s->num_kv_rows);
  }
  if (k_cache) plane(k_cache, 64 * 256, 256, 256, 16, s->num_key_rows);
  p.kept = kept;
  p.new_len = new_len;
  p.from = page_table;
  p.to = new_page_table ? new_page_table : page_table;
  p.budget = s->budget;
  p.pages_from = s->pages_per_seq;
  p.pages_to = p.to == p.from ? s->pages_per_seq : s->new_pages_per_seq;
  void* args[] = {&p};
  const cudaError_t e = launch_pdl((const void*)smla_evict_compact_kernel, dim3((unsigned)ctas, (unsigned)s->batch),
                                   dim3(kCpThreads), 0, stream, args);
  return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

}  // namespace smla

extern "C" {

smla_status sparse_mla_evict_select(const smla_evict_shape* shape, const float* acc, const int32_t* ctx_len,
                                    int32_t* kept, int32_t* new_len, float* acc_out, void* stream) {
  const smla_status st = smla::check_select(shape, acc, ctx_len, kept, new_len, acc_out);
  if (st != SMLA_OK) return st;
  return smla::run_select(shape, acc, ctx_len, kept, new_len, acc_out, static_cast<cudaStream_t>(stream));
}

smla_status sparse_mla_evict_compact(const smla_evict_shape* shape, const int32_t* kept, const int32_t* new_len,
                                     const int32_t* page_table, const int32_t* new_page_table, void* kv_cache,
                                     float* kv_row_scale, void* k_cache, void* stream) {
  const smla_status st = smla::check_compact(shape, kept, new_len, page_table, new_page_table, kv_cache, kv_row_scale, k_cache);
  if (st != SMLA_OK) return st;
  return smla::run_compact(shape, kept, new_len, page_table, new_page_table, kv_cache, kv_row_scale, k_cache,
                           static_cast<cudaStream_t>(stream));
}

smla_status sparse_mla_evict(const smla_evict_shape* shape, const float* acc, const int32_t* ctx_len, int32_t* kept,
                             int32_t* new_len, float* acc_out, const int32_t* page_table,
                             const int32_t* new_page_table, void* kv_cache, float* kv_row_scale, void* k_cache,
                             void* stream) {
  smla_status st = smla::check_select(shape, acc, ctx_len, kept, new_len, acc_out);
  if (st == SMLA_OK)
    st = smla::check_compact(shape, kept, new_len, page_table, new_page_table, kv_cache, kv_row_scale, k_cache);
  if (st == SMLA_OK) st = smla::run_select(shape, acc, ctx_len, kept, new_len, acc_out, static_cast<cudaStream_t>(stream));
  if (st != SMLA_OK) return st;
  return smla::run_compact(shape, kept, new_len, page_table, new_page_table, kv_cache, kv_row_scale, k_cache,
                           static_cast<cudaStream_t>(stream));
}

}  // extern "C"
