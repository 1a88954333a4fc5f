// Eviction: which cache positions a sequence keeps, by the attention weight
// they accumulated, and the compaction of its paged caches to them.  Included
// by sparse_mla.cu after indexer.cuh (same translation unit).

namespace smla {

constexpr int kEvThreads = 1024;       // selection
constexpr int kEvPer = 8;              // weights per thread and tile

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

// A cluster of CTAs per sequence, each thread holding eight weights of a tile of
// ctas x 8,192 positions.  Radix select of the budget-th largest key by digits
// of 11, 11 and 10 bits: each CTA counts its keys in shared memory, adds its
// counts that are not zero (a few hundred of 2,048) to every CTA's sums
// (distributed shared memory; reading all counts of all CTAs instead took 4,100
// cycles a digit), and all pick the same digit; it ends as soon as all keys
// that start with the digits so far are kept.  Then
// every key above the selection is kept and the lowest positions equal to it;
// the CTAs exchange their counts to know where their kept positions go.
// Contexts of one tile (65,536 positions with eight CTAs) read the weights
// once; longer ones read them again for each digit and for the compaction,
// which walks the tiles upwards and writes, once all CTAs have read a tile, at
// or below where it was read: acc_out may be acc.
constexpr int kEvMaxCtas = 8;          // the portable cluster size

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void red_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void evict_sync(int ctas) {
  if (ctas > 1) cluster_sync_all();
  else __syncthreads();
}
// Warp 0: exclusive prefix sums, in place, of the 32 kPer counts v[]; returns
// the total to every lane.
template <int kPer>
__device__ __forceinline__ int prefix_counts(int* v) {
  const int lane = threadIdx.x & 31;
  int x[kPer], sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    x[k] = v[kPer * lane + k];
    sum += x[k];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  int run = incl - sum;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    v[kPer * lane + k] = run;
    run += x[k];
  }
  return __shfl_sync(0xffffffffu, incl, 31);
}

template <bool kLong>     // more than one tile
__global__ void __launch_bounds__(kEvThreads, 1) smla_evict_select_kernel(const SelectParams p) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t total[3][2048]; // by digit: the sums of all CTAs' counts
  __shared__ int cnt[32 * kEvPer];    // [k][warp] counts, then their prefix sums
  __shared__ int wsum[32];
  __shared__ int s_total[2][2];       // [tile parity]: this CTA's keys equal to the selection, and its kept keys
  __shared__ uint32_t s_digit;
  __shared__ int s_need, s_cnt;
  grid_dep_wait();
  grid_dep_launch();
  const int rank = blockIdx.x, ctas = gridDim.x, b = blockIdx.y;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int n = p.ctx_len[b];
  if (n < 0 || n > p.max_ctx) {
    if (t == 0) atomicOr(&g_error_word, 4u);
    n = n < 0 ? 0 : p.max_ctx;
  }
  const float* acc = p.acc + (size_t)b * p.max_ctx;
  float* out = p.acc_out + (size_t)b * p.max_ctx;
  int32_t* kept = p.kept + (size_t)b * p.budget;
  if (n <= p.budget) {
    evict_sync(ctas);                 // new_len may be ctx_len, which every CTA of the cluster has read by here
    for (int i = rank * kEvThreads + t; i < p.budget; i += ctas * kEvThreads) kept[i] = i < n ? i : -1;
    if (out != acc)
      for (int i = rank * kEvThreads + t; i < n; i += ctas * kEvThreads) out[i] = acc[i];
    if (rank == 0 && t == 0) p.new_len[b] = n;
    return;
  }
  const int tail = n - p.recent, tile = ctas * kEvThreads * kEvPer;
  float w[kEvPer];
  uint32_t key[kEvPer];
  int base = 0;                       // this CTA's first position of the tile at hand
  auto valid = [&](int k) -> bool { return base + k * kEvThreads + t < n; };
  auto load = [&](int first) {
    base = first + rank * kEvThreads * kEvPer;
#pragma unroll
    for (int k = 0; k < kEvPer; ++k) w[k] = valid(k) ? acc[base + k * kEvThreads + t] : 0.f;
#pragma unroll
    for (int k = 0; k < kEvPer; ++k) key[k] = evict_key(w[k], base + k * kEvThreads + t, p.sinks, tail);
  };
  load(0);
  if (ctas > 1) {
    for (int i = t; i < 3 * 2048; i += kEvThreads) total[0][i] = 0;
    cluster_sync_all();               // all sums zero before any CTA adds to them
  }
  uint32_t prefix = 0, mask = 0;
  int need = p.budget, eq_count = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t dmask = pass == 2 ? 1023u : 2047u;
    hist[t] = 0;
    hist[t + 1024] = 0;
    __syncthreads();
#pragma unroll 1
    for (int first = 0; first < (kLong ? n : 1); first += tile) {
      if (kLong && (pass > 0 || first > 0)) load(first);
#pragma unroll
      for (int k = 0; k < kEvPer; ++k) {
        // weights of zero and protected positions, which may be most, would
        // queue at one counter each: one atomic for those of a warp
        const bool in = valid(k) && (key[k] & mask) == prefix;
        const uint32_t digit = (key[k] >> shift) & dmask;
        const bool zero = in && key[k] == 0x80000000u, fixed = in && key[k] == 0xFFFFFFFFu;
        const unsigned zeros = __ballot_sync(0xffffffffu, zero), fixeds = __ballot_sync(0xffffffffu, fixed);
        if (zero || fixed) {
          const unsigned same = zero ? zeros : fixeds;
          if (lane == __ffs(same) - 1) atomicAdd(&hist[digit], (uint32_t)__popc(same));
        } else if (in) {
          atomicAdd(&hist[digit], 1u);
        }
      }
    }
    __syncthreads();
    if (ctas > 1) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t c = hist[t + 1024 * u], a = smem_u32(&total[pass][t + 1024 * u]);
        if (c)
          for (int r = 0; r < ctas; ++r) red_cluster_u32(mapa_shared(a, (uint32_t)r), c);
      }
      cluster_sync_all();
    }
    radix_pick2048(ctas > 1 ? total[pass] : hist, need, wsum, &s_digit, &s_need, &s_cnt);
    prefix |= s_digit << shift;
    mask |= dmask << shift;
    need = s_need;
    eq_count = s_cnt;
    __syncthreads();
    if (eq_count == need) break;      // every key that starts with these digits is kept (the same in all CTAs)
  }
  // Ranks in position order (k, warp, lane) and across the cluster's CTAs.
  // cnt receives the CTA's exclusive counts; returns what the lower CTAs count,
  // *all what the whole tile does.
  const unsigned lt = (1u << lane) - 1u;
  auto ranks = [&](const unsigned (&m)[kEvPer], int* slot, int* all) -> int {
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < kEvPer; ++k) cnt[k * 32 + warp] = __popc(m[k]);
    }
    __syncthreads();
    if (warp == 0) {
      const int sum = prefix_counts<kEvPer>(cnt);
      if (lane == 0) *slot = sum;
    }
    evict_sync(ctas);
    // lane r reads CTA r's count
    const int c = lane < ctas ? (int)ld_cluster_u32(mapa_shared(smem_u32(slot), (uint32_t)lane)) : 0;
    *all = __reduce_add_sync(0xffffffffu, c);
    return __reduce_add_sync(0xffffffffu, lane < rank ? c : 0);
  };
  int written = 0, ties = 0;          // kept, and equal to the selection, in the tiles before
  unsigned selm[kEvPer];
#pragma unroll 1
  for (int first = 0, turn = 0; first < (kLong ? n : 1); first += tile, turn ^= 1) {
    if (kLong) load(first);
    int all;
    if (eq_count == need) {
#pragma unroll
      for (int k = 0; k < kEvPer; ++k) selm[k] = __ballot_sync(0xffffffffu, valid(k) && (key[k] & mask) >= prefix);
    } else {
      unsigned eqm[kEvPer];
#pragma unroll
      for (int k = 0; k < kEvPer; ++k) eqm[k] = __ballot_sync(0xffffffffu, valid(k) && key[k] == prefix);
      const int off = ties + ranks(eqm, &s_total[turn][0], &all);
#pragma unroll
      for (int k = 0; k < kEvPer; ++k) {
        const int rk = off + cnt[k * 32 + warp] + __popc(eqm[k] & lt);
        selm[k] = __ballot_sync(0xffffffffu, valid(k) && (key[k] > prefix || (key[k] == prefix && rk < need)));
      }
      ties += all;
      __syncthreads();   // every rank read before cnt is reused
    }
    const int off = written + ranks(selm, &s_total[turn][1], &all);   // (all CTAs have read the tile by here)
#pragma unroll
    for (int k = 0; k < kEvPer; ++k) {
      const int i = base + k * kEvThreads + t;
      if ((selm[k] >> lane) & 1u) {
        const int pos = off + cnt[k * 32 + warp] + __popc(selm[k] & lt);
        if (pos < p.budget) {
          kept[pos] = i;
          out[pos] = w[k];
        }
      }
      if (!kLong && i >= p.budget && i < n) out[i] = 0.f;
    }
    written += all;
    if (kLong) __syncthreads();       // cnt read before the next tile counts
  }
  if (kLong) {
    evict_sync(ctas);                 // every tile read before the rest is cleared
    for (int i = p.budget + rank * kEvThreads + t; i < n; i += ctas * kEvThreads) out[i] = 0.f;
  }
  if (rank == 0 && t == 0) p.new_len[b] = p.budget;
  if (ctas > 1) cluster_sync_all();   // no CTA leaves while its counts may be read
}

// ------------------------------------------------------------ compaction
// A cache as planes: each a run of bytes per row, 64 rows to a page, moved in
// columns of 2^log2_lanes units of 16 bytes (row scales and scale blocks: one
// unit of four or eight bytes).
struct EvictPlane {
  uint8_t* base;
  long long page_stride;     // bytes from page to page
  int row_stride;            // bytes from row to row in a page
  int unit, log2_lanes;      // bytes per thread, threads per row
  int slot0;                 // first slot of the plane; a slot is a column
  int pages;                 // pages in the plane
};
struct CompactParams {
  EvictPlane plane[3];
  int planes;
  const int32_t* kept;
  const int32_t* new_len;
  const int32_t* from;       // page table of the source
  const int32_t* to;         // of the destination (the same: in place)
  int budget, pages_from, pages_to;
  int ctas;                  // CTAs per sequence and column (in place: a cluster)
};

constexpr int kCpThreads = 256;
constexpr int kCpBatch = 8;            // rows a thread has in flight
constexpr int kCpMaxRows = 1024;       // rows per CTA and step
constexpr int kCpPages = 512;          // pages of a sequence held in shared memory (the rest read as needed)

template <int kUnit> struct UnitOf;
template <> struct UnitOf<16> { using T = uint4; };
template <> struct UnitOf<8> { using T = uint2; };
template <> struct UnitOf<4> { using T = uint32_t; };

// Moves row kept[i] to row i, i < n, for one column of a plane, in steps of
// ctas x R rows, R per CTA.
//
// In place: kept[i] >= i, so writing rows [i, i + R) destroys only sources that
// rows up to i + R - 1 needed.  A barrier per step, of the CTAs (a cluster) that
// share the column, puts all of the step's reads before any of its writes, and
// rows read later lie above them.  (Columns need no order among themselves.)
// Between CTAs it releases and acquires: nothing less orders one CTA's reads
// before another's writes, although it waits for the last step's writes too.
// With new pages nothing has to wait.
//
// Each step's physical rows are worked out once, by one thread per row and a
// step ahead (kept position -> page -> row, both page tables in shared
// memory), so the moving threads wait for one memory latency a step and
// spend few instructions on addresses.  Column widths, 32 x 4,096 fp8 rows and
// keys: 64 / 128 bytes 52 / 53 us in place and 47 / 42 us into new pages; 32
// bytes 67 / 65.  Bulk copies of whole rows through shared memory were two to
// three times as slow.
template <int kUnit, bool kInPlace>
__device__ __forceinline__ void compact_column(const CompactParams& p, const EvictPlane& pl, const int* s_from, const int* s_to,
                                               int2 (*s_rows)[kCpMaxRows], int column, int n) {
  using U = typename UnitOf<kUnit>::T;
  constexpr int kBatch = kUnit == 16 ? kCpBatch : kCpMaxRows / kCpThreads;
  const int b = blockIdx.y, t = threadIdx.x, rank = blockIdx.x % p.ctas;
  const int32_t* kept = p.kept + (size_t)b * p.budget;
  const int rows = kCpThreads >> pl.log2_lanes;     // rows per batch element
  const int r0 = t >> pl.log2_lanes;
  const int mine = rows * kBatch;                   // rows per CTA and step, at most kCpMaxRows
  const int step = mine * p.ctas;
  const int col = ((column << pl.log2_lanes) + (t & ((1 << pl.log2_lanes) - 1))) * kUnit;
  const bool live = col < pl.row_stride;
  bool outside = false;
  // (source, destination) of this CTA's rows of the step at `base`; -1: nothing moves
  auto prepare = [&](int base, int2* to_rows) {
    for (int j = t; j < mine; j += kCpThreads) {
      const int i = base + rank * mine + j;
      int2 r = make_int2(-1, -1);
      if (i < n) {
        const int o = __ldg(kept + i);
        if (o >= 0 && !(kInPlace && o == i)) {
          const int ps = o >> 6, pd = i >> 6;
          const int fp = ps < p.pages_from ? (ps < kCpPages ? s_from[ps] : __ldg(p.from + (size_t)b * p.pages_from + ps)) : -1;
          const int tp = pd < p.pages_to ? (pd < kCpPages ? s_to[pd] : __ldg(p.to + (size_t)b * p.pages_to + pd)) : -1;
          if (fp >= 0 && tp >= 0 && fp < pl.pages && tp < pl.pages) r = make_int2(fp * 64 + (o & 63), tp * 64 + (i & 63));
          else outside = true;
        }
      }
      to_rows[j] = r;
    }
  };
  prepare(0, s_rows[0]);
  int buf = 0;
  for (int base = 0; base < n; base += step, buf ^= 1) {
    __syncthreads();
    U v[kBatch];
    int to[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int2 r = live ? s_rows[buf][k * rows + r0] : make_int2(-1, -1);
      to[k] = r.y;
      if (r.y >= 0)
        v[k] = *reinterpret_cast<const U*>(pl.base + (r.x >> 6) * pl.page_stride + (uint32_t)((r.x & 63) * pl.row_stride + col));
    }
    if (base + step < n) prepare(base + step, s_rows[buf ^ 1]);
    if (kInPlace) evict_sync(p.ctas);
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (to[k] >= 0)
        *reinterpret_cast<U*>(pl.base + (to[k] >> 6) * pl.page_stride + (uint32_t)((to[k] & 63) * pl.row_stride + col)) = v[k];
  }
  if (outside) atomicOr(&g_error_word, 4u);
}

template <bool kInPlace>
__global__ void __launch_bounds__(kCpThreads, 4) smla_evict_compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int s_from[kCpPages], s_to[kCpPages];
  __shared__ int2 s_rows[2][kCpMaxRows];
  grid_dep_wait();
  const int b = blockIdx.y;
  const int n = min(p.new_len[b], p.budget);
  for (int i = threadIdx.x; i < kCpPages; i += kCpThreads) {
    if (i < p.pages_from) s_from[i] = __ldg(p.from + (size_t)b * p.pages_from + i);
    if (i < p.pages_to) s_to[i] = __ldg(p.to + (size_t)b * p.pages_to + i);
  }
  __syncthreads();
  const int slot = blockIdx.x / p.ctas;
  int k = p.planes - 1;
  while (slot < p.plane[k].slot0) --k;
  const EvictPlane& pl = p.plane[k];
  const int column = slot - pl.slot0;
  if (pl.unit == 16) compact_column<16, kInPlace>(p, pl, s_from, s_to, s_rows, column, n);
  else if (pl.unit == 8) compact_column<8, kInPlace>(p, pl, s_from, s_to, s_rows, column, n);
  else compact_column<4, kInPlace>(p, pl, s_from, s_to, s_rows, column, n);
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
  int ctas = 1;
  while (ctas < kEvMaxCtas && ctas * kEvThreads * kEvPer < s->max_ctx) ctas *= 2;
  const void* kern = ctas * kEvThreads * kEvPer < s->max_ctx ? (const void*)smla_evict_select_kernel<true>
                                                             : (const void*)smla_evict_select_kernel<false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)s->batch);
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kern, args);
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
  const int sms = device_sm_count();
  if (sms <= 0) return SMLA_ERR_CUDA;
  const bool in_place = !new_page_table || new_page_table == page_table;
  const int log2_lanes = in_place ? 2 : 3;          // columns of 64 or 128 bytes
  int slots = 0;
  auto plane = [&](void* base, long long page_stride, int row_stride, int unit, long long rows) {
    const int lg = unit == 16 ? log2_lanes : 0;
    p.plane[p.planes++] = {static_cast<uint8_t*>(base), page_stride, row_stride, unit, lg, slots, (int)(rows / 64)};
    slots += (row_stride + (unit << lg) - 1) / (unit << lg);
  };
  if (s->kv_dtype == SMLA_KV_BF16) {
    plane(kv, 64ll * kRowBytesBf16, kRowBytesBf16, 16, s->num_kv_rows);
  } else if (s->kv_dtype == SMLA_KV_FP8_E4M3_ROWSCALE) {
    plane(kv, 64ll * kRowBytesFp8, kRowBytesFp8, 16, s->num_kv_rows);
    plane(kv_row_scale, 64 * 4, 4, 4, s->num_kv_rows);
  } else {
    plane(kv, kDsv4Page, kDsv4Slot, 16, s->num_kv_rows);
    plane(static_cast<uint8_t*>(kv) + kDsv4ScaleOff, kDsv4Page, 8, 8, s->num_kv_rows);
  }
  if (k_cache) plane(k_cache, 64 * 256, 256, 16, s->num_key_rows);
  // In place a cluster per column: as many CTAs (a power of two, at most eight)
  // as leave three to an SM (one sequence of 65,536 -> 8,192 bf16 rows: 30 us
  // with one CTA, 9 with eight).  New pages: a CTA per step.
  const int step_rows = (kCpThreads >> log2_lanes) * kCpBatch;
  p.ctas = 1;
  if (in_place) {
    while (p.ctas < 8 && (long long)s->batch * slots * p.ctas * 2 <= 3 * sms && s->budget > step_rows * p.ctas) p.ctas *= 2;
  } else {
    p.ctas = (s->budget + step_rows - 1) / step_rows;
  }
  p.kept = kept;
  p.new_len = new_len;
  p.from = page_table;
  p.to = in_place ? page_table : new_page_table;
  p.budget = s->budget;
  p.pages_from = s->pages_per_seq;
  p.pages_to = p.to == p.from ? s->pages_per_seq : s->new_pages_per_seq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slots * p.ctas), (unsigned)s->batch);
  cfg.blockDim = dim3(kCpThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)p.ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = in_place && p.ctas > 1 ? 2 : 1;
  void* args[] = {&p};
  const void* kern = in_place ? (const void*)smla_evict_compact_kernel<true> : (const void*)smla_evict_compact_kernel<false>;
  return cudaLaunchKernelExC(&cfg, kern, args) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
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
