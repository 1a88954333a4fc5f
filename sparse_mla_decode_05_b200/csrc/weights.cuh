// Attention weights: how much of the decode's attention each listed cache row
// received, and the sum of that over steps per cache position.  Included by
// sparse_mla.cu (same translation unit).
//
//   w[r, j]   = sum_h exp(scale * <q[r, h], k_j> - lse[r, h])      (0 for padding)
//   acc[b, p] = decay * acc[b, p] + sum over (t, j) with indices[b, t, j] = p of w[b, t, j]

namespace smla {

constexpr int kWtTile = 128;                       // entries per CTA (MMA M)
constexpr int kWtThreads = 256;
constexpr int kWtAtomK = kWtTile * 128;            // 64 dims of the rows: 128 rows x 128 B
constexpr int kWtAtomQ = kH * 128;                 // 64 dims of the query: 64 heads x 128 B
constexpr int kWtSmemK = 0;
constexpr int kWtSmemQ = kWtSmemK + kAtoms * kWtAtomK;
constexpr int kWtSmemRow = kWtSmemQ + kAtoms * kWtAtomQ;   // int  [128] physical row or -1
constexpr int kWtSmemScale = kWtSmemRow + kWtTile * 4;     // f32  [128] row scale
constexpr int kWtSmemLse = kWtSmemScale + kWtTile * 4;     // f32  [64]  lse
constexpr int kWtSmemPart = kWtSmemLse + kH * 4;           // f32  [128] the upper 32 heads' sums
constexpr int kWtSmemBar = kWtSmemPart + kWtTile * 4;
constexpr int kWtSmemTmem = kWtSmemBar + 8;
constexpr int kWtSmemBytes = kWtSmemTmem + 8;
static_assert(kWtSmemBytes <= 232448, "exceeds the 227 KB per-CTA shared memory of sm_100");
constexpr uint32_t kIdescWt = make_idesc(128, 64, false, false);

struct WeightsParams {
  const uint8_t* q;
  const uint8_t* kv;
  const float* kv_row_scale;
  const int32_t* page_table;
  const int32_t* indices;
  const float* lse;
  float* out;
  int topk, tok_per_seq, page_size, pages_per_seq, num_kv_rows;
  float scale;
};

// physical row of an index entry of decode row `drow`; -1: padding, or (with
// error bit 2) an entry outside its range
template <class P>
__device__ __forceinline__ int resolve_row(const P& p, int idx, int drow) {
  if (idx < 0) return -1;
  long long r = idx;
  if (p.page_size) {
    if (idx >= (long long)p.pages_per_seq * 64) r = -1;
    else {
      const long long page = __ldg(p.page_table + (size_t)(drow / p.tok_per_seq) * p.pages_per_seq + (idx >> 6));
      r = page < 0 ? -1 : page * 64 + (idx & 63);
    }
  }
  if (r < 0 || r >= p.num_kv_rows) {
    atomicOr(&g_error_word, 4u);
    return -1;
  }
  return (int)r;
}

// One CTA per (decode row, tile of 128 entries): rows and query into shared
// memory as bf16 (128-byte swizzle), D[128 entries x 64 heads] = K Q^T in
// tensor memory, then two threads per entry sum exp over 32 heads each.
template <int kKind>
__global__ void __launch_bounds__(kWtThreads, 1) smla_weights_kernel(const __grid_constant__ WeightsParams p) {
  constexpr bool kDsv4 = kKind == kKindDsv4, kFp8 = kKind == kKindFp8;
  constexpr int kQK = kDsv4 ? 512 : kDqk;
  constexpr int kQAtoms = kQK / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int drow = blockIdx.y, e0 = blockIdx.x * kWtTile;
  const uint32_t bar = sbase + kWtSmemBar;
  grid_dep_wait();
  if (sbase & 1023u) {
    if (t == 0) atomicOr(&g_error_word, 2u);
    return;
  }
  if (t == 0) {
    mbar_init(bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    tmem_alloc(sbase + kWtSmemTmem, 64);
    tmem_relinquish();
  }
  int* s_row = reinterpret_cast<int*>(smem + kWtSmemRow);
  float* s_scale = reinterpret_cast<float*>(smem + kWtSmemScale);
  float* s_lse = reinterpret_cast<float*>(smem + kWtSmemLse);
  float* s_part = reinterpret_cast<float*>(smem + kWtSmemPart);
  if (t < kWtTile) {
    const int idx = e0 + t < p.topk ? __ldg(p.indices + (size_t)drow * p.topk + e0 + t) : -1;
    const int r = resolve_row(p, idx, drow);
    s_row[t] = r;
    s_scale[t] = kFp8 && r >= 0 ? __ldg(p.kv_row_scale + r) : 1.f;
  } else if (t < kWtTile + kH) {
    // a head without any valid entry has lse -inf and takes no part
    const float l = __ldg(p.lse + (size_t)drow * kH + t - kWtTile);
    s_lse[t - kWtTile] = l == -INFINITY ? INFINITY : l;
  }
  const uint8_t* q = p.q + (size_t)drow * kH * kQK * 2;
  for (int c = t; c < kH * kQK / 8; c += kWtThreads) {
    const int h = c / (kQK / 8), j = c % (kQK / 8);
    cp_async_16(sbase + kWtSmemQ + (j >> 3) * kWtAtomQ + sw128_off(h, j & 7), q + (size_t)c * 16, 16u);
  }
  __syncthreads();
  if constexpr (kKind == kKindBf16) {
    for (int c = t; c < kWtTile * (kQK / 8); c += kWtThreads) {
      const int e = c / (kQK / 8), j = c % (kQK / 8);
      const int r = s_row[e];
      cp_async_16(sbase + kWtSmemK + (j >> 3) * kWtAtomK + sw128_off(e, j & 7),
                  p.kv + (size_t)(r >= 0 ? r : 0) * kRowBytesBf16 + j * 16, r >= 0 ? 16u : 0u);
    }
  } else {
    // 36 chunks of 16 bytes per row: 16 codes each, or (DeepSeek-V4, from
    // chunk 28 on) eight bf16 dims
    for (int c = t; c < kWtTile * 36; c += kWtThreads) {
      const int e = c / 36, j = c % 36;
      const int r = s_row[e];
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      const uint8_t* src = kDsv4 ? p.kv + (size_t)(r >> 6) * kDsv4Page + (r & 63) * kDsv4Slot : p.kv + (size_t)r * 576;
      if (r >= 0) v = *reinterpret_cast<const uint4*>(src + j * 16);
      if (kDsv4 && j >= 28) {
        st_shared_v4(sbase + kWtSmemK + 7 * kWtAtomK + sw128_off(e, j - 28), v);
        continue;
      }
      uint32_t s2 = 0x3F803F80u;
      if (kDsv4 && r >= 0)
        s2 = ue8m0_bf16x2(p.kv[(size_t)(r >> 6) * kDsv4Page + kDsv4ScaleOff + (r & 63) * 8 + (j >> 2)]);
      uint4 lo, hi;
      e4m3x4_to_bf16x4_scaled(v.x, s2, lo.x, lo.y);
      e4m3x4_to_bf16x4_scaled(v.y, s2, lo.z, lo.w);
      e4m3x4_to_bf16x4_scaled(v.z, s2, hi.x, hi.y);
      e4m3x4_to_bf16x4_scaled(v.w, s2, hi.z, hi.w);
      const uint32_t atom = sbase + kWtSmemK + (j >> 2) * kWtAtomK;
      st_shared_v4(atom + sw128_off(e, 2 * (j & 3)), lo);
      st_shared_v4(atom + sw128_off(e, 2 * (j & 3) + 1), hi);
    }
  }
  cp_async_wait_all();
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kWtSmemTmem);
  if (warp == 0) {
    const uint64_t da = sw128_desc(sbase + kWtSmemK, 16, 1024), db = sw128_desc(sbase + kWtSmemQ, 16, 1024);
    for (int ks = 0; ks < kQK / 16; ++ks) {
      const uint64_t ao = (uint64_t)((ks >> 2) * (kWtAtomK >> 4) + (ks & 3) * 2);
      const uint64_t bo = (uint64_t)((ks >> 2) * (kWtAtomQ >> 4) + (ks & 3) * 2);
      if (ks == 0) mma_set_elect(tmem, da + ao, db + bo, kIdescWt);
      else mma_acc_elect(tmem, da + ao, db + bo, kIdescWt);
    }
    commit_elect(bar);
  }
  const bool ok = mbar_wait(bar, 0);
  tc_fence_after();
  const int e = (warp & 3) * 32 + lane, half = warp >> 2;
  float sum = 0.f;
  if (ok) {
    float x[32];
    tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 32u * (uint32_t)half, x);
    tmem_wait_ld();
    // scale q.k - lse in one rounding, in natural units: where a weight is
    // large the difference is small, so what the exponential is taken of is
    // known to its own last bits, not to those of the lse
    const float k = p.scale * s_scale[e];
#pragma unroll
    for (int h = 0; h < 32; ++h) sum += ex2(1.44269504f * fmaf(x[h], k, -s_lse[32 * half + h]));
  }
  if (half) s_part[e] = sum;
  tc_fence_before();
  __syncthreads();
  if (!half && e0 + e < p.topk) p.out[(size_t)drow * p.topk + e0 + e] = s_row[e] >= 0 ? sum + s_part[e] : 0.f;
  if (warp == 0) tmem_dealloc(tmem, 64);
}

// ---------------------------------------------------------- accumulation
// One CTA per (sequence, range of kAcRange positions).  The entries of the
// sequence that fall into the range are summed in 64-bit fixed point in
// shared memory: integer addition is associative, so the result does not
// depend on the order of the atomics, whatever positions repeat.  The unit is
// 2^-s for all ranges of a sequence, s as large as keeps (entries x largest
// |weight|) below 2^62: sums keep at least 46 bits below the largest weight.
constexpr int kAcRange = 4096;
constexpr int kAcThreads = 512;

struct AccumulateParams {
  const int32_t* indices;
  const float* weights;
  float* acc;
  int entries, max_ctx;      // entries: tokens x topk of a sequence
  int log2_entries;          // entries <= 2^log2_entries
  float decay;
};

__global__ void __launch_bounds__(kAcThreads) smla_accumulate_kernel(const AccumulateParams p) {
  __shared__ long long sum[kAcRange];
  __shared__ uint32_t bad[kAcRange / 32];     // positions that got a NaN or an infinity
  __shared__ int s_max;
  grid_dep_wait();
  const int t = threadIdx.x, b = blockIdx.y, p0 = blockIdx.x * kAcRange;
  const int32_t* idx = p.indices + (size_t)b * p.entries;
  const float* w = p.weights + (size_t)b * p.entries;
  for (int i = t; i < kAcRange; i += kAcThreads) sum[i] = 0;
  for (int i = t; i < kAcRange / 32; i += kAcThreads) bad[i] = 0;
  if (t == 0) s_max = 0;
  __syncthreads();
  // largest finite |weight| (as bits) of the sequence's entries
  int m = 0;
  bool outside = false;
  for (int i = t; i < p.entries; i += kAcThreads) {
    const int at = __ldg(idx + i), v = __float_as_int(fabsf(__ldg(w + i)));
    outside |= at >= p.max_ctx;
    if (at >= 0 && at < p.max_ctx && v < 0x7F800000) m = max(m, v);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((t & 31) == 0 && m > 0) atomicMax(&s_max, m);
  if (outside && p0 == 0) atomicOr(&g_error_word, 4u);
  __syncthreads();
  m = s_max;
  // largest < 2^(e + 1): the unit's exponent
  const int e = m >= 0x800000 ? (m >> 23) - 127 : -126;
  const int s = 62 - p.log2_entries - (e + 1);
  if (m > 0 || p.decay != 1.0f) {
    const double up = ldexp(1.0, s), down = ldexp(1.0, -s);
    for (int i = t; i < p.entries; i += kAcThreads) {
      int at = __ldg(idx + i);
      if (at < p0 || at >= p.max_ctx || at - p0 >= kAcRange) continue;
      at -= p0;
      const float v = __ldg(w + i);
      if (fabsf(v) < INFINITY) atomicAdd(reinterpret_cast<unsigned long long*>(&sum[at]), (unsigned long long)__double2ll_rn((double)v * up));
      else atomicOr(&bad[at >> 5], 1u << (at & 31));
    }
    __syncthreads();
    for (int i = t; i < kAcRange && p0 + i < p.max_ctx; i += kAcThreads) {
      float* a = p.acc + (size_t)b * p.max_ctx + p0 + i;
      const bool nan = (bad[i >> 5] >> (i & 31)) & 1u;
      if (sum[i] == 0 && !nan && p.decay == 1.0f) continue;
      const float r = (float)fma((double)*a, (double)p.decay, (double)sum[i] * down);
      *a = nan ? __int_as_float(0x7FC00000) : r;
    }
  }
}

// ------------------------------------------------------------------ host
template <int kKind>
static cudaError_t launch_weights(WeightsParams& p, int rows, cudaStream_t stream) {
  static volatile int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(smla_weights_kernel<kKind>, cudaFuncAttributeMaxDynamicSharedMemorySize, kWtSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = 1;
  }
  void* args[] = {&p};
  return launch_pdl((const void*)smla_weights_kernel<kKind>, dim3((unsigned)((p.topk + kWtTile - 1) / kWtTile), (unsigned)rows),
                    dim3(kWtThreads), kWtSmemBytes, stream, args);
}

static smla_status run_weights(const smla_shape* s, const void* q, const void* kv, const float* kv_row_scale,
                               const int32_t* page_table, const int32_t* indices, const float* lse, float scale,
                               float* weights, cudaStream_t stream) {
  const smla_status st = validate_shape(s);
  if (st != SMLA_OK) return st;
  const bool fp8 = s->kv_dtype == SMLA_KV_FP8_E4M3_ROWSCALE;
  if (!q || !kv || !indices || !lse || !weights) return SMLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(indices, 4) || !aligned(lse, 4) || !aligned(weights, 4))
    return SMLA_ERR_INVALID_ARG;
  if (fp8 != (kv_row_scale != nullptr) || (fp8 && !aligned(kv_row_scale, 4))) return SMLA_ERR_INVALID_ARG;
  if (s->page_size && (!page_table || !aligned(page_table, 4))) return SMLA_ERR_INVALID_ARG;
  if (!(scale == scale) || isinf(scale)) return SMLA_ERR_INVALID_ARG;
  WeightsParams p;
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint8_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv);
  p.kv_row_scale = kv_row_scale;
  p.page_table = page_table;
  p.indices = indices;
  p.lse = lse;
  p.out = weights;
  p.topk = s->topk;
  p.tok_per_seq = tokens_of(s);
  p.page_size = s->page_size;
  p.pages_per_seq = s->pages_per_seq;
  p.num_kv_rows = (int)s->num_kv_rows;
  p.scale = scale;
  const cudaError_t e = fp8 ? launch_weights<kKindFp8>(p, rows_of(s), stream)
                            : (s->kv_dtype == SMLA_KV_DSV4_PAGED ? launch_weights<kKindDsv4>(p, rows_of(s), stream)
                                                                : launch_weights<kKindBf16>(p, rows_of(s), stream));
  return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

static smla_status run_accumulate(int batch, int64_t entries, int max_ctx, const int32_t* indices, const float* weights,
                                  float decay, float* acc, cudaStream_t stream) {
  if (batch < 1 || batch > 65535 || entries < 1 || entries > (1 << 28) || max_ctx < 1 || max_ctx > (1 << 20))
    return SMLA_ERR_INVALID_ARG;
  if (!(decay >= 0.0f && decay <= 1.0f)) return SMLA_ERR_INVALID_ARG;
  if (!indices || !weights || !acc || !aligned(indices, 4) || !aligned(weights, 4) || !aligned(acc, 4))
    return SMLA_ERR_INVALID_ARG;
  AccumulateParams p;
  memset(&p, 0, sizeof(p));
  p.indices = indices;
  p.weights = weights;
  p.acc = acc;
  p.entries = (int)entries;
  p.max_ctx = max_ctx;
  while ((1ll << p.log2_entries) < entries) ++p.log2_entries;
  p.decay = decay;
  void* args[] = {&p};
  const cudaError_t e = launch_pdl((const void*)smla_accumulate_kernel,
                                   dim3((unsigned)((max_ctx + kAcRange - 1) / kAcRange), (unsigned)batch), dim3(kAcThreads), 0,
                                   stream, args);
  return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

}  // namespace smla

extern "C" {

smla_status sparse_mla_attn_weights(const smla_shape* shape, const void* q, const void* kv_cache,
                                    const float* kv_row_scale, const int32_t* page_table, const int32_t* indices,
                                    const float* lse, float scale, float* weights, void* stream) {
  return smla::run_weights(shape, q, kv_cache, kv_row_scale, page_table, indices, lse, scale, weights,
                           static_cast<cudaStream_t>(stream));
}

smla_status sparse_mla_accumulate_weights(int32_t batch, int64_t entries, int32_t max_ctx, const int32_t* indices,
                                          const float* weights, float decay, float* acc, void* stream) {
  return smla::run_accumulate(batch, entries, max_ctx, indices, weights, decay, acc, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
