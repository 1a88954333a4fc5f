// Attention weights: how much of the decode's attention each listed cache row
// received, and the sum of that over steps per cache position.  Included by
// sparse_mla.cu (same translation unit).
//
//   w[r, j]   = sum_h exp(scale * <q[r, h], k_j> - lse[r, h])      (0 for padding)
//   acc[b, p] = decay * acc[b, p] + sum over (t, j) with indices[b, t, j] = p of w[b, t, j]

namespace smla {

constexpr int kWtEpiWarps = 8;
constexpr int kWtRing = 8;                         // tiles whose rows and scales are kept
// Shared-memory operands are 128-byte-swizzled atoms of [rows][128 B]; the
// last 64 bytes of a 576-byte fp8 row are a 64-byte-swizzled atom [rows][64 B].
template <int kKind>
struct WtCfg {
  static constexpr bool kFp8 = kKind == kKindFp8;
  static constexpr int kQK = kKind == kKindDsv4 ? 512 : kDqk;
  static constexpr int kRowBytes = kFp8 ? kQK : 2 * kQK;           // of an operand row
  // Entries per tile = MMA M.  The tensor cores take as long for 64 rows as
  // for 128: fp8 rows, whose bytes arrive fastest per MMA, need the full rate
  // (64 rows: 47.8 us on the batch of 128, the MMAs busy 63 % of it).
  static constexpr int kM = kFp8 ? 128 : 64;
  static constexpr int kAtom = kM * 128;                           // 128 bytes of each of the rows
  static constexpr int kStages = 2;
  static constexpr int kStageBytes = kM * kRowBytes;
  static constexpr int kCopyWarps = kKind == kKindDsv4 ? 16 : 8;
  static constexpr int kRows = kM / kCopyWarps;                    // rows of a tile per copy warp
  // fp8: eight warps more help the epilogue warps to stage the query.  Staged by
  // eight, a row's query took 10,000 cycles, longer than two stages of copies
  // last; by the copy warps too, it held up the copies.
  static constexpr int kHelpers = kFp8 ? 8 : 0;
  static constexpr int kThreads = 32 * (1 + kWtEpiWarps + kCopyWarps + kHelpers);
  static constexpr int kQWarps = kWtEpiWarps + kHelpers;           // that stage the query
  static constexpr int kQHeads = kH / kQWarps;
  static constexpr int kQRows = kFp8 ? 128 : 64;                   // fp8: the heads' high parts, then their low parts
  static constexpr int kQBytes = kQRows * kRowBytes;
  static constexpr int kMmaN = kQRows;
  // bf16 operands: the K steps go to four accumulators, added in the epilogue.
  // The tensor cores cut every update of an accumulator to fp32, an error in
  // proportion to its value and all of one sign; in a quarter each, partial
  // sums are a quarter as large (one sequence, scores up to 20: relative
  // error of the weights 7.7e-6 with one accumulator, 1.4e-6 with four; 1 % of
  // the time).  DeepSeek-V4 rows, short of registers, take two; fp8 rows take
  // half the steps, in two parts already.
  static constexpr int kAccs = kFp8 ? 1 : (kKind == kKindBf16 ? 4 : 2);
  static constexpr int kN = kAccs * kMmaN;                         // columns of a score buffer
  static constexpr uint32_t kTmem = 2 * kN;
  static constexpr int kSmemQ = kStages * kStageBytes;
  static constexpr int kSmemRow = kSmemQ + kQBytes;                // int  [kWtRing][kM] physical row or -1
  static constexpr int kSmemScale = kSmemRow + kWtRing * kM * 4;   // f32  [kWtRing][kM] row scale (fp8)
  static constexpr int kSmemLse = kSmemScale + kWtRing * kM * 4;   // f32  [2][64] by row parity
  static constexpr int kSmemK = kSmemLse + 2 * 64 * 4;             // f32  [2][64] scale, over the query's power of two
  static constexpr int kSmemBar = kSmemK + 2 * 64 * 4;
  static constexpr int kSmemTmem = kSmemBar + 8 * 16;
  static constexpr int kSmemBytes = kSmemTmem + 16;
  static_assert(kSmemBytes <= 232448, "exceeds the 227 KB per-CTA shared memory of sm_100");
  static_assert(kSmemQ % 1024 == 0 && kStageBytes % 1024 == 0, "swizzled operands need 1024-byte aligned atoms");
  // Reuse of the row / scale ring: tile t + stages + 2 is copied after MMA(t + 2) has completed, which waited for
  // the epilogue of tile t to have read its slot.
  static_assert(kWtRing >= kStages + 2, "row ring");
};
constexpr uint32_t kIdescWt = make_idesc(64, 64, false, false), kIdescWt8 = make_idesc_e4m3(128, 128, false);
// barriers
constexpr int WB_FULL = 0, WB_EMPTY = 4, WB_SF = 8, WB_SE = 10, WB_Q = 12, WB_FIN = 13, WB_ROW = 14;

// Shared-memory matrix descriptor, 64-byte swizzle (layout type 4), K-major:
// rows of 64 B, 8-row groups 512 B apart.
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(512 >> 4) << 32) | (1ull << 46) | (4ull << 61);
}
__device__ __forceinline__ uint32_t sw64_off(int r, int j) { return (uint32_t)(r * 64 + ((j ^ ((r >> 1) & 3)) << 4)); }
// byte offset of 16-byte chunk c (0..35) of row r of a 576-byte-row operand of `rows` rows
template <int kRows>
__device__ __forceinline__ uint32_t wt_off8(int r, int c) {
  return c < 32 ? (uint32_t)((c >> 3) * (kRows * 128)) + sw128_off(r, c & 7)
                : (uint32_t)(4 * kRows * 128) + sw64_off(r, c - 32);
}

struct WeightsParams {
  const uint8_t* q;
  const uint8_t* kv;
  const float* kv_row_scale;
  const int32_t* page_table;
  const int32_t* indices;
  const float* lse;
  float* out;
  int topk, tok_per_seq, page_size, pages_per_seq, num_kv_rows;
  int ntiles;                // tiles per decode row
  long long total;           // rows x ntiles
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

// 32 lanes x 16 columns: thread t reads columns [c, c+16) of lane base+t.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// x (f16x2, |x| < 448) = hi + lo in e4m3x2: hi = e4m3(x), lo = e4m3(x - hi)
__device__ __forceinline__ void split_e4m3x2_f16(uint32_t x, uint32_t& hi, uint32_t& lo) {
  uint16_t h, l;
  uint32_t h16, r16;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(x));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h16) : "h"(h));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r16) : "r"(x), "r"(h16));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(r16));
  hi = h;
  lo = l;
}

// kHeads heads of a row's query (h0 ..) into the B operand, by one warp.
// bf16 caches: as they are.  fp8: times the power of two that brings the
// head's largest |q| into [128, 256), split into e4m3 high and low parts
// (exact for the bf16 values whose parts are e4m3 normals, within 2^-10 of the
// scaled value otherwise); s_k[h] receives scale over that power.  This runs
// once per row between two rows' products, at a warp's own pace (a few cycles
// an instruction), so it is spread over as many warps as there are and kept
// short: bf16 pairs are scaled as pairs and split as f16 pairs.
template <int kKind, int kHeads>
__device__ __forceinline__ void wt_stage_query(const WeightsParams& p, uint8_t* smem, uint32_t sbase, int row, int h0,
                                               int lane, float* s_k) {
  using C = WtCfg<kKind>;
  constexpr int kChunks = C::kQK / 8;               // 16-byte chunks of a head
  const uint8_t* q = p.q + ((size_t)row * kH + h0) * (C::kQK * 2);
  const uint32_t qb = sbase + C::kSmemQ;
  if constexpr (!C::kFp8) {
    for (int c = lane; c < kHeads * kChunks; c += 32) {
      const int h = c / kChunks, j = c - h * kChunks;
      cp_async_16(qb + (uint32_t)((j >> 3) * (C::kQRows * 128)) + sw128_off(h0 + h, j & 7), q + (size_t)c * 16, 16u);
    }
    cp_async_wait_all();
  } else {
    // lane l: chunks l, 32 + l and, of lanes 0-7, 64 + l
    uint4 v[kHeads][3];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const uint4* src = reinterpret_cast<const uint4*>(q + (size_t)i * (C::kQK * 2));
      v[i][0] = __ldg(src + lane);
      v[i][1] = __ldg(src + 32 + lane);
      v[i][2] = lane < 8 ? __ldg(src + 64 + lane) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i;
      // largest magnitude (bf16 bits order as the magnitudes do)
      uint32_t m2 = 0;
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        m2 = __vmaxu2(m2, v[i][u].x & 0x7FFF7FFFu);
        m2 = __vmaxu2(m2, v[i][u].y & 0x7FFF7FFFu);
        m2 = __vmaxu2(m2, v[i][u].z & 0x7FFF7FFFu);
        m2 = __vmaxu2(m2, v[i][u].w & 0x7FFF7FFFu);
      }
      const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
      int sq = m ? 134 - (int)(m >> 7) : 0;          // 7 - floor(log2 m)
      sq = sq > 120 ? 120 : (sq < -120 ? -120 : sq);
      const uint32_t up = (uint32_t)(127 + sq) * 0x00800080u;       // 2^sq as a bf16 pair
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        if (u == 2 && lane >= 8) continue;
        const uint32_t w4[4] = {v[i][u].x, v[i][u].y, v[i][u].z, v[i][u].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t y = bf16x2_mul(w4[k], up);
          split_e4m3x2_f16(pack_f16x2(__uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u)), hi[k], lo[k]);
        }
        // eight codes: half of 16-byte chunk (32 u + lane) / 2 of the row
        const int c = (32 * u + lane) >> 1;
        const uint32_t at = (uint32_t)(8 * (lane & 1));
        *reinterpret_cast<uint2*>(smem + C::kSmemQ + wt_off8<C::kQRows>(h, c) + at) =
            make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
        *reinterpret_cast<uint2*>(smem + C::kSmemQ + wt_off8<C::kQRows>(64 + h, c) + at) =
            make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
      }
      if (lane == 0) s_k[h] = p.scale * pow2i(-sq);
    }
  }
}

// The decode rows' tiles are laid end to end and shared out
// evenly over one CTA per SM; every tile's weights are its own, so nothing is
// merged.  Warp roles: one MMA issuer; eight epilogue warps, which also
// stage the query of each row the CTA meets (for fp8 rows with eight more);
// the copy warps.
//  * Copy warps resolve and gather kRows rows each of every tile by 16-byte
//    cp.async (lane = chunk of one row, the rows' last 64 bytes merged):
//    conflict-free in the swizzled atoms, two tiles ahead.
//  * S[entries x 64 heads] = K Q^T in tensor memory, two buffers.  fp8 rows
//    are multiplied as stored (kind::f8f6f4) by the query scaled per head by
//    a power of two and split into e4m3 high and low parts, as in the decode:
//    columns 0-63 and 64-127 of the buffer.
//  * Epilogue warps 0-3 take the even tiles, 4-7 the odd ones; a thread has one
//    entry: of 128-entry tiles all heads, of 64-entry tiles 32, the other 32
//    being its partner's, sixteen lanes on.
template <int kKind>
__global__ void __launch_bounds__(WtCfg<kKind>::kThreads, 1) smla_weights_kernel(const __grid_constant__ WeightsParams p) {
  using C = WtCfg<kKind>;
  constexpr bool kFp8 = C::kFp8, kDsv4 = kKind == kKindDsv4;
  constexpr int kStages = C::kStages, kM = C::kM, kRows = C::kRows, kAtom = C::kAtom;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto BAR = [&](int i) -> uint32_t { return sbase + C::kSmemBar + 8u * (uint32_t)i; };
  if (sbase & 1023u) {
    grid_dep_wait();
    if (threadIdx.x == 0) atomicOr(&g_error_word, 2u);
    return;
  }
  // this CTA's tiles
  const int nt = p.ntiles;
  const long long g0 = (long long)blockIdx.x * p.total / gridDim.x, g1 = (long long)(blockIdx.x + 1) * p.total / gridDim.x;
  const int count = (int)(g1 - g0);
  const int row0 = (int)(g0 / nt), tin0 = (int)(g0 % nt);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      // a copying thread's copies (fp8, bf16), and each copy warp's row numbers or converted rows
      mbar_init(BAR(WB_FULL + i), C::kCopyWarps + (kDsv4 ? 0 : 32 * C::kCopyWarps));
      mbar_init(BAR(WB_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(WB_SF + i), 1);
      mbar_init(BAR(WB_SE + i), kWtEpiWarps / 2);
    }
    mbar_init(BAR(WB_Q), C::kQWarps);
    mbar_init(BAR(WB_FIN), 1);
    mbar_init(BAR(WB_ROW), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    tmem_alloc(sbase + C::kSmemTmem, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::kSmemTmem);
  int* s_row = reinterpret_cast<int*>(smem + C::kSmemRow);
  float* s_scale = reinterpret_cast<float*>(smem + C::kSmemScale);
  float* s_lse = reinterpret_cast<float*>(smem + C::kSmemLse);
  float* s_k = reinterpret_cast<float*>(smem + C::kSmemK);
  auto wait_all = [&](int bar, int parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(BAR(bar), (uint32_t)parity));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = true;
    int tin = tin0, seg = 0;
    for (int t = 0; ok && t < count; ++t, tin = tin + 1 == nt ? 0 : tin + 1) {
      const int stage = t % kStages, buf = t & 1;
      if (t == 0 || tin == 0) ok = wait_all(WB_Q, seg++ & 1);
      if (ok && t >= 2) ok = wait_all(WB_SE + buf, ((t >> 1) - 1) & 1);
      if (ok) ok = wait_all(WB_FULL + stage, (t / kStages) & 1);
      if (!ok) break;
      tc_fence_after();
      fence_proxy_async_smem();    // the copies (generic proxy) before the tensor core's reads
      const uint32_t d = tmem + (uint32_t)(buf * C::kN);
      const uint32_t a = sbase + (uint32_t)(stage * C::kStageBytes), b = sbase + C::kSmemQ;
      if constexpr (kFp8) {
        const uint32_t idesc = kIdescWt8;
        const uint64_t da = sw128_desc(a, 16, 1024), db = sw128_desc(b, 16, 1024);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          mma8_ss_elect(d, da + (uint64_t)((k >> 2) * (kAtom >> 4) + (k & 3) * 2),
                        db + (uint64_t)((k >> 2) * (C::kQRows * 128 >> 4) + (k & 3) * 2), idesc, k > 0);
        const uint64_t ta = sw64_desc(a + 4 * kAtom), tb = sw64_desc(b + 4 * C::kQRows * 128);
#pragma unroll
        for (int k = 0; k < 2; ++k) mma8_ss_elect(d, ta + (uint64_t)(2 * k), tb + (uint64_t)(2 * k), idesc, true);
      } else {
        const uint32_t idesc = kIdescWt;
        const uint64_t da = sw128_desc(a, 16, 1024), db = sw128_desc(b, 16, 1024);
#pragma unroll
        for (int k = 0; k < C::kQK / 16; ++k) {
          const uint64_t off = (uint64_t)((k >> 2) * (kAtom >> 4) + (k & 3) * 2);
          constexpr int kPart = C::kQK / 16 / C::kAccs;                // K steps per accumulator
          const uint32_t dk = d + (uint32_t)(k / kPart * C::kMmaN);
          if (k % kPart == 0) mma_set_elect(dk, da + off, db + off, idesc);
          else mma_acc_elect(dk, da + off, db + off, idesc);
        }
      }
      commit_elect(BAR(WB_EMPTY + stage));
      commit_elect(BAR(WB_SF + buf));
      if (tin + 1 == nt) commit_elect(BAR(WB_ROW));    // the row's last products: its query may go
    }
    // every MMA issued has completed before teardown
    commit_elect(BAR(WB_FIN));
    mbar_wait(BAR(WB_FIN), 0);
  } else if (warp <= kWtEpiWarps) {
    // -------------------------------------------------------------- epilogue
    const int ew = warp - 1, group = ew >> 2, quarter = warp & 3;
    const int e = kM == 128 ? 32 * quarter + lane : 16 * quarter + (lane & 15), half = kM == 128 ? 0 : lane >> 4;
    bool ok = true;
    int row = row0, tin = tin0, seg = 0;
    for (int t = 0; ok && t < count; ++t) {
      if (t == 0 || tin == 0) {
        // the row's query, once the last row's products are done
        if (t > 0) ok = wait_all(WB_ROW, (seg - 1) & 1);
        if (!ok) break;
        const int h0 = 8 * ew, sb = (seg & 1) * 64;
        // the query of the row after this one, into L2 ahead of its use
        if (ew == 0 && lane == 0 && t + nt - tin < count)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.q + (size_t)(row + 1) * kH * C::kQK * 2),
                       "r"(kH * C::kQK * 2) : "memory");
        if (lane < 8) {
          // a head without any valid entry has lse -inf and takes no part
          const float l = __ldg(p.lse + (size_t)row * kH + h0 + lane);
          s_lse[sb + h0 + lane] = l == -INFINITY ? INFINITY : l;
          if (!kFp8) s_k[sb + h0 + lane] = p.scale;
        }
        wt_stage_query<kKind, C::kQHeads>(p, smem, sbase, row, C::kQHeads * ew, lane, s_k + sb);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(WB_Q));
        ++seg;
      }
      if ((t & 1) == group) {
        ok = wait_all(WB_SF + group, (t >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const int rs = (t % kWtRing) * kM + e;
        const int r = s_row[rs];
        const float rsc = kFp8 ? s_scale[rs] : 1.f;
        const uint32_t d = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(group * C::kN);
        const float* lse = s_lse + ((seg - 1) & 1) * 64 + 32 * half;
        const float* kh = s_k + ((seg - 1) & 1) * 64 + 32 * half;
        // scale q.k - lse in natural units and one rounding: where a weight is
        // large the difference is small, so the exponential is taken of a
        // number known to its own last bits, not to those of the lse
        auto weigh = [&](const float* x, const float* l, const float* k) -> float {   // 16 heads
          float sum = 0.f;
#pragma unroll
          for (int h = 0; h < 16; h += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(l + h), k4 = *reinterpret_cast<const float4*>(k + h);
            sum += ex2(1.44269504f * fmaf(x[h] * rsc, k4.x, -l4.x)) + ex2(1.44269504f * fmaf(x[h + 1] * rsc, k4.y, -l4.y)) +
                   (ex2(1.44269504f * fmaf(x[h + 2] * rsc, k4.z, -l4.z)) + ex2(1.44269504f * fmaf(x[h + 3] * rsc, k4.w, -l4.w)));
          }
          return sum;
        };
        auto taken = [&]() {      // the score buffer has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(WB_SE + group));
        };
        float sum = 0.f;
        if constexpr (kFp8) {
          // 16 heads at a time: high parts from column 16 g, low parts from 64 + 16 g
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float x[16], lo[16];
            tmem_ld_32x32b_x16(d + 16u * (uint32_t)g, x);
            tmem_ld_32x32b_x16(d + 64u + 16u * (uint32_t)g, lo);
            tmem_wait_ld();
            if (g == 3) taken();
#pragma unroll
            for (int h = 0; h < 16; ++h) x[h] += lo[h];
            sum += weigh(x, lse + 16 * g, kh + 16 * g);
          }
        } else {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float x[16], y[16];
            tmem_ld_16x32bx2_x16(d + 16u * (uint32_t)g, x);
#pragma unroll
            for (int a = 1; a < C::kAccs; ++a) {
              tmem_ld_16x32bx2_x16(d + (uint32_t)(a * C::kMmaN) + 16u * (uint32_t)g, y);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < 16; ++h) x[h] += y[h];
            }
            if (g == 1) taken();
            sum += weigh(x, lse + 16 * g, kh + 16 * g);
          }
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        }
        const int at = tin * kM + e;
        if (half == 0 && at < p.topk) p.out[(size_t)row * p.topk + at] = r >= 0 ? sum : 0.f;
      }
      if (++tin == nt) {
        tin = 0;
        ++row;
      }
    }
  } else if (C::kHelpers > 0 && warp > kWtEpiWarps + C::kCopyWarps) {
    // ---------------------------------------------------------- query helpers
    const int hw = warp - 1 - C::kCopyWarps;          // 8 .. 15: their place among the staging warps
    int row = row0, tin = tin0, seg = 0;
    for (int t = 0; t < count; t += nt - tin, tin = 0, ++row, ++seg) {
      if (t > 0 && !wait_all(WB_ROW, (seg - 1) & 1)) break;
      wt_stage_query<kKind, C::kQHeads>(p, smem, sbase, row, C::kQHeads * hw, lane, s_k + (seg & 1) * 64);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(WB_Q));
    }
  } else {
    // ------------------------------------------------------------- copy warps
    const int cw = warp - 1 - kWtEpiWarps, first = kRows * cw;     // rows first .. first + kRows - 1 of a tile
    // lanes l, l + kRows, ... hold row first + l: the entry of tile t + 3, its
    // rows of tiles t + 2 and t + 1, and tile t's row being copied, so that
    // neither the entry nor its page is waited for
    struct Cursor {
      int row, tin;
    };
    Cursor c2{row0, tin0};
    auto next = [&](Cursor c) -> Cursor { return c.tin + 1 == nt ? Cursor{c.row + 1, 0} : Cursor{c.row, c.tin + 1}; };
    auto entry = [&](Cursor c, int t) -> int {
      const int at = c.tin * kM + first + (lane & (kRows - 1));
      return t < count && at < p.topk ? __ldg(p.indices + (size_t)c.row * p.topk + at) : -1;
    };
    // DeepSeek-V4: a tile's part in registers.  Lane l has chunk l (16 codes, or
    // from chunk 28 on eight bf16 dims) of each of the warp's rows and the scale
    // of its 64 dims; lanes 0 - 15 also one of the rows' last four chunks.
    uint4 va[kRows + 1], vb[kRows + 1];
    uint32_t sa[kRows], sb[kRows];
    auto dsv4_load = [&](int rows, uint4 (&v)[kRows + 1], uint32_t (&sc)[kRows]) {
#pragma unroll
      for (int u = 0; u <= kRows; ++u) {
        const int r = __shfl_sync(0xffffffffu, rows, u < kRows ? u : (lane >> 2) & (kRows - 1));
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (u < kRows) sc[u] = 127u;
        if (r < 0 || (u == kRows && lane >= 4 * kRows)) continue;
        const uint8_t* page = p.kv + (size_t)(r >> 6) * kDsv4Page;
        v[u] = __ldg(reinterpret_cast<const uint4*>(page + (r & 63) * kDsv4Slot + 16 * (u < kRows ? lane : 32 + (lane & 3))));
        if (u < kRows && lane < 28) sc[u] = __ldg(page + kDsv4ScaleOff + (r & 63) * 8 + (lane >> 2));
      }
    };
    const int i0 = entry(c2, 0);
    c2 = next(c2);
    const int i1 = entry(c2, 1);
    int r0 = resolve_row(p, i0, row0), r1 = resolve_row(p, i1, c2.row);
    c2 = next(c2);
    int i2 = entry(c2, 2);
    // one tile: true unless a wait gave up.  (DeepSeek-V4: stores `now`, loads the
    // next tile's part into `then`; the two swap from tile to tile, as moving
    // registers would wait for the loads.)
    auto copy_tile = [&](int t, uint4 (&now)[kRows + 1], uint32_t (&snow)[kRows], uint4 (&then)[kRows + 1],
                         uint32_t (&sthen)[kRows]) -> bool {
      const int stage = t % kStages, rs = (t % kWtRing) * kM;
      const int r2 = resolve_row(p, i2, c2.row);
      c2 = next(c2);
      i2 = entry(c2, t + 3);
      const uint32_t base = sbase + (uint32_t)(stage * C::kStageBytes);
      if constexpr (kDsv4) {
        // codes to bf16 on the way
        dsv4_load(r1, then, sthen);
        if (t >= kStages && !wait_all(WB_EMPTY + stage, ((t / kStages) - 1) & 1)) return false;
        const int g = lane >> 2;
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int tok = first + u;
          if (lane < 28) {
            const uint32_t s2 = ue8m0_bf16x2(snow[u]);
            uint4 lo, hi;
            e4m3x4_to_bf16x4_scaled(now[u].x, s2, lo.x, lo.y);
            e4m3x4_to_bf16x4_scaled(now[u].y, s2, lo.z, lo.w);
            e4m3x4_to_bf16x4_scaled(now[u].z, s2, hi.x, hi.y);
            e4m3x4_to_bf16x4_scaled(now[u].w, s2, hi.z, hi.w);
            st_shared_v4(base + g * kAtom + sw128_off(tok, 2 * (lane & 3)), lo);
            st_shared_v4(base + g * kAtom + sw128_off(tok, 2 * (lane & 3) + 1), hi);
          } else {
            st_shared_v4(base + 7 * kAtom + sw128_off(tok, lane - 28), now[u]);
          }
        }
        if (lane < 4 * kRows) st_shared_v4(base + 7 * kAtom + sw128_off(first + g, 4 + (lane & 3)), now[kRows]);
        if (lane < kRows) s_row[rs + first + lane] = r0;
        fence_proxy_async_smem();
      } else {
        if (t >= kStages && !wait_all(WB_EMPTY + stage, ((t / kStages) - 1) & 1)) return false;
        // one instruction per row and 512 bytes, then the rows' tails
        // together.  Absent rows read nothing and are zero.
#pragma unroll
        for (int rr = 0; rr < kRows; ++rr) {
          const int r = __shfl_sync(0xffffffffu, r0, rr);
          const uint32_t n = r >= 0 ? 16u : 0u;
          const uint8_t* src = p.kv + (size_t)(r >= 0 ? r : 0) * C::kRowBytes + lane * 16;
          if constexpr (kFp8) {
            cp_async_16(base + wt_off8<kM>(first + rr, lane), src, n);
          } else {
            const uint32_t at = base + (uint32_t)((lane >> 3) * kAtom) + sw128_off(first + rr, lane & 7);
            cp_async_16(at, src, n);
            cp_async_16(at + 4 * kAtom, src + 512, n);
          }
        }
        if constexpr (kFp8) {
#pragma unroll
          for (int hh = 0; hh < kRows / 8; ++hh) {
            const int rr = 8 * hh + (lane >> 2), r = __shfl_sync(0xffffffffu, r0, rr);
            cp_async_16(base + wt_off8<kM>(first + rr, 32 + (lane & 3)),
                        p.kv + (size_t)(r >= 0 ? r : 0) * C::kRowBytes + 512 + (lane & 3) * 16, r >= 0 ? 16u : 0u);
          }
          // the row's scale rides along (a copy of four bytes)
          if (lane < kRows)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(s_scale + rs + first + lane)),
                         "l"(p.kv_row_scale + (r0 >= 0 ? r0 : 0)) : "memory");
        } else {
#pragma unroll
          for (int hh = 0; hh < kRows / 4; ++hh) {
            const int rr = 4 * hh + (lane >> 3), r = __shfl_sync(0xffffffffu, r0, rr);
            cp_async_16(base + 8 * kAtom + sw128_off(first + rr, lane & 7),
                        p.kv + (size_t)(r >= 0 ? r : 0) * C::kRowBytes + 1024 + (lane & 7) * 16, r >= 0 ? 16u : 0u);
          }
        }
        if (lane < kRows) s_row[rs + first + lane] = r0;
        cp_async_mbar_arrive_noinc(BAR(WB_FULL + stage));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(WB_FULL + stage));
      r0 = r1;
      r1 = r2;
      return true;
    };
    if constexpr (kDsv4) {
      dsv4_load(r0, va, sa);
      for (int t = 0; t < count; t += 2)
        if (!copy_tile(t, va, sa, vb, sb) || (t + 1 < count && !copy_tile(t + 1, vb, sb, va, sa))) break;
    } else {
      for (int t = 0; t < count; ++t)
        if (!copy_tile(t, va, sa, vb, sb)) break;
    }
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, C::kTmem);
}

// ---------------------------------------------------------- accumulation
// One CTA per (sequence, range of kRange positions).  The entries of the
// sequence that fall into the range are summed in 64-bit fixed point in
// shared memory: integer addition is associative, so the result does not
// depend on the order of the atomics, whatever positions repeat.  The unit is
// 2^-s for all ranges of a sequence, s as large as keeps (entries x largest
// |weight|) below 2^62: sums keep at least 46 bits below the largest weight.
// Every CTA reads the sequence's whole list (from L2 after the first); what
// bounds a call is its chain of latencies, so the list's first kAcKeep entries
// per thread and the range's old sums are all loaded at the start (batch 16 x
// 512 entries: 4.7 us with the loads where they are used, 2.3 now).
constexpr int kAcThreads = 512;
constexpr int kAcKeep = 8;             // entries per thread held in registers

struct AccumulateParams {
  const int32_t* indices;
  const float* weights;
  float* acc;
  int entries, max_ctx;      // entries: tokens x topk of a sequence
  int log2_entries;          // entries <= 2^log2_entries
  float decay;
};

template <int kRange>
__global__ void __launch_bounds__(kAcThreads) smla_accumulate_kernel(const AccumulateParams p) {
  constexpr int kPos = kRange / kAcThreads;
  __shared__ long long sum[kRange];
  __shared__ uint32_t bad[kRange / 32];     // positions that got a NaN or an infinity
  __shared__ int s_max;
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x, b = blockIdx.y, p0 = blockIdx.x * kRange;
  const int32_t* idx = p.indices + (size_t)b * p.entries;
  const float* w = p.weights + (size_t)b * p.entries;
  float* acc = p.acc + (size_t)b * p.max_ctx + p0;
  const int here = min(kRange, p.max_ctx - p0);
  int at[kAcKeep];
  float wt[kAcKeep], old[kPos];
#pragma unroll
  for (int j = 0; j < kAcKeep; ++j) {
    const int i = j * kAcThreads + t;
    at[j] = i < p.entries ? __ldg(idx + i) : -1;
    wt[j] = i < p.entries ? __ldg(w + i) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < kPos; ++j) old[j] = j * kAcThreads + t < here ? acc[j * kAcThreads + t] : 0.f;
#pragma unroll
  for (int j = 0; j < kPos; ++j) sum[j * kAcThreads + t] = 0;
  if (t < kRange / 32) bad[t] = 0;
  if (t == 0) s_max = 0;
  __syncthreads();
  // largest finite |weight| (as bits) of the sequence's entries; at least the
  // smallest number where any entry is NaN or infinite
  int m = 0;
  bool outside = false;
  auto look = [&](int pos, float v) {
    const int bits = __float_as_int(fabsf(v));
    outside |= pos >= p.max_ctx;
    if (pos >= 0 && pos < p.max_ctx) m = max(m, bits < 0x7F800000 ? bits : 1);
  };
#pragma unroll
  for (int j = 0; j < kAcKeep; ++j) look(at[j], wt[j]);
  for (int i = kAcKeep * kAcThreads + t; i < p.entries; i += kAcThreads) look(__ldg(idx + i), __ldg(w + i));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((t & 31) == 0 && m > 0) atomicMax(&s_max, m);
  if (outside && p0 == 0) atomicOr(&g_error_word, 4u);
  __syncthreads();
  m = s_max;
  if (m == 0 && p.decay == 1.0f) return;
  // largest < 2^(e + 1): the unit's exponent
  const int e = m >= 0x800000 ? (m >> 23) - 127 : -126;
  const int s = 62 - p.log2_entries - (e + 1);
  auto power = [](int k) -> double { return __longlong_as_double((long long)(1023 + k) << 52); };
  const double up = power(s), down = power(-s);
  auto add = [&](int pos, float v) {
    if (pos < p0 || pos - p0 >= here) return;
    pos -= p0;
    if (fabsf(v) < INFINITY) {
      // 64 bits as two native 32-bit additions with the carry between them
      const unsigned long long x = (unsigned long long)__double2ll_rn((double)v * up);
      uint32_t* at2 = reinterpret_cast<uint32_t*>(&sum[pos]);
      const uint32_t before = atomicAdd(at2, (uint32_t)x);
      const uint32_t high = (uint32_t)(x >> 32) + (before + (uint32_t)x < before ? 1u : 0u);
      if (high) atomicAdd(at2 + 1, high);
    } else {
      atomicOr(&bad[pos >> 5], 1u << (pos & 31));
    }
  };
#pragma unroll
  for (int j = 0; j < kAcKeep; ++j) add(at[j], wt[j]);
  for (int i = kAcKeep * kAcThreads + t; i < p.entries; i += kAcThreads) add(__ldg(idx + i), __ldg(w + i));
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPos; ++j) {
    const int i = j * kAcThreads + t;
    if (i >= here) continue;
    const long long v = sum[i];
    const bool nan = (bad[i >> 5] >> (i & 31)) & 1u;
    if (v == 0 && !nan && p.decay == 1.0f) continue;
    const float r = (float)fma((double)old[j], (double)p.decay, (double)v * down);
    acc[i] = nan ? __int_as_float(0x7FC00000) : r;
  }
}

// ------------------------------------------------------------------ host
template <int kKind>
static cudaError_t launch_weights(WeightsParams& p, cudaStream_t stream) {
  static volatile int done[64] = {0};
  constexpr int bytes = WtCfg<kKind>::kSmemBytes;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(smla_weights_kernel<kKind>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = 1;
  }
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  void* args[] = {&p};
  return launch_pdl((const void*)smla_weights_kernel<kKind>, dim3((unsigned)(p.total < sms ? p.total : sms)),
                    dim3(WtCfg<kKind>::kThreads), bytes, stream, args);
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
  const int m = fp8 ? WtCfg<kKindFp8>::kM : (s->kv_dtype == SMLA_KV_DSV4_PAGED ? WtCfg<kKindDsv4>::kM : WtCfg<kKindBf16>::kM);
  p.ntiles = (s->topk + m - 1) / m;
  p.total = (long long)rows_of(s) * p.ntiles;
  p.scale = scale;
  const cudaError_t e = fp8 ? launch_weights<kKindFp8>(p, stream)
                            : (s->kv_dtype == SMLA_KV_DSV4_PAGED ? launch_weights<kKindDsv4>(p, stream)
                                                                : launch_weights<kKindBf16>(p, stream));
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
  // Narrow ranges while each CTA has an SM to itself (every CTA reads the whole
  // list).  1,024 / 2,048 / 4,096 positions: 16 x 512 entries 2.3 / 2.7 / 3.3 us,
  // 64 x 4,096 entries 6.2 / 5.1 / 3.9, both over 8,192 positions, in a graph.
  const int sms = device_sm_count();
  if (sms <= 0) return SMLA_ERR_CUDA;
  int range = 1024;
  auto ranges = [&]() -> long long { return (max_ctx + range - 1) / range; };
  while (range < 4096 && batch * ranges() > sms) range *= 2;
  const void* kern = range == 1024 ? (const void*)smla_accumulate_kernel<1024>
                                   : (range == 2048 ? (const void*)smla_accumulate_kernel<2048> : (const void*)smla_accumulate_kernel<4096>);
  const cudaError_t e = launch_pdl(kern, dim3((unsigned)ranges(), (unsigned)batch), dim3(kAcThreads), 0, stream, args);
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
