// Attention weights: how much of the decode's attention each listed cache row
// received, and the sum of that over steps per cache position.  Included by
// sparse_mla.cu (same translation unit).
//
//   w[r, j]   = sum_h exp(scale * <q[r, h], k_j> - lse[r, h])      (0 for padding)
//   acc[b, p] = decay * acc[b, p] + sum over (t, j) with indices[b, t, j] = p of w[b, t, j]

namespace smla {

constexpr int kWtEpiWarps = 8;
constexpr int kWtRing = 8;                         // tiles whose rows and scales are kept
// Shared-memory operands are 128-byte-swizzled atoms of [rows][128 B].  Of a
// 576-byte fp8 row the last 64 bytes, of a DeepSeek-V4 row's 448 codes the last
// 64, are a 64-byte-swizzled atom [rows][64 B]; its 64 bf16 dims follow in an
// atom of their own.
template <int kKind>
struct WtCfg {
  static constexpr bool kFp8 = kKind == kKindFp8, kDsv4 = kKind == kKindDsv4;
  static constexpr bool kCodes = kFp8 || kDsv4;                    // multiplied as stored
  static constexpr int kQK = kDsv4 ? 512 : kDqk;
  static constexpr int kRowBytes = kCodes ? 576 : 2 * kQK;         // of an operand row
  // Entries per tile = MMA M.  The tensor cores take as long for 64 rows as
  // for 128: rows of codes, whose bytes arrive fastest per MMA, need the full rate
  // (64 rows: 47.8 us on the batch of 128, the MMAs busy 63 % of it).
  static constexpr int kM = kCodes ? 128 : 64;
  static constexpr int kAtom = kM * 128;                           // 128 bytes of each of the rows
  static constexpr int kStages = 2;
  static constexpr int kStageBytes = kM * kRowBytes;
  static constexpr int kCopyWarps = 8;
  static constexpr int kRows = kM / kCopyWarps;                    // rows of a tile per copy warp
  // Codes: eight warps more help the epilogue warps to stage the query.  Staged by
  // eight, a row's query took 10,000 cycles, longer than two stages of copies
  // last; by the copy warps too, it held up the copies.
  static constexpr int kHelpers = kCodes ? 8 : 0;
  static constexpr int kThreads = 32 * (1 + kWtEpiWarps + kCopyWarps + kHelpers);
  static constexpr int kQWarps = kWtEpiWarps + kHelpers;           // that stage the query
  static constexpr int kQHeads = kH / kQWarps;
  static constexpr int kQRows = kFp8 ? 128 : 64;                   // fp8: the heads' high parts, then their low parts
  static constexpr int kQPart = 64 * 448;                          // DeepSeek-V4: high parts, low parts, then the bf16 dims
  static constexpr int kQBytes = kDsv4 ? 2 * kQPart + 64 * 128 : kQRows * kRowBytes;
  static constexpr int kMmaN = kQRows;
  // bf16 operands: the K steps go to four accumulators, added in the epilogue.
  // The tensor cores cut every update of an accumulator to fp32, an error in
  // proportion to its value and all of one sign; in a quarter each, partial
  // sums are a quarter as large (one sequence, scores up to 20: relative
  // error of the weights 7.7e-6 with one accumulator, 1.4e-6 with four; 1 % of
  // the time).  fp8 rows take half the steps, in two parts already.
  // DeepSeek-V4 rows: one accumulator per scale group, whose scales the epilogue
  // applies, and one for the bf16 dims: all of tensor memory, so one buffer.
  static constexpr int kAccs = kFp8 ? 1 : (kDsv4 ? 8 : 4);
  static constexpr int kN = kAccs * kMmaN;                         // columns of a score buffer
  static constexpr int kBufs = kDsv4 ? 1 : 2;
  static constexpr uint32_t kTmem = kBufs * kN;
  static constexpr int kSmemQ = kStages * kStageBytes;
  static constexpr int kSmemRow = kSmemQ + kQBytes;                // int  [kWtRing][kM] physical row or -1
  static constexpr int kSmemScale = kSmemRow + kWtRing * kM * 4;   // [kWtRing][kM] scales (codes)
  static constexpr int kScaleBytes = kDsv4 ? 8 : 4;                // DeepSeek-V4: the row's block of scales
  static constexpr int kSmemLse = kSmemScale + kWtRing * kM * kScaleBytes;   // f32  [2][64] by row parity
  static constexpr int kSmemK = kSmemLse + 2 * 64 * 4;             // f32  [2][64] scale, over the query's power of two
  static constexpr int kSmemPart = kSmemK + 2 * 64 * 4;            // f32  [2][kM] sums of heads 32-63 (DeepSeek-V4), by tile parity
  static constexpr int kSmemBar = kSmemPart + (kDsv4 ? 2 * kM * 4 : 0);
  static constexpr int kSmemTmem = kSmemBar + 8 * 24;
  static constexpr int kSmemBytes = kSmemTmem + 16;
  static_assert(kSmemBytes <= 232448, "exceeds the 227 KB per-CTA shared memory of sm_100");
  static_assert(kSmemQ % 1024 == 0 && kStageBytes % 1024 == 0, "swizzled operands need 1024-byte aligned atoms");
  // Reuse of the row / scale ring: tile t + stages + 2 is copied after MMA(t + 2) has completed, which waited for
  // the epilogue of tile t to have read its slot.
  static_assert(kWtRing >= kStages + 2, "row ring");
};
constexpr uint32_t kIdescWt = make_idesc(64, 64, false, false), kIdescWt8 = make_idesc_e4m3(128, 128, false);
constexpr uint32_t kIdescWtGroup = make_idesc_e4m3(128, 64, false), kIdescWtRope = make_idesc(128, 64, false, false);
constexpr uint32_t kIdescWtLow = kIdescWtGroup | (1u << 10);         // B e5m2 (format 1 in bits 10-12)
// barriers
constexpr int WB_FULL = 0, WB_EMPTY = 4, WB_SF = 8, WB_SE = 10, WB_Q = 12, WB_FIN = 13, WB_ROW = 14, WB_PART = 16;

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

// and of a DeepSeek-V4 slot: 28 chunks of codes, then eight of bf16 dims
template <int kRows>
__device__ __forceinline__ uint32_t wt_off_codes(int r, int c) {
  return c < 24 ? (uint32_t)((c >> 3) * (kRows * 128)) + sw128_off(r, c & 7) : (uint32_t)(3 * kRows * 128) + sw64_off(r, c - 24);
}
template <int kRows>
__device__ __forceinline__ uint32_t wt_off_slot(int r, int c) {
  return c < 28 ? wt_off_codes<kRows>(r, c) : (uint32_t)(448 * kRows) + sw128_off(r, c - 28);
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
// x (f16x2, |x| < 448) = hi + lo: hi = e4m3(x), lo = e4m3(x - hi), or e5m2(x - hi)
template <bool kLowE5m2>
__device__ __forceinline__ void split_f16(uint32_t x, uint32_t& hi, uint32_t& lo) {
  uint16_t h, l;
  uint32_t h16, r16;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(x));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h16) : "h"(h));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r16) : "r"(x), "r"(h16));
  if constexpr (kLowE5m2) asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(l) : "r"(r16));
  else asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(r16));
  hi = h;
  lo = l;
}

// kHeads heads of a row's query (h0 ..) into the B operand, by one warp.
// bf16 caches: as they are.  Codes: times the power of two that brings the
// head's largest |q| into [128, 256), split into a high and a low part.  fp8 rows:
// both e4m3, as in the decode (exact for the bf16 values whose parts are e4m3
// normals, within 2^-10 of the scaled value otherwise).  DeepSeek-V4: the low part
// is e5m2, which holds the up to three significant bits that e4m3 leaves of a
// bf16 value over a range 2^8 times as wide (one dim of 300 beside N(0, 1) ones:
// largest error of a weight 6e-6 to 1.5e-5 of it, with an e4m3 low part 5e-4 to
// 1e-3): exact down to 2^-6 of the scaled value, within 2^-14 below; the decode
// multiplies these queries as bf16, and its lse comes from there.  s_k[h] receives
// scale over that power.  This runs once per row between two rows' products, at a
// warp's own pace (a few cycles an instruction), so it is spread over as many
// warps as there are and kept short: bf16 pairs are scaled as pairs and split as
// f16 pairs.  (DeepSeek-V4's last 64 dims are scaled alike and stay bf16.)
template <int kKind, int kHeads>
__device__ __forceinline__ void wt_stage_query(const WeightsParams& p, uint8_t* smem, uint32_t sbase, int row, int h0,
                                               int lane, float* s_k) {
  using C = WtCfg<kKind>;
  constexpr int kChunks = C::kQK / 8;               // 16-byte chunks of a head
  const uint8_t* q = p.q + ((size_t)row * kH + h0) * (C::kQK * 2);
  const uint32_t qb = sbase + C::kSmemQ;
  if constexpr (!C::kCodes) {
    for (int c = lane; c < kHeads * kChunks; c += 32) {
      const int h = c / kChunks, j = c - h * kChunks;
      cp_async_16(qb + (uint32_t)((j >> 3) * (C::kQRows * 128)) + sw128_off(h0 + h, j & 7), q + (size_t)c * 16, 16u);
    }
    cp_async_wait_all();
  } else {
    // lane l: chunks l, 32 + l and, where there are 72, of lanes 0-7, 64 + l
    constexpr int kUnits = C::kDsv4 ? 2 : 3;
    uint4 v[kHeads][kUnits];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const uint4* src = reinterpret_cast<const uint4*>(q + (size_t)i * (C::kQK * 2));
      v[i][0] = __ldg(src + lane);
      v[i][1] = __ldg(src + 32 + lane);
      if constexpr (kUnits == 3) v[i][2] = lane < 8 ? __ldg(src + 64 + lane) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i;
      // largest magnitude (bf16 bits order as the magnitudes do)
      uint32_t m2 = 0;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
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
      for (int u = 0; u < kUnits; ++u) {
        if (u == 2 && lane >= 8) continue;
        const uint32_t w4[4] = {v[i][u].x, v[i][u].y, v[i][u].z, v[i][u].w};
        if (C::kDsv4 && u == 1 && lane >= 24) {
          st_shared_v4(qb + 2 * C::kQPart + sw128_off(h, lane - 24),
                       make_uint4(bf16x2_mul(w4[0], up), bf16x2_mul(w4[1], up), bf16x2_mul(w4[2], up), bf16x2_mul(w4[3], up)));
          continue;
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t y = bf16x2_mul(w4[k], up);
          split_f16<C::kDsv4>(pack_f16x2(__uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u)), hi[k], lo[k]);
        }
        // eight codes: half of 16-byte chunk (32 u + lane) / 2 of the row
        const int c = (32 * u + lane) >> 1;
        const uint32_t at = (uint32_t)(8 * (lane & 1));
        if constexpr (C::kDsv4) {
          uint8_t* dst = smem + C::kSmemQ + wt_off_codes<64>(h, c) + at;
          *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
          *reinterpret_cast<uint2*>(dst + C::kQPart) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
        } else {
          *reinterpret_cast<uint2*>(smem + C::kSmemQ + wt_off8<C::kQRows>(h, c) + at) =
              make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
          *reinterpret_cast<uint2*>(smem + C::kSmemQ + wt_off8<C::kQRows>(64 + h, c) + at) =
              make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
        }
      }
      if (lane == 0) s_k[h] = p.scale * pow2i(-sq);
    }
  }
}

// The decode rows' tiles are laid end to end and shared out
// evenly over one CTA per SM; every tile's weights are its own, so nothing is
// merged.  Warp roles: one MMA issuer; eight epilogue warps, which also
// stage the query of each row the CTA meets (for codes with eight more);
// the copy warps.
//  * Copy warps resolve and gather kRows rows each of every tile by 16-byte
//    cp.async (lane = chunk of one row, the rows' last 64 bytes merged):
//    conflict-free in the swizzled atoms, two tiles ahead.
//  * S[entries x 64 heads] = K Q^T in tensor memory, two buffers.  fp8 rows
//    are multiplied as stored (kind::f8f6f4) by the query scaled per head by
//    a power of two and split into e4m3 high and low parts, as in the decode:
//    columns 0-63 and 64-127 of the buffer.  DeepSeek-V4 codes too, each group
//    of 64 dims into 64 columns of its own, high and low parts added there
//    (converting the codes to bf16 instead took 14,400 instructions per 64
//    entries, 79 us on 128 x 2,048 entries against 40 so; relative error 1.1e-7
//    then, 0.7e-7 so).
//  * Epilogue warps 0-3 take the even tiles, 4-7 the odd ones; a thread has one
//    entry: of 128-entry tiles all heads, of 64-entry tiles 32, the other 32
//    being its partner's, sixteen lanes on.  DeepSeek-V4 (one buffer): all eight
//    take every tile, warps 4-7 heads 32-63, and hand their sums to warps 0-3.
template <int kKind>
__global__ void __launch_bounds__(WtCfg<kKind>::kThreads, 1) smla_weights_kernel(const __grid_constant__ WeightsParams p) {
  using C = WtCfg<kKind>;
  constexpr bool kFp8 = C::kFp8, kDsv4 = C::kDsv4;
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
      // a copying thread's copies, and each copy warp's row numbers
      mbar_init(BAR(WB_FULL + i), 33 * C::kCopyWarps);
      mbar_init(BAR(WB_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(WB_SF + i), 1);
      mbar_init(BAR(WB_SE + i), kWtEpiWarps / C::kBufs);
    }
    mbar_init(BAR(WB_Q), C::kQWarps);
    mbar_init(BAR(WB_FIN), 1);
    mbar_init(BAR(WB_ROW), 1);
    for (int i = 0; i < 8; ++i) mbar_init(BAR(WB_PART + i), 1);
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
      const int stage = t % kStages, buf = t % C::kBufs;
      if (t == 0 || tin == 0) ok = wait_all(WB_Q, seg++ & 1);
      if (ok && t >= C::kBufs) ok = wait_all(WB_SE + buf, (t / C::kBufs - 1) & 1);
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
      } else if constexpr (kDsv4) {
#pragma unroll
        for (int g = 0; g < 7; ++g) {
          const uint32_t dg = d + (uint32_t)(64 * g);
          // the group's 64 bytes of a row: half an atom, or the 64-byte one
          const uint64_t da = g < 6 ? sw128_desc(a + (g >> 1) * kAtom, 16, 1024) + (uint64_t)((g & 1) * 4) : sw64_desc(a + 3 * kAtom);
          const uint32_t bg = b + (g < 6 ? (g >> 1) : 3) * 8192;
          const uint64_t dh = g < 6 ? sw128_desc(bg, 16, 1024) + (uint64_t)((g & 1) * 4) : sw64_desc(bg);
          const uint64_t dl = dh + (uint64_t)(C::kQPart >> 4);
          mma8_ss_elect(dg, da, dh, kIdescWtGroup, false);
          mma8_ss_elect(dg, da + 2, dh + 2, kIdescWtGroup, true);
          mma8_ss_elect(dg, da, dl, kIdescWtLow, true);
          mma8_ss_elect(dg, da + 2, dl + 2, kIdescWtLow, true);
        }
        const uint64_t ra = sw128_desc(a + 448 * kM, 16, 1024), rb = sw128_desc(b + 2 * C::kQPart, 16, 1024);
        mma_set_elect(d + 448u, ra, rb, kIdescWtRope);
#pragma unroll
        for (int k = 1; k < 4; ++k) mma_acc_elect(d + 448u, ra + (uint64_t)(2 * k), rb + (uint64_t)(2 * k), kIdescWtRope);
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
          if (!C::kCodes) s_k[sb + h0 + lane] = p.scale;
        }
        wt_stage_query<kKind, C::kQHeads>(p, smem, sbase, row, C::kQHeads * ew, lane, s_k + sb);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(WB_Q));
        ++seg;
      }
      if (C::kBufs == 1 || (t & 1) == group) {
        const int buf = C::kBufs == 1 ? 0 : group;
        ok = wait_all(WB_SF + buf, (t / C::kBufs) & 1);
        if (!ok) break;
        tc_fence_after();
        const int rs = (t % kWtRing) * kM + e;
        const int r = s_row[rs];
        const float rsc = kFp8 ? s_scale[rs] : 1.f;
        const uint32_t d = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(buf * C::kN);
        const int hp = kDsv4 ? group : half;                     // which 32 heads
        const float* lse = s_lse + ((seg - 1) & 1) * 64 + 32 * hp;
        const float* kh = s_k + ((seg - 1) & 1) * 64 + 32 * hp;
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
          if (lane == 0) mbar_arrive(BAR(WB_SE + buf));
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
        } else if constexpr (kDsv4) {
          // the entry's scales: bytes 2^(e - 127), e = 0 a subnormal
          const uint2 sc = *reinterpret_cast<const uint2*>(smem + C::kSmemScale + rs * 8);
          auto group_scale = [&](int g) -> float {
            const uint32_t ex = ((g < 4 ? sc.x : sc.y) >> (8 * (g & 3))) & 0xFFu;
            return __uint_as_float(ex ? ex << 23 : 0x00400000u);
          };
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float x[16], y[16], z[16];
            const uint32_t dh = d + (uint32_t)(32 * group + 16 * hh);
            tmem_ld_32x32b_x16(dh + 448u, x);              // the bf16 dims
            tmem_ld_32x32b_x16(dh, y);
            tmem_wait_ld();
            const float s0 = group_scale(0);
#pragma unroll
            for (int h = 0; h < 16; ++h) x[h] = fmaf(y[h], s0, x[h]);
#pragma unroll
            for (int g = 1; g < 7; g += 2) {
              tmem_ld_32x32b_x16(dh + 64u * (uint32_t)g, y);
              tmem_ld_32x32b_x16(dh + 64u * (uint32_t)(g + 1), z);
              tmem_wait_ld();
              if (hh == 1 && g == 5) taken();
              const float sy = group_scale(g), sz = group_scale(g + 1);
#pragma unroll
              for (int h = 0; h < 16; ++h) x[h] = fmaf(z[h], sz, fmaf(y[h], sy, x[h]));
            }
            sum += weigh(x, lse + 16 * hh, kh + 16 * hh);
          }
          // One sum per entry: warps 4-7 hand theirs to warps 0-3, by slots and
          // barriers of the tile's parity.  Both are free again at tile t: its
          // products waited for warps 0-3 to let go of tile t - 1's, after they had
          // ended tile t - 2.  (By one barrier, warps 4-7 could complete tile t + 1's
          // phase while warps 0-3, who let go of the products before they wait
          // here, had not yet seen tile t's.)
          float* part = reinterpret_cast<float*>(smem + C::kSmemPart) + (t & 1) * kM + e;
          if (group == 1) {
            *part = sum;
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(WB_PART + 4 * (t & 1) + quarter));
          } else {
            ok = wait_all(WB_PART + 4 * (t & 1) + quarter, (t >> 1) & 1);
            if (!ok) break;
            sum += *part;
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
        if (half == 0 && (!kDsv4 || group == 0) && at < p.topk) p.out[(size_t)row * p.topk + at] = r >= 0 ? sum : 0.f;
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
    const int i0 = entry(c2, 0);
    c2 = next(c2);
    const int i1 = entry(c2, 1);
    int r0 = resolve_row(p, i0, row0), r1 = resolve_row(p, i1, c2.row);
    c2 = next(c2);
    int i2 = entry(c2, 2);
    for (int t = 0; t < count; ++t) {
      const int stage = t % kStages, rs = (t % kWtRing) * kM;
      const int r2 = resolve_row(p, i2, c2.row);
      c2 = next(c2);
      i2 = entry(c2, t + 3);
      const uint32_t base = sbase + (uint32_t)(stage * C::kStageBytes);
      if (t >= kStages && !wait_all(WB_EMPTY + stage, ((t / kStages) - 1) & 1)) break;
      // one instruction per row and 512 bytes, then the rows' tails
      // together.  Absent rows read nothing and are zero.
      auto row_at = [&](int r) -> const uint8_t* {
        const uint32_t at = (uint32_t)(r >= 0 ? r : 0);
        if constexpr (kDsv4) return p.kv + (size_t)(at >> 6) * kDsv4Page + (at & 63u) * kDsv4Slot;
        else return p.kv + (size_t)at * C::kRowBytes;
      };
#pragma unroll
      for (int rr = 0; rr < kRows; ++rr) {
        const int r = __shfl_sync(0xffffffffu, r0, rr);
        const uint32_t n = r >= 0 ? 16u : 0u;
        const uint8_t* src = row_at(r) + lane * 16;
        if constexpr (kFp8) {
          cp_async_16(base + wt_off8<kM>(first + rr, lane), src, n);
        } else if constexpr (kDsv4) {
          cp_async_16(base + wt_off_slot<kM>(first + rr, lane), src, n);
        } else {
          const uint32_t at = base + (uint32_t)((lane >> 3) * kAtom) + sw128_off(first + rr, lane & 7);
          cp_async_16(at, src, n);
          cp_async_16(at + 4 * kAtom, src + 512, n);
        }
      }
      if constexpr (C::kCodes) {
#pragma unroll
        for (int hh = 0; hh < kRows / 8; ++hh) {
          const int rr = 8 * hh + (lane >> 2), r = __shfl_sync(0xffffffffu, r0, rr), c = 32 + (lane & 3);
          cp_async_16(base + (kDsv4 ? wt_off_slot<kM>(first + rr, c) : wt_off8<kM>(first + rr, c)), row_at(r) + c * 16,
                      r >= 0 ? 16u : 0u);
        }
        // the row's scales ride along (a copy of four or eight bytes)
        if (lane < kRows) {
          const uint32_t dst = sbase + (uint32_t)(C::kSmemScale + (rs + first + lane) * C::kScaleBytes);
          const uint32_t at = (uint32_t)(r0 >= 0 ? r0 : 0);
          if constexpr (kDsv4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst),
                         "l"(p.kv + (size_t)(at >> 6) * kDsv4Page + kDsv4ScaleOff + (at & 63u) * 8) : "memory");
          else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(p.kv_row_scale + at) : "memory");
        }
      } else {
#pragma unroll
        for (int hh = 0; hh < kRows / 4; ++hh) {
          const int rr = 4 * hh + (lane >> 3), r = __shfl_sync(0xffffffffu, r0, rr);
          cp_async_16(base + 8 * kAtom + sw128_off(first + rr, lane & 7), row_at(r) + 1024 + (lane & 7) * 16, r >= 0 ? 16u : 0u);
        }
      }
      if (lane < kRows) s_row[rs + first + lane] = r0;
      cp_async_mbar_arrive_noinc(BAR(WB_FULL + stage));
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(WB_FULL + stage));
      r0 = r1;
      r1 = r2;
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
// depend on the order of the atomics, whatever positions repeat.  Each position
// has a unit of its own, 2^-s, s as large as keeps (entries x its largest
// |weight|) below 2^62: a sum keeps 61 - log2(entries, rounded up to a power of
// two) bits below that weight (49 of 4,096 entries, 33 of 2^28), whatever weight
// other positions got (with one unit for a whole sequence, 5e-14 beside a 64 was lost).
// So the range's entries are gone through twice, for the largest weights and
// for the sums.
// Every CTA reads the sequence's whole list (from L2 after the first); what
// bounds a call is its chain of latencies, so the list's first kAcKeep entries
// per thread and the range's old sums are all loaded at the start (batch 16 x
// 512 entries: 4.7 us with the loads where they are used, 2.3 so).
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
  __shared__ uint32_t top[kRange];          // the largest |weight|, as bits (at most 48 KB in all)
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
  for (int j = 0; j < kPos; ++j) {
    sum[j * kAcThreads + t] = 0;
    top[j * kAcThreads + t] = 0;
  }
  __syncthreads();
  bool any = false, outside = false;
  // place of an entry in the range; -1: it takes no part in the sums
  auto look = [&](int entry, float v) -> int {
    outside |= entry >= p.max_ctx;
    const uint32_t pos = (uint32_t)entry - (uint32_t)p0, bits = __float_as_uint(fabsf(v));
    if (pos >= (uint32_t)here || bits == 0) return -1;
    any = true;
    atomicMax(&top[pos], bits);                      // (an infinity or a NaN stands above all numbers)
    return bits < 0x7F800000u ? (int)pos : -1;
  };
#pragma unroll
  for (int j = 0; j < kAcKeep; ++j) at[j] = look(at[j], wt[j]);
  for (int i = kAcKeep * kAcThreads + t; i < p.entries; i += kAcThreads) look(__ldg(idx + i), __ldg(w + i));
  if (outside && p0 == 0) atomicOr(&g_error_word, 4u);
  if (!__syncthreads_or(any) && p.decay == 1.0f) return;
  // a number of exponent field f is below 2^(f - 126) (subnormal ones: as of field 1)
  const int s0 = 62 - p.log2_entries + 126;
  auto field = [&](int pos) -> int { return max((int)(top[pos] >> 23), 1); };
  auto power = [](int k) -> double { return __hiloint2double((1023 + k) << 20, 0); };
  auto add = [&](int pos, float v) {
    // 64 bits as two native 32-bit additions with the carry between them
    const unsigned long long x = (unsigned long long)__double2ll_rn((double)v * power(s0 - field(pos)));
    uint32_t* at2 = reinterpret_cast<uint32_t*>(&sum[pos]);
    const uint32_t before = atomicAdd(at2, (uint32_t)x);
    const uint32_t high = (uint32_t)(x >> 32) + (before + (uint32_t)x < before ? 1u : 0u);
    if (high) atomicAdd(at2 + 1, high);
  };
#pragma unroll
  for (int j = 0; j < kAcKeep; ++j)
    if (at[j] >= 0) add(at[j], wt[j]);
  for (int i = kAcKeep * kAcThreads + t; i < p.entries; i += kAcThreads) {
    const uint32_t pos = (uint32_t)__ldg(idx + i) - (uint32_t)p0;
    const float v = __ldg(w + i);
    if (pos < (uint32_t)here && fabsf(v) < INFINITY) add((int)pos, v);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPos; ++j) {
    const int i = j * kAcThreads + t;
    if (i >= here) continue;
    const long long v = sum[i];
    const bool nan = top[i] >= 0x7F800000u;
    if (v == 0 && !nan && p.decay == 1.0f) continue;
    const float r = (float)fma((double)old[j], (double)p.decay, (double)v * power(field(i) - s0));
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
  // list).  1,024 / 2,048 / 4,096 positions: 16 x 512 entries 2.3 / 2.6 / 3.1 us,
  // 64 x 4,096 entries 6.8 / 4.4 / 3.8, both over 8,192 positions, in a graph.
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
