// Cache append: new tokens' rows, normalised, rotated and encoded, into the
// cache layouts that the decode reads.  Included by sparse_mla.cu after
// rope.cuh (same translation unit).
//
// One token (row x of 576 dims; 512 for DeepSeek-V4 pages):
//   x[0:512]  -> w x / sqrt(mean(x[0:512]^2) + eps)        (with a weight)
//   last 64   -> turned by the token's position             (with a table)
//   row       -> bf16, or e4m3 codes with the row scale amax / 448, or
//                DeepSeek-V4: 448 e4m3 codes with a power-of-two scale per
//                64 dims, then 64 bf16 dims
// All of it in fp32 with one rounding at the end (the scale is a rounding of
// its own): the row is read once and written once.

namespace smla {

constexpr int kApWarps = 4;            // warps per CTA, one token per warp at a time
constexpr int kApCtas = 6;             // CTAs per SM (80 registers a thread)
constexpr int kApStages = 3;           // rows of its run that a warp has under way

static_assert(sizeof(smla_append_shape) == 56 && offsetof(smla_append_shape, x_dtype) == 24, "smla_append_shape layout");

struct AppendParams {
  const void* x;
  const float* norm_weight;       // [512] or null
  const int32_t* positions;       // [tokens] (with a rotation)
  const int32_t* slots;           // [tokens]
  const int32_t* seq;             // [tokens] or null
  const int32_t* page_table;      // [batch, pages_per_seq] (paged)
  uint8_t* kv;
  float* kv_row_scale;
  long long tokens, x_stride, num_kv_rows;
  int page_size, pages_per_seq, batch, tok_per_seq;
  float eps;
  int rotate;
  int run;                        // consecutive tokens per warp, at most 32
  smla_rope_table table;
};

// eight consecutive elements, as stored
template <typename T, bool kVec>
__device__ __forceinline__ RopeVec<T, 8> ap_load8(const T* src) {
  RopeVec<T, 8> r;
  if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = src[i];
  } else {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(src)[i];
  }
  return r;
}
// two fp32 at a time (the packed instructions issue once for both)
__device__ __forceinline__ void ap_mul2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void ap_fma2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 d, {%0, %1};\n\t"
      "fma.rn.f32x2 d, a, b, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void ap_scale8(float (&v)[8], float s) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) ap_mul2(v[j], v[j + 1], s, s);
}
__device__ __forceinline__ void ap_mul8(float (&v)[8], const float (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) ap_mul2(v[j], v[j + 1], w[j], w[j + 1]);
}
__device__ __forceinline__ float ap_rcp(float x) {     // within one ulp
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x (not negative) in [2^-96, 2^96): two integer instructions
__device__ __forceinline__ bool ap_ordinary(float x) {
  return __float_as_uint(x) - (31u << 23) < (192u << 23);
}
// eight fp32 -> eight e4m3 codes
__device__ __forceinline__ uint2 ap_codes8(const float (&v)[8]) {
  return make_uint2(pack_e4m3x2(v[0], v[1]) | (pack_e4m3x2(v[2], v[3]) << 16),
                    pack_e4m3x2(v[4], v[5]) | (pack_e4m3x2(v[6], v[7]) << 16));
}
__device__ __forceinline__ float ap_amax8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}
// The UE8M0 byte of a group: the smallest e with amax <= 448 * 2^(e - 127),
// at least 1.  amax = 1.m * 2^k and 448 = 1.75 * 2^8, so e - 127 is k - 8
// while the significand is at most 1.75 and k - 7 above it.
__device__ __forceinline__ uint32_t ap_ue8m0(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : (e > 254 ? 254 : e));
}

// One warp per token.  Lane l holds dims 8 l .. 8 l + 7 and 256 + 8 l .. +7
// of the 512 normalised dims, and pair l of the 64 rotated ones (read on
// its own: for DeepSeek-V4 pages those are dims 448 - 511, which lanes 24 -
// 31 hold too for the mean square).  A group of 64 dims is eight lanes.
//
// A warp takes a run of up to 32 consecutive tokens: their places are worked
// out once, a token per lane, and the rows come by bulk copies into a ring of
// kApStages rows of the warp's own, so that a token's arithmetic waits neither
// for its row nor for its place and holds no registers for rows to come.
// (Rows that are not 16-byte aligned are loaded as they are needed: 65,536
// tokens into fp8 rows 33 us, against 25.)
template <typename T, int kKind, bool kVec>
__global__ void __launch_bounds__(kApWarps * 32, kApCtas) smla_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr bool kDsv4 = kKind == kKindDsv4;
  constexpr int kR = kDsv4 ? 448 : 512;                // first rotated dim
  constexpr int kWidth = kDsv4 ? kDv : kDqk;
  constexpr int kRowB = kWidth * (int)sizeof(T);
  __shared__ __align__(16) uint8_t s_x[kVec ? kApWarps * kApStages * kRowB : 16];
  __shared__ __align__(8) unsigned long long s_bar[kApWarps * kApStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t bar = smem_u32(s_bar + warp * kApStages);
  if (kVec) {
    if (lane == 0) {
      for (int k = 0; k < kApStages; ++k) mbar_init(bar + 8u * (uint32_t)k, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
  }
  grid_dep_wait();
  const long long first = ((long long)blockIdx.x * kApWarps + warp) * p.run;
  const int count = (int)min((long long)p.run, p.tokens - first);
  if (count <= 0) return;
  const T* xs = static_cast<const T*>(p.x) + first * p.x_stride;
  auto fetch = [&](int j) {
    const int st = j % kApStages;
    mbar_arrive_expect_tx(bar + 8u * (uint32_t)st, kRowB);
    bulk_load_g2s(smem_u32(s_x) + (uint32_t)((warp * kApStages + st) * kRowB), xs + j * p.x_stride, kRowB,
                  bar + 8u * (uint32_t)st);
  };
  if (kVec && lane == 0)
    for (int j = 0; j < min(count, kApStages); ++j) fetch(j);
  // lane j: the place of the run's token j and its position.  Slots are
  // physical rows, or positions through the page table of the token's
  // sequence, as the decode's index entries are.  A place: the row, or -1
  // (skipped, or out of range and reported)
  int place = -1, position = 0;
  if (lane < count) {
    const long long i = first + lane;
    const int slot = __ldg(p.slots + i);
    if (p.rotate) position = __ldg(p.positions + i);
    long long row = slot;
    if (p.page_size && slot >= 0) {
      const int seq = p.seq ? __ldg(p.seq + i) : (int)((uint32_t)i / (uint32_t)p.tok_per_seq);
      row = -2;
      if (seq >= 0 && seq < p.batch && (slot >> 6) < p.pages_per_seq) {
        const int page = __ldg(p.page_table + (long long)seq * p.pages_per_seq + (slot >> 6));
        if (page >= 0) row = (long long)page * 64 + (slot & 63);
      }
    }
    if (slot >= 0 && (row < 0 || row >= p.num_kv_rows)) {
      atomicOr(&g_error_word, 4u);
      row = -1;
    }
    place = row >= 0 ? (int)row : -1;
  }
  const bool inter = p.table.layout == SMLA_ROPE_INTERLEAVED;
  const int da = kR + (inter ? 2 * lane : lane), db = inter ? da + 1 : da + 32;
  const unsigned long long turn = p.table.step[lane];
  float w0[8], w1[8], wa = 1.f, wb = 1.f;
  if (p.norm_weight) {
    rope_unpack<float, 8>(ap_load8<float, true>(p.norm_weight + 8 * lane), w0);
    rope_unpack<float, 8>(ap_load8<float, true>(p.norm_weight + 256 + 8 * lane), w1);
    if (kDsv4) {
      wa = __ldg(p.norm_weight + da);
      wb = __ldg(p.norm_weight + db);
    }
  }
  int j = 0;
  for (; j < count; ++j) {
    const long long row = __shfl_sync(0xffffffffu, place, j);
    const int pos = __shfl_sync(0xffffffffu, position, j);
    const T* x = xs + j * p.x_stride;
    if constexpr (kVec) {
      const int st = j % kApStages;
      if (!__all_sync(0xffffffffu, mbar_wait(bar + 8u * (uint32_t)st, (uint32_t)((j / kApStages) & 1)))) break;
      x = reinterpret_cast<const T*>(s_x + (warp * kApStages + st) * kRowB);
    }
    const RopeVec<T, 8> x0 = ap_load8<T, kVec>(x + 8 * lane), x1 = ap_load8<T, kVec>(x + 256 + 8 * lane);
    const T xa = x[da], xb = x[db];
    if (kVec) {
      __syncwarp();                                    // the ring's row has been read by all lanes
      if (lane == 0 && j + kApStages < count) fetch(j + kApStages);
    }
    if (row < 0) continue;                             // no place: nothing is written
    float v0[8], v1[8];
    rope_unpack<T, 8>(x0, v0);
    rope_unpack<T, 8>(x1, v1);
    float a = RopeIo<T>::get(xa), b = RopeIo<T>::get(xb), r = 1.f;
    if (p.norm_weight) {
      float ss = 0.f, ss1 = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        ap_fma2(ss, ss1, v0[j], v0[j + 1], v0[j], v0[j + 1]);
        ap_fma2(ss, ss1, v1[j], v1[j + 1], v1[j], v1[j + 1]);
      }
      ss += ss1;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      // (1 / rms goes to the row's largest value and to the final scaling of
      // fp8 rows, not to every element on the way)
      r = rsqrtf(ss * (1.0f / 512.0f) + p.eps);
      ap_mul8(v0, w0);
      ap_mul8(v1, w1);
      if (kDsv4) {
        a = a * r * wa;
        b = b * r * wb;
      }
    }
    if (p.rotate) {
      float c, s;
      rope_sincos(turn, pos, p.table.mscale, c, s);
      const float ra = fmaf(a, c, -b * s);
      b = fmaf(a, s, b * c);
      a = ra;
    }
    if constexpr (kKind == kKindBf16) {
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.kv) + row * kDqk;
      if (p.norm_weight) {
        ap_scale8(v0, r);
        ap_scale8(v1, r);
      }
      *reinterpret_cast<uint4*>(dst + 8 * lane) = make_uint4(pack_bf16x2(v0[0], v0[1]), pack_bf16x2(v0[2], v0[3]),
                                                             pack_bf16x2(v0[4], v0[5]), pack_bf16x2(v0[6], v0[7]));
      *reinterpret_cast<uint4*>(dst + 256 + 8 * lane) = make_uint4(
          pack_bf16x2(v1[0], v1[1]), pack_bf16x2(v1[2], v1[3]), pack_bf16x2(v1[4], v1[5]), pack_bf16x2(v1[6], v1[7]));
      if (inter) {
        *reinterpret_cast<uint32_t*>(dst + da) = pack_bf16x2(a, b);
      } else {
        dst[da] = __float2bfloat16_rn(a);
        dst[db] = __float2bfloat16_rn(b);
      }
    } else if constexpr (kKind == kKindFp8) {
      // (magnitudes order as their bits do)
      const float latent = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(fmaxf(ap_amax8(v0), ap_amax8(v1)))));
      const float rope = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(fmaxf(fabsf(a), fabsf(b)))));
      const float m = fmaxf(latent * r, rope);
      // a row of zeros keeps scale 1; a scale below the normal range would
      // lose bits, so it stops at 2^-126
      // (m / 448 by its remainder: correctly rounded)
      const float m448 = m * (1.0f / 448.0f);
      const float scale = m > 0.f ? fmaxf(fmaf(fmaf(-m448, 448.0f, m), 1.0f / 448.0f, m448), 1.1754943508222875e-38f) : 1.0f;
      uint8_t* dst = p.kv + row * kRowBytesFp8;
      // x / scale.  Normalised values: by way of the reciprocal (of the largest
      // of them, where that sets the scale: 1 / rms then cancels), within
      // 2^-22, far inside the half step of 2^-4 that the codes round by.  Values as
      // they came have few bits, and can lie on the border between two codes
      // exactly: their quotient is corrected by its remainder, which one fma
      // gives without rounding (P. Markstein, IBM J. Res. Dev. 34 (1990) 111).
      const float inv = ap_rcp(scale);
      auto exact = [&](float x) -> float {
        const float q = x * inv;
        return fmaf(fmaf(-q, scale, x), inv, q);
      };
      if (p.norm_weight) {
        // (One factor only while it is an ordinary number: rows of tiny values
        // would make it infinite, and 0 times infinity a NaN.)
        float f = r * inv;
        if (latent * r >= rope && scale > 1.1754943508222875e-38f && ap_ordinary(latent)) {
          const float y = ap_rcp(latent);
          f = 448.0f * fmaf(fmaf(-latent, y, 1.0f), y, y);
        } else if (!ap_ordinary(f)) {
          ap_scale8(v0, r);
          ap_scale8(v1, r);
          f = inv;
        }
        ap_scale8(v0, f);
        ap_scale8(v1, f);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v0[j] = exact(v0[j]);
          v1[j] = exact(v1[j]);
        }
      }
      *reinterpret_cast<uint2*>(dst + 8 * lane) = ap_codes8(v0);
      *reinterpret_cast<uint2*>(dst + 256 + 8 * lane) = ap_codes8(v1);
      const uint32_t ab = pack_e4m3x2(exact(a), exact(b));
      if (inter) {
        *reinterpret_cast<uint16_t*>(dst + da) = (uint16_t)ab;
      } else {
        dst[da] = (uint8_t)ab;
        dst[db] = (uint8_t)(ab >> 8);
      }
      if (lane == 0) p.kv_row_scale[row] = scale;
    } else {
      // groups 0-3 are lanes 8 g .. 8 g + 7 of v0, groups 4-6 those of v1
      float m0 = ap_amax8(v0) * r, m1 = ap_amax8(v1) * r;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
      }
      const uint32_t e0 = ap_ue8m0(m0), e1 = ap_ue8m0(m1);
      // 2^(127 - e) is a normal number for e <= 253 and halves once more for
      // 254; the product with it is exact
      auto down = [&](float (&v)[8], uint32_t e) {
        const float f = e < 254 ? pow2i(127 - (int)e) : 0.5f * pow2i(-126);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * r * f;
      };
      down(v0, e0);
      down(v1, e1);
      uint8_t* page = p.kv + (row >> 6) * (long long)kDsv4Page;
      uint8_t* dst = page + (row & 63) * kDsv4Slot;
      *reinterpret_cast<uint2*>(dst + 8 * lane) = ap_codes8(v0);
      if (lane < 24) *reinterpret_cast<uint2*>(dst + 256 + 8 * lane) = ap_codes8(v1);
      __nv_bfloat16* rope = reinterpret_cast<__nv_bfloat16*>(dst + kDsv4Nope);
      if (inter) {
        *reinterpret_cast<uint32_t*>(rope + da - kR) = pack_bf16x2(a, b);
      } else {
        rope[da - kR] = __float2bfloat16_rn(a);
        rope[db - kR] = __float2bfloat16_rn(b);
      }
      uint2 block = make_uint2(0u, 0u);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        block.x |= __shfl_sync(0xffffffffu, e0, 8 * g) << (8 * g);
        if (g < 3) block.y |= __shfl_sync(0xffffffffu, e1, 8 * g) << (8 * g);
      }
      if (lane == 0) *reinterpret_cast<uint2*>(page + kDsv4ScaleOff + (row & 63) * 8) = block;
    }
  }
  // a wait gave up: the rows under way land (or run out of time too) before the
  // shared memory is left
  if (kVec)
    for (int k = j; k < min(count, j + kApStages); ++k)
      mbar_wait(bar + 8u * (uint32_t)(k % kApStages), (uint32_t)((k / kApStages) & 1));
}

// ------------------------------------------------------------------ host
template <typename T, int kKind>
static cudaError_t launch_append(AppendParams& p, bool vec, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // runs as long as fill the resident warps once, at most 32 tokens
  const long long resident = (long long)kApCtas * kApWarps * sms;
  p.run = (int)((p.tokens + resident - 1) / resident);
  if (p.run > 32) p.run = 32;
  const long long per_cta = (long long)kApWarps * p.run;
  void* args[] = {&p};
  const void* kern = vec ? (const void*)smla_append_kernel<T, kKind, true> : (const void*)smla_append_kernel<T, kKind, false>;
  return launch_pdl(kern, dim3((unsigned)((p.tokens + per_cta - 1) / per_cta)), dim3(kApWarps * 32), 0, stream, args);
}
template <typename T>
static cudaError_t launch_append_kind(AppendParams& p, int kv_dtype, bool vec, cudaStream_t stream) {
  if (kv_dtype == SMLA_KV_BF16) return launch_append<T, kKindBf16>(p, vec, stream);
  if (kv_dtype == SMLA_KV_FP8_E4M3_ROWSCALE) return launch_append<T, kKindFp8>(p, vec, stream);
  return launch_append<T, kKindDsv4>(p, vec, stream);
}

static smla_status run_append(const smla_append_shape* s, const void* x, const float* norm_weight,
                              const smla_rope_table* table, const int32_t* positions, const int32_t* slots,
                              const int32_t* seq, const int32_t* page_table, void* kv, float* kv_row_scale,
                              cudaStream_t stream) {
  if (!s) return SMLA_ERR_INVALID_ARG;
  const bool fp8 = s->kv_dtype == SMLA_KV_FP8_E4M3_ROWSCALE, dsv4 = s->kv_dtype == SMLA_KV_DSV4_PAGED;
  if (s->kv_dtype != SMLA_KV_BF16 && !fp8 && !dsv4) return SMLA_ERR_UNSUPPORTED;
  if (s->x_dtype < SMLA_DTYPE_BF16 || s->x_dtype > SMLA_DTYPE_FP32) return SMLA_ERR_UNSUPPORTED;
  if (s->page_size != 0 && s->page_size != 64) return SMLA_ERR_UNSUPPORTED;
  if (s->num_kv_rows < 1 || s->num_kv_rows > 0x7FFFFFFFLL) return SMLA_ERR_INVALID_ARG;
  if (dsv4 && (s->page_size != 64 || s->num_kv_rows % 64 != 0)) return SMLA_ERR_UNSUPPORTED;
  if (s->tokens < 0 || s->tokens > 0x7FFFFFFFLL || s->reserved != 0) return SMLA_ERR_INVALID_ARG;
  const int width = dsv4 ? kDv : kDqk;
  if (s->tokens > 1 && s->x_stride != 0 && s->x_stride < width) return SMLA_ERR_INVALID_ARG;
  if (!(s->eps >= 0) || isinf(s->eps)) return SMLA_ERR_INVALID_ARG;
  if (table) {
    const smla_status st = validate_rope_table(table);
    if (st != SMLA_OK) return st;
    if (table->rope_dim != 64) return SMLA_ERR_UNSUPPORTED;
  }
  if (s->page_size) {
    if (s->pages_per_seq < 1 || s->batch < 1) return SMLA_ERR_INVALID_ARG;
    // without a sequence per token, the tokens are shared out evenly
    if (!seq && s->tokens % s->batch != 0) return SMLA_ERR_INVALID_ARG;
  }
  if (fp8 != (kv_row_scale != nullptr)) return SMLA_ERR_INVALID_ARG;
  if (s->tokens == 0) return SMLA_OK;
  const int size = dtype_bytes(s->x_dtype);
  if (!x || !slots || !kv || (table && !positions) || (s->page_size && !page_table)) return SMLA_ERR_INVALID_ARG;
  if (!aligned(x, size) || !aligned(kv, 16) || !aligned(slots, 4) || (fp8 && !aligned(kv_row_scale, 4)) ||
      (norm_weight && !aligned(norm_weight, 16)) || (table && !aligned(positions, 4)) || (seq && !aligned(seq, 4)) ||
      (s->page_size && !aligned(page_table, 4)))
    return SMLA_ERR_INVALID_ARG;
  AppendParams p;
  memset(&p, 0, sizeof(p));
  p.x = x;
  p.norm_weight = norm_weight;
  p.positions = positions;
  p.slots = slots;
  p.seq = seq;
  p.page_table = page_table;
  p.kv = static_cast<uint8_t*>(kv);
  p.kv_row_scale = kv_row_scale;
  p.tokens = s->tokens;
  p.x_stride = s->tokens > 1 ? s->x_stride : 0;
  p.num_kv_rows = s->num_kv_rows;
  p.page_size = s->page_size;
  p.pages_per_seq = s->pages_per_seq;
  p.batch = s->batch;
  p.tok_per_seq = s->page_size && !seq ? (int)(s->tokens / s->batch) : 1;
  p.eps = s->eps;
  p.rotate = table != nullptr;
  if (table) p.table = *table;
  const bool vec = aligned(x, 16) && (p.x_stride * size) % 16 == 0;
  cudaError_t e;
  if (s->x_dtype == SMLA_DTYPE_BF16) e = launch_append_kind<__nv_bfloat16>(p, s->kv_dtype, vec, stream);
  else if (s->x_dtype == SMLA_DTYPE_FP16) e = launch_append_kind<__half>(p, s->kv_dtype, vec, stream);
  else e = launch_append_kind<float>(p, s->kv_dtype, vec, stream);
  return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

}  // namespace smla

extern "C" {

smla_status sparse_mla_cache_append(const smla_append_shape* shape, const void* x, const float* norm_weight,
                                    const smla_rope_table* table, const int32_t* positions, const int32_t* slots,
                                    const int32_t* seq, const int32_t* page_table, void* kv_cache,
                                    float* kv_row_scale, void* stream) {
  return smla::run_append(shape, x, norm_weight, table, positions, slots, seq, page_table, kv_cache, kv_row_scale,
                          static_cast<cudaStream_t>(stream));
}

}  // extern "C"
