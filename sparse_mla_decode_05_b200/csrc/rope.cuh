// Rotary positions: the rotation of part of each head by its token's
// position, and the table of frequencies it works from.  Included by
// sparse_mla.cu (same translation unit).
//
// Pair (a, b) of a head at position p, with frequency f_i radians per
// position:
//   y_a = m (a cos(p f_i) - b sin(p f_i)),  y_b = m (a sin(p f_i) + b cos(p f_i))
// and with `transpose` the angle's sign turned, which is the gradient of
// that map (and its inverse when m = 1).  The pairs are (2 i, 2 i + 1)
// (interleaved) or (i, i + rope_dim / 2) (half).
//
// Angles.  p f_i in fp32 loses the angle of far positions (2^-24 of
// thousands of turns), so the table holds each frequency as a 64-bit
// fraction of a turn, f_i / (2 pi) * 2^64, and the kernel multiplies it by
// the position modulo 2^64: whole turns drop out of the product exactly,
// negative positions included.  What remains is rounded to 32 bits of a turn
// (1.5e-9 rad), so cos and sin are within a few fp32 roundings of their
// values at any int32 position.

namespace smla {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;          // head rows whose loads a thread has in flight

static_assert(sizeof(smla_rope_table) == 16 + 8 * SMLA_ROPE_MAX_DIM / 2 && offsetof(smla_rope_table, step) == 16,
              "smla_rope_table layout");
static_assert(sizeof(smla_rope_shape) == 64 && offsetof(smla_rope_shape, x_token_stride) == 32, "smla_rope_shape layout");

// cos and sin of position p at table entry `step`, times m.  The fraction of a
// turn is split into the nearest quarter and a rest of at most an eighth
// either way; sin and cos of the rest (at most pi / 4) are their Taylor
// series up to x^9 and x^8 (truncation below 2^-28 and 2^-25), turned by the
// quarter.  Within 2^-22 of the values by the roundings (1.4 x 2^-24 measured), in
// about half the instructions of a general sincos, as the reduction is already
// done by the integer product.
__device__ __forceinline__ void rope_sincos(unsigned long long step, int p, float m, float& c, float& s) {
  const unsigned long long turn = step * (unsigned long long)(long long)p;
  const uint32_t t = (uint32_t)((turn + 0x80000000ull) >> 32);         // 2^-32 turns
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const float x = (float)(int)(t - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi 2^-32
  const float x2 = x * x;
  float sx = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);                  // 1 / 9!, -1 / 7!
  sx = fmaf(x2, sx, 8.3333333e-3f);                                    // 1 / 5!
  sx = fmaf(x2, sx, -0.16666667f);                                     // -1 / 3!
  sx = fmaf(x * x2, sx, x);
  float cx = fmaf(x2, 2.4801587e-5f, -1.3888889e-3f);                  // 1 / 8!, -1 / 6!
  cx = fmaf(x2, cx, 4.1666667e-2f);                                    // 1 / 4!
  cx = fmaf(x2, cx, -0.5f);
  cx = fmaf(x2, cx, 1.0f);
  // a quarter turn on: (cos, sin) -> (-sin, cos)
  const float ca = (quarter & 1u) ? sx : cx, sa = (quarter & 1u) ? cx : sx;
  c = __uint_as_float(__float_as_uint(ca * m) ^ (((quarter + 1u) & 2u) << 30));
  s = __uint_as_float(__float_as_uint(sa * m) ^ ((quarter & 2u) << 30));
}

// Element types: a vector is 16 bytes (kV elements), or one element.
template <typename T> struct RopeIo;
template <> struct RopeIo<__nv_bfloat16> {
  __device__ static float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  __device__ static __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct RopeIo<__half> {
  __device__ static float get(__half v) { return __half2float(v); }
  __device__ static __half put(float v) { return __float2half_rn(v); }
};
template <> struct RopeIo<float> {
  __device__ static float get(float v) { return v; }
  __device__ static float put(float v) { return v; }
};
template <typename T, int kN>
struct alignas(sizeof(T) * kN) RopeVec {
  T v[kN];
};

struct RopeParams {
  const void* x;
  void* y;
  const int32_t* positions;     // [tokens]
  long long xt, xh, yt, yh;     // strides in elements
  int tokens, heads, groups;    // groups: threads per (token, unit) over the heads
  int offset, pairs;            // rotated dims [offset, offset + 2 pairs)
  int rot_units, copy_units;    // units of a head row
  int left;                     // copied units that lie before the rotated dims
  float sign;
  smla_rope_table table;
};

// kN elements from / to fp32, two at a time where they are 16 bits wide
template <typename T, int kN>
__device__ __forceinline__ void rope_unpack(const RopeVec<T, kN>& r, float (&v)[kN]) {
  if constexpr (sizeof(T) == 2 && kN % 2 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = RopeIo<T>::get(r.v[i]);
  }
}
template <typename T, int kN>
__device__ __forceinline__ RopeVec<T, kN> rope_pack(const float (&v)[kN]) {
  RopeVec<T, kN> r;
  if constexpr (sizeof(T) == 2 && kN % 2 == 0) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      else w[i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) r.v[i] = RopeIo<T>::put(v[i]);
  }
  return r;
}

// Items (token, head group, unit), unit fastest, so that a warp's lanes cover
// whole head rows.  A thread takes the heads g, g + groups, ... of its item:
// cos and sin are computed once for them all, and kRopeBatch rows' loads are
// in flight together.  kN > 1: 16-byte units, of kN / 2 pairs (interleaved)
// or of kN elements of each half; kN = 1: one pair, element by element.
// Every thread also passes on its share of the dims outside the rotation, so
// that the lanes of a warp do the same work.
template <typename T, int kN, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) smla_rope_kernel(const __grid_constant__ RopeParams p) {
  using V = RopeVec<T, kN>;
  constexpr bool kTwo = !kInter || kN == 1;      // the pair's halves are two loads
  constexpr int kPairs = kTwo ? kN : kN / 2;
  grid_dep_wait();
  const uint32_t per_token = (uint32_t)p.groups * (uint32_t)p.rot_units;
  const unsigned long long item = (unsigned long long)blockIdx.x * kRopeThreads + threadIdx.x;
  // (the host keeps tokens * per_token below 2^32)
  const uint32_t tok = (uint32_t)item / per_token, rest = (uint32_t)item % per_token;
  const int g = (int)(rest / (uint32_t)p.rot_units), u = (int)(rest % (uint32_t)p.rot_units);
  if (item >= (unsigned long long)p.tokens * per_token) return;
  const T* x = static_cast<const T*>(p.x) + (long long)tok * p.xt;
  T* y = static_cast<T*>(p.y) + (long long)tok * p.yt;
  const int pos = __ldg(p.positions + tok);
  const int pair0 = u * kPairs;
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    rope_sincos(p.table.step[pair0 + j], pos, p.table.mscale, c[j], s[j]);
    s[j] *= p.sign;
  }
  const int d0 = p.offset + (kInter ? 2 * pair0 : pair0);
  for (int h0 = g; h0 < p.heads; h0 += kRopeBatch * p.groups) {
    V a[kRopeBatch], b[kRopeBatch];
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (h0 + i * p.groups < p.heads) {
        const T* row = x + (long long)(h0 + i * p.groups) * p.xh + d0;
        a[i] = *reinterpret_cast<const V*>(row);
        if constexpr (kTwo) b[i] = *reinterpret_cast<const V*>(row + (kInter ? 1 : p.pairs));
      }
    }
    // dims outside the rotation (when y is not x), passed on
    for (int k = u; k < p.copy_units; k += p.rot_units) {
      const int d = k < p.left ? k * kN : p.offset + 2 * p.pairs + (k - p.left) * kN;
      V v[kRopeBatch];
#pragma unroll
      for (int i = 0; i < kRopeBatch; ++i)
        if (h0 + i * p.groups < p.heads) v[i] = *reinterpret_cast<const V*>(x + (long long)(h0 + i * p.groups) * p.xh + d);
#pragma unroll
      for (int i = 0; i < kRopeBatch; ++i)
        if (h0 + i * p.groups < p.heads) *reinterpret_cast<V*>(y + (long long)(h0 + i * p.groups) * p.yh + d) = v[i];
    }
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (h0 + i * p.groups < p.heads) {
        T* row = y + (long long)(h0 + i * p.groups) * p.yh + d0;
        float va[kN], vb[kN];
        rope_unpack<T, kN>(a[i], va);
        if constexpr (kTwo) rope_unpack<T, kN>(b[i], vb);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          float& ra = kTwo ? va[j] : va[(2 * j) % kN];
          float& rb = kTwo ? vb[j] : va[(2 * j + 1) % kN];
          const float u0 = ra, u1 = rb;
          ra = fmaf(u0, c[j], -u1 * s[j]);
          rb = fmaf(u0, s[j], u1 * c[j]);
        }
        *reinterpret_cast<V*>(row) = rope_pack<T, kN>(va);
        if constexpr (kTwo) *reinterpret_cast<V*>(row + (kInter ? 1 : p.pairs)) = rope_pack<T, kN>(vb);
      }
    }
  }
}

// ------------------------------------------------------------------ host
static smla_status validate_rope_table(const smla_rope_table* t) {
  if (!t) return SMLA_ERR_INVALID_ARG;
  if (t->rope_dim < 2 || t->rope_dim > SMLA_ROPE_MAX_DIM || t->rope_dim % 2) return SMLA_ERR_INVALID_ARG;
  if (t->layout != SMLA_ROPE_INTERLEAVED && t->layout != SMLA_ROPE_HALF) return SMLA_ERR_INVALID_ARG;
  if (!(t->mscale == t->mscale) || isinf(t->mscale)) return SMLA_ERR_INVALID_ARG;
  return SMLA_OK;
}

static int dtype_bytes(int dtype) { return dtype == SMLA_DTYPE_FP32 ? 4 : 2; }

template <typename T, int kN, bool kInter>
static cudaError_t launch_rope_as(const RopeParams& prm, long long tokens, cudaStream_t stream) {
  RopeParams p = prm;
  // chunks of tokens whose items stay below 2^31
  const long long per_token = (long long)p.groups * p.rot_units;
  const long long most = ((1ll << 31) - kRopeThreads) / per_token;
  long long left = tokens;
  while (left > 0) {
    p.tokens = (int)(left < most ? left : most);
    const long long items = (long long)p.tokens * per_token;
    void* args[] = {&p};
    const cudaError_t e = launch_pdl((const void*)smla_rope_kernel<T, kN, kInter>,
                                     dim3((unsigned)((items + kRopeThreads - 1) / kRopeThreads)), dim3(kRopeThreads), 0,
                                     stream, args);
    if (e != cudaSuccess) return e;
    left -= p.tokens;
    p.x = static_cast<const T*>(p.x) + (long long)p.tokens * p.xt;
    p.y = static_cast<T*>(p.y) + (long long)p.tokens * p.yt;
    p.positions += p.tokens;
  }
  return cudaSuccess;
}

template <typename T>
static cudaError_t launch_rope(RopeParams p, const smla_rope_shape* s, bool inter, bool in_place, cudaStream_t stream) {
  constexpr int kV = 16 / (int)sizeof(T);
  const int rot = 2 * p.pairs;
  const int before = in_place ? 0 : s->offset, after = in_place ? 0 : s->dim - s->offset - rot;
  // 16-byte units where every edge they start from is a multiple of 16 bytes
  // (8,192 x 64 heads x 64 dims of rows 144 bytes apart: 32.5 us, element by
  // element 44.4)
  auto mult = [&](long long elements) { return elements % kV == 0; };
  const bool vec = (reinterpret_cast<uintptr_t>(p.x) % 16) == 0 && (reinterpret_cast<uintptr_t>(p.y) % 16) == 0 &&
                   mult(p.xt) && mult(p.xh) && mult(p.yt) && mult(p.yh) && mult(s->offset) && mult(after) &&
                   mult(inter ? rot : p.pairs);
  const int n = vec ? kV : 1;                       // elements per copied unit
  p.rot_units = vec ? (inter ? rot : p.pairs) / kV : p.pairs;
  p.left = before / n;
  p.copy_units = p.left + after / n;
  // Heads per thread: up to 16 share a thread's cos and sin where there is
  // enough other work to fill the device, fewer for a few tokens.  Measured
  // with 1 / 4 / 16 heads per thread (64 heads x 64 dims, interleaved, in a
  // graph): 128 tokens 2.2 / 2.1 / 3.9 us, 256 3.2 / 2.2 / 3.9, 1,024 9.0 / 4.1 /
  // 4.0, 2,048 16.1 / 6.4 / 5.5, 16,384 125 / 49 / 44; 16 tokens 1.85 / 2.06 / 3.9.
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const long long work = s->tokens * s->heads * p.rot_units, fill = 2048ll * sms;
  const int per = 3 * work >= 5 * fill ? 16 : (3 * work >= fill ? 4 : 1);
  p.groups = (s->heads + per - 1) / per;
  if (vec)
    return inter ? launch_rope_as<T, kV, true>(p, s->tokens, stream) : launch_rope_as<T, kV, false>(p, s->tokens, stream);
  return inter ? launch_rope_as<T, 1, true>(p, s->tokens, stream) : launch_rope_as<T, 1, false>(p, s->tokens, stream);
}

// Rows of `width` elements at two strides share no memory: one dim's stride
// clears all that the other one spans (a dim of size one spans nothing).
static bool rows_apart(long long s0, long long n0, long long s1, long long n1, int width) {
  const long long a0 = s0 < 0 ? -s0 : s0, a1 = s1 < 0 ? -s1 : s1;
  const long long most = 1ll << 62;
  auto span = [&](long long stride, long long n) -> long long {     // of n rows
    return stride > 0 && n - 1 > (most - width) / stride ? most : (n - 1) * stride + width;
  };
  if (n0 <= 1) return n1 <= 1 || a1 >= width;
  if (n1 <= 1) return a0 >= width;
  return (a1 >= width && a0 >= span(a1, n1)) || (a0 >= width && a1 >= span(a0, n0));
}

static smla_status run_rope(const smla_rope_shape* s, const smla_rope_table* t, const void* x, const int32_t* positions,
                            void* y, cudaStream_t stream) {
  if (!s) return SMLA_ERR_INVALID_ARG;
  const smla_status st = validate_rope_table(t);
  if (st != SMLA_OK) return st;
  if (s->dtype < SMLA_DTYPE_BF16 || s->dtype > SMLA_DTYPE_FP32) return SMLA_ERR_UNSUPPORTED;
  if (s->tokens < 0 || s->heads < 1 || s->heads > 65536 || s->dim < 2 || s->dim > 65536) return SMLA_ERR_INVALID_ARG;
  if (s->offset < 0 || s->offset > s->dim - t->rope_dim) return SMLA_ERR_INVALID_ARG;
  if ((s->transpose != 0 && s->transpose != 1) || s->reserved != 0) return SMLA_ERR_INVALID_ARG;
  if (s->tokens == 0) return SMLA_OK;
  const int size = dtype_bytes(s->dtype);
  if (!x || !y || !positions || !aligned(x, size) || !aligned(y, size) || !aligned(positions, 4))
    return SMLA_ERR_INVALID_ARG;
  // rows of y do not meet (two would be written to one place); in place the
  // layouts are the same
  if (!rows_apart(s->y_token_stride, s->tokens, s->y_head_stride, s->heads, s->dim)) return SMLA_ERR_INVALID_ARG;
  const bool in_place = x == y;
  if (in_place && ((s->tokens > 1 && s->x_token_stride != s->y_token_stride) ||
                   (s->heads > 1 && s->x_head_stride != s->y_head_stride)))
    return SMLA_ERR_INVALID_ARG;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.x = x;
  p.y = y;
  p.positions = positions;
  // the stride of a dim of size one is never used
  p.xt = s->tokens > 1 ? s->x_token_stride : 0;
  p.yt = s->tokens > 1 ? s->y_token_stride : 0;
  p.xh = s->heads > 1 ? s->x_head_stride : 0;
  p.yh = s->heads > 1 ? s->y_head_stride : 0;
  p.heads = s->heads;
  p.offset = s->offset;
  p.pairs = t->rope_dim / 2;
  p.sign = s->transpose ? -1.0f : 1.0f;
  p.table = *t;
  const bool inter = t->layout == SMLA_ROPE_INTERLEAVED;
  cudaError_t e;
  if (s->dtype == SMLA_DTYPE_BF16) e = launch_rope<__nv_bfloat16>(p, s, inter, in_place, stream);
  else if (s->dtype == SMLA_DTYPE_FP16) e = launch_rope<__half>(p, s, inter, in_place, stream);
  else e = launch_rope<float>(p, s, inter, in_place, stream);
  return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

}  // namespace smla

extern "C" {

smla_status sparse_mla_rope_init(const smla_rope_config* c, smla_rope_table* table) {
  if (!c || !table) return SMLA_ERR_INVALID_ARG;
  if (c->rope_dim < 2 || c->rope_dim > SMLA_ROPE_MAX_DIM || c->rope_dim % 2) return SMLA_ERR_INVALID_ARG;
  if (c->layout != SMLA_ROPE_INTERLEAVED && c->layout != SMLA_ROPE_HALF) return SMLA_ERR_INVALID_ARG;
  auto positive = [](double v) { return v > 0 && !isinf(v); };
  if (!positive(c->base) || !(c->mscale == c->mscale) || isinf(c->mscale)) return SMLA_ERR_INVALID_ARG;
  if (c->scaling != SMLA_ROPE_SCALING_NONE && !positive(c->factor)) return SMLA_ERR_INVALID_ARG;
  const int d = c->rope_dim;
  double lo = 0, hi = 1;
  if (c->scaling == SMLA_ROPE_SCALING_YARN) {
    if (c->original_ctx < 1 || !positive(c->beta_fast) || !positive(c->beta_slow) || c->base <= 1)
      return SMLA_ERR_INVALID_ARG;
    // the pair that turns r times over the original context
    auto pair_of = [&](double r) {
      return d * log(c->original_ctx / (r * 6.283185307179586)) / (2 * log(c->base));
    };
    lo = fmax(floor(pair_of(c->beta_fast)), 0.0);
    hi = fmin(ceil(pair_of(c->beta_slow)), d - 1.0);
  } else if (c->scaling != SMLA_ROPE_SCALING_NONE && c->scaling != SMLA_ROPE_SCALING_LINEAR) {
    return SMLA_ERR_UNSUPPORTED;
  }
  memset(table, 0, sizeof(*table));
  table->rope_dim = d;
  table->layout = c->layout;
  table->mscale = (float)c->mscale;
  for (int i = 0; i < d / 2; ++i) {
    long double f = powl((long double)c->base, -2.0L * i / d);
    if (c->scaling == SMLA_ROPE_SCALING_LINEAR) f /= c->factor;
    if (c->scaling == SMLA_ROPE_SCALING_YARN) {
      const double r = fmin(1.0, fmax(0.0, (i - lo) / fmax(hi - lo, 0.001)));
      f = f * (1.0L - r) + f / c->factor * r;
    }
    long double turns = f / 6.283185307179586476925286766559L;
    turns -= floorl(turns);
    const long double step = roundl(turns * 18446744073709551616.0L);   // 2^64
    table->step[i] = step >= 18446744073709551616.0L ? 0ull : (uint64_t)step;
  }
  return SMLA_OK;
}

smla_status sparse_mla_rope(const smla_rope_shape* shape, const smla_rope_table* table, const void* x,
                            const int32_t* positions, void* y, void* stream) {
  return smla::run_rope(shape, table, x, positions, y, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
