// 8-bit codes of rows with one scale a row, with SwiGLU before them where the
// rows are an expert's gate and up values, and the inverse.
//
// Mathematics.  For a row v (or v = silu(g) u of its halves) with largest
// magnitude A:  scale = A / 127,  code = v * 127 / A rounded to the nearest
// whole number, ties to even.  A row with A < 2^-100 is zeros; one that holds an
// infinity or NaN gets scale NaN and codes 0, so that its products are NaN.
// The quotient is taken in fp32; where it lies so near the middle of two codes
// that its rounding may decide, the sign of v * 127 - middle * A does: codes are
// those of exact arithmetic.  (With SwiGLU those of the fp32 results silu(g) u,
// which are within 2^-21 of the 64-bit ones.)
//
// One pass: a row's values stay in registers between its maximum and its
// codes (up to 8192 values, 32 a thread; longer rows are read twice).  Bound:
// HBM, 2 or 4 bytes in and one out a value, and close to it the instructions:
// two values an fp32 instruction and, of 16-bit values, two magnitudes a
// comparison.  8192 x 6144 bf16 24.5 us (6.2 TB/s of 6.79 copied; one value an
// instruction 34), fp32 8192 x 4096 26 us (6.5), SwiGLU of 16384 x 2048 bf16 33.9 us
// (5.0: exponentials, and 31.0 without the look at middles, with codes one off
// next to some); back to bf16, 8192 x 6144, 24 us (6.3).  Rows that are not 16-byte
// aligned move value by value: 48, 63 and 117 us.
#include "mx4_common.cuh"

namespace colimoe {
namespace {

constexpr int IQ_T = 256;   // threads of a CTA
constexpr int IQ_FEW = 600; // rows of a small call
constexpr int IQ_U = 4;     // 8-value units a thread holds
constexpr float IQ_TINY = 7.8886090522101181e-31f;  // 2^-100

// 8 values at p, of which n exist; VEC: whole units start on 16-byte boundaries
template <typename TY, bool VEC>
__device__ __forceinline__ Raw8<TY> load_unit(const TY* p, int n) {
  if (VEC && n >= 8) return load8<TY, true>(p, 8);
  return load8<TY, false>(p, n);
}

// Two fp32 operations an instruction (x: the pair's first)
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// silu(g) u of two values; exp of -|g| alone, so that nothing overflows on the way
__device__ __forceinline__ float2 swiglu2(float2 g, float2 u) {
  const float2 x = make_float2(expf(-fabsf(g.x)), expf(-fabsf(g.y))), y = add2(x, both(1.f));
  float2 q;  // (of 1 to 2: within a unit)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.x) : "f"(y.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.y) : "f"(y.y));
  const float2 n = make_float2(g.x >= 0.f ? 1.f : x.x, g.y >= 0.f ? 1.f : x.y);
  return mul2(mul2(g, mul2(n, q)), u);
}

template <typename TY, bool SW>
__device__ __forceinline__ void unit_values(const Raw8<TY>& a, const Raw8<TY>& b, float* v) {
  floats8(a, v);
  if (SW) {
    float u[8];
    floats8(b, u);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 h = swiglu2(make_float2(v[i], v[i + 1]), make_float2(u[i], u[i + 1]));
      v[i] = h.x;
      v[i + 1] = h.y;
    }
  }
}

constexpr float IQ_MAGIC = 12582912.f;  // 1.5 * 2^23: adding it rounds to whole numbers, ties to even, into the low bits

// How a quotient's rounding to fp32 is kept from turning a code
//   SNAP    16-bit values: with A = b 2^j and v = a 2^i, a and b whole numbers of
//           at most 11 bits, the quotient 127 a / (b 2^(j-i)) is the middle of two codes or at
//           least 1 / (254 a) > 2^-19 of itself away from it, and v * inv is at
//           most 2^-24 from the exact one.  c - (c - v * inv) with c = 9 v * inv
//           is that rounded to a multiple of 8 of its units: the middle where the
//           exact quotient is one, and else on its side
//   DECIDE  fp32 values, also those of SwiGLU: near a middle the exact sign decides
enum { SNAP, DECIDE };

// 8 codes in two words
template <int MODE>
__device__ __forceinline__ uint2 codes8(const float* v, float inv, float amax) {
  float r[8];
  float far = 0.f;  // from a whole number, at most
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 x = make_float2(v[i], v[i + 1]);
    float2 q;
    if (MODE == SNAP) {
      const float2 c = mul2(x, both(9.f * inv)), d = fma2(x, both(-inv), c);
      q = add2(fma2(d, both(-1.f), c), both(IQ_MAGIC));
    } else {
      const float2 t = mul2(x, both(inv));
      q = add2(t, both(IQ_MAGIC));
      const float2 off = fma2(add2(q, both(-IQ_MAGIC)), both(-1.f), t);
      far = fmaxf(far, fmaxf(fabsf(off.x), fabsf(off.y)));
    }
    r[i] = q.x;
    r[i + 1] = q.y;
  }
  if (MODE == DECIDE && far > 0.49996f) {  // (the quotient is within 127 * 2^-23 of the exact one)
    // v * 127 - (low + 1/2) * A to its sign: the product and its rounding
    // error, then a difference of near numbers, exact as they cancel.  (Scaled
    // down, so that nothing overflows.)  Rare in fp32 values; 16-bit values, whose quotients
    // often are middles, took 48 us this way when the other took 34 (8192 x 6144, before two values an instruction).
    const float f = amax > 1e30f ? 0x1p-10f : 1.f, a = amax * f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = v[i] * inv, low = floorf(t), h = low + 0.5f, p = h * a;
      const float d = fmaf(v[i] * f, 127.f, -p) - fmaf(h, a, -p);
      const float code = d > 0.f || (d == 0.f && ((int)low & 1)) ? low + 1.f : low;
      if (fabsf(t - h) < 4e-5f) r[i] = code + IQ_MAGIC;
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __byte_perm(__float_as_uint(r[4 * h]), __float_as_uint(r[4 * h + 1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(r[4 * h + 2]), __float_as_uint(r[4 * h + 3]), 0x0040);
    w[h] = __byte_perm(lo, hi, 0x5410);
  }
  return make_uint2(w[0], w[1]);
}

template <bool VEC>
__device__ __forceinline__ void store_codes(int8_t* p, int n, uint2 w) {
  if (VEC && n >= 8) {
    *reinterpret_cast<uint2*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (int8_t)((i < 4 ? w.x >> (8 * i) : w.y >> (8 * i - 32)) & 0xffu);
  }
}

struct QuantParams {
  const void* x;
  long long ldx;
  int T, K;
  int8_t* codes;
  long long ldc;
  float* scales;
};

// the largest of m and 8 magnitudes, NaN if one is
__device__ __forceinline__ uint32_t max_bits(uint32_t m, const float* v) {
  float f = __uint_as_float(m);
#pragma unroll
  for (int i = 0; i < 8; i += 2) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(f) : "f"(v[i]), "f"(v[i + 1]));
  return __float_as_uint(f);
}
// factor of a row's codes from the bits of its largest magnitude (0: no codes), and its scale
__device__ __forceinline__ float row_inv(uint32_t bits) {
  const float a = __uint_as_float(bits);
  return bits >= 0x7f800000u || a < IQ_TINY ? 0.f : __fdiv_rn(127.f, a);
}
__device__ __forceinline__ float row_scale(uint32_t bits) {
  const float a = __uint_as_float(bits);
  return bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : a < IQ_TINY ? 0.f : __fdiv_rn(a, 127.f);
}
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// What a thread keeps of a unit: the values as they came, or after SwiGLU; and
// the largest magnitude of units, as the bits of a float.  Magnitudes of 16-bit
// values are compared as they are, two an instruction.  (Loads beyond a row give zeros.)
template <typename TY, bool SW>
struct Held {
  Raw8<TY> raw;
  __device__ __forceinline__ void values(float* v) const { floats8(raw, v); }
  __device__ __forceinline__ uint32_t join(uint32_t m) const {
    if constexpr (sizeof(TY) == 4) {
      float v[8];
      values(v);
      return max_bits(m, v);
    }
    const uint32_t w[4] = {raw.q[0].x, raw.q[0].y, raw.q[0].z, raw.q[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max16x2(m, w[j] & 0x7fff7fffu);
    return m;
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) {
    if constexpr (sizeof(TY) == 4) return m;
    const uint16_t top = (uint16_t)max(m & 0xffffu, m >> 16);
    return __float_as_uint(to_f32(*reinterpret_cast<const TY*>(&top)));
  }
};
template <typename TY>
struct Held<TY, true> {
  float h[8];
  __device__ __forceinline__ void values(float* v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = h[i];
  }
  __device__ __forceinline__ uint32_t join(uint32_t m) const { return max_bits(m, h); }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
};

// ROW: threads of a row; LONG: rows of any length, read twice
template <typename TY, bool VEC, bool SW, int ROW, bool LONG>
__global__ void __launch_bounds__(IQ_T, sizeof(TY) == 2 && VEC && !SW && !LONG ? 6 : 4) i8_quantize_kernel(const QuantParams P) {
  __shared__ __align__(16) uint32_t s_max[IQ_T / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in = threadIdx.x % ROW;
  pdl_wait();
  pdl_trigger();
  const long long t = (long long)blockIdx.x * (IQ_T / ROW) + threadIdx.x / ROW;
  if (t >= P.T) return;  // (all threads of a row)
  const TY* src = static_cast<const TY*>(P.x) + t * P.ldx;
  int8_t* dst = P.codes + t * P.ldc;
  const int K = P.K;
  auto reduce = [&](uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (ROW > 32) {
      constexpr int W = ROW / 32;
      if (lane == 0) s_max[warp] = m;
      named_bar(1 + warp / W, ROW);
      if constexpr (W == 2) {
        const uint2 a = *reinterpret_cast<const uint2*>(s_max + warp / W * W);
        m = max(a.x, a.y);
      } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
          const uint4 a = *reinterpret_cast<const uint4*>(s_max + warp / W * W + i);
          m = max(m, max(max(a.x, a.y), max(a.z, a.w)));
        }
      }
    }
    return m;
  };
  if (!LONG) {
    const int units = (K + ROW * 8 - 1) / (ROW * 8);  // of a thread; the branches on it are uniform
    Held<TY, SW> x[IQ_U];
    uint32_t m = 0;
    if constexpr (SW) {
      Raw8<TY> a[IQ_U], b[IQ_U];
#pragma unroll
      for (int u = 0; u < IQ_U; ++u) {
        const int k = (in + u * ROW) * 8;
        if (u < units) {
          a[u] = load_unit<TY, VEC>(src + k, K - k);
          b[u] = load_unit<TY, VEC>(src + K + k, K - k);
        }
      }
#pragma unroll
      for (int u = 0; u < IQ_U; ++u)
        if (u < units) unit_values<TY, SW>(a[u], b[u], x[u].h);
    } else {
#pragma unroll
      for (int u = 0; u < IQ_U; ++u) {
        const int k = (in + u * ROW) * 8;
        if (u < units) x[u].raw = load_unit<TY, VEC>(src + k, K - k);
      }
    }
#pragma unroll
    for (int u = 0; u < IQ_U; ++u)
      if (u < units) m = x[u].join(m);
    m = reduce(Held<TY, SW>::bits(m));
    const float inv = row_inv(m), amax = __uint_as_float(m);
    if (in == 0) P.scales[t] = row_scale(m);
#pragma unroll
    for (int u = 0; u < IQ_U; ++u) {
      const int k = (in + u * ROW) * 8;
      if (u < units && k < K) {
        float v[8];
        x[u].values(v);
        store_codes<VEC>(dst + k, K - k, inv > 0.f ? codes8<SW || sizeof(TY) == 4 ? DECIDE : SNAP>(v, inv, amax) : make_uint2(0, 0));
      }
    }
  } else {
    uint32_t m = 0;
#pragma unroll 4
    for (int k = in * 8; k < K; k += ROW * 8) {
      float v[8];
      unit_values<TY, SW>(load_unit<TY, VEC>(src + k, K - k), load_unit<TY, VEC>(src + (SW ? K : 0) + k, SW ? K - k : 0), v);
      m = max_bits(m, v);
    }
    m = reduce(m);
    const float inv = row_inv(m), amax = __uint_as_float(m);
    if (in == 0) P.scales[t] = row_scale(m);
#pragma unroll 2
    for (int k = in * 8; k < K; k += ROW * 8) {
      float v[8];
      unit_values<TY, SW>(load_unit<TY, VEC>(src + k, K - k), load_unit<TY, VEC>(src + (SW ? K : 0) + k, SW ? K - k : 0), v);
      store_codes<VEC>(dst + k, K - k, inv > 0.f ? codes8<SW || sizeof(TY) == 4 ? DECIDE : SNAP>(v, inv, amax) : make_uint2(0, 0));
    }
  }
}

template <typename TY, bool VEC>
__global__ void __launch_bounds__(IQ_T) i8_dequantize_kernel(const int8_t* __restrict__ codes, long long ldc, const float* __restrict__ scales, int T,
                                                             int K, int units, TY* __restrict__ out, long long ldo) {
  constexpr int U = 4;
  pdl_wait();
  pdl_trigger();
  const long long tasks = (long long)T * units, first = (long long)blockIdx.x * (IQ_T * U) + threadIdx.x;
  uint2 w[U];
  float s[U];
  long long row[U];
  int at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long task = first + u * IQ_T;
    w[u] = make_uint2(0, 0);
    s[u] = 0.f;
    at[u] = K;
    if (task >= tasks) continue;
    row[u] = tasks <= 0xffffffffLL ? (long long)((uint32_t)task / (uint32_t)units) : task / units;  // (a 64-bit division costs as much as the rest)
    at[u] = (int)(task - row[u] * units) * 8;
    const int n = K - at[u];
    const int8_t* p = codes + row[u] * ldc + at[u];
    s[u] = __ldg(scales + row[u]);
    if (VEC && n >= 8) {
      w[u] = __ldcs(reinterpret_cast<const uint2*>(p));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) (i < 4 ? w[u].x : w[u].y) |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = K - at[u];
    if (n <= 0) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the byte with its sign bit flipped is code + 128, the low byte of the float 2^23 + code + 128
      const uint32_t b = __byte_perm(i < 4 ? w[u].x ^ 0x80808080u : w[u].y ^ 0x80808080u, 0x4b000000u, 0x7650 | (i & 3));
      v[i] = (__uint_as_float(b) - 8388736.f) * s[u];
    }
    TY* dst = out + row[u] * ldo + at[u];
    if (VEC && n >= 8) store8<TY, true>(dst, 8, v);
    else store8<TY, false>(dst, n, v);
  }
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? COLI_OK : COLI_ECUDA; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename TY, bool VEC, bool SW>
cudaError_t quantize_v(const QuantParams& P, cudaStream_t st) {
  auto go = [&](auto kernel, int row) { return launch_pdl(kernel, (unsigned)(((long long)P.T * row + IQ_T - 1) / IQ_T), IQ_T, 0, st, P); };
  // As few threads a row as hold it; calls whose rows leave SMs idle that way take
  // 128 at least (600 rows of 1024: 1.66 us, with 32 threads a row 1.89; but 2400
  // rows 3.1 and 2.2, 16384 rows 16.4 and 7.3).
  const int least = P.T <= IQ_FEW ? 128 : 32;
  if (least <= 32 && P.K <= 32 * 8 * IQ_U) return go(i8_quantize_kernel<TY, VEC, SW, 32, false>, 32);
  if (least <= 64 && P.K <= 64 * 8 * IQ_U) return go(i8_quantize_kernel<TY, VEC, SW, 64, false>, 64);
  if (P.K <= 128 * 8 * IQ_U) return go(i8_quantize_kernel<TY, VEC, SW, 128, false>, 128);
  if (P.K <= 256 * 8 * IQ_U) return go(i8_quantize_kernel<TY, VEC, SW, 256, false>, 256);
  return launch_pdl(i8_quantize_kernel<TY, VEC, SW, IQ_T, true>, (unsigned)P.T, IQ_T, 0, st, P);
}
template <typename TY>
cudaError_t quantize_t(const QuantParams& P, bool vec, bool sw, cudaStream_t st) {
  if (vec) return sw ? quantize_v<TY, true, true>(P, st) : quantize_v<TY, true, false>(P, st);
  return sw ? quantize_v<TY, false, true>(P, st) : quantize_v<TY, false, false>(P, st);
}
template <typename TY>
cudaError_t dequantize_t(const int8_t* codes, long long ldc, const float* scales, int T, int K, void* out, long long ldo, bool vec, cudaStream_t st) {
  const int units = (K + 7) / 8;
  const long long grid = ((long long)T * units + IQ_T * 4 - 1) / (IQ_T * 4);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return vec ? launch_pdl(i8_dequantize_kernel<TY, true>, (unsigned)grid, IQ_T, 0, st, codes, ldc, scales, T, K, units, static_cast<TY*>(out), ldo)
             : launch_pdl(i8_dequantize_kernel<TY, false>, (unsigned)grid, IQ_T, 0, st, codes, ldc, scales, T, K, units, static_cast<TY*>(out), ldo);
}

int check(const void* x, int32_t type, int64_t ldx, int64_t width, int32_t T, int32_t K, const int8_t* codes, int64_t ldc, const float* scales) {
  if (!float_type(type) || T < 0 || K < 1 || ldx < width || ldc < K) return COLI_EINVAL;
  if (K > COLI_I8_MAX_K) return COLI_EUNSUPPORTED;
  if (T == 0) return COLI_OK;
  if (!x || !codes || !scales) return COLI_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return COLI_EALIGN;
  return COLI_OK;
}

}  // namespace
}  // namespace colimoe

using namespace colimoe;

extern "C" int coli_i8_quantize(const void* x, int32_t x_type, int64_t ldx, int32_t T, int32_t K, int32_t act, int8_t* codes, int64_t ldc,
                                float* scales, cudaStream_t stream) {
  if (act != COLI_ACT_NONE && act != COLI_ACT_SWIGLU) return COLI_EINVAL;
  const bool sw = act == COLI_ACT_SWIGLU;
  const int rc = check(x, x_type, ldx, sw ? 2 * (int64_t)K : K, T, K, codes, ldc, scales);
  if (rc || T == 0) return rc;
  const QuantParams P{x, ldx, T, K, codes, ldc, scales};
  const bool vec = rows_aligned(x, ldx, x_type) && ldc % 8 == 0 && (!sw || (K * type_bytes(x_type)) % 16 == 0);
  if (x_type == COLI_F32) return rc_of(quantize_t<float>(P, vec, sw, stream));
  if (x_type == COLI_BF16) return rc_of(quantize_t<__nv_bfloat16>(P, vec, sw, stream));
  return rc_of(quantize_t<__half>(P, vec, sw, stream));
}

extern "C" int coli_i8_dequantize(const int8_t* codes, int64_t ldc, const float* scales, int32_t T, int32_t K, void* out, int32_t out_type,
                                  int64_t ldo, cudaStream_t stream) {
  const int rc = check(out, out_type, ldo, K, T, K, codes, ldc, scales);
  if (rc || T == 0) return rc;
  const bool vec = rows_aligned(out, ldo, out_type) && ldc % 8 == 0;
  if (out_type == COLI_F32) return rc_of(dequantize_t<float>(codes, ldc, scales, T, K, out, ldo, vec, stream));
  if (out_type == COLI_BF16) return rc_of(dequantize_t<__nv_bfloat16>(codes, ldc, scales, T, K, out, ldo, vec, stream));
  return rc_of(dequantize_t<__half>(codes, ldc, scales, T, K, out, ldo, vec, stream));
}
