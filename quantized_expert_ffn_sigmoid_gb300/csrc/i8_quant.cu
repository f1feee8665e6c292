// 8-bit codes of rows with one scale a row, with SwiGLU before them where the
// rows are an expert's gate and up values, and the inverse.
//
// Mathematics.  For a row v (or v = silu(g) u of its halves) with largest
// magnitude A:  scale = A / 127,  code = v * 127 / A rounded to the nearest
// whole number, ties to even.  A row with A < 2^-100 is zeros; one that holds an
// infinity or NaN gets scale NaN and codes 0, so that its products are NaN.
// The quotient is taken in fp32; a value whose quotient lies so near the middle
// of two codes that fp32 may turn it is decided by the sign of
// v * 127 - middle * A, whose terms are exact in 64 bits: codes are those of
// exact arithmetic.  (With SwiGLU the values themselves are fp32 results.)
//
// One pass: a row's values stay in registers between its maximum and its
// codes (up to 8192 values, 32 a thread; longer rows are read twice).  Bound:
// HBM, 2 or 4 bytes in and one out a value.
#include "mx4_common.cuh"

namespace colimoe {
namespace {

constexpr int IQ_T = 256;   // threads of a CTA
constexpr int IQ_U = 4;     // 8-value units a thread holds
constexpr float IQ_TINY = 7.8886090522101181e-31f;  // 2^-100

// 8 values at p, of which n exist; VEC: whole units start on 16-byte boundaries
template <typename TY, bool VEC>
__device__ __forceinline__ Raw8<TY> load_unit(const TY* p, int n) {
  if (VEC && n >= 8) return load8<TY, true>(p, 8);
  return load8<TY, false>(p, n);
}

// silu(g) u; exp of -|g| alone, so that nothing overflows on the way
__device__ __forceinline__ float swiglu(float g, float u) {
  const float x = expf(-fabsf(g)), q = __fdividef(1.f, 1.f + x);
  return g * (g >= 0.f ? q : x * q) * u;
}

template <typename TY, bool SW>
__device__ __forceinline__ void unit_values(const Raw8<TY>& a, const Raw8<TY>& b, float* v) {
  floats8(a, v);
  if (SW) {
    float u[8];
    floats8(b, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = swiglu(v[i], u[i]);
  }
}

// t rounded to a whole number, as the low byte of the result's bits
constexpr float IQ_MAGIC = 12582912.f;  // 1.5 * 2^23: adding it rounds to whole numbers, ties to even

template <bool SW>
__device__ __forceinline__ uint32_t code_of(float v, float inv, float amax) {
  const float t = v * inv;
  float r = t + IQ_MAGIC;
  if (!SW) {
    const float d = t - (r - IQ_MAGIC);
    // (the quotient is within 127 * 2^-23 of the exact one)
    if (fabsf(d) > 0.49996f) {
      const float low = floorf(t);  // t is near low + 1/2
      const double s = (double)v * 127.0 - ((double)low + 0.5) * (double)amax;
      const float c = s > 0.0 || (s == 0.0 && ((int)low & 1)) ? low + 1.f : low;
      r = c + IQ_MAGIC;
    }
  }
  return __float_as_uint(r) & 0xffu;
}

template <bool SW>
__device__ __forceinline__ uint2 codes8(const float* v, float inv, float amax) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[h] |= code_of<SW>(v[4 * h + i], inv, amax) << (8 * i);
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

__device__ __forceinline__ uint32_t max_bits(const float* v, int n) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, i < n ? __float_as_uint(v[i]) & 0x7fffffffu : 0u);
  return m;
}
// scale and factor of a row from the bits of its largest magnitude
__device__ __forceinline__ float row_scale(uint32_t bits, float* inv) {
  const float a = __uint_as_float(bits);
  *inv = 0.f;
  if (bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  if (a < IQ_TINY) return 0.f;
  *inv = __fdiv_rn(127.f, a);
  return __fdiv_rn(a, 127.f);
}

// ROW: threads of a row (a warp, or the CTA); LONG: rows of any length, read twice
template <typename TY, bool VEC, bool SW, int ROW, bool LONG>
__global__ void __launch_bounds__(IQ_T) i8_quantize_kernel(const QuantParams P) {
  __shared__ uint32_t s_max[IQ_T / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in = threadIdx.x % ROW;
  pdl_wait();
  pdl_trigger();
  const long long t = (long long)blockIdx.x * (IQ_T / ROW) + threadIdx.x / ROW;
  if (t >= P.T) return;  // (whole warps of rows, or the CTA)
  const TY* src = static_cast<const TY*>(P.x) + t * P.ldx;
  int8_t* dst = P.codes + t * P.ldc;
  const int K = P.K;
  auto reduce = [&](uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (ROW > 32) {
      if (lane == 0) s_max[warp] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < IQ_T / 32; ++i) m = max(m, s_max[i]);
    }
    return m;
  };
  if (!LONG) {
    float v[IQ_U][8];
    {
      Raw8<TY> a[IQ_U], b[SW ? IQ_U : 1];
#pragma unroll
      for (int u = 0; u < IQ_U; ++u) {
        const int k = (in + u * ROW) * 8;
        a[u] = load_unit<TY, VEC>(src + k, K - k);
        if (SW) b[u] = load_unit<TY, VEC>(src + K + k, K - k);
      }
#pragma unroll
      for (int u = 0; u < IQ_U; ++u) unit_values<TY, SW>(a[u], b[SW ? u : 0], v[u]);
    }
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < IQ_U; ++u) m = max(m, max_bits(v[u], K - (in + u * ROW) * 8));
    m = reduce(m);
    float inv;
    const float scale = row_scale(m, &inv), amax = __uint_as_float(m);
    if (in == 0) P.scales[t] = scale;
#pragma unroll
    for (int u = 0; u < IQ_U; ++u) {
      const int k = (in + u * ROW) * 8;
      if (k < K) store_codes<VEC>(dst + k, K - k, inv > 0.f ? codes8<SW>(v[u], inv, amax) : make_uint2(0, 0));
    }
  } else {
    uint32_t m = 0;
#pragma unroll 4
    for (int k = in * 8; k < K; k += ROW * 8) {
      float v[8];
      unit_values<TY, SW>(load_unit<TY, VEC>(src + k, K - k), load_unit<TY, VEC>(src + (SW ? K : 0) + k, SW ? K - k : 0), v);
      m = max(m, max_bits(v, K - k));
    }
    m = reduce(m);
    float inv;
    const float scale = row_scale(m, &inv), amax = __uint_as_float(m);
    if (in == 0) P.scales[t] = scale;
#pragma unroll 2
    for (int k = in * 8; k < K; k += ROW * 8) {
      float v[8];
      unit_values<TY, SW>(load_unit<TY, VEC>(src + k, K - k), load_unit<TY, VEC>(src + (SW ? K : 0) + k, SW ? K - k : 0), v);
      store_codes<VEC>(dst + k, K - k, inv > 0.f ? codes8<SW>(v, inv, amax) : make_uint2(0, 0));
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
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long task = first + u * IQ_T;
    w[u] = make_uint2(0, 0);
    s[u] = 0.f;
    if (task >= tasks) continue;
    const long long t = task / units;
    const int k = (int)(task - t * units) * 8, n = K - k;
    const int8_t* p = codes + t * ldc + k;
    s[u] = __ldg(scales + t);
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
    const long long task = first + u * IQ_T;
    if (task >= tasks) continue;
    const long long t = task / units;
    const int k = (int)(task - t * units) * 8, n = K - k;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the byte with its sign bit flipped is code + 128, the low byte of the float 2^23 + code + 128
      const uint32_t b = ((i < 4 ? w[u].x : w[u].y) >> (8 * (i & 3)) & 0xffu) ^ 0x80u;
      v[i] = (__uint_as_float(0x4b000000u | b) - 8388736.f) * s[u];
    }
    if (VEC && n >= 8) store8<TY, true>(out + t * ldo + k, 8, v);
    else store8<TY, false>(out + t * ldo + k, n, v);
  }
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? COLI_OK : COLI_ECUDA; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename TY, bool VEC, bool SW>
cudaError_t quantize_v(const QuantParams& P, cudaStream_t st) {
  if (P.K <= 32 * 8 * IQ_U) {
    const long long grid = ((long long)P.T + IQ_T / 32 - 1) / (IQ_T / 32);
    return launch_pdl(i8_quantize_kernel<TY, VEC, SW, 32, false>, (unsigned)grid, IQ_T, 0, st, P);
  }
  if (P.K <= IQ_T * 8 * IQ_U) return launch_pdl(i8_quantize_kernel<TY, VEC, SW, IQ_T, false>, (unsigned)P.T, IQ_T, 0, st, P);
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
