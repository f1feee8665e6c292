// MX4 quantisation of rows and its inverse (the format: mx4_common.cuh).
//
// Both are one pass over the data and bound by HBM: 2 (bf16) or 4 (fp32)
// bytes in and 17/32 bytes out per element, or the reverse.  A lane holds 8
// consecutive elements (one or two 16-byte loads), so a block of 32 is four
// neighbouring lanes and its maximum two shuffles; a warp takes 2048
// consecutive elements of one row, all loads of every lane in flight before
// the first use.  8192 x 6144 bf16 there and back take 43.7 us (45.4 with
// 1024 elements a warp, 50.2 with 512).  Two kinds of calls take 512 a warp:
//   few       fewer than 32 long warps for every SM, where the shorter chain
//             counts (6144 bf16 there and back, short and long warps: one row
//             2.5 and 3.6 us, 1280 rows 10.6 and 11.4, 1792 rows 13.6 both,
//             2432 rows 17.1 and 16.0)
//   ragged    rows that would leave over a quarter of the long warps empty
//             (52 M elements, short and long: K = 512 52 and 110 us, 1024 52
//             and 66, 2560 52 and 58, 4128 56.5 both; but 1536 52.3 and 51.8,
//             5120 52.2 and 49.5, 6176 55.1 and 53.2)
#include "mx4_common.cuh"

namespace {

using namespace colimoe;

constexpr int QT = 256;      // threads per CTA

// QU: 8-element units per lane
template <typename T, bool VEC, int QU>
__global__ void __launch_bounds__(QT) quantize_kernel(const T* __restrict__ x, long long ldx, int rows, int K,
                                                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int QW = 256 * QU;  // elements per warp and step
  const int lane = threadIdx.x & 31;
  const int per_row = (K + QW - 1) / QW;
  const long long tasks = (long long)rows * per_row, step = (long long)gridDim.x * (QT / 32);
  pdl_wait();
  pdl_trigger();
  for (long long task = (long long)blockIdx.x * (QT / 32) + (threadIdx.x >> 5); task < tasks; task += step) {
    const long long row = task / per_row;
    const int k0 = (int)(task - row * per_row) * QW + lane * 8;
    const T* src = x + row * ldx;
    Raw8<T> r[QU];
#pragma unroll
    for (int u = 0; u < QU; ++u) r[u] = load8<T, VEC>(src + k0 + u * 256, K - (k0 + u * 256));
#pragma unroll
    for (int u = 0; u < QU; ++u) {
      const int k = k0 + u * 256;
      float v[8];
      floats8(r[u], v);
      uint32_t b;
      const uint32_t w = mx4_quant8(v, &b);
      if (k < K) {  // K % 32 == 0: a block's four lanes are in or out together
        reinterpret_cast<uint32_t*>(codes)[(row * K + k) / 8] = w;
        if ((lane & 3) == 0) scales[(row * K + k) / MXB] = (uint8_t)b;
      }
    }
  }
}

template <typename T, bool VEC, int QU>
__global__ void __launch_bounds__(QT) dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                        int rows, int K, T* __restrict__ out, long long ldo) {
  constexpr int QW = 256 * QU;  // elements per warp and step
  const int lane = threadIdx.x & 31;
  const int per_row = (K + QW - 1) / QW;
  const long long tasks = (long long)rows * per_row, step = (long long)gridDim.x * (QT / 32);
  pdl_wait();
  pdl_trigger();
  for (long long task = (long long)blockIdx.x * (QT / 32) + (threadIdx.x >> 5); task < tasks; task += step) {
    const long long row = task / per_row;
    const int k0 = (int)(task - row * per_row) * QW + lane * 8;
    uint32_t w[QU], b[QU];
#pragma unroll
    for (int u = 0; u < QU; ++u) {
      const int k = k0 + u * 256;
      if (k < K) {
        w[u] = reinterpret_cast<const uint32_t*>(codes)[(row * K + k) / 8];
        b[u] = scales[(row * K + k) / MXB];
      }
    }
#pragma unroll
    for (int u = 0; u < QU; ++u) {
      const int k = k0 + u * 256;
      if (k < K) {
        const float s = mx4_scale(b[u]);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = mx4_code((w[u] >> (4 * i)) & 15u) * s;
        store8<T, VEC>(out + row * ldo + k, 8, v);
      }
    }
  }
}

// A CTA per 8 warp tasks: the hardware deals them out as CTAs end (a grid of
// resident CTAs that stride over the tasks left a sixth of the last round idle)
unsigned grid_for(long long rows, int K, int units) {
  const long long tasks = rows * ((K + 256 * units - 1) / (256 * units));
  const long long blocks = (tasks + QT / 32 - 1) / (QT / 32);
  return (unsigned)(blocks < 0x7fffffffLL ? blocks : 0x7fffffffLL);
}
constexpr int FEW = 2, MANY = 8;  // units per lane
bool many(long long rows, int K) {
  const long long per_row = (K + 256 * MANY - 1) / (256 * MANY);
  return rows * per_row >= 32LL * device_sms() && 4LL * K >= 3 * per_row * (256 * MANY);
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? COLI_OK : COLI_ECUDA; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int QU>
cudaError_t quantize_u(const T* x, long long ldx, int rows, int K, uint8_t* codes, uint8_t* scales, bool vec, cudaStream_t st) {
  const unsigned grid = grid_for(rows, K, QU);
  return vec ? launch_pdl(quantize_kernel<T, true, QU>, grid, QT, 0, st, x, ldx, rows, K, codes, scales)
             : launch_pdl(quantize_kernel<T, false, QU>, grid, QT, 0, st, x, ldx, rows, K, codes, scales);
}
template <typename T, int QU>
cudaError_t dequantize_u(const uint8_t* codes, const uint8_t* scales, int rows, int K, T* out, long long ldo, bool vec, cudaStream_t st) {
  const unsigned grid = grid_for(rows, K, QU);
  return vec ? launch_pdl(dequantize_kernel<T, true, QU>, grid, QT, 0, st, codes, scales, rows, K, out, ldo)
             : launch_pdl(dequantize_kernel<T, false, QU>, grid, QT, 0, st, codes, scales, rows, K, out, ldo);
}
template <typename T>
cudaError_t quantize(const void* x, long long ldx, int rows, int K, uint8_t* codes, uint8_t* scales, bool vec, cudaStream_t st) {
  const T* xt = static_cast<const T*>(x);
  return many(rows, K) ? quantize_u<T, MANY>(xt, ldx, rows, K, codes, scales, vec, st) : quantize_u<T, FEW>(xt, ldx, rows, K, codes, scales, vec, st);
}
template <typename T>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int K, void* out, long long ldo, bool vec, cudaStream_t st) {
  T* ot = static_cast<T*>(out);
  return many(rows, K) ? dequantize_u<T, MANY>(codes, scales, rows, K, ot, ldo, vec, st) : dequantize_u<T, FEW>(codes, scales, rows, K, ot, ldo, vec, st);
}

int check(const void* x, int32_t type, int64_t ld, int32_t T, int32_t K, const void* codes, const void* scales) {
  if (!float_type(type) || T < 0 || K <= 0 || K % MXB || ld < K) return COLI_EINVAL;
  if (K > COLI_MX4_MAX_K) return COLI_EUNSUPPORTED;
  if (T == 0) return COLI_OK;
  if (!x || !codes || !scales) return COLI_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return COLI_EALIGN;
  return COLI_OK;
}

}  // namespace

extern "C" int coli_mx4_quantize(const void* x, int32_t x_type, int64_t ldx, int32_t T, int32_t K, uint8_t* codes,
                                 uint8_t* scales, cudaStream_t stream) {
  const int rc = check(x, x_type, ldx, T, K, codes, scales);
  if (rc || T == 0) return rc;
  const bool vec = rows_aligned(x, ldx, x_type);
  if (x_type == COLI_F32) return rc_of(quantize<float>(x, ldx, T, K, codes, scales, vec, stream));
  if (x_type == COLI_BF16) return rc_of(quantize<__nv_bfloat16>(x, ldx, T, K, codes, scales, vec, stream));
  return rc_of(quantize<__half>(x, ldx, T, K, codes, scales, vec, stream));
}

extern "C" int coli_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t T, int32_t K, void* out,
                                   int32_t out_type, int64_t ldo, cudaStream_t stream) {
  const int rc = check(out, out_type, ldo, T, K, codes, scales);
  if (rc || T == 0) return rc;
  const bool vec = rows_aligned(out, ldo, out_type);
  if (out_type == COLI_F32) return rc_of(dequantize<float>(codes, scales, T, K, out, ldo, vec, stream));
  if (out_type == COLI_BF16) return rc_of(dequantize<__nv_bfloat16>(codes, scales, T, K, out, ldo, vec, stream));
  return rc_of(dequantize<__half>(codes, scales, T, K, out, ldo, vec, stream));
}
