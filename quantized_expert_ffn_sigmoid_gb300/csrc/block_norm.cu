// coli_moe_block_norm: the norm, gate and residual add behind a block fused
// with the norm before the next one, optionally with the MX4 codes of its
// result (mx4_common.cuh).
//
//   r  = y * rsqrt(mean(y^2) + eps) * post_w     (post_w NULL: r = y)
//   x' = x + res_scale * gate * r                (gate NULL: 1; y NULL: x' = x)
//   n  = x' * rsqrt(mean(x'^2) + eps) * pre_w    (pre_w NULL: no weight)
//
// One pass: a row stays in registers between its two reductions, so x, y and
// gate are read once and x', n and the codes written once; bound by HBM (a
// single row by its load, two reductions and store).  All arithmetic is fp32;
// n and its codes are formed from the unrounded x'.
#include "mx4_common.cuh"

namespace {

using namespace colimoe;

struct NormParams {
  const void* x;
  const void* y;
  const void* gate;
  const float* post_w;
  const float* pre_w;
  void* x_out;
  void* n_out;
  uint8_t* codes;
  uint8_t* scales;
  long long ldx, ldy, ldg, ldxo, ldno;
  int rows, H;
  float res_scale, eps;
};

// sum over the threads of a row: a warp, or the whole CTA through `red`
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (WARP) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  // every warp sums the same partials in the same order
  v = warp_sum(lane < nw ? red[lane] : 0.f);
  return v;
}

// 8 weights, which every row reads again: cached loads
template <bool VEC>
__device__ __forceinline__ void load_w(const float* p, int n, float* v) {
  if (VEC) {
    if (n <= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      return;
    }
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __ldg(p + i) : 0.f;
  }
}

// U units of 8 elements per thread; WARP: one row per warp, else per CTA.
// Every load of the row (x, y and gate) is issued before the first reduction.
template <typename T, typename TN, int U, int THREADS, int CTAS, bool VEC, bool WARP>
__global__ void __launch_bounds__(THREADS, CTAS) norm_kernel(const NormParams P) {
  __shared__ float red[2][32];
  const int H = P.H;
  const int nthr = WARP ? 32 : (int)blockDim.x, t = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const long long row = WARP ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (long long)blockIdx.x;
  pdl_wait();
  pdl_trigger();
  if (row >= P.rows) return;  // (whole warps; a CTA's row always exists)
  Raw8<T> xr[U], yr[U], gr[U];
  const bool with_y = P.y != nullptr, gated = P.gate != nullptr;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = (u * nthr + t) * 8;
    xr[u] = load8<T, VEC>(static_cast<const T*>(P.x) + row * P.ldx + k, H - k);
    if (with_y) yr[u] = load8<T, VEC>(static_cast<const T*>(P.y) + row * P.ldy + k, H - k);
    if (gated) gr[u] = load8<T, VEC>(static_cast<const T*>(P.gate) + row * P.ldg + k, H - k);
  }
  float c = P.res_scale, ss = 0.f;
  if (P.post_w) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[8];
      floats8(yr[u], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += y[i] * y[i];
    }
    c *= rsqrtf(row_sum<WARP>(ss, red[0]) / (float)H + P.eps);
  }
  float x[U][8];
  ss = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = (u * nthr + t) * 8, n = H - k;
    floats8(xr[u], x[u]);
    if (with_y) {
      float y[8], w[8];
      floats8(yr[u], y);
      if (P.post_w) {
        load_w<VEC>(P.post_w + k, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= w[i];
      }
      if (gated) {
        floats8(gr[u], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] += c * y[i];
    }
    if (P.x_out && n > 0) store8<T, VEC>(static_cast<T*>(P.x_out) + row * P.ldxo + k, n, x[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[u][i] * x[u][i];
  }
  if (!P.n_out && !P.codes) return;
  c = rsqrtf(row_sum<WARP>(ss, red[1]) / (float)H + P.eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = (u * nthr + t) * 8, n = H - k;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[u][i] * c;
    if (P.pre_w) {
      float w[8];
      load_w<VEC>(P.pre_w + k, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= w[i];
    }
    if (P.n_out && n > 0) store8<TN, VEC>(static_cast<TN*>(P.n_out) + row * P.ldno + k, n, v);
    if (P.codes) {  // H % 32 == 0: a block's four lanes are in or out together
      uint32_t b;
      const uint32_t q = mx4_quant8(v, &b);
      if (n > 0) {
        reinterpret_cast<uint32_t*>(P.codes)[(row * H + k) / 8] = q;
        if ((t & 3) == 0) P.scales[(row * H + k) / MXB] = (uint8_t)b;
      }
    }
  }
}

template <typename T, typename TN, int U, int THREADS, int CTAS>
cudaError_t launch_u(const NormParams& P, bool vec, unsigned block, cudaStream_t st) {
  const unsigned grid = (unsigned)P.rows;
  return vec ? launch_pdl(norm_kernel<T, TN, U, THREADS, CTAS, true, false>, grid, block, 0, st, P)
             : launch_pdl(norm_kernel<T, TN, U, THREADS, CTAS, false, false>, grid, block, 0, st, P);
}

// Threads of a row: one warp up to 512 elements (no barrier).  Beyond, with no
// more rows than SMs, a CTA with one unit per thread, the shortest chain.
// With more rows two units per thread and three CTAs of up to 384 threads on
// an SM, which cover each other's reductions: 4096 x 6144 bf16 with codes and
// their values take 59 us, against 63 with three units and 256 threads, 66
// with one unit and 768, 74 with 256 threads and the registers unbounded.
// Those threads hold 768 units, H = 6144; longer rows take four units a thread
// and up to 512 threads (111 registers in bf16, 124 in fp32: two CTAs an SM up
// to H = 8192, one beyond).  4096 rows with y, gate, both
// norms and codes, of the copy rate: bf16 H = 6144 47.4 us (84 %), 7168 68.9
// (67 %), 8192 72.9 (73 %), 16384 153.5 (69 %); fp32 90.4 (86 %), 100.1
// (90 %), 111.5 (93 %), 256.1 (81 %).
template <typename T, typename TN>
cudaError_t launch(const NormParams& P, bool vec, cudaStream_t st) {
  const int units = (P.H + 7) / 8;
  if (units <= 64) {
    const unsigned grid = (unsigned)(((long long)P.rows + 7) / 8);
    return vec ? launch_pdl(norm_kernel<T, TN, 2, 256, 1, true, true>, grid, 256, 0, st, P)
               : launch_pdl(norm_kernel<T, TN, 2, 256, 1, false, true>, grid, 256, 0, st, P);
  }
  auto threads = [&](int u) { return (unsigned)(((units + u - 1) / u + 31) / 32 * 32); };
  if (P.rows <= device_sms())
    return units <= 1024 ? launch_u<T, TN, 1, 1024, 1>(P, vec, threads(1), st) : launch_u<T, TN, 2, 1024, 1>(P, vec, threads(2), st);
  if (units <= 768) return launch_u<T, TN, 2, 384, 3>(P, vec, threads(2), st);
  return launch_u<T, TN, 4, 512, 1>(P, vec, threads(4), st);
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? COLI_OK : COLI_ECUDA; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

extern "C" int coli_moe_block_norm(const coli_moe_norm_args* a, int32_t T, int32_t H, cudaStream_t stream) {
  if (!a || T < 0 || H <= 0 || !float_type(a->type)) return COLI_EINVAL;
  if (H > COLI_NORM_MAX_H) return COLI_EUNSUPPORTED;
  if (a->n_out && a->n_type != a->type && a->n_type != COLI_F32) return COLI_EINVAL;
  if (!a->codes != !a->scales) return COLI_EINVAL;
  if (a->codes && H % MXB) return COLI_EINVAL;
  if ((a->post_w || a->gate) && !a->y) return COLI_EINVAL;
  if (!(a->eps >= 0.f) || a->ldx < H || (a->y && a->ldy < H) || (a->gate && a->ld_gate != 0 && a->ld_gate < H) ||
      (a->x_out && a->ld_x_out < H) || (a->n_out && a->ld_n_out < H))
    return COLI_EINVAL;
  if (T == 0) return COLI_OK;
  if (!a->x || (!a->x_out && !a->n_out && !a->codes)) return COLI_EINVAL;
  const void* ptrs[] = {a->x, a->y, a->post_w, a->gate, a->pre_w, a->x_out, a->n_out, a->codes, a->scales};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return COLI_EALIGN;
  const int32_t nt = a->n_out ? a->n_type : a->type;
  const bool vec = H % 8 == 0 && rows_aligned(a->x, a->ldx, a->type) && (!a->y || rows_aligned(a->y, a->ldy, a->type)) &&
                   (!a->gate || rows_aligned(a->gate, a->ld_gate, a->type)) &&
                   (!a->x_out || rows_aligned(a->x_out, a->ld_x_out, a->type)) &&
                   (!a->n_out || rows_aligned(a->n_out, a->ld_n_out, nt));
  NormParams P{a->x, a->y, a->gate, a->post_w, a->pre_w, a->x_out, a->n_out, a->codes, a->scales,
               a->ldx, a->ldy, a->ld_gate, a->ld_x_out, a->ld_n_out, T, H, a->res_scale, a->eps};
  if (a->type == COLI_F32) return rc_of(launch<float, float>(P, vec, stream));
  if (a->type == COLI_BF16)
    return rc_of(nt == COLI_F32 ? launch<__nv_bfloat16, float>(P, vec, stream) : launch<__nv_bfloat16, __nv_bfloat16>(P, vec, stream));
  return rc_of(nt == COLI_F32 ? launch<__half, float>(P, vec, stream) : launch<__half, __half>(P, vec, stream));
}
