// Products of MX4 rows, grouped by expert: the grouped product and the two
// passes of the MX4 expert layer.
#include "mx4_layer.cuh"

namespace colimoe {

constexpr int SR = 32;   // result rows of a tile (one MX4 block of h)
constexpr int SP = 32;   // activation rows of a tile
constexpr int ST = 256;

__device__ __forceinline__ float mx4_value(const uint8_t* codes, const uint8_t* scales, long long row, int pitch, int k) {
  const uint32_t b = codes[(row * pitch + k) / 2];
  return mx4_code((k & 1) ? b >> 4 : b & 15u) * mx4_scale(scales[(row * pitch + k) / MXB]);
}

// Tile of SR result rows x SP activation rows, K in steps of one block; each
// thread holds 4 rows of one activation row.
template <int MODE>
__global__ void __launch_bounds__(ST) mx4_gemm_simple(const Mx4Gemm A) {
  constexpr int NW = MODE == MX4_GATE_UP ? 2 : 1;
  __shared__ float sw[NW][SR][MXB + 1], sx[SP][MXB + 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, p = tid & 31, rg = tid >> 5;
  const int n_ent = mx4_entries<MODE>(A);
  if ((int)blockIdx.y >= n_ent) return;
  const Mx4Entry e = mx4_entry<MODE>(A, blockIdx.y);
  const int r0 = blockIdx.x * SR;
  if (r0 >= e.rows) return;
  const uint8_t* wc = e.shared ? A.shc : A.wc;
  const uint8_t* wsc = e.shared ? A.shs : A.wsc;
  const long long wrow = mx4_weight_row<MODE>(e) + r0;
  for (int p0 = 0; p0 < e.count; p0 += SP) {
    float acc[NW][4] = {};
    for (int k0 = 0; k0 < e.K; k0 += MXB) {
      __syncthreads();
      for (int i = tid; i < SR * MXB; i += ST) {
        const int r = i / MXB, k = i % MXB;
        for (int w = 0; w < NW; ++w)
          sw[w][r][k] = r0 + r < e.rows ? mx4_value(wc, wsc, wrow + r + (long long)w * e.rows, e.K, k0 + k) : 0.f;
        sx[r][k] = p0 + r < e.count ? mx4_value(A.xc, A.xs, e.row0 + p0 + r, A.xpitch, k0 + k) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < MXB; ++k) {
        const float x = sx[p][k];
        for (int w = 0; w < NW; ++w)
          for (int j = 0; j < 4; ++j) acc[w][j] += x * sw[w][rg * 4 + j][k];
      }
    }
    if (MODE == MX4_GATE_UP) {
      __syncthreads();
      for (int j = 0; j < 4; ++j) {
        const float g = acc[0][j], u = acc[NW - 1][j];
        sw[0][rg * 4 + j][p] = g / (1.f + expf(-g)) * u;
      }
      __syncthreads();
      // a row's block of 32 h values: four lanes of eight
      const int q = tid >> 2, i8 = (tid & 3) * 8;
      if (q < SP) {
        float v[8];
        for (int i = 0; i < 8; ++i) v[i] = sw[0][i8 + i][q];
        uint32_t b;
        const uint32_t w = mx4_quant8(v, &b);
        if (p0 + q < e.count) {
          const long long row = e.row0 + p0 + q;
          reinterpret_cast<uint32_t*>(A.ws + A.L.hq)[(row * A.L.imax + r0 + i8) / 8] = w;
          if (i8 == 0) (A.ws + A.L.hs)[(row * A.L.imax + r0) / MXB] = (uint8_t)b;
          if (b == 255u) atomicOr(reinterpret_cast<uint32_t*>(A.ws), COLI_STATUS_NONFINITE);
        }
      }
    } else if (p0 + p < e.count) {
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + rg * 4 + j;
        if (r < e.rows) store_typed(A.y, A.y_type, (e.row0 + p0 + p) * A.ldy + r, acc[0][j]);
      }
    }
  }
}

cudaError_t launch_mx4_gemm(const Mx4Gemm& A, Mx4Mode mode, cudaStream_t st) {
  const int rows = mode == MX4_PRODUCT ? A.N : mode == MX4_GATE_UP ? A.L.imax : A.cfg.hidden;
  const dim3 grid((rows + SR - 1) / SR, mode == MX4_PRODUCT ? A.G : A.L.n_ent_max);
  if (mode == MX4_PRODUCT) mx4_gemm_simple<MX4_PRODUCT><<<grid, ST, 0, st>>>(A);
  else if (mode == MX4_GATE_UP) mx4_gemm_simple<MX4_GATE_UP><<<grid, ST, 0, st>>>(A);
  else mx4_gemm_simple<MX4_DOWN><<<grid, ST, 0, st>>>(A);
  return cudaGetLastError();
}

}  // namespace colimoe
