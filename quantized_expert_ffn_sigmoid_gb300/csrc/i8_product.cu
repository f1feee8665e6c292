// Products of 8-bit codes with a scale for each token and each channel, grouped
// by expert: the entry point and the kernel of calls with few rows (the
// others: i8_gemm.cu).
//
// Mathematics.  y[p][n] = sx[row] * sw[g][n] * sum_k x[row][k] w[g][n][k], the sum
// exact in 32-bit integers (K up to 131071 products of at most 2^14), so every
// path and every split of the sum gives the same bits.
//
// Few rows (up to 8): a stream of the weights through 4-way integer dots, with
// the codes of the group's rows in shared memory.  A warp takes R weight rows
// (2, or 4 where 3 or more activation rows reuse the loads from shared memory),
// each lane 16 bytes of every 512; the lanes' sums meet in redux.  Bound: HBM;
// 4096 x 6144 against one row 6.0 us (25 MB, in L2 here; 9.9 us cold), 8 experts' of
// 256 for one position 41.7 us (4.8 TB/s: the last CTAs' tail).
#include "i8_product.cuh"

namespace colimoe {
namespace {

constexpr int IS_WARPS = 8, IS_T = 32 * IS_WARPS;
// Codes of a row held in shared memory at a time: 48 KB for eight rows.  Each further
// part costs two barriers, half a microsecond (1 row against 4096 x 6144 4.8 us, x 6160
// 5.3, x 8192 5.8, x 12288 7.0).
constexpr int IS_KC = 6144;

// 16 codes at p of which n exist (the others 0)
__device__ __forceinline__ uint4 codes16(const int8_t* p, int n) {
  if (n >= 16) return __ldcs(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) w[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int c) {
  c = dp4a_ss(a.x, b.x, c);
  c = dp4a_ss(a.y, b.y, c);
  c = dp4a_ss(a.z, b.z, c);
  return dp4a_ss(a.w, b.w, c);
}

template <typename T>
__device__ __forceinline__ void put(void* y, long long at, float v) { static_cast<T*>(y)[at] = from_f32<T>(v); }
__device__ __forceinline__ void put_any(void* y, int32_t type, long long at, float v) {
  if (type == COLI_F32) put<float>(y, at, v);
  else if (type == COLI_BF16) put<__nv_bfloat16>(y, at, v);
  else put<__half>(y, at, v);
}

// One block of weight rows against up to MT activation rows p0 ..
template <int MT, int R>
__device__ __forceinline__ void stream_block(const I8Params& A, int g, int p0, int nt, int block, const int* s_row, uint4* sx) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n0 = (block * IS_WARPS + warp) * R;
  int acc[R][MT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[r][t] = 0;
  for (int kc = 0; kc < A.K; kc += IS_KC) {
    const int span = min(IS_KC, A.K - kc), units = (span + 15) / 16;
    __syncthreads();  // (the last block's or chunk's codes are no longer read)
    for (int i = threadIdx.x; i < MT * units; i += IS_T) {
      const int t = i / units, u = i - t * units;
      const int row = t < nt ? s_row[p0 + t] : -1;
      sx[t * (IS_KC / 16) + u] = codes16(A.x + (row < 0 ? 0 : row) * A.ldx + kc + 16 * u, row < 0 ? 0 : span - 16 * u);
    }
    __syncthreads();
    if (n0 < A.N) {
      const int8_t* w = A.w + g * A.wgroup + (long long)n0 * A.ldw + kc;
      const int8_t* wr[R];
#pragma unroll
      for (int r = 0; r < R; ++r) wr[r] = w + (n0 + r < A.N ? r * A.ldw : 0);
      auto dots = [&](int u, const uint4* b) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const uint4 a = sx[t * (IS_KC / 16) + u];
#pragma unroll
          for (int r = 0; r < R; ++r) acc[r][t] = dot16(a, b[r], acc[r][t]);
        }
      };
      // U units of every row under way together
      constexpr int U = R == 2 ? 4 : 2;
      const int whole = span / 16;
      int u = lane;
      for (; u + (U - 1) * 32 < whole; u += U * 32) {
        uint4 b[U][R];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int r = 0; r < R; ++r) b[i][r] = __ldcs(reinterpret_cast<const uint4*>(wr[r]) + u + 32 * i);
#pragma unroll
        for (int i = 0; i < U; ++i) dots(u + 32 * i, b[i]);
      }
      for (; u < whole; u += 32) {
        uint4 b[R];
#pragma unroll
        for (int r = 0; r < R; ++r) b[r] = __ldcs(reinterpret_cast<const uint4*>(wr[r]) + u);
        dots(u, b);
      }
      if (u < units) {
        uint4 b[R];
#pragma unroll
        for (int r = 0; r < R; ++r) b[r] = codes16(wr[r] + 16 * u, span - 16 * u);
        dots(u, b);
      }
    }
  }
  if (n0 >= A.N) return;
  int mine = 0;  // lane r * MT + t
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int s = __reduce_add_sync(0xffffffffu, acc[r][t]);
      if (lane == r * MT + t) mine = s;
    }
  const int r = lane / MT, t = lane % MT;
  if (r < R && t < nt && n0 + r < A.N) {
    const int row = s_row[p0 + t];
    const float sx_ = row < 0 ? __uint_as_float(0x7fc00000u) : __ldcg(A.xs + row);
    put_any(A.y, A.y_type, (long long)(p0 + t) * A.ldy + n0 + r, i8_value(mine, sx_, __ldg(A.ws_ + g * A.wsgroup + n0 + r)));
  }
}

__global__ void __launch_bounds__(IS_T, 2) i8_stream(const I8Params A) {
  extern __shared__ __align__(16) uint4 sm_x[];  // [rows][IS_KC / 16]
  __shared__ int s_group[I8_FEW];                // group of each row of y (G: of none)
  __shared__ int s_row[I8_FEW];                  // its activation row (-1: out of range)
  __shared__ int s_seg[I8_FEW + 1], s_nseg;      // runs of rows of one group
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < I8_FEW) s_group[threadIdx.x] = A.offsets ? A.G + 1 : 1;
  __syncthreads();
  if (A.offsets)  // the first offset beyond a row ends its group
    for (int g = threadIdx.x; g <= A.G; g += IS_T) {
      const int o = i8_offset(A, g);
      for (int p = 0; p < A.P && p < o; ++p) atomicMin(&s_group[p], g);
    }
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0, last = -1;
    for (int p = 0; p < A.P; ++p) {
      const int g = s_group[p] - 1;  // -1: before the first group, G: behind the last
      s_group[p] = g;
      const bool live = g >= 0 && g < A.G;
      const int row = !live ? -1 : A.rows ? __ldcg(A.rows + p) : p;
      s_row[p] = row < 0 || row >= A.X ? -1 : row;
      if (live && s_row[p] < 0 && blockIdx.x == 0) atomicOr(reinterpret_cast<uint32_t*>(A.ws), COLI_STATUS_BADIDX);
      if (g != last) s_seg[n++] = p;
      last = g;
    }
    s_seg[n] = A.P;
    s_nseg = n;
  }
  __syncthreads();
  const int nseg = s_nseg;
  int first = 0;  // blocks before this segment
  for (int s = 0; s < nseg; ++s) {
    const int p0 = s_seg[s], nt = s_seg[s + 1] - p0, g = s_group[p0];
    if (g < 0 || g >= A.G) continue;
    const int rows = nt <= 2 ? 2 : 4, blocks = (A.N + IS_WARPS * rows - 1) / (IS_WARPS * rows);
    // the CTAs take the blocks of all segments in turn
    int b = (int)blockIdx.x - first % (int)gridDim.x;
    if (b < 0) b += gridDim.x;
    for (; b < blocks; b += gridDim.x) {
      if (nt == 1) stream_block<1, 2>(A, g, p0, nt, b, s_row, sm_x);
      else if (nt == 2) stream_block<2, 2>(A, g, p0, nt, b, s_row, sm_x);
      else if (nt <= 4) stream_block<4, 4>(A, g, p0, nt, b, s_row, sm_x);
      else stream_block<8, 4>(A, g, p0, nt, b, s_row, sm_x);
    }
    first += blocks;
  }
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? COLI_OK : COLI_ECUDA; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

cudaError_t launch_i8_stream(const I8Params& A, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int held = A.P <= 2 ? A.P : A.P <= 4 ? 4 : 8;
  const size_t smem = (size_t)held * IS_KC;
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(raised.load(std::memory_order_acquire) >> dev & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(i8_stream, cudaFuncAttributeMaxDynamicSharedMemorySize, I8_FEW * IS_KC);
    if (e != cudaSuccess) return e;
    raised.fetch_or(1ull << dev, std::memory_order_release);
  }
  const long long blocks = (long long)((A.N + 2 * IS_WARPS - 1) / (2 * IS_WARPS)) * (A.P < A.G ? A.P : A.G);
  return launch_pdl(i8_stream, (unsigned)(blocks < 2LL * sms ? blocks : 2LL * sms), IS_T, smem, st, A);
}

}  // namespace colimoe

using namespace colimoe;

extern "C" size_t coli_i8_product_workspace_size(int32_t max_P, int32_t K) {
  if (max_P < 0 || K < 1 || K > COLI_I8_MAX_K) return 0;
  return i8_ws_bytes(max_P, K);
}

extern "C" int coli_i8_product(const coli_i8_product_args* a, cudaStream_t stream) {
  if (!a) return COLI_EINVAL;
  if (a->P < 0 || a->x_rows < 0 || a->G < 1 || a->N < 1 || a->K < 1 || !float_type(a->y_type) || a->ldx < a->K || a->ldw < a->K || a->ldy < a->N)
    return COLI_EINVAL;
  if (a->G > 1 && (a->w_group < 0 || a->w_scale_group < 0)) return COLI_EINVAL;
  if (a->K > COLI_I8_MAX_K || a->G > COLI_I8_MAX_GROUPS || a->P > 0x7fffffff / 64 || a->N > 0x7fffffff / 64) return COLI_EUNSUPPORTED;
  if (!a->offsets && a->G != 1) return COLI_EINVAL;
  if (!a->rows && a->P > a->x_rows) return COLI_EINVAL;
  if (a->P == 0) return COLI_OK;
  if ((a->x_rows > 0 && (!a->x_codes || !a->x_scales)) || !a->w_codes || !a->w_scales || !a->y || !a->ws) return COLI_EINVAL;
  const void* ptrs[] = {a->x_codes, a->x_scales, a->rows, a->w_codes, a->w_scales, a->offsets, a->y, a->ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return COLI_EALIGN;
  if (a->ldx % 16 || a->ldw % 16 || (a->G > 1 && a->w_group % 16)) return COLI_EALIGN;
  if (a->ws_bytes < (i8_few(a->P, a->G) ? WS_HEADER_BYTES : i8_ws_bytes(a->P, a->K))) return COLI_EWORKSPACE;
  I8Params A{};
  A.x = a->x_codes;
  A.ldx = a->ldx;
  A.xs = a->x_scales;
  A.X = a->x_rows;
  A.rows = a->rows;
  A.P = a->P;
  A.w = a->w_codes;
  A.ldw = a->ldw;
  A.wgroup = a->G > 1 ? a->w_group : 0;
  A.ws_ = a->w_scales;
  A.wsgroup = a->G > 1 ? a->w_scale_group : 0;
  A.G = a->G;
  A.N = a->N;
  A.K = a->K;
  A.offsets = a->offsets;
  A.y = a->y;
  A.y_type = a->y_type;
  A.ldy = a->ldy;
  A.ws = static_cast<uint8_t*>(a->ws);
  return rc_of(i8_few(a->P, a->G) ? launch_i8_stream(A, stream) : launch_i8_gemm(A, stream));
}
