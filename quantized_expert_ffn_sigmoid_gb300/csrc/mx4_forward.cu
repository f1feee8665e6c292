// Dispatch and combine of the MX4 expert layer, and the entry points of the
// grouped product and the layer.
//
// The layer: x in MX4, one copy of a token's row per expert it goes to, rows
// of one expert consecutive; gate/up products with SwiGLU and MX4 of h; down
// products; y = sum_j w_j o_j + sum_s o_s in fixed order.
#include "mx4_layer.cuh"

namespace colimoe {

constexpr int TT = 1024;  // threads of the table kernel

// exclusive scan of one int per thread over 1024 threads
__device__ int scan1024(int v, int* part /*33*/, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = part[lane];
    int wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += n;
    }
    part[lane] = wi - w;
    if (lane == 31) part[32] = wi;
  }
  __syncthreads();
  const int r = part[warp] + inc - v;
  *total = part[32];
  __syncthreads();
  return r;
}

// Entries (distinct experts ascending, then the shared ones) with their row
// ranges, and the row of every (token, slot).  The order of rows inside an
// expert's range is the order of shared-memory atomics and may differ from
// call to call; no result depends on it, since every row's products are
// computed alike wherever the row stands.
__global__ void __launch_bounds__(TT) mx4_tables(const coli_moe_cfg c, const Mx4Layout L, const int32_t* __restrict__ idx, int T,
                                                 uint8_t* __restrict__ ws) {
  __shared__ int cnt[MAX_E], off[MAX_E], part[33];
  const int tid = threadIdx.x, E = c.n_experts, np = T * c.top_k;
  int32_t* slot = reinterpret_cast<int32_t*>(ws + L.slot);
  int32_t* ent_expert = reinterpret_cast<int32_t*>(ws + L.ent_expert);
  int32_t* ent_count = reinterpret_cast<int32_t*>(ws + L.ent_count);
  int32_t* ent_offset = reinterpret_cast<int32_t*>(ws + L.ent_offset);
  int32_t* hdr = reinterpret_cast<int32_t*>(ws + L.hdr);
  cnt[tid] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  bool bad = false;
  for (int p = tid; p < np; p += TT) {
    const int e = idx[p];
    const bool in = e >= 0 && e < E;
    bad |= !in && e != -1;
    slot[p] = in && ep_owned(c, e) ? atomicAdd(&cnt[e], 1) : -1;
  }
  if (bad) atomicOr(reinterpret_cast<uint32_t*>(ws), COLI_STATUS_BADIDX);
  __syncthreads();
  int pairs, uniq;
  const int v = tid < E ? cnt[tid] : 0;
  const int o = scan1024(v, part, &pairs);
  const int ent = scan1024(v > 0 ? 1 : 0, part, &uniq);
  off[tid] = o;
  if (v > 0) {
    ent_expert[ent] = tid;
    ent_count[ent] = v;
    ent_offset[ent] = o;
  }
  const int ns = c.n_shared;
  if (tid < ns) {
    ent_expert[uniq + tid] = E + tid;
    ent_count[uniq + tid] = T;
    ent_offset[uniq + tid] = pairs + tid * T;
  }
  if (tid == 0) {
    ent_offset[uniq + ns] = pairs + ns * T;
    hdr[MH_NENT] = uniq + ns;
    hdr[MH_NUNIQ] = uniq;
    hdr[MH_NPAIRS] = pairs + ns * T;
  }
  __syncthreads();
  for (int p = tid; p < np; p += TT) {  // the same thread as above wrote slot[p]
    const int r = slot[p];
    if (r >= 0) slot[p] = off[idx[p]] + r;
  }
}

// MX4 of each token's row (or the caller's codes), written to every row of
// the token's experts.  A warp takes 1024 elements of one token.
template <typename T, int TYPE>
__global__ void __launch_bounds__(256) mx4_gather(const coli_moe_cfg c, const Mx4Layout L, const T* __restrict__ x,
                                                  const uint8_t* __restrict__ x_scales, int rows, uint8_t* __restrict__ ws) {
  const int lane = threadIdx.x & 31, H = c.hidden, k = c.top_k, ns = c.n_shared;
  const int per_row = (H + 1023) / 1024;
  const long long tasks = (long long)rows * per_row, step = (long long)gridDim.x * 8;
  pdl_wait();
  pdl_trigger();
  const int32_t* hdr = reinterpret_cast<const int32_t*>(ws + L.hdr);
  const int32_t* slot = reinterpret_cast<const int32_t*>(ws + L.slot);
  const int shared0 = __ldcg(hdr + MH_NPAIRS) - ns * rows;
  uint32_t* xq = reinterpret_cast<uint32_t*>(ws + L.xq);
  uint8_t* xs = ws + L.xs;
  for (long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); task < tasks; task += step) {
    const int t = (int)(task / per_row);
    const int k0 = (int)(task - (long long)t * per_row) * 1024 + lane * 8;
    uint32_t w[4] = {}, b[4] = {};
    if constexpr (TYPE == COLI_MX4) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k0 + u * 256 < H) {
          const long long at = (long long)t * H + k0 + u * 256;
          w[u] = reinterpret_cast<const uint32_t*>(x)[at / 8];
          b[u] = x_scales[at / MXB];
        }
    } else {
      float v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (k0 + u * 256 < H) {
          load8<T, true>(x + (long long)t * H + k0 + u * 256, 8, v[u]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = mx4_quant8(v[u], &b[u]);
    }
    bool bad = false;
    for (int j = 0; j < k + ns; ++j) {
      const int r = j < k ? __ldcg(slot + (long long)t * k + j) : shared0 + (j - k) * rows + t;
      if (r < 0) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k0 + u * 256 < H) {
          const long long at = (long long)r * H + k0 + u * 256;
          xq[at / 8] = w[u];
          if ((lane & 3) == 0) xs[at / MXB] = (uint8_t)b[u];
          bad |= b[u] == 255u;
        }
    }
    if (bad) atomicOr(reinterpret_cast<uint32_t*>(ws), COLI_STATUS_NONFINITE);
  }
}

// y[t] = sum_j w[t][j] o[row(t, j)] + sum_s o[shared row of t], in this order
__global__ void __launch_bounds__(256) mx4_combine(const coli_moe_cfg c, const Mx4Layout L, const uint8_t* __restrict__ ws, int T,
                                                   const float* __restrict__ topk_w, void* __restrict__ y, int32_t y_type) {
  const int H = c.hidden, k = c.top_k, ns = c.n_shared, h4 = H / 4;
  pdl_wait();
  pdl_trigger();
  const int32_t* slot = reinterpret_cast<const int32_t*>(ws + L.slot);
  const int shared0 = __ldcg(reinterpret_cast<const int32_t*>(ws + L.hdr) + MH_NPAIRS) - ns * T;
  const float* o = reinterpret_cast<const float*>(ws + L.o);
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < (long long)T * h4; i += (long long)gridDim.x * 256) {
    const int t = (int)(i / h4), c4 = (int)(i - (long long)t * h4);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < k + ns; ++j) {
      const int r = j < k ? __ldcg(slot + (long long)t * k + j) : shared0 + (j - k) * T + t;
      if (r < 0) continue;
      const float w = j < k ? topk_w[(long long)t * k + j] : 1.f;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(o + (long long)r * H) + c4);
      a.x += w * v.x; a.y += w * v.y; a.z += w * v.z; a.w += w * v.w;
    }
    if (y_type == COLI_F32) {
      reinterpret_cast<float4*>(y)[i] = a;
    } else {
      const float v[4] = {a.x, a.y, a.z, a.w};
      uint32_t p[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (y_type == COLI_BF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
          p[q] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(v[2 * q], v[2 * q + 1]);
          p[q] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      reinterpret_cast<uint2*>(y)[i] = make_uint2(p[0], p[1]);
    }
  }
}

cudaError_t launch_mx4_dispatch(const coli_moe_cfg& c, const Mx4Layout& L, const void* x, int32_t x_type, const uint8_t* x_scales,
                                int T, const int32_t* idx, uint8_t* ws, cudaStream_t st) {
  const cudaError_t e = launch_pdl(mx4_tables, 1, TT, 0, st, c, L, idx, T, ws);
  if (e != cudaSuccess) return e;
  const int sms = device_sms() > 0 ? device_sms() : 152;
  const long long tasks = (long long)T * ((c.hidden + 1023) / 1024);
  long long blocks = (tasks + 7) / 8;
  if (blocks > 8LL * sms) blocks = 8LL * sms;
  const unsigned grid = (unsigned)blocks;
  if (x_type == COLI_F32)
    return launch_pdl(mx4_gather<float, COLI_F32>, grid, 256, 0, st, c, L, static_cast<const float*>(x), x_scales, T, ws);
  if (x_type == COLI_BF16)
    return launch_pdl(mx4_gather<__nv_bfloat16, COLI_BF16>, grid, 256, 0, st, c, L, static_cast<const __nv_bfloat16*>(x), x_scales, T, ws);
  if (x_type == COLI_F16)
    return launch_pdl(mx4_gather<__half, COLI_F16>, grid, 256, 0, st, c, L, static_cast<const __half*>(x), x_scales, T, ws);
  return launch_pdl(mx4_gather<uint8_t, COLI_MX4>, grid, 256, 0, st, c, L, static_cast<const uint8_t*>(x), x_scales, T, ws);
}

cudaError_t launch_mx4_combine(const coli_moe_cfg& c, const Mx4Layout& L, const uint8_t* ws, int T, const float* topk_w, void* y,
                               int32_t y_type, cudaStream_t st) {
  const long long n4 = (long long)T * (c.hidden / 4);
  const int sms = device_sms() > 0 ? device_sms() : 152;
  long long blocks = (n4 + 255) / 256;
  if (blocks > 8LL * sms) blocks = 8LL * sms;
  return launch_pdl(mx4_combine, (unsigned)blocks, 256, 0, st, c, L, ws, T, topk_w, y, y_type);
}

}  // namespace colimoe

using namespace colimoe;

namespace {

int rc_of(cudaError_t e) { return e == cudaSuccess ? COLI_OK : COLI_ECUDA; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The layer limits of coli_moe_forward apply (coli_moe_workspace_size is 0
// outside them); the MX4 container is the 4-bit one with its own scales.
int check_mx4_cfg(const coli_moe_cfg* cfg, int32_t T, coli_moe_cfg* out) {
  if (!cfg || T < 0 || coli_moe_workspace_size(cfg, T) == 0) return COLI_EINVAL;
  if (cfg->weight_bits != 4 || cfg->group_size != 0) return COLI_EINVAL;
  *out = *cfg;
  if (out->ep_size <= 1) out->ep_size = 1;
  if (out->ep_rank != 0) out->n_shared = 0;  // the shared experts belong to shard 0
  if (out->n_shared == 0) out->shared_inter = out->inter;
  // rows and table indices are 32-bit
  const long long P = (long long)T * (out->top_k + out->n_shared);
  return P <= 0x7fffffffLL / 64 ? COLI_OK : COLI_EUNSUPPORTED;
}

}  // namespace

extern "C" int coli_mx4_product(const uint8_t* x_codes, const uint8_t* x_scales, int32_t P, const uint8_t* w_codes,
                                const uint8_t* w_scales, int32_t G, int32_t N, int32_t K, const int32_t* offsets, void* y,
                                int32_t y_type, int64_t ldy, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (P < 0 || G < 1 || N < 1 || K < 1 || K % MXB || !float_type(y_type) || ldy < N) return COLI_EINVAL;
  if (G > COLI_MX4_MAX_GROUPS || (long long)G * N > 0x7fffffffLL || P > 0x7fffffff / 64) return COLI_EUNSUPPORTED;
  if (!offsets && G != 1) return COLI_EINVAL;
  if (P == 0) return COLI_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !y || !ws) return COLI_EINVAL;
  if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) ||
      !aligned16(ws) || (reinterpret_cast<uintptr_t>(offsets) & 3u))
    return COLI_EALIGN;
  if (ws_bytes < WS_HEADER_BYTES) return COLI_EWORKSPACE;
  Mx4Gemm A{};
  A.xc = x_codes;
  A.xs = x_scales;
  A.wc = w_codes;
  A.wsc = w_scales;
  A.offsets = offsets;
  A.G = G;
  A.N = N;
  A.K = A.xpitch = K;
  A.P = P;
  A.y = y;
  A.y_type = y_type;
  A.ldy = ldy;
  A.ws = static_cast<uint8_t*>(ws);
  return rc_of(launch_mx4_gemm(A, MX4_PRODUCT, stream));
}

extern "C" size_t coli_mx4_workspace_size(const coli_moe_cfg* cfg, int32_t max_T) {
  coli_moe_cfg c;
  if (check_mx4_cfg(cfg, max_T, &c) != COLI_OK) return 0;
  // one workspace serves coli_moe_route and coli_mx4_forward
  const size_t moe = coli_moe_workspace_size(cfg, max_T), mx = make_mx4_layout(c, max_T).total;
  return moe > mx ? moe : mx;
}

extern "C" int coli_mx4_forward(const coli_moe_cfg* cfg, const coli_mx4_weights* weights, const void* x, int32_t x_type,
                                const uint8_t* x_scales, int32_t T, const int32_t* topk_idx, const float* topk_w, void* y,
                                int32_t y_type, void* ws, size_t ws_bytes, cudaStream_t stream) {
  coli_moe_cfg c;
  int rc = check_mx4_cfg(cfg, T, &c);
  if (rc) return rc;
  if ((!float_type(x_type) && x_type != COLI_MX4) || !float_type(y_type)) return COLI_EINVAL;
  if (T == 0) return COLI_OK;
  if (!weights || !weights->experts || !weights->expert_scales) return COLI_EINVAL;
  if (c.n_shared > 0 && (!weights->shared || !weights->shared_scales)) return COLI_EINVAL;
  if (!x || !topk_idx || !topk_w || !y || !ws || (x_type == COLI_MX4) != (x_scales != nullptr)) return COLI_EINVAL;
  const void* ptrs[] = {weights->experts, weights->expert_scales, x, topk_idx, topk_w, y, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return COLI_EALIGN;
  if (x_scales && !aligned16(x_scales)) return COLI_EALIGN;
  if (c.n_shared > 0 && (!aligned16(weights->shared) || !aligned16(weights->shared_scales))) return COLI_EALIGN;
  const Mx4Layout L = make_mx4_layout(c, T);
  if (ws_bytes < L.total) return COLI_EWORKSPACE;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  if ((rc = rc_of(launch_mx4_dispatch(c, L, x, x_type, x_scales, T, topk_idx, w8, stream)))) return rc;
  Mx4Gemm A{};
  A.wc = weights->experts;
  A.wsc = weights->expert_scales;
  A.shc = weights->shared;
  A.shs = weights->shared_scales;
  A.P = L.P;
  A.ws = w8;
  A.L = L;
  A.cfg = c;
  A.xc = w8 + L.xq;
  A.xs = w8 + L.xs;
  A.xpitch = c.hidden;
  if ((rc = rc_of(launch_mx4_gemm(A, MX4_GATE_UP, stream)))) return rc;
  A.xc = w8 + L.hq;
  A.xs = w8 + L.hs;
  A.xpitch = L.imax;
  A.y = w8 + L.o;
  A.y_type = COLI_F32;
  A.ldy = c.hidden;
  if ((rc = rc_of(launch_mx4_gemm(A, MX4_DOWN, stream)))) return rc;
  return rc_of(launch_mx4_combine(c, L, w8, T, topk_w, y, y_type, stream));
}
