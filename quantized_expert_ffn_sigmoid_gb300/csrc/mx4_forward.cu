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
  int32_t* ent_offset = reinterpret_cast<int32_t*>(ws + L.ent_offset);
  int32_t* hdr = reinterpret_cast<int32_t*>(ws + L.hdr);
  cnt[tid] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  for (int u = tid; u < L.n_ent_max; u += TT) reinterpret_cast<uint32_t*>(ws + L.ready)[u] = 0u;
  if (tid == 0) *reinterpret_cast<uint32_t*>(ws + L.claim) = 0u;
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
    ent_offset[ent] = o;
  }
  const int ns = c.n_shared;
  if (tid < ns) {
    ent_expert[uniq + tid] = E + tid;
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

// MX4 of one unit (8 elements a lane, 256 a warp) of a token's row, or the
// caller's codes: the lane's codes and its block's scale byte.
template <typename T>
__device__ __forceinline__ uint32_t unit_codes(const T* x, const uint8_t* x_scales, long long at, bool in, uint32_t* b) {
  if constexpr (sizeof(T) == 1) {  // codes
    *b = in ? x_scales[at / MXB] : 0u;
    return in ? reinterpret_cast<const uint32_t*>(x)[at / 8] : 0u;
  } else {
    float v[8];
    floats8(load8<T, true>(x + at, in ? 8 : 0), v);
    return mx4_quant8(v, b);
  }
}

// Writes a lane's U units (codes w, scale bytes b, elements k0 + 256 u) to the
// rows that lanes 0 .. n-1 hold in `row` (-1: none).
template <int U>
__device__ __forceinline__ void scatter_units(uint8_t* ws, const Mx4Layout& L, int H, const uint32_t* w, const uint32_t* b, int k0,
                                              int row, int n) {
  const int lane = threadIdx.x & 31;
  uint32_t* xq = reinterpret_cast<uint32_t*>(ws + L.xq);
  uint8_t* xs = ws + L.xs;
  bool bad = false;
  for (int j = 0; j < n; ++j) {
    const int r = __shfl_sync(0xffffffffu, row, j);
    if (r < 0) continue;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u * 256 < H) {
        const long long at = (long long)r * H + k0 + u * 256;
        xq[at / 8] = w[u];
        if ((lane & 3) == 0) xs[at / MXB] = (uint8_t)b[u];
        bad |= b[u] == 255u;
      }
  }
  if (bad) atomicOr(reinterpret_cast<uint32_t*>(ws), COLI_STATUS_NONFINITE);
}

// MX4 of each token's row, written to every row of the token's experts.  A
// warp takes 1024 elements of one token.
template <typename T>
__global__ void __launch_bounds__(256) mx4_gather(const coli_moe_cfg c, const Mx4Layout L, const T* __restrict__ x,
                                                  const uint8_t* __restrict__ x_scales, int rows, uint8_t* __restrict__ ws) {
  const int lane = threadIdx.x & 31, H = c.hidden, k = c.top_k, ns = c.n_shared;
  const int per_row = (H + 1023) / 1024;
  const long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (task >= (long long)rows * per_row) return;
  const int t = (int)(task / per_row), k0 = (int)(task - (long long)t * per_row) * 1024 + lane * 8;
  const int32_t* slot = reinterpret_cast<const int32_t*>(ws + L.slot);
  const int shared0 = __ldcg(reinterpret_cast<const int32_t*>(ws + L.hdr) + MH_NPAIRS) - ns * rows;
  uint32_t w[4], b[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) w[u] = unit_codes(x, x_scales, (long long)t * H + k0 + u * 256, k0 + u * 256 < H, &b[u]);
  for (int j0 = 0; j0 < k + ns; j0 += 32) {
    const int j = j0 + lane;
    const int row = j < k ? __ldcg(slot + (long long)t * k + j) : shared0 + (j - k) * rows + t;
    scatter_units<4>(ws, L, H, w, b, k0, row, min(32, k + ns - j0));
  }
}

// Tables and activations of calls of few pairs in one launch: every CTA works
// out all pairs' rows by itself (in the order of (expert, pair), from the at
// most PREP_PAIRS ids in shared memory), CTA 0 writes the tables, and each
// warp quantises 256 elements of one token.
constexpr int PREP_PAIRS = 256;
template <typename T>
__global__ void __launch_bounds__(256) mx4_prep_small(const coli_moe_cfg c, const Mx4Layout L, const T* __restrict__ x,
                                                      const uint8_t* __restrict__ x_scales, int rows, const int32_t* __restrict__ idx,
                                                      uint8_t* __restrict__ ws) {
  __shared__ int4 s_keys[PREP_PAIRS / 4];
  __shared__ int s_row[PREP_PAIRS], s_expert[PREP_PAIRS + 1], s_leads[8];
  const int tid = threadIdx.x, lane = tid & 31, H = c.hidden, E = c.n_experts, k = c.top_k, ns = c.n_shared, np = rows * k;
  constexpr int NONE = 0x7fffffff;
  pdl_wait();
  pdl_trigger();
  // this warp's activations are on their way while the pairs are sorted
  const int per_row = H / 256 + (H % 256 ? 1 : 0);
  const int task = blockIdx.x * 8 + (tid >> 5);
  const int t = task / per_row, k0 = (task - t * per_row) * 256 + lane * 8;
  uint32_t w[1], b[1];
  w[0] = unit_codes(x, x_scales, (long long)t * H + k0, t < rows && k0 < H, &b[0]);
  bool bad = false;
  int key = NONE;
  if (tid < np) {
    const int e = idx[tid];
    const bool in = e >= 0 && e < E;
    bad = !in && e != -1;
    if (in && ep_owned(c, e)) key = e * PREP_PAIRS + tid;
  }
  reinterpret_cast<int*>(s_keys)[tid] = key;
  if (bad && blockIdx.x == 0) atomicOr(reinterpret_cast<uint32_t*>(ws), COLI_STATUS_BADIDX);
  const int pairs = __syncthreads_count(key != NONE);
  // a pair's row: the keys below its own
  int row = 0;
  if (key != NONE)
#pragma unroll 4
    for (int q = 0; q < (np + 3) / 4; ++q) {
      const int4 o = s_keys[q];
      row += (o.x < key) + (o.y < key) + (o.z < key) + (o.w < key);
    }
  s_row[tid] = key == NONE ? -1 : row;
  if (blockIdx.x == 0) {
    // entries: runs of one expert among the rows
    int32_t* ent_expert = reinterpret_cast<int32_t*>(ws + L.ent_expert);
    int32_t* ent_offset = reinterpret_cast<int32_t*>(ws + L.ent_offset);
    int32_t* hdr = reinterpret_cast<int32_t*>(ws + L.hdr);
    for (int u = tid; u < L.n_ent_max; u += 256) reinterpret_cast<uint32_t*>(ws + L.ready)[u] = 0u;
    if (tid == 0) *reinterpret_cast<uint32_t*>(ws + L.claim) = 0u;
    if (key != NONE) s_expert[row + 1] = key / PREP_PAIRS;
    if (tid == 0) s_expert[0] = -1;
    __syncthreads();
    const bool lead = tid < pairs && s_expert[tid + 1] != s_expert[tid];
    const unsigned leads = __ballot_sync(0xffffffffu, lead);
    if (lane == 0) s_leads[tid >> 5] = __popc(leads);
    const int uniq = __syncthreads_count(lead);
    if (lead) {
      int entry = __popc(leads & ((1u << lane) - 1u));
      for (int v = 0; v < tid >> 5; ++v) entry += s_leads[v];
      ent_expert[entry] = s_expert[tid + 1];
      ent_offset[entry] = tid;
    }
    if (tid < ns) ent_expert[uniq + tid] = E + tid;
    if (tid <= ns) ent_offset[uniq + tid] = pairs + tid * rows;
    if (tid == 0) {
      hdr[MH_NENT] = uniq + ns;
      hdr[MH_NUNIQ] = uniq;
      hdr[MH_NPAIRS] = pairs + ns * rows;
    }
    if (tid < np) reinterpret_cast<int32_t*>(ws + L.slot)[tid] = s_row[tid];
  } else {
    __syncthreads();
  }
  if (t >= rows) return;  // (whole warps)
  for (int j0 = 0; j0 < k + ns; j0 += 32) {
    const int j = j0 + lane;
    const int r = j < k ? s_row[t * k + j] : pairs + (j - k) * rows + t;
    scatter_units<1>(ws, L, H, w, b, k0, r, min(32, k + ns - j0));
  }
}

// y[t] = sum_j w[t][j] o[row(t, j)] + sum_s o[shared row of t], in this order.
// B rows' loads in flight per thread: 12 up to two CTAs an SM, where one round
// trip to L2 is what counts, 3 beyond, where bandwidth is and the registers
// have to leave room for threads.  Layer calls of 8 experts and a shared one,
// inter 128, with 12 and with 3: 48 CTAs 24.9 and 26.1 us, 128 26.1 and 27.3,
// 256 30.9 and 32.0, 288 34.4 and 34.3, 384 36.8 and 35.8, 768 47.6 and 43.6,
// 1536 61.1 and 53.7.
template <int B>
__global__ void __launch_bounds__(256) mx4_combine(const coli_moe_cfg c, const Mx4Layout L, const uint8_t* __restrict__ ws, int T,
                                                   const float* __restrict__ topk_w, void* __restrict__ y, int32_t y_type) {
  const int H = c.hidden, k = c.top_k, ns = c.n_shared, h4 = H / 4;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(i / h4), c4 = (int)(i - (long long)t * h4);
  pdl_wait();
  pdl_trigger();
  if (t >= T) return;
  const int32_t* slot = reinterpret_cast<const int32_t*>(ws + L.slot) + (long long)t * k;
  const int shared0 = __ldcg(reinterpret_cast<const int32_t*>(ws + L.hdr) + MH_NPAIRS) - ns * T;
  const float* o = reinterpret_cast<const float*>(ws + L.o);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < k + ns; j0 += B) {
    int r[B];
    float w[B];
    float4 v[B];
#pragma unroll
    for (int q = 0; q < B; ++q) {
      const int j = j0 + q;
      r[q] = j < k ? __ldcg(slot + j) : j < k + ns ? shared0 + (j - k) * T + t : -1;
      w[q] = j < k ? __ldg(topk_w + (long long)t * k + j) : 1.f;
    }
#pragma unroll
    for (int q = 0; q < B; ++q)
      if (r[q] >= 0) v[q] = __ldcs(reinterpret_cast<const float4*>(o + (long long)r[q] * H) + c4);
#pragma unroll
    for (int q = 0; q < B; ++q)
      if (r[q] >= 0) {
        a.x += w[q] * v[q].x; a.y += w[q] * v[q].y; a.z += w[q] * v[q].z; a.w += w[q] * v[q].w;
      }
  }
  if (y_type == COLI_F32) {
    reinterpret_cast<float4*>(y)[i] = a;
  } else if (y_type == COLI_BF16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a.x, a.y), q = __floats2bfloat162_rn(a.z, a.w);
    reinterpret_cast<uint2*>(y)[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
  } else {
    const __half2 p = __floats2half2_rn(a.x, a.y), q = __floats2half2_rn(a.z, a.w);
    reinterpret_cast<uint2*>(y)[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
  }
}

template <typename T>
cudaError_t dispatch(const coli_moe_cfg& c, const Mx4Layout& L, const T* x, const uint8_t* x_scales, int rows, const int32_t* idx,
                     uint8_t* ws, cudaStream_t st) {
  if (rows * c.top_k <= PREP_PAIRS && rows <= PREP_PAIRS) {
    const unsigned tasks = (unsigned)rows * (unsigned)((c.hidden + 255) / 256);
    return launch_pdl(mx4_prep_small<T>, (tasks + 7) / 8, 256, 0, st, c, L, x, x_scales, rows, idx, ws);
  }
  const cudaError_t e = launch_pdl(mx4_tables, 1, TT, 0, st, c, L, idx, rows, ws);
  if (e != cudaSuccess) return e;
  const long long tasks = (long long)rows * ((c.hidden + 1023) / 1024);
  return launch_pdl(mx4_gather<T>, (unsigned)((tasks + 7) / 8), 256, 0, st, c, L, x, x_scales, rows, ws);
}

cudaError_t launch_mx4_dispatch(const coli_moe_cfg& c, const Mx4Layout& L, const void* x, int32_t x_type, const uint8_t* x_scales,
                                int T, const int32_t* idx, uint8_t* ws, cudaStream_t st) {
  if (x_type == COLI_F32) return dispatch(c, L, static_cast<const float*>(x), x_scales, T, idx, ws, st);
  if (x_type == COLI_BF16) return dispatch(c, L, static_cast<const __nv_bfloat16*>(x), x_scales, T, idx, ws, st);
  if (x_type == COLI_F16) return dispatch(c, L, static_cast<const __half*>(x), x_scales, T, idx, ws, st);
  return dispatch(c, L, static_cast<const uint8_t*>(x), x_scales, T, idx, ws, st);
}

cudaError_t launch_mx4_combine(const coli_moe_cfg& c, const Mx4Layout& L, const uint8_t* ws, int T, const float* topk_w, void* y,
                               int32_t y_type, cudaStream_t st) {
  const long long blocks = ((long long)T * (c.hidden / 4) + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return blocks <= 2LL * device_sms() ? launch_pdl(mx4_combine<12>, (unsigned)blocks, 256, 0, st, c, L, ws, T, topk_w, y, y_type)
                                      : launch_pdl(mx4_combine<3>, (unsigned)blocks, 256, 0, st, c, L, ws, T, topk_w, y, y_type);
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
  if (K > COLI_MX4_MAX_K || G > COLI_MX4_MAX_GROUPS || (long long)G * N > 0x7fffffffLL || P > 0x7fffffff / 64) return COLI_EUNSUPPORTED;
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
  return rc_of(launch_mx4_product(A, stream));
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
  A.y = w8 + L.o;
  A.y_type = COLI_F32;
  A.ldy = c.hidden;
  if ((rc = rc_of(launch_mx4_layer(A, stream)))) return rc;
  return rc_of(launch_mx4_combine(c, L, w8, T, topk_w, y, y_type, stream));
}
