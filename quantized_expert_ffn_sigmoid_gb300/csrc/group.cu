// The routed pairs in expert order, and the weighted sum that brings their
// results back to the positions.
//
// Grouping is a stable counting sort of T * top_k ids: pairs of one expert
// stand together, in the order of their positions, so results do not depend on
// the order of any atomic.  A CTA of 32 warps takes a run of pairs, each warp a
// consecutive part of it: the warp counts its part per expert (pairs of one
// expert within a warp's 32 find each other by match), a scan over the warps and
// one over the experts give every warp its first place per expert, and a second
// pass over the part hands the places out.  More pairs than one CTA takes are
// counted first by a kernel of their own; each CTA then sums the counts of the
// CTAs before it.  Bound: latency (131072 pairs are 1.5 MB in all): 256 pairs over
// 256 experts 3.9 us, 131072 10.6 us, of which 4 are the first kernel.
//
// The sum is one pass: a thread owns 8 consecutive values of a position and
// adds the slots' terms in their order in fp32 registers, then rounds once.
// Bound: HBM (each pair's row is read once): 2048 positions of 8 pairs of 6144 bf16
// values 34.7 us, 7.2 TB/s with what is still in L2 (of 6143 values, one a load, 86 us);
// 32 positions 3.0 us.
#include "mx4_common.cuh"

namespace colimoe {
namespace {

constexpr int GR_WARPS = 32, GR_THREADS = 32 * GR_WARPS;
// Up to GR_ONE pairs one CTA does it all (2048 pairs 6.9 us, in two runs 7.6);
// beyond, runs of at least GR_RUN (4096 pairs 8.3 us, in runs of 2048 9.6).
constexpr int GR_ONE = 2048, GR_RUN = 1024;
constexpr int GR_CTAS = 128;      // CTAs at most, while runs stay below 2^20 pairs
constexpr int GR_MAX_RUN = 1 << 20;

struct GroupParams {
  const int32_t* idx;
  long long n;        // pairs
  int k, E, ep_rank, ep_size, local;  // local: experts of this shard
  int run, ctas;
  int32_t *offsets, *rows, *slots, *counts;  // counts [ctas][local]
  uint32_t* status;
};

// group of a pair, -1 for skipped slots
__device__ __forceinline__ int group_of(const GroupParams& P, long long pair, bool* bad) {
  const int e = __ldcg(P.idx + pair);
  if (e < 0 || e >= P.E) {
    *bad |= e != -1;
    return -1;
  }
  if (P.ep_size <= 1) return e;
  return e % P.ep_size == P.ep_rank ? e / P.ep_size : -1;
}

__global__ void __launch_bounds__(GR_THREADS) group_count(const GroupParams P) {
  extern __shared__ int sm_count[];
  pdl_wait();
  pdl_trigger();
  for (int e = threadIdx.x; e < P.local; e += GR_THREADS) sm_count[e] = 0;
  __syncthreads();
  const long long first = (long long)blockIdx.x * P.run, last = min(first + P.run, P.n);
  bool bad = false;
  for (long long p = first + threadIdx.x; p < last; p += GR_THREADS) {
    const int g = group_of(P, p, &bad);
    if (g >= 0) atomicAdd(&sm_count[g], 1);  // (counts alone: their order is free)
  }
  __syncthreads();
  for (int e = threadIdx.x; e < P.local; e += GR_THREADS) P.counts[(long long)blockIdx.x * P.local + e] = sm_count[e];
}

// MULTI: group_count has run over the same runs
template <bool MULTI>
__global__ void __launch_bounds__(GR_THREADS) group_scatter(const GroupParams P) {
  extern __shared__ int sm_hist[];       // [warps][local], then [local] first places and [local] totals
  __shared__ int s_warp[GR_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, L = P.local;
  int* hist = sm_hist + warp * L;
  int* base = sm_hist + GR_WARPS * L;
  for (int i = tid; i < GR_WARPS * L; i += GR_THREADS) sm_hist[i] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const long long first = (long long)blockIdx.x * P.run, last = min(first + P.run, P.n);
  const int part = (P.run + GR_THREADS - 1) / GR_THREADS * 32;  // pairs of a warp
  const long long w0 = first + (long long)warp * part, w1 = min(w0 + part, last);
  bool bad = false;
  for (long long p0 = w0; p0 < w1; p0 += 32) {
    const int g = p0 + lane < w1 ? group_of(P, p0 + lane, &bad) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, g);
    if (g >= 0 && lane == __ffs(same) - 1) hist[g] += __popc(same);
    __syncwarp();
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0 && P.status) atomicOr(P.status, COLI_STATUS_BADIDX);
  __syncthreads();
  // per expert: the warps' first places within this run, and the run's own
  // (experts ascending over the threads, so the scan below is over experts)
  const int e = tid;
  if (MULTI) {
    // the other runs' counts: threads share an expert's, all loads under way together
    for (int i = tid; i < 2 * L; i += GR_THREADS) base[i] = 0;
    __syncthreads();
    int wide = 32;
    while (wide < L) wide *= 2;  // threads for one run's counts
    const int c = tid % wide, rows = GR_THREADS / wide;
    if (c < L) {
      int all = 0, ahead = 0;
      for (int b0 = tid / wide; b0 < P.ctas; b0 += 16 * rows) {
        int v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = b0 + i * rows < P.ctas ? __ldcg(P.counts + (long long)(b0 + i * rows) * L + c) : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          all += v[i];
          ahead += b0 + i * rows < (int)blockIdx.x ? v[i] : 0;
        }
      }
      atomicAdd(&base[c], ahead);  // (sums of whole numbers: their order is free)
      atomicAdd(&base[L + c], all);
    }
    __syncthreads();
  }
  int total = 0, before = 0;
  if (e < L) {
    int c[GR_WARPS];
#pragma unroll
    for (int w = 0; w < GR_WARPS; ++w) c[w] = sm_hist[w * L + e];
#pragma unroll
    for (int w = 0; w < GR_WARPS; ++w) {
      sm_hist[w * L + e] = total;
      total += c[w];
    }
    if (MULTI) {
      before = base[e];
      total = base[L + e];
    }
  }
  int scan = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) s_warp[warp] = scan;
  __syncthreads();
  if (warp == 0) {
    int v = s_warp[lane];
    const int own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    s_warp[lane] = v - own;
  }
  __syncthreads();
  scan += s_warp[warp];
  if (e < L) {
    base[e] = scan - total + before;
    if (blockIdx.x == 0) {
      P.offsets[e + 1] = scan;
      if (e == 0) P.offsets[0] = 0;
    }
  }
  __syncthreads();
  for (long long p0 = w0; p0 < w1; p0 += 32) {
    const long long p = p0 + lane;
    const int g = p < w1 ? group_of(P, p, &bad) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, g);
    int place = -1;
    if (g >= 0) place = base[g] + hist[g] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (g >= 0 && lane == __ffs(same) - 1) hist[g] += __popc(same);
    __syncwarp();
    if (p < w1) {
      P.slots[p] = place;
      if (place >= 0) P.rows[place] = (int)((uint32_t)p / (uint32_t)P.k);
    }
  }
}

int group_run(long long n) {
  long long run = (n + GR_CTAS - 1) / GR_CTAS;
  run = (run + GR_THREADS - 1) / GR_THREADS * GR_THREADS;
  if (n <= GR_ONE) return GR_ONE;
  return (int)(run < GR_RUN ? GR_RUN : run > GR_MAX_RUN ? GR_MAX_RUN : run);
}
int group_ctas(long long n) { const int run = group_run(n); return (int)((n + run - 1) / run); }

// ---------------------------------------------------------------- weighted sum
struct CombineParams {
  const void* o;
  long long ldo;
  int P;
  const int32_t* slots;
  const float* w;
  int T, k, H, units;
  const void* add;
  long long ld_add;
  void* y;
  long long ldy;
};

constexpr int CB_T = 256;

template <typename TO, typename TY, bool VEC>
__global__ void __launch_bounds__(CB_T) combine_kernel(const CombineParams P) {
  pdl_wait();
  pdl_trigger();
  const long long task = (long long)blockIdx.x * CB_T + threadIdx.x;
  const long long t = task <= 0xffffffffLL ? (long long)((uint32_t)task / (uint32_t)P.units) : task / P.units;
  if (t >= P.T) return;
  const int h = (int)(task - t * P.units) * 8, n = P.H - h;
  const int32_t* slot = P.slots + t * P.k;
  const float* w = P.w + t * P.k;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  if (P.add) {
    const Raw8<TY> r = load8<TY, VEC>(static_cast<const TY*>(P.add) + t * P.ld_add + h, n);
    floats8(r, acc);
  }
  constexpr int U = 4;  // slots whose rows are under way together
  for (int j0 = 0; j0 < P.k; j0 += U) {
    Raw8<TO> r[U];
    float f[U];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = j0 + u < P.k ? __ldcg(slot + j0 + u) : -1;
      live[u] = (unsigned)s < (unsigned)P.P;
      f[u] = live[u] ? __ldcg(w + j0 + u) : 0.f;
      r[u] = load8<TO, VEC>(static_cast<const TO*>(P.o) + (live[u] ? s : 0) * P.ldo + h, live[u] ? n : 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live[u]) continue;
      float v[8];
      floats8(r[u], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(f[u], v[i], acc[i]);
    }
  }
  store8<TY, VEC>(static_cast<TY*>(P.y) + t * P.ldy + h, n, acc);
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? COLI_OK : COLI_ECUDA; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename TO, typename TY>
cudaError_t launch_combine(const CombineParams& P, bool vec, cudaStream_t st) {
  const long long grid = ((long long)P.T * P.units + CB_T - 1) / CB_T;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return vec ? launch_pdl(combine_kernel<TO, TY, true>, (unsigned)grid, CB_T, 0, st, P) : launch_pdl(combine_kernel<TO, TY, false>, (unsigned)grid, CB_T, 0, st, P);
}
template <typename TO>
cudaError_t combine_to(const CombineParams& P, int32_t y_type, bool vec, cudaStream_t st) {
  if (y_type == COLI_F32) return launch_combine<TO, float>(P, vec, st);
  if (y_type == COLI_BF16) return launch_combine<TO, __nv_bfloat16>(P, vec, st);
  return launch_combine<TO, __half>(P, vec, st);
}

}  // namespace
}  // namespace colimoe

using namespace colimoe;

extern "C" size_t coli_moe_group_workspace_size(int32_t max_T, int32_t top_k, int32_t n_experts) {
  if (max_T < 0 || top_k < 1 || top_k > MAX_TOPK || n_experts < 1 || n_experts > MAX_E) return 0;
  const long long n = (long long)max_T * top_k;
  if (n > 0x7fffffffLL) return 0;
  // (CTAs grow with the pairs up to GR_CTAS, and beyond it once runs are at their longest)
  const long long ctas = n > (long long)GR_CTAS * GR_MAX_RUN ? group_ctas(n) : GR_CTAS;
  return align_up(WS_HEADER_BYTES + (size_t)ctas * n_experts * 4, 256);
}

extern "C" int coli_moe_group(const int32_t* topk_idx, int32_t T, int32_t top_k, int32_t n_experts, int32_t ep_rank, int32_t ep_size,
                              int32_t* offsets, int32_t* rows, int32_t* slots, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (T < 0 || top_k < 1 || n_experts < 1 || ep_size < 0 || ep_size > n_experts || ep_rank < 0 || ep_rank >= (ep_size > 1 ? ep_size : 1)) return COLI_EINVAL;
  if (top_k > MAX_TOPK || n_experts > MAX_E || (long long)T * top_k > 0x7fffffffLL) return COLI_EUNSUPPORTED;
  if (!offsets || !ws || (T > 0 && (!topk_idx || !rows || !slots))) return COLI_EINVAL;
  const void* ptrs[] = {topk_idx, offsets, rows, slots, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return COLI_EALIGN;
  if (ws_bytes < coli_moe_group_workspace_size(T, top_k, n_experts)) return COLI_EWORKSPACE;
  GroupParams P{};
  P.idx = topk_idx;
  P.n = (long long)T * top_k;
  P.k = top_k;
  P.E = n_experts;
  P.ep_rank = ep_rank;
  P.ep_size = ep_size;
  P.local = ep_size <= 1 ? n_experts : (n_experts - ep_rank + ep_size - 1) / ep_size;
  P.run = group_run(P.n);
  P.ctas = P.n > 0 ? group_ctas(P.n) : 1;  // no positions: every offset is 0
  P.offsets = offsets;
  P.rows = rows;
  P.slots = slots;
  P.counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + WS_HEADER_BYTES);
  P.status = static_cast<uint32_t*>(ws);
  const size_t smem = (size_t)(GR_WARPS + 2) * P.local * 4;
  static std::atomic<uint64_t> raised{0};  // the shared-memory limit, once a device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return COLI_ECUDA;
  if (!(raised.load(std::memory_order_acquire) >> dev & 1)) {
    const int most = (GR_WARPS + 2) * MAX_E * 4;
    if (cudaFuncSetAttribute(group_scatter<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
        cudaFuncSetAttribute(group_scatter<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
      return COLI_ECUDA;
    raised.fetch_or(1ull << dev, std::memory_order_release);
  }
  if (P.ctas == 1) return rc_of(launch_pdl(group_scatter<false>, 1u, GR_THREADS, smem, stream, P));
  const cudaError_t e = launch_pdl(group_count, (unsigned)P.ctas, GR_THREADS, (size_t)P.local * 4, stream, P);
  if (e != cudaSuccess) return COLI_ECUDA;
  return rc_of(launch_pdl(group_scatter<true>, (unsigned)P.ctas, GR_THREADS, smem, stream, P));
}

extern "C" int coli_moe_combine(const void* o, int32_t o_type, int64_t ldo, int32_t P, const int32_t* slots, const float* topk_w, int32_t T,
                                int32_t top_k, int32_t H, const void* add, int64_t ld_add, void* y, int32_t y_type, int64_t ldy, cudaStream_t stream) {
  if (T < 0 || P < 0 || top_k < 1 || H < 1 || !float_type(o_type) || !float_type(y_type) || ldo < H || ldy < H || (add && ld_add < H)) return COLI_EINVAL;
  if (T == 0) return COLI_OK;
  if (!slots || !topk_w || !y || (P > 0 && !o)) return COLI_EINVAL;
  const void* ptrs[] = {o, slots, topk_w, add, y};
  for (const void* p : ptrs)
    if (!aligned16(p)) return COLI_EALIGN;
  CombineParams C{};
  C.o = o;
  C.ldo = ldo;
  C.P = P;
  C.slots = slots;
  C.w = topk_w;
  C.T = T;
  C.k = top_k;
  C.H = H;
  C.units = (H + 7) / 8;
  C.add = add;
  C.ld_add = ld_add;
  C.y = y;
  C.ldy = ldy;
  const bool vec = H % 8 == 0 && rows_aligned(o, ldo, o_type) && rows_aligned(y, ldy, y_type) && (!add || rows_aligned(add, ld_add, y_type));
  if (o_type == COLI_F32) return rc_of(combine_to<float>(C, y_type, vec, stream));
  if (o_type == COLI_BF16) return rc_of(combine_to<__nv_bfloat16>(C, y_type, vec, stream));
  return rc_of(combine_to<__half>(C, y_type, vec, stream));
}
