// Selection of experts from scores: softmax or sigmoid, a bias for balance,
// groups, top-k, weights from the unbiased scores.
//
// Mathematics, per position with logits l[e]:
//     s = softmax(l) or 1 / (1 + exp(-l));   v = s + bias
//     group score = the best v of the group, or the sum of its two best
//     the topk_group best groups stay (ties to the lower group)
//     the top_k best v of these, ties to the lower id;  w = s_sel [/ sum s_sel] * scaling
// An expert whose logit or bias is -inf takes no part.  Without a bias the
// logits rank the experts: scores are monotone in them, and where scores
// underflow or saturate to one value the logits still tell them apart.  They
// rank the groups by the groups' two best logits: by the best, or by the sum of
// their scores, of which sums that are equal in fp32 are told apart by
// sum_rest, their distance from 0, 1 or 2.
//
// One warp a position, E / 32 experts a lane (expert lane + 32 i) in registers.
// Scores become integers of the same order (0: takes no part), so that maxima are
// single warp reductions (redux).  The top-k first bounds the k-th best by the
// k-th best of the lanes' best, then ranks the few keys that reach the bound, a
// lane each; only where more than 32 do (many equal ones) it goes round by round.
// Groups of whole warps take two reductions each; others are scanned by one lane
// each in shared memory.  All sums are fp32.
//
// Bound: instructions (about 870 a position of 256 experts with groups and a bias;
// 16384 of them 14.6 us, issue slots 78 % busy, where their 17 MB would take 2.6;
// groups without a bias 16.9 us, softmax without groups 9.9 us; one position 2.7 us,
// from its hidden state 8.2).
#include "mx4_common.cuh"

namespace colimoe {
cudaError_t launch_route_partials(const float* x, int T, int H, const float* wr, int E, float* part, uint32_t* status, int* splits, cudaStream_t st);

namespace {

struct SelectParams {
  const void* x;      // logits, or the router product's partial sums [splits][T][E]
  long long ldx;
  int splits;
  const float* bias;
  int T, E, G, per, keep, k, softmax, top2, renorm;
  uint32_t gmul;      // e / per as (e * gmul) >> 20: exact for e < 1024
  float scaling;
  int32_t* idx;
  float* w;
  uint32_t* status;   // may be null
};

// floats as unsigned integers of the same order; -0 counts as +0
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// What tells sums of two scores apart that fp32 does not, as a + b unevaluated
// (logits l1 >= l2, without a bias; `sum` is the sum in fp32, f2 the score of l2):
//   softmax, and sigmoids near 0     log(e^l1 + e^l2) = l1 + log(1 + e^(l2 - l1))
//   one sigmoid near 1               s1 + s2 - 1 = s2 - sigmoid(-l1)
//   both                             -log(2 - s1 - s2) -> l2 - log(1 + e^(l2 - l1))
// Equal logits give equal values, so that the lower group comes first.
__device__ __forceinline__ float2 sum_rest(float l1, float l2, float f2, float sum, int softmax) {
  float a, b;
  if (softmax || sum < 0.5f || sum >= 1.5f) {
    const float t = log1pf(expf(l2 - l1));
    a = softmax || sum < 0.5f ? l1 : l2;
    b = softmax || sum < 0.5f ? t : -t;
  } else {
    a = f2;
    b = -__fdividef(1.f, 1.f + expf(l1));
  }
  const float hi = a + b, c = hi - a;
  return make_float2(hi, (a - (hi - c)) + (b - c));
}

// V: experts a lane; PART: x holds partial sums of the router product; LOGIT: no
// bias, the logits rank (kernels of their own: with both in one, 16384 positions
// of 256 experts with groups and a bias took 16.4 us instead of 14.6)
template <int V, typename TY, bool PART, bool LOGIT>
__global__ void __launch_bounds__(128, V <= 8 ? 8 : 1) select_kernel(const SelectParams P) {
  extern __shared__ float sm_sel[];  // [warps][E] scores, where groups are not whole warps
  __shared__ __align__(16) uint32_t s_keys[4][32];  // candidates: keys, ids and scores
  __shared__ uint2 s_rest[4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  uint32_t* keys = s_keys[warp];
  uint2* rest = s_rest[warp];
  const int E = P.E;
  const float NONE = -INFINITY;
  pdl_wait();  // (the bias too may come from the kernel before: it is what a balancing step updates)
  pdl_trigger();
  float b[V];
  bool bias_bad = false, bias_odd = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    b[i] = !LOGIT && e < E ? __ldg(P.bias + e) : 0.f;
    bias_bad |= !(b[i] < INFINITY);
    bias_odd |= !(fabsf(b[i]) < INFINITY);
  }
  for (long long t = (long long)blockIdx.x * warps + warp; t < P.T; t += (long long)gridDim.x * warps) {
    float l[V], s[V];
    if (PART) {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = lane + 32 * i < E ? 0.f : NONE;
      const float* p = static_cast<const float*>(P.x) + t * E;
      for (int z = 0; z < P.splits; ++z, p += (long long)P.T * E)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (lane + 32 * i < E) l[i] += __ldcg(p + lane + 32 * i);
    } else {
      const TY* p = static_cast<const TY*>(P.x) + t * P.ldx;
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = lane + 32 * i < E ? to_f32(p[lane + 32 * i]) : NONE;
    }
    // Whether any expert takes no part; looked at one by one only where a logit
    // or bias is not finite (0 * l is NaN then) or registers are left over.
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) z = fmaf(l[i], 0.f, z);
    bool some_none = false;
    if (__any_sync(0xffffffffu, bias_odd || z != z) || E != 32 * V) {
      bool bad = bias_bad, none = E != 32 * V;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (PART) bad |= l[i] == NONE && lane + 32 * i < E;  // (a product that is not finite masks nothing)
        bad |= !(l[i] < INFINITY);
        none |= l[i] == NONE || b[i] == NONE;
      }
      if (__any_sync(0xffffffffu, bad)) {
        if (lane < P.k) {
          P.idx[t * P.k + lane] = -1;
          P.w[t * P.k + lane] = 0.f;
        }
        if (lane == 0 && P.status) atomicOr(P.status, COLI_STATUS_NONFINITE);
        continue;
      }
      some_none = __any_sync(0xffffffffu, none);
    }
    // Where the logits alone rank the experts, scores are needed of the selected
    // only (softmax: also for its sum, which renormalised weights do without).
    const bool late = LOGIT && P.keep == P.G && (!P.softmax || P.renorm);
    float m = NONE, inv = 0.f;  // of a softmax: largest logit, 1 / sum
    if (late) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = l[i];
    } else if (P.softmax) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
      m = warp_max(m);
      if (m == NONE) m = 0.f;  // no expert takes part
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = expf(l[i] - m);
        sum += s[i];
      }
      sum = warp_sum(sum);
      inv = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= inv;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = __fdividef(1.f, 1.f + expf(-l[i]));  // (0 from where the exponential overflows)
    }
    uint32_t key[V];
    auto make_keys = [&]() {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = order_key(LOGIT ? l[i] : s[i] + b[i]);
      if (some_none)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (l[i] == NONE || b[i] == NONE) key[i] = 0u;
    };
    if (P.keep < P.G) {
      float group = NONE, second = NONE;  // lane g: score of group g; without a bias its best logits, for sums two
      const bool sums = LOGIT && P.top2, add = !LOGIT && P.top2;
      const bool whole = P.per % 32 == 0;
      if (whole) {
        make_keys();
        if (P.G == V && P.per == 32) {
          // a group a register: at each exchange a lane keeps half of the groups
          // and takes its neighbour's share of them, then all lanes of one group join
          uint32_t a1[V], a2[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            a1[i] = key[i];
            a2[i] = 0u;
          }
          int o = 1;
#pragma unroll
          for (int n = V / 2; n >= 1; n /= 2, o *= 2) {
            const bool high = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
              const uint32_t r1 = __shfl_xor_sync(0xffffffffu, high ? a1[i] : a1[i + n], o), k1 = high ? a1[i + n] : a1[i];
              const uint32_t r2 = n == V / 2 ? 0u : __shfl_xor_sync(0xffffffffu, high ? a2[i] : a2[i + n], o), k2 = n == V / 2 ? 0u : high ? a2[i + n] : a2[i];
              a1[i] = max(k1, r1);
              a2[i] = max(min(k1, r1), max(k2, r2));
            }
          }
          for (; o < 32; o *= 2) {
            const uint32_t r1 = __shfl_xor_sync(0xffffffffu, a1[0], o), r2 = __shfl_xor_sync(0xffffffffu, a2[0], o);
            a2[0] = max(min(a1[0], r1), max(a2[0], r2));
            a1[0] = max(a1[0], r1);
          }
          // lane g looks at a lane that holds group g (its bits in the other order)
          const int from = V > 1 ? (int)(__brev((uint32_t)lane) >> (32 - (31 - __clz(V)))) : 0;
          const float score = a1[0] == 0u ? NONE : key_value(a1[0]) + (add && a2[0] ? key_value(a2[0]) : 0.f);
          group = __shfl_sync(0xffffffffu, score, from & 31);
          if (lane >= P.G) group = NONE;
          if (sums) second = __shfl_sync(0xffffffffu, a2[0] ? key_value(a2[0]) : NONE, from & 31);
        } else {
          const int span = P.per / 32;
          uint32_t a1 = 0, a2 = 0;  // the group's two best
          int g = 0, in = 0;
  #pragma unroll
          for (int i = 0; i < V; ++i) {
            const uint32_t m1 = __reduce_max_sync(0xffffffffu, key[i]);
            uint32_t m2 = 0;
            if (P.top2) {
              const uint32_t who = __ballot_sync(0xffffffffu, key[i] == m1);
              m2 = __reduce_max_sync(0xffffffffu, lane == __ffs(who) - 1 ? 0u : key[i]);
            }
            a2 = max(max(a2, m2), min(a1, m1));
            a1 = max(a1, m1);
            if (++in == span) {
              if (lane == g) {
                group = a1 == 0 ? NONE : key_value(a1) + (add && a2 ? key_value(a2) : 0.f);
                second = a2 ? key_value(a2) : NONE;
              }
              a1 = a2 = 0;
              in = 0;
              ++g;
            }
          }
        }
      } else {
        float* row = sm_sel + warp * E;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (lane + 32 * i < E) row[lane + 32 * i] = LOGIT || l[i] == NONE ? l[i] : s[i] + b[i];
        __syncwarp();
        if (lane < P.G) {
          for (int j = 0; j < P.per; ++j) {
            const float v = row[lane * P.per + j];
            second = fmaxf(second, fminf(group, v));
            group = fmaxf(group, v);
          }
          group += add && second != NONE ? second : 0.f;
        }
        __syncwarp();
      }
      const float first = group;
      float f2 = 0.f;
      if (sums && first != NONE) {
        auto f = [&](float v) { return P.softmax ? expf(v - m) * inv : __fdividef(1.f, 1.f + expf(-v)); };
        f2 = second == NONE ? 0.f : f(second);
        group = f(first) + f2;
        if (group < 0x1p-100f) group = 0.f;  // (subnormal numbers lose bits: sum_rest has them)
      }
      const uint32_t mk = group == NONE ? 0u : order_key(group);
      int before = 0;
      for (int g = 0; g < P.G; ++g) {
        const uint32_t other = __shfl_sync(0xffffffffu, mk, g);
        before += other > mk || (other == mk && g < lane);
      }
      // (sums have the upper bit of their keys set: no lane's number is one)
      if (sums && __any_sync(0xffffffffu, __popc(__match_any_sync(0xffffffffu, mk ? mk : (uint32_t)lane)) > 1)) {
        const float2 r = mk ? sum_rest(first, second, f2, group, P.softmax) : make_float2(0.f, 0.f);
        before = 0;
        for (int g = 0; g < P.G; ++g) {
          const uint32_t other = __shfl_sync(0xffffffffu, mk, g);
          const float hi = __shfl_sync(0xffffffffu, r.x, g), lo = __shfl_sync(0xffffffffu, r.y, g);
          const bool equal = other == mk && hi == r.x;
          before += other > mk || (other == mk && hi > r.x) || (equal && lo > r.y) || (equal && lo == r.y && g < lane);
        }
      }
      const uint32_t kept = __ballot_sync(0xffffffffu, lane < P.G && before < P.keep);
      if (!whole) make_keys();
      if (whole) {
        int g = 0, in = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (!(kept >> g & 1u)) key[i] = 0u;
          if (++in == P.per / 32) {
            in = 0;
            ++g;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const uint32_t g = ((uint32_t)(lane + 32 * i) * P.gmul) >> 20;
          if (g >= 32 || !(kept >> g & 1u)) key[i] = 0u;
        }
      }
    } else {
      make_keys();
    }
    // The k-th of the lanes' best (or one further down, where some are equal)
    // bounds the k-th best of all from below.  What reaches it goes to shared memory.
    uint32_t top = 0, bound = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, key[i]);
    for (int j = 0; j < P.k; ++j) {
      bound = __reduce_max_sync(0xffffffffu, top);
      top = top == bound ? 0u : top;
    }
    bound = max(bound, 1u);
    int own = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) own += key[i] >= bound;
    int at = own;  // places up to and with this lane's
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += v;
    }
    const int n = __shfl_sync(0xffffffffu, at, 31);
    at -= own;
    keys[lane] = 0u;
    __syncwarp();
    if (n <= 32) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (key[i] >= bound) {
          keys[at] = key[i];
          rest[at] = make_uint2(lane + 32 * i, __float_as_uint(s[i]));
          ++at;
        }
      }
    }
    __syncwarp();
    auto score_of = [&](float logit, float best) { return P.softmax ? expf(logit - best) : __fdividef(1.f, 1.f + expf(-logit)); };
    int my_id = -1, slot = lane;
    float my_w = 0.f, sum = 0.f;
    if (n <= 32) {
      // a lane each: its place is how many come before it
      const uint32_t k0 = keys[lane];
      const uint2 c = lane < n ? rest[lane] : make_uint2(~0u, 0u);
      my_id = (int)c.x;
      my_w = __uint_as_float(c.y);
      if (late) {
        const float best = key_value(__reduce_max_sync(0xffffffffu, k0));
        my_w = lane < n ? score_of(my_w, best) : 0.f;
      }
      int before = 0, same = 0;
      for (int j = 0; j < n; j += 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(keys + j);
        before += (q.x > k0) + (q.y > k0) + (q.z > k0) + (q.w > k0);
        same += (q.x == k0) + (q.y == k0) + (q.z == k0) + (q.w == k0);
      }
      if (__any_sync(0xffffffffu, lane < n && same > 1))  // of equal keys the lower id comes first
        for (int j = 0; j < n; ++j) before += keys[j] == k0 && rest[j].x < c.x;
      if (lane < n) slot = before;
      sum = warp_sum(slot < P.k ? my_w : 0.f);
    } else {
      // many equal ones: round by round the best key and the lowest id that has it
      float most = 0.f;
      for (int j = 0; j < P.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        if (best == 0u) break;  // no more experts take part
        uint32_t id = 0xffffu;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if (key[i] == best) id = lane + 32 * i;
        id = __reduce_min_sync(0xffffffffu, id);
        const int at = id >> 5;
        float sv = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i == at) {
            sv = s[i];
            if (lane == (int)(id & 31u)) key[i] = 0u;
          }
        sv = __shfl_sync(0xffffffffu, sv, id & 31u);
        if (j == 0) most = sv;
        if (late) sv = score_of(sv, most);
        sum += sv;
        if (lane == j) {
          my_id = (int)id;
          my_w = sv;
        }
      }
    }
    __syncwarp();  // (the candidates are read: the next position's may come)
    if (P.renorm) my_w = sum > 0.f ? __fdiv_rn(my_w, sum) : 0.f;
    if (slot < P.k) {
      P.idx[t * P.k + slot] = my_id;
      P.w[t * P.k + slot] = my_w * P.scaling;
    }
  }
}

template <typename TY, bool PART, bool LOGIT>
cudaError_t launch_select_t(const SelectParams& P, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int warps = 4;  // (against one: 600 positions 3.1 us and 3.2, 16384 15.8 and 19.0)
  long long grid = ((long long)P.T + warps - 1) / warps;
  if (grid > 16LL * sms) grid = 16LL * sms;
  const size_t smem = P.keep < P.G && P.per % 32 ? (size_t)warps * P.E * 4 : 0;
  auto go = [&](auto kernel) { return launch_pdl(kernel, (unsigned)grid, 32u * warps, smem, st, P); };
  if (P.E <= 32) return go(select_kernel<1, TY, PART, LOGIT>);
  if (P.E <= 64) return go(select_kernel<2, TY, PART, LOGIT>);
  if (P.E <= 128) return go(select_kernel<4, TY, PART, LOGIT>);
  if (P.E <= 256) return go(select_kernel<8, TY, PART, LOGIT>);
  if (P.E <= 512) return go(select_kernel<16, TY, PART, LOGIT>);
  return go(select_kernel<32, TY, PART, LOGIT>);
}
template <typename TY, bool PART>
cudaError_t launch_select(const SelectParams& P, cudaStream_t st) {
  return P.bias ? launch_select_t<TY, PART, false>(P, st) : launch_select_t<TY, PART, true>(P, st);
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? COLI_OK : COLI_ECUDA; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int SELECT_MAX_T = 65535 * 64;  // positions of a product: the grid's second dimension is tiles of 64

size_t partial_bytes(int T, int H, int E) {
  const size_t splits = T <= ROUTE_GEMV_MAX_T ? (size_t)GEMV_SPLITS : (size_t)route_ksplits(T, H, E);
  return splits * (size_t)T * (size_t)E * 4;
}

}  // namespace
}  // namespace colimoe

using namespace colimoe;

extern "C" size_t coli_moe_select_workspace_size(int32_t max_T, int32_t hidden, int32_t n_experts) {
  if (max_T < 0 || max_T > SELECT_MAX_T || hidden < 1 || hidden % 16 || n_experts < 1 || n_experts > MAX_E) return 0;
  // (fewer positions can take more splits, and then more room in all)
  const size_t few = partial_bytes(max_T < ROUTE_GEMV_MAX_T ? max_T : ROUTE_GEMV_MAX_T, hidden, n_experts);
  size_t most = few;
  // splits fall with the number of 64-row tiles: the largest product is at the end of some tile
  for (long long t = 64; t < (long long)max_T + 64 && most < (size_t)-1; t += 64) {
    const int T = (int)(t < max_T ? t : max_T);
    const size_t n = partial_bytes(T, hidden, n_experts);
    if (n > most) most = n;
    if (route_ksplits(T, hidden, n_experts) == 1) {  // from here on it grows with T
      const size_t last = (size_t)max_T * n_experts * 4;
      if (last > most) most = last;
      break;
    }
  }
  return align_up(WS_HEADER_BYTES + most, 256);
}

extern "C" int coli_moe_select(const coli_moe_select_args* a, int32_t T, cudaStream_t stream) {
  if (!a || T < 0) return COLI_EINVAL;
  if (a->n_experts < 1 || a->n_groups < 1 || a->top_k < 1) return COLI_EINVAL;
  if (a->n_experts > MAX_E || a->n_groups > MAX_GROUPS || a->top_k > MAX_TOPK) return COLI_EUNSUPPORTED;
  if (a->n_experts % a->n_groups || a->topk_group < 1 || a->topk_group > a->n_groups) return COLI_EINVAL;
  if (a->top_k > a->topk_group * (a->n_experts / a->n_groups)) return COLI_EINVAL;
  if ((a->score != COLI_SCORE_SIGMOID && a->score != COLI_SCORE_SOFTMAX) || (a->group_score != COLI_GROUP_TOP2 && a->group_score != COLI_GROUP_MAX))
    return COLI_EINVAL;
  if (!(a->scaling == a->scaling)) return COLI_EINVAL;
  const bool product = a->router_w != nullptr;
  if (product ? a->type != COLI_F32 || a->hidden < 1 || a->hidden % 16 || a->ldx != a->hidden : !float_type(a->type) || a->ldx < a->n_experts)
    return COLI_EINVAL;
  if (product && T > SELECT_MAX_T) return COLI_EUNSUPPORTED;
  if (T == 0) return COLI_OK;
  if (!a->x || !a->topk_idx || !a->topk_w || (product && !a->ws)) return COLI_EINVAL;
  const void* ptrs[] = {a->x, a->router_w, a->bias, a->topk_idx, a->topk_w, a->ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return COLI_EALIGN;
  if (a->ws && a->ws_bytes < 256) return COLI_EWORKSPACE;
  if (product && a->ws_bytes < WS_HEADER_BYTES + partial_bytes(T, a->hidden, a->n_experts)) return COLI_EWORKSPACE;
  SelectParams P{};
  P.x = a->x;
  P.ldx = a->ldx;
  P.bias = a->bias;
  P.T = T;
  P.E = a->n_experts;
  P.G = a->n_groups;
  P.per = a->n_experts / a->n_groups;
  P.keep = a->topk_group;
  P.k = a->top_k;
  P.softmax = a->score == COLI_SCORE_SOFTMAX;
  P.top2 = a->group_score == COLI_GROUP_TOP2;
  P.renorm = a->renorm != 0;
  P.gmul = (1u << 20) / (uint32_t)P.per + 1u;
  P.scaling = a->scaling;
  P.idx = a->topk_idx;
  P.w = a->topk_w;
  P.status = static_cast<uint32_t*>(a->ws);
  if (product) {
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a->ws) + WS_HEADER_BYTES);
    const cudaError_t e = launch_route_partials(static_cast<const float*>(a->x), T, a->hidden, a->router_w, a->n_experts, part, P.status, &P.splits, stream);
    if (e != cudaSuccess) return COLI_ECUDA;
    P.x = part;
    return rc_of(launch_select<float, true>(P, stream));
  }
  if (a->type == COLI_F32) return rc_of(launch_select<float, false>(P, stream));
  if (a->type == COLI_BF16) return rc_of(launch_select<__nv_bfloat16, false>(P, stream));
  return rc_of(launch_select<__half, false>(P, stream));
}
