// Workspace layout and the parameter block of the MX4 products: what the
// dispatch, product and combine kernels of coli_mx4_forward share.
#pragma once
#include "mx4_common.cuh"

namespace colimoe {

struct Mx4Layout {
  int T, P, n_ent_max, imax;
  size_t hdr, ent_expert, ent_count, ent_offset, slot, xq, xs, hq, hs, o, total;
};
enum Mx4Hdr { MH_NENT = 0, MH_NUNIQ, MH_NPAIRS, MH_FIELDS = 8 };

// c is normalised: n_shared 0 on shards that own no shared experts
inline Mx4Layout make_mx4_layout(const coli_moe_cfg& c, int T) {
  Mx4Layout L{};
  const size_t k = (size_t)c.top_k, ns = (size_t)c.n_shared, H = (size_t)c.hidden;
  L.T = T;
  const size_t P = (size_t)T * (k + ns);
  L.P = (int)P;
  const size_t routed = (size_t)T * k < (size_t)c.n_experts ? (size_t)T * k : (size_t)c.n_experts;
  L.n_ent_max = (int)(routed + ns);
  L.imax = c.n_shared > 0 && c.shared_inter > c.inter ? c.shared_inter : c.inter;
  size_t off = WS_HEADER_BYTES;  // status and counter words, as in every workspace of this library
  auto take = [&](size_t bytes) { const size_t r = off; off = align_up(off + bytes, 256); return r; };
  L.hdr = take(4 * MH_FIELDS);
  L.ent_expert = take(4 * (size_t)L.n_ent_max);
  L.ent_count = take(4 * (size_t)L.n_ent_max);
  L.ent_offset = take(4 * ((size_t)L.n_ent_max + 1));
  L.slot = take(4 * (size_t)T * k);
  L.xq = take(P * H / 2);
  L.xs = take(P * H / MXB);
  L.hq = take(P * L.imax / 2);
  L.hs = take(P * L.imax / MXB);
  L.o = take(4 * P * H);
  L.total = off;
  return L;
}

enum Mx4Mode { MX4_PRODUCT = 0, MX4_GATE_UP = 1, MX4_DOWN = 2 };

// One launch of grouped products.  Row p of the activations belongs to the
// entry whose range holds p; an entry names the weight matrix.
//   MX4_PRODUCT  entry g = group g, rows offsets[g] .. offsets[g + 1] (offsets
//                NULL: one group of all rows), weights [G][N][K]; y = product
//   MX4_GATE_UP  entries from the workspace tables, records of gate | up | down
//                with row pitch K = H; the result is h = silu(g) * u in MX4
//   MX4_DOWN     the same entries, K = the expert's intermediate size, rows of
//                the record's down part; the result is o in fp32
struct Mx4Gemm {
  const uint8_t *xc, *xs;    // activation codes [P][xpitch / 2] and scales [P][xpitch / 32]
  const uint8_t *wc, *wsc;   // weights of the groups, or the routed records
  const uint8_t *shc, *shs;  // shared records
  const int32_t* offsets;    // MX4_PRODUCT
  int G, N, K, P, xpitch;
  void* y;
  int32_t y_type;
  long long ldy;
  uint8_t* ws;               // workspace: status word at 0
  Mx4Layout L;
  coli_moe_cfg cfg;
};

// what one entry is
struct Mx4Entry {
  int rec;      // group, routed record or shared record
  int shared;
  int row0;     // first activation row
  int count;    // activation rows
  int K;        // reduction length
  int rows;     // weight rows of the result (gate/up: h rows)
};

// Entry u.  Offsets from the caller are clamped to [0, P] and to ascending
// order, so that no value of theirs reaches outside the arrays.
template <int MODE>
__device__ __forceinline__ Mx4Entry mx4_entry(const Mx4Gemm& A, int u) {
  Mx4Entry e;
  if (MODE == MX4_PRODUCT) {
    int a = 0, b = A.P;
    if (A.offsets) {
      a = min(max(__ldcg(A.offsets + u), 0), A.P);
      b = min(max(__ldcg(A.offsets + u + 1), a), A.P);
    }
    e.rec = u;
    e.shared = 0;
    e.row0 = a;
    e.count = b - a;
    e.K = A.K;
    e.rows = A.N;
  } else {
    const int32_t* hdr = reinterpret_cast<const int32_t*>(A.ws + A.L.hdr);
    const int ex = __ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.ent_expert) + u);
    e.shared = u >= __ldcg(hdr + MH_NUNIQ);
    e.rec = e.shared ? ex - A.cfg.n_experts : ep_local(A.cfg, ex);
    e.row0 = __ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.ent_offset) + u);
    e.count = __ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.ent_count) + u);
    const int inter = e.shared ? A.cfg.shared_inter : A.cfg.inter;
    e.K = MODE == MX4_GATE_UP ? A.cfg.hidden : inter;
    e.rows = MODE == MX4_GATE_UP ? inter : A.cfg.hidden;
  }
  return e;
}
template <int MODE>
__device__ __forceinline__ int mx4_entries(const Mx4Gemm& A) {
  return MODE == MX4_PRODUCT ? A.G : __ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.hdr) + MH_NENT);
}
// Row of the weights, counted in rows of pitch e.K, that holds result row 0 of
// entry e (gate/up: the gate rows; the up rows follow e.rows later).  A record
// is gate, up, down: 3 * inter rows of pitch hidden, or 3 * hidden rows of
// pitch inter of which the last third are the down rows.
template <int MODE>
__device__ __forceinline__ long long mx4_weight_row(const Mx4Entry& e) {
  if (MODE == MX4_DOWN) return (long long)e.rec * 3 * e.rows + 2LL * e.rows;
  return (long long)e.rec * (MODE == MX4_GATE_UP ? 3 : 1) * e.rows;
}

__device__ __forceinline__ void store_typed(void* y, int32_t type, long long i, float v) {
  if (type == COLI_F32) static_cast<float*>(y)[i] = v;
  else if (type == COLI_BF16) static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(y)[i] = __float2half_rn(v);
}

cudaError_t launch_mx4_dispatch(const coli_moe_cfg& c, const Mx4Layout& L, const void* x, int32_t x_type, const uint8_t* x_scales,
                                int T, const int32_t* idx, uint8_t* ws, cudaStream_t st);
cudaError_t launch_mx4_gemm(const Mx4Gemm& A, Mx4Mode mode, cudaStream_t st);
cudaError_t launch_mx4_combine(const coli_moe_cfg& c, const Mx4Layout& L, const uint8_t* ws, int T, const float* topk_w, void* y,
                               int32_t y_type, cudaStream_t st);

}  // namespace colimoe
