// Workspace layout and the parameter block of the MX4 products: what the
// dispatch, product and combine kernels of coli_mx4_forward share.
#pragma once
#include "mx4_common.cuh"

namespace colimoe {

struct Mx4Layout {
  int T, P, n_ent_max, imax;
  size_t hdr, claim, ready, ent_expert, ent_offset, slot, xq, xs, hq, hs, o, total;
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
  L.claim = take(4);                           // next item of the products
  L.ready = take(4 * (size_t)L.n_ent_max);  // gate/up items done per entry; both zeroed by the dispatch
  L.ent_expert = take(4 * (size_t)L.n_ent_max);
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

// One launch of products.
//   product  row p of the activations belongs to group g, rows offsets[g] ..
//            offsets[g + 1] (offsets NULL: one group of all rows); weights
//            [G][N][K]; y = product
//   layer    entries from the workspace tables; gate/up items write h in MX4,
//            down items the per-row outputs o in fp32 (y, ldy = hidden)
struct Mx4Gemm {
  const uint8_t *xc, *xs;    // activation codes [P][xpitch / 2] and scales [P][xpitch / 32]
  const uint8_t *wc, *wsc;   // weights of the groups, or the routed records
  const uint8_t *shc, *shs;  // shared records
  const int32_t* offsets;
  int G, N, K, P, xpitch;
  void* y;
  int32_t y_type;
  long long ldy;
  uint8_t* ws;               // workspace: status word at 0
  Mx4Layout L;
  coli_moe_cfg cfg;
};

cudaError_t launch_mx4_dispatch(const coli_moe_cfg& c, const Mx4Layout& L, const void* x, int32_t x_type, const uint8_t* x_scales,
                                int T, const int32_t* idx, uint8_t* ws, cudaStream_t st);
cudaError_t launch_mx4_product(const Mx4Gemm& A, cudaStream_t st);
cudaError_t launch_mx4_layer(const Mx4Gemm& A, cudaStream_t st);
cudaError_t launch_mx4_combine(const coli_moe_cfg& c, const Mx4Layout& L, const uint8_t* ws, int T, const float* topk_w, void* y,
                               int32_t y_type, cudaStream_t st);

}  // namespace colimoe
