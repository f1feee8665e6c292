// Products of MX4 rows, grouped by expert, on the block-scaled 4-bit tensor
// core instruction (tcgen05.mma kind::mxf4): the grouped product and the two
// passes of the MX4 expert layer.
//
// Mathematics.  y[p][n] = sum_b 2^(sx[p][b] + sw[n][b] - 254) * sum_{k in b}
// x[p][k] w[n][k] with b the blocks of 32.  The instruction takes 4-bit codes
// of both operands as they are stored, one scale byte per 32 of them and row,
// multiplies K = 64 at a time and accumulates in fp32, so packed rows go from
// global memory to the tensor core without conversion.
//
// Layout.  Weight rows are the M side (128 TMEM lanes), activation rows the N
// side (16 to 128 columns): a weight is read from HBM once per 128 activation
// rows of its expert, and with few rows the kernel is a pure weight stream.
// Gate/up tiles pair 64 gate rows with the same 64 up rows.  K runs in stages
// of 512 (256 bytes of a row: two 128-byte swizzled boxes per operand).
//
// One persistent CTA per SM, thirteen warps:
//   warps 0-3  scales: bytes of the stage's rows by cp.async two stages ahead,
//              then into tensor memory.  Row r of a 128-row tile is lane r % 32,
//              column r / 32 (the four bytes of K / 128 in one 32-bit column),
//              repeated in all four lane quarters, one quarter per warp;
//   warps 4-7  epilogue: accumulators to y, or SwiGLU and MX4 of h;
//   warp 8     MMA issuer;
//   warps 9-12 TMA producers of the codes, one for each 128-byte half of a
//              stage of each operand (one thread issues a box of 8 KB every
//              190 cycles, which alone held a stage back to 1150 cycles).
// Two accumulators, so a tile's epilogue overlaps the next tile's products.
// Every wait is bounded; an expired one sets COLI_STATUS_TIMEOUT and the rest
// of the launch drains.
#include <cstdlib>
#include "mx4_layer.cuh"
#include "tcgen05.cuh"
#include "tensormap.cuh"

namespace colimoe {

constexpr int GM = 128;                  // weight rows of a tile
constexpr int GK = 512;                  // K of a stage
constexpr uint32_t GABYTES = GM * GK / 2;  // 32 KB of weight codes per stage
constexpr int GSR = 4;                   // ring of scale bytes in shared memory (two stages ahead + two)
constexpr int GTHREADS = 416;
constexpr int GW_EPI = 4, GW_MMA = 8, GW_TMA = 9;
constexpr int GEC = 8;                   // columns exchanged at a time between gate and up lanes
constexpr int GMAXENT = MAX_E + MAX_SHARED;
constexpr uint32_t GTMEM = 512;
constexpr int G_MAX_SMEM = 227 * 1024;   // dynamic shared memory of a CTA

struct Mx4Maps {
  CUtensorMap w, w_sh;   // 128 bytes x 128 rows (gate/up: 64) of weight codes (routed or grouped, shared)
  CUtensorMap x[4];      // 128 bytes x 16, 32, 64, 128 rows of activation codes, up to the tile's
};

// tile capacity on the N side and what follows from it
struct Mx4Tile {
  int n;          // activation rows per tile: 16, 32, 64 or 128
  int stages;
};
__host__ __device__ inline uint32_t g_stage(int n) { return GABYTES + (uint32_t)n * (GK / 2); }
__host__ __device__ inline uint32_t g_scale_slot(int n) { return (uint32_t)(GM + (n <= 32 ? 32 : GM)) * (GK / MXB); }
constexpr uint32_t GSCOLS = 32;  // TMEM columns of one stage's scales: 4 x K / 128 x 4 for each operand
struct Mx4Smem {
  uint32_t scales, pre, row0, ent, ex, bars, total;
};
__host__ __device__ inline Mx4Smem g_smem(const Mx4Tile& t) {
  Mx4Smem s;
  uint32_t at = g_stage(t.n) * (uint32_t)t.stages;
  s.scales = at;  at += g_scale_slot(t.n) * GSR;
  s.ex = at;      at += GM * (GEC + 1) * 4;
  s.bars = at;    at += 256;
  s.pre = at;     at += (GMAXENT + 1) * 4;
  s.row0 = at;    at += (GMAXENT + 1) * 4;
  s.ent = at;     at += GMAXENT * 2;
  s.total = at + 1024;  // alignment slack
  return s;
}

// kind::mxf4, E2M1 x E2M1, UE8M0 scales, both K-major, M = 128; the scale data
// ids (which half of the four bytes of a column) are added per instruction
__device__ __forceinline__ uint32_t mx4_idesc(int n) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(GM >> 7) << 27);
}
__device__ __forceinline__ void umma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc) : "memory");
}
__device__ __forceinline__ void tmem_ld8_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
}

// 16 scale bytes of a row from byte `at` on, of which the first `valid` exist
// (the rest become 0, the scale of codes that are 0), to shared memory.
// unit: the alignment that the rows' pitch allows for the copies.
__device__ __forceinline__ void copy_scales(uint8_t* dst, const uint8_t* row, int at, int valid, int unit) {
  if (unit == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(valid > 0 ? row + at : row), "r"(valid > 0 ? 16 : 0) : "memory");
  } else if (unit == 4) {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst + i)), "l"(valid > i ? row + at + i : row), "r"(valid > i ? 4 : 0) : "memory");
  } else {
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < valid) w[i / 4] |= (uint32_t)row[at + i] << (8 * (i % 4));
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// One element of y per lane and column: 16 columns (activation rows) of the
// warp's 32 result rows, consecutive lanes to consecutive elements of y.
template <typename T>
__device__ __forceinline__ void store_cols(T* y, long long ldy, const uint32_t* v, int n) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) y[i * ldy] = from_f32<T>(__uint_as_float(v[i]));
}

template <int MODE>
__global__ void __launch_bounds__(GTHREADS, 1) mx4_gemm(const __grid_constant__ Mx4Maps maps, const Mx4Gemm A, const Mx4Tile T) {
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<size_t>(sm_raw), 1024));
  const Mx4Smem S = g_smem(T);
  const uint32_t STAGE = g_stage(T.n);
  const int NST = T.stages;
  int* s_pre = reinterpret_cast<int*>(sm + S.pre);        // [entries + 1] first item of an entry
  int* s_row0 = reinterpret_cast<int*>(sm + S.row0);      // [entries + 1] first activation row
  uint16_t* s_ent = reinterpret_cast<uint16_t*>(sm + S.ent);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S.bars);  // [NST] codes landed, scales in TMEM
  uint64_t* empty = full + 8;                                 // [NST] the stage's products are done
  uint64_t* acc_full = empty + 8;                             // [2]
  uint64_t* acc_empty = acc_full + 2;                         // [2]
  uint64_t* fin = acc_empty + 2;
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(fin + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_taddr + 1);
  uint32_t* status = reinterpret_cast<uint32_t*>(A.ws);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int RT = MODE == MX4_GATE_UP ? GM / 2 : GM;   // result rows of a tile

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 4 + 4);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(fin, 1);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == GW_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_taddr)), "n"(GTMEM) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  // items: (entry, row tile, tile of activation rows), the last fastest, so
  // that neighbouring items share weight rows, which L2 then serves once
  const int n_ent = mx4_entries<MODE>(A);
  const int n_uniq = MODE == MX4_PRODUCT ? n_ent : __ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.hdr) + MH_NUNIQ);
  for (int u = tid; u <= n_ent; u += GTHREADS) {
    if (MODE == MX4_PRODUCT) {
      s_row0[u] = A.offsets ? min(max(__ldcg(A.offsets + u), 0), A.P) : u * A.P;
    } else {
      s_row0[u] = __ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.ent_offset) + u);
      if (u < n_ent) s_ent[u] = (uint16_t)__ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.ent_expert) + u);
    }
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0, top = 0;
    for (int base = 0; base <= n_ent; base += 32) {
      const int u = base + lane;
      // ascending first rows: the running maximum (the caller's offsets need not be)
      int a = u <= n_ent ? s_row0[u] : 0;
      a = max(a, top);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, a, o);
        if (lane >= o) a = max(a, v);
      }
      top = __shfl_sync(0xffffffffu, a, 31);
      const int next = u + 1 <= n_ent ? max(s_row0[u + 1], a) : a;
      int items = 0;
      if (u < n_ent) {
        const int rows = MODE == MX4_PRODUCT ? A.N : MODE == MX4_DOWN ? A.cfg.hidden : u >= n_uniq ? A.cfg.shared_inter : A.cfg.inter;
        items = ((rows + RT - 1) / RT) * ((next - a + T.n - 1) / T.n);
      }
      int inc = items;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      __syncwarp();
      if (u <= n_ent) {
        s_pre[u] = run + inc - items;
        s_row0[u] = a;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
      __syncwarp();
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t taddr = *s_taddr;
  const uint32_t acc_cols = T.n < 32 ? 32 : T.n;
  const uint32_t sc_col0 = 2 * acc_cols;
  const int n_items = s_pre[n_ent];

  struct Item {
    int row0, ntok;     // activation rows
    int r0, rows;       // first result row of the tile, result rows of the matrix
    int K, nst, shared;
    long long wrow;     // weight row (of pitch K) of result row r0; gate/up: up rows `rows` later
  };
  auto item_at = [&](int item) {
    int lo = 0, hi = n_ent - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pre[mid] <= item) lo = mid; else hi = mid - 1;
    }
    Item it;
    const int cnt = s_row0[lo + 1] - s_row0[lo];
    const int ntn = (cnt + T.n - 1) / T.n;
    const int local = item - s_pre[lo], m = local / ntn, nt = local - m * ntn;
    it.row0 = s_row0[lo] + nt * T.n;
    it.ntok = min(T.n, cnt - nt * T.n);
    it.r0 = m * RT;
    Mx4Entry e;
    if (MODE == MX4_PRODUCT) {
      it.shared = 0;
      it.K = A.K;
      it.rows = A.N;
      e.rec = lo;
    } else {
      it.shared = lo >= n_uniq;
      const int inter = it.shared ? A.cfg.shared_inter : A.cfg.inter;
      it.K = MODE == MX4_GATE_UP ? A.cfg.hidden : inter;
      it.rows = MODE == MX4_GATE_UP ? inter : A.cfg.hidden;
      e.rec = it.shared ? s_ent[lo] - A.cfg.n_experts : ep_local(A.cfg, s_ent[lo]);
    }
    e.rows = it.rows;
    it.wrow = mx4_weight_row<MODE>(e) + it.r0;
    it.nst = (it.K + GK - 1) / GK;
    return it;
  };

  if (warp < GW_EPI) {
    // ---------------------------------------------------------------- scales
    const int unit = A.K % 512 == 0 && A.cfg.hidden % 512 == 0 && A.cfg.inter % 512 == 0 && A.cfg.shared_inter % 512 == 0 ? 16
                     : A.K % 128 == 0 ? 4 : 1;   // (the layer's sizes are multiples of 128; A.K is 0 there)
    const uint32_t slot = g_scale_slot(T.n);
    const bool wide = T.n > 32;
    // copies run ahead of their use, over item boundaries
    int p_item = blockIdx.x, p_st = 0;
    uint32_t pc = 0;
    Item pit;
    if (p_item < n_items) pit = item_at(p_item);
    auto fetch = [&]() {
      if (p_item < n_items) {
        uint8_t* dst = sm + S.scales + (pc % GSR) * slot;
        const int at = p_st * (GK / MXB);
        {
          const int pitch = pit.K / MXB;
          const uint8_t* base = pit.shared ? A.shs : A.wsc;
          // gate/up: threads 64..127 hold the up rows of threads 0..63
          const int r = MODE == MX4_GATE_UP ? tid & 63 : tid;
          const bool live = pit.r0 + r < pit.rows;
          const long long row = pit.wrow + r + (MODE == MX4_GATE_UP && tid >= 64 ? pit.rows : 0);
          copy_scales(dst + tid * 16, live ? base + row * pitch : base, at, live ? pitch - at : 0, unit);
        }
        if (tid < (wide ? GM : 32)) {
          const int pitch = A.xpitch / MXB, len = pit.K / MXB;
          const bool live = tid < pit.ntok;
          copy_scales(dst + (GM + tid) * 16, live ? A.xs + (long long)(pit.row0 + tid) * pitch : A.xs, at, live ? len - at : 0, unit);
        }
        if (++p_st == pit.nst) {
          p_st = 0;
          p_item += gridDim.x;
          if (p_item < n_items) pit = item_at(p_item);
        }
      }
      ++pc;
      cp_async_commit();
    };
    fetch();
    fetch();
    uint32_t gs = 0;
    const uint32_t lane0 = taddr + ((uint32_t)(32 * warp) << 16) + sc_col0;
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
      const int nst = item_at(item).nst;
      for (int st = 0; st < nst; ++st, ++gs) {
        fetch();
        cp_async_wait<2>();
        named_bar(1, 128);  // the stage's bytes are there, and every thread is past the slot before it
        const uint4* src = reinterpret_cast<const uint4*>(sm + S.scales + (gs % GSR) * slot);
        uint32_t a[16], b[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // rows 32 c + lane: word j is K / 128 of the stage
          const uint4 v = src[32 * c + lane];
          a[c] = v.x; a[4 + c] = v.y; a[8 + c] = v.z; a[12 + c] = v.w;
        }
        if (wide) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 v = src[GM + 32 * c + lane];
            b[c] = v.x; b[4 + c] = v.y; b[8 + c] = v.z; b[12 + c] = v.w;
          }
        } else {
          const uint4 v = src[GM + lane];  // at most 32 rows: one column of each four
#pragma unroll
          for (int c = 0; c < 16; ++c) b[c] = 0;
          b[0] = v.x; b[4] = v.y; b[8] = v.z; b[12] = v.w;
        }
        const uint32_t s = gs % NST;
        pf_wait(&empty[s], ((gs / NST) & 1u) ^ 1u, status, s_abort);
        tmem_fence_after();
        __syncwarp();
        tmem_st16(lane0 + s * GSCOLS, a);
        tmem_st16(lane0 + s * GSCOLS + 16, b);
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
    }
    cp_async_wait<0>();
  } else if (warp >= GW_TMA) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producers
      const int h = (warp - GW_TMA) & 1;         // 128-byte half of the stage
      const bool weights = warp - GW_TMA < 2;
      const uint64_t stream = policy_evict_first();
      uint32_t gs = 0;
      bool go = true;
      for (int item = blockIdx.x; item < n_items && go; item += gridDim.x) {
        const Item it = item_at(item);
        const CUtensorMap* wm = it.shared ? &maps.w_sh : &maps.w;
        const int w0 = (int)it.wrow, n16 = (it.ntok + 15) / 16;
        for (int st = 0; st < it.nst; ++st, ++gs) {
          const uint32_t s = gs % NST;
          if (!pf_wait(&empty[s], ((gs / NST) & 1u) ^ 1u, status, s_abort)) { go = false; break; }
          const int x = st * (GK / 2) + h * 128;
          if (x >= it.K / 2) {  // nothing of the row in this half: no products either
            mbar_arrive(&full[s]);
            continue;
          }
          uint8_t* dst = sm + (size_t)s * STAGE;
          if (weights) {
            dst += h * (GABYTES / 2);
            mbar_arrive_expect_tx(&full[s], GABYTES / 2);
            if (MODE == MX4_GATE_UP) {
              tma_load_2d_hint(dst, wm, x, w0, &full[s], stream);
              tma_load_2d_hint(dst + GABYTES / 4, wm, x, w0 + it.rows, &full[s], stream);
            } else if (MODE == MX4_DOWN) {
              tma_load_2d_hint(dst, wm, x, w0, &full[s], stream);
            } else {
              tma_load_2d(dst, wm, x, w0, &full[s]);
            }
          } else {
            dst += GABYTES + h * T.n * 128;
            mbar_arrive_expect_tx(&full[s], (uint32_t)n16 * 2048);
            int row = 0;
#pragma unroll
            for (int i = 3; i >= 0; --i)  // the rows in boxes of 128, 64, 32, 16
              if (n16 >> i & 1) {
                tma_load_2d(dst + row * 128, &maps.x[i], x, it.row0 + row, &full[s]);
                row += 16 << i;
              }
          }
        }
      }
      // every copy issued has landed before the CTA can exit; a stage's phase
      // also needs the other warps, so after an abort this wait is bounded
      for (uint32_t k = gs > (uint32_t)NST ? gs - NST : 0; k < gs; ++k)
        for (uint32_t i = 0; i < SPIN_LIMIT && !mbar_try_wait(&full[k % NST], (k / NST) & 1u); ++i) {
        }
    }
  } else if (warp == GW_MMA) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      uint32_t gs = 0, n = 0;
      for (int item = blockIdx.x; item < n_items; item += gridDim.x, ++n) {
        const Item it = item_at(item);
        const uint32_t idesc = mx4_idesc((it.ntok + 15) & ~15);
        const uint32_t buf = n & 1u, d = taddr + buf * acc_cols;
        bool ok = pf_wait_poll(&acc_empty[buf], ((n >> 1) & 1u) ^ 1u, status, s_abort);
        for (int st = 0; st < it.nst; ++st, ++gs) {
          const uint32_t s = gs % NST;
          ok = ok && pf_wait_poll(&full[s], (gs / NST) & 1u, status, s_abort);
          if (ok) {  // (aborted: the results are flagged invalid; issue nothing)
            tmem_fence_after();
            const uint32_t a0 = smem_u32(sm + (size_t)s * STAGE), b0 = a0 + GABYTES;
            const uint32_t sa = taddr + sc_col0 + s * GSCOLS, sb = sa + 16;
            // kept short: this thread's instructions are on the pipeline's critical path
            const uint64_t da = umma_desc_sw128(a0), db = umma_desc_sw128(b0);
            const uint32_t bh = (uint32_t)T.n * 8;  // second box of B, in descriptor units of 16 bytes
            const int steps = min(GK / 64, (it.K - st * GK + 63) / 64);
            if (steps == GK / 64) {
#pragma unroll
              for (int k = 0; k < GK / 64; ++k)
                umma_mx4(d, da + (k >> 2) * (GABYTES / 32) + (k & 3) * 2, db + (k >> 2) * bh + (k & 3) * 2,
                         idesc | ((k & 1) * ((2u << 4) | (2u << 29))), sa + 4 * (k >> 1), sb + 4 * (k >> 1), k ? 1u : (uint32_t)(st != 0));
            } else {
              for (int k = 0; k < steps; ++k)
                umma_mx4(d, da + (k >> 2) * (GABYTES / 32) + (k & 3) * 2, db + (k >> 2) * bh + (k & 3) * 2,
                         idesc | ((k & 1) * ((2u << 4) | (2u << 29))), sa + 4 * (k >> 1), sb + 4 * (k >> 1), (st | k) != 0);
            }
          }
          umma_commit(&empty[s]);
        }
        umma_commit(&acc_full[buf]);
      }
      // every MMA issued has completed before the accumulators are freed
      umma_commit(fin);
      for (uint32_t i = 0; i < SPIN_LIMIT && !mbar_try_wait(fin, 0u); ++i) {
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp - GW_EPI, r = q * 32 + lane;
    const uint32_t lane0 = taddr + ((uint32_t)(32 * q) << 16);
    uint32_t n = 0;
    for (int item = blockIdx.x; item < n_items; item += gridDim.x, ++n) {
      const Item it = item_at(item);
      const uint32_t buf = n & 1u, d = lane0 + buf * acc_cols;
      pf_wait(&acc_full[buf], (n >> 1) & 1u, status, s_abort);
      tmem_fence_after();
      __syncwarp();
      if (MODE == MX4_GATE_UP) {
        // lanes 0-63 hold gate rows, 64-127 up rows: through shared memory, GEC
        // columns at a time; then warps 0, 1 take the first half of the columns
        // and warps 2, 3 the second, each warp one MX4 block of 32 h rows
        float* ex = reinterpret_cast<float*>(sm + S.ex);
        const int blk = q & 1, c0 = (q >> 1) * (GEC / 2), hr = blk * 32 + lane;
        uint8_t* hq = A.ws + A.L.hq;
        uint8_t* hs = A.ws + A.L.hs;
        for (int c = 0; c < it.ntok; c += GEC) {
          uint32_t v[GEC];
          tmem_ld8_nowait(d + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < GEC; ++i) ex[r * (GEC + 1) + i] = __uint_as_float(v[i]);
          named_bar(2, 128);
#pragma unroll
          for (int i = 0; i < GEC / 2; ++i) {
            const float g = ex[hr * (GEC + 1) + c0 + i], u = ex[(64 + hr) * (GEC + 1) + c0 + i];
            const float h = __fdiv_rn(g, 1.0f + expf(-g)) * u;
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu);
            const uint32_t b = mx4_scale_byte(m);
            const float hv = b == 255u ? 0.f : h * mx4_inv(b);
            const float up = __shfl_down_sync(0xffffffffu, hv, 1);
            if (c + c0 + i < it.ntok) {
              const long long at = (long long)(it.row0 + c + c0 + i) * A.L.imax + it.r0 + blk * 32;
              if ((lane & 1) == 0) hq[at / 2 + lane / 2] = (uint8_t)mx4_pack2(hv, up);
              if (lane == 0) {
                hs[at / MXB] = (uint8_t)b;
                if (b == 255u) atomicOr(status, COLI_STATUS_NONFINITE);
              }
            }
          }
          named_bar(2, 128);
        }
      } else {
        const bool live = it.r0 + r < it.rows;
        for (int c = 0; c < it.ntok; c += 16) {
          uint32_t v[16];
          tmem_ld16_nowait(d + c, v);
          tmem_wait_ld();
          const int nc = live ? it.ntok - c : 0;
          const long long at = (long long)(it.row0 + c) * A.ldy + it.r0 + r;
          if (A.y_type == COLI_F32) store_cols(static_cast<float*>(A.y) + at, A.ldy, v, nc);
          else if (A.y_type == COLI_BF16) store_cols(static_cast<__nv_bfloat16*>(A.y) + at, A.ldy, v, nc);
          else store_cols(static_cast<__half*>(A.y) + at, A.ldy, v, nc);
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == GW_MMA)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(GTMEM) : "memory");
}

// ---------------------------------------------------------------- host
namespace {

bool encode_bytes(CUtensorMap* m, const void* base, size_t row_bytes, size_t rows, uint32_t box_rows) {
  return encode_rows_sw(m, base, row_bytes, rows, 128, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE>
cudaError_t launch_mode(const Mx4Gemm& A, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // most rows an entry can hold
  const int most = MODE == MX4_PRODUCT ? A.P : A.L.T;
  Mx4Tile T;
  const int n_env = getenv("MXN") ? atoi(getenv("MXN")) : 0;
  T.n = most <= 16 ? 16 : most <= 32 ? 32 : most <= 64 ? 64 : 128;
  if (n_env && n_env < T.n) T.n = n_env;
  T.stages = T.n == 128 ? 3 : T.n == 64 ? 4 : 5;
  const Mx4Smem S = g_smem(T);
  if (S.total > (uint32_t)G_MAX_SMEM) return cudaErrorInvalidConfiguration;
  Mx4Maps maps{};
  const coli_moe_cfg& c = A.cfg;
  const size_t pitch = MODE == MX4_PRODUCT ? A.K : MODE == MX4_GATE_UP ? c.hidden : c.inter;
  const size_t rows = MODE == MX4_PRODUCT ? (size_t)A.G * A.N : (size_t)ep_records(c) * 3 * (MODE == MX4_GATE_UP ? c.inter : c.hidden);
  const uint32_t box = MODE == MX4_GATE_UP ? 64 : 128;
  bool ok = encode_bytes(&maps.w, A.wc, pitch / 2, rows, box);
  for (int i = 0; ok && 16 << i <= T.n; ++i) ok = encode_bytes(&maps.x[i], A.xc, A.xpitch / 2, A.P, 16u << i);
  maps.w_sh = maps.w;
  if (ok && MODE != MX4_PRODUCT && c.n_shared > 0)
    ok = encode_bytes(&maps.w_sh, A.shc, (MODE == MX4_GATE_UP ? c.hidden : c.shared_inter) / 2,
                      (size_t)c.n_shared * 3 * (MODE == MX4_GATE_UP ? c.shared_inter : c.hidden), box);
  if (!ok) return cudaErrorInvalidValue;
  // the kernel's shared-memory limit is raised once per device, to the most any tile needs
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(raised.load(std::memory_order_acquire) >> dev & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(mx4_gemm<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, G_MAX_SMEM);
    if (e != cudaSuccess) return e;
    raised.fetch_or(1ull << dev, std::memory_order_release);
  }
  return launch_pdl(mx4_gemm<MODE>, (unsigned)sms, GTHREADS, S.total, st, maps, A, T);
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4Gemm& A, Mx4Mode mode, cudaStream_t st) {
  return mode == MX4_PRODUCT ? launch_mode<MX4_PRODUCT>(A, st) : mode == MX4_GATE_UP ? launch_mode<MX4_GATE_UP>(A, st) : launch_mode<MX4_DOWN>(A, st);
}

}  // namespace colimoe
