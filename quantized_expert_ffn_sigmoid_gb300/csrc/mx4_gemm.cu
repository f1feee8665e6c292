// Products of MX4 rows, grouped by expert, on the block-scaled 4-bit tensor
// core instruction (tcgen05.mma kind::mxf4): the grouped product, and both
// passes of the MX4 expert layer in one launch.
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
// Items are (entry, row tile, tile of activation rows), the last fastest, so
// that neighbouring items share weight rows, which L2 then serves once.  The
// layer's items are all gate/up items, then all down items, claimed in order
// from a counter: a CTA that claims a down item knows that every gate/up item
// is claimed by a running CTA, so its wait for the entry's h (a counter per
// entry) ends however many CTAs are resident; meanwhile the down weights
// already stream into the ring.
//
// One persistent CTA per SM, 22 warps meeting at mbarriers:
//   warps 0-3   scales into tensor memory.  Row r of a 128-row tile is lane
//               r % 32, column r / 32 (the four bytes of K / 128 in one 32-bit
//               column), repeated in all four lane quarters, one per warp;
//   warps 4-7 and 18-21  epilogue: accumulators to y, or SwiGLU and MX4 of h.
//               Two sets of four, taking the columns of a tile in turn: with
//               one set a gate/up tile of 64 columns took 18,000 cycles,
//               longer than its products;
//   warp 8      MMA issuer;
//   warps 9-12  TMA producers of the codes, one for each 128-byte half of a
//               stage of each operand (one thread issues a box of 8 KB every
//               190 cycles, which alone held a stage back to 1150 cycles);
//   warp 13     schedule: claims and decodes items ahead of their use;
//   warps 14-17 copy the stage's scale bytes, one row of each operand per
//               thread, with cp.async (16 bytes where the rows allow it) or,
//               for rows that begin anywhere, through registers.
//               Apart from the warps that use them, or a stage takes the sum
//               of both latencies (1650 cycles).
// Two accumulators, so a tile's epilogue overlaps the next tile's products.
//
// Bounds and measurements (GB300; 6.68 TB/s copy and 1920 TFLOP/s bf16
// measured; a range is what several of them gave).  The layer of 256 experts,
// 6144 x 2048, 8 of them and a shared one per position, streams its experts:
// 32 positions 463-487 us, 6.8 to 7.1 TB/s of weights; 4 positions 97-104 us,
// 6.1 to 6.5 TB/s; one position 39-41 us, of which 27
// are the weights' and the rest the dispatch and combine launches, the first
// tile's latency and the end of the down items; 2048 positions 985-1005 us, 779 for
// the weights and 136 for o, which is written and read once.  Products of 8192
// x 4096 x 6144: 102-105 us, 4.0 PFLOP/s; a stage takes 1100 cycles, of which the
// instructions 640, the rest the time until its 68 KB have arrived, which
// three stages do not cover.  4096 rows over 32 groups, 4096 x 6144: 90-92 us,
// 5.3 TB/s.
// Every wait is bounded; an expired one sets COLI_STATUS_TIMEOUT and the rest
// of the launch drains.
#include <algorithm>
#include "mx4_layer.cuh"
#include "tcgen05.cuh"
#include "tensormap.cuh"

namespace colimoe {

constexpr int GM = 128;                  // weight rows of a tile
constexpr int GK = 512;                  // K of a stage
constexpr uint32_t GABYTES = GM * GK / 2;  // 32 KB of weight codes per stage
constexpr int GIR = 4;                   // ring of items
constexpr uint32_t GAHEAD = 3;           // stages left to request when the next item is claimed
constexpr int GTHREADS = 704;
constexpr int GW_EPI = 4, GW_MMA = 8, GW_TMA = 9, GW_SCHED = 13, GW_COPY = 14, GW_EPI2 = 18;
constexpr int GROLES = 21;               // warps that read an item
constexpr int GEC = 8;                   // columns exchanged at a time between gate and up lanes
constexpr uint32_t GSCOLS = 32;          // TMEM columns of one stage's scales: 4 x K / 128 x 4 for each operand
constexpr uint32_t GTMEM = 512;
constexpr int G_MAX_SMEM = 227 * 1024;   // dynamic shared memory of a CTA

template <bool LAYER>
struct Mx4Maps {
  // 128 bytes x 16, 32, 64, 128 rows of activation codes, up to the tile's
  CUtensorMap x[4];
  // 128 bytes x 128 rows of weight codes
  CUtensorMap w[1];
};
template <>
struct Mx4Maps<true> {
  CUtensorMap x[4], h[4];    // h: of the down items
  CUtensorMap w[2], wd[2];   // gate/up (64 rows) and down; [1]: of the shared experts
};

// tile capacity on the N side and what follows from it
struct Mx4Tile {
  int n;          // activation rows per tile: 16, 32, 64 or 128
  int entries;    // most entries of the launch
  int stages;     // as many as fit
};

// one item, as the schedule warp leaves it for the others
struct __align__(16) Mx4Item {
  int row0, ntok;     // activation rows
  int r0, rows;       // first result row of the tile, result rows of the matrix
  int K, nst;         // reduction length, stages (0: no more items)
  int wrow;           // weight row (of pitch K) of result row r0; gate/up: up rows `rows` later
  int shared, down;
  int entry, ready;   // down: entry whose h must be complete, gate/up items that complete it
  int pad;
};

__host__ __device__ inline uint32_t g_stage(int n) { return GABYTES + (uint32_t)n * (GK / 2); }
// scale bytes of a stage: 16 per row, the activation rows up to a multiple of 32
__host__ __device__ inline uint32_t g_scale_slot(int n) { return (uint32_t)(GM + (n <= 32 ? 32 : n)) * (GK / MXB); }
struct Mx4Smem {
  uint32_t scales, ex, bars, items, tiles, row0, ent, total;
};
__host__ __device__ inline Mx4Smem g_smem(const Mx4Tile& t) {
  Mx4Smem s;
  uint32_t at = g_stage(t.n) * (uint32_t)t.stages;
  s.scales = at;  at += g_scale_slot(t.n) * (uint32_t)t.stages;
  s.ex = at;      at += 2 * GM * (GEC + 1) * 4;
  s.bars = at;    at += 320;
  s.items = at;   at += GIR * sizeof(Mx4Item);
  s.tiles = at;   at += (uint32_t)(t.entries + 1) * 4;
  s.row0 = at;    at += (uint32_t)(t.entries + 1) * 4;
  s.ent = at;     at += (uint32_t)t.entries * 2;
  s.total = at + 1024;  // alignment slack
  return s;
}

// kind::mxf4, E2M1 x E2M1, UE8M0 scales, both K-major, M = 128; the scale data
// ids (which half of the four bytes of a column) are added per instruction
__device__ __forceinline__ uint32_t mx4_idesc(int n) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(GM >> 7) << 27);
}
// Issued by the lane whose `leader` is set; executed by a whole converged
// warp, so that the operands stay in uniform registers.
__device__ __forceinline__ void umma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t acc,
                                         uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %6, 0;\n\t"
      "setp.ne.u32 q, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "r"(leader) : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(leader) : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void tmem_ld8_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
}

// 16 scale bytes of a row from byte `at` on, of which the first `valid` exist
// (the rest become 0, the scale of codes that are 0), to shared memory; rows
// of whole 32-bit words, copied as wide as their address allows.
__device__ __forceinline__ void copy_scales(uint8_t* dst, const uint8_t* row, int at, int valid) {
  if (((reinterpret_cast<uintptr_t>(row + at) & 15u) == 0) && (valid >= 16 || valid <= 0)) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(valid > 0 ? row + at : row), "r"(valid > 0 ? 16 : 0) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst + i)), "l"(valid > i ? row + at + i : row), "r"(valid > i ? 4 : 0) : "memory");
  }
}

// The same for rows that begin anywhere (K not a multiple of 128), through
// registers: the aligned words that hold the bytes, put in place by shifts.
// end: of the array, past which no word reaches.
struct ScaleWords {
  uint32_t w[5];
};
__device__ __forceinline__ ScaleWords load_scales(const uint8_t* row, int at, int valid, const uint8_t* end) {
  ScaleWords s;
  const uint8_t* p = row + at;
  const uint32_t a = (uint32_t)reinterpret_cast<uintptr_t>(p) & 3u;
  const uint8_t* q = p - a;  // (not before the array, whose base is aligned)
  if (q + 20 <= end) {  // all but the last bytes of the array (what is beyond `valid` is masked later)
#pragma unroll
    for (int i = 0; i < 5; ++i) s.w[i] = valid > 0 ? __ldg(reinterpret_cast<const uint32_t*>(q) + i) : 0u;
    return s;
  }
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    uint32_t v = 0;
    if (valid > 0 && q + 4 * i < end) {
      v = q[4 * i];
      if (q + 4 * i + 1 < end) v |= (uint32_t)q[4 * i + 1] << 8;
      if (q + 4 * i + 2 < end) v |= (uint32_t)q[4 * i + 2] << 16;
      if (q + 4 * i + 3 < end) v |= (uint32_t)q[4 * i + 3] << 24;
    }
    s.w[i] = v;
  }
  return s;
}
__device__ __forceinline__ void put_scales(uint8_t* dst, const ScaleWords& s, const uint8_t* row, int at, int valid) {
  const uint32_t a = (uint32_t)reinterpret_cast<uintptr_t>(row + at) & 3u;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = valid - 4 * i;  // bytes of this word that exist
    o[i] = __funnelshift_r(s.w[i], s.w[i + 1], 8 * a) & (n >= 4 ? 0xffffffffu : n > 0 ? (1u << (8 * n)) - 1u : 0u);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}

// One element of y per lane and column: 16 columns (activation rows) of the
// warp's 32 result rows, consecutive lanes to consecutive elements of y.
template <typename T>
__device__ __forceinline__ void store_cols(T* y, long long ldy, const uint32_t* v, int n) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) y[i * ldy] = from_f32<T>(__uint_as_float(v[i]));
}

// silu(g) = g / (1 + exp(-g)) in fp32, the quotient taken of operands a
// quarter as large (exact): 1 + exp(-g) passes 2^126, beyond which the fast
// division returns 0, for g < -87.3, while silu(g) is a normal number down to
// -88.7.  expf, not __expf, whose error grows with |g|.  Over every float g
// with |g| < 88.7 the result is within 4.6 units of 2^-24 (g / (1 + expf(-g))
// with an IEEE division: 4.2; fast exponential and division: 66, all of the
// value below -87.3).  It costs the layer what those do (256 experts of 1024 x
// 128 at 128 positions 46.2 us against 46.0, 8 of 1024 x 2048 at 1792 95.6
// against 92.9); the IEEE division, 51.9 and 107.1.
__device__ __forceinline__ float silu(float g) { return __fdividef(0.25f * g, fmaf(0.25f, expf(-g), 0.25f)); }

// GEC columns of a gate/up tile by one set of epilogue warps: lanes 0-63 hold
// gate rows, 64-127 up rows.  Through shared memory warps 0 and 1 take the
// first half of the columns and warps 2 and 3 the second, each warp 32 h rows:
// one MX4 block a column.  r: lane of the tile; n: columns from here on that
// exist; codes, scales: of the block in the first column's h row, the next
// column's `pitch` values further.
__device__ __forceinline__ void swiglu_cols(float* ex, int bar, uint32_t tmem, int r, int n, uint8_t* codes, uint8_t* scales, int pitch,
                                            uint32_t* status) {
  const int lane = r & 31, c0 = (r >> 6) * (GEC / 2), hr = r & 63;
  uint32_t v[GEC];
  tmem_ld8_nowait(tmem, v);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < GEC; ++i) ex[r * (GEC + 1) + i] = __uint_as_float(v[i]);
  named_bar(bar, 128);
  // every value before the first store, or the columns run one after the
  // other (byte stores may alias anything)
  uint32_t code[GEC / 2], byte[GEC / 2];
#pragma unroll
  for (int i = 0; i < GEC / 2; ++i) {
    const float g = ex[hr * (GEC + 1) + c0 + i], u = ex[(64 + hr) * (GEC + 1) + c0 + i];
    const float h = silu(g) * u;
    byte[i] = mx4_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu));
    const float hv = byte[i] == 255u ? 0.f : h * mx4_inv(byte[i]);
    code[i] = mx4_pack2(hv, __shfl_down_sync(0xffffffffu, hv, 1));
  }
  named_bar(bar, 128);  // the exchange space is free
  codes += c0 * (pitch / 2) + lane / 2;
  scales += c0 * (pitch / MXB);
#pragma unroll
  for (int i = 0; i < GEC / 2; ++i) {
    if (c0 + i < n) {
      if ((lane & 1) == 0) codes[i * (pitch / 2)] = (uint8_t)code[i];
      if (lane == 0) {
        scales[i * (pitch / MXB)] = (uint8_t)byte[i];
        if (byte[i] == 255u) atomicOr(status, COLI_STATUS_NONFINITE);
      }
    }
  }
}

// A bounded wait that gives up at once after any wait of the CTA has expired
// (the abort flag), so that a broken pipeline drains.  Without a suspend-time
// hint, with which a thread wakes late, and not polling, which takes issue
// slots from the epilogue: one position took 45.3 us against 47.2 with the
// scale writers and the MMA warp polling.
__device__ __forceinline__ bool gwait(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* abort) {
  for (uint32_t i = 0; i < SPIN_LIMIT; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  atomicOr(status, COLI_STATUS_TIMEOUT);
  return false;
}

// Waits until the entry's gate/up items are complete (bounded, as gwait).
__device__ __forceinline__ void wait_ready(const uint32_t* ready, int target, uint32_t* status, volatile int* abort) {
  for (uint32_t i = 0; i < SPIN_LIMIT; ++i) {
    if (ld_acquire_u32(ready) >= (uint32_t)target) return;
    if (*abort) return;
    __nanosleep(100);
  }
  *abort = 1;
  atomicOr(status, COLI_STATUS_TIMEOUT);
}

// An arrival of this thread at `bar` once all its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Named barrier of `threads` threads that also ANDs a predicate over them.
__device__ __forceinline__ bool named_bar_and(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"((uint32_t)v), "r"(id), "r"(threads) : "memory");
  return r != 0;
}

// LAYER: both passes of the expert layer; otherwise a grouped product
template <bool LAYER>
__global__ void __launch_bounds__(GTHREADS, 1) mx4_gemm(const __grid_constant__ Mx4Maps<LAYER> maps, const Mx4Gemm A, const Mx4Tile T) {
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<size_t>(sm_raw), 1024));
  const Mx4Smem S = g_smem(T);
  const uint32_t STAGE = g_stage(T.n);
  const int NST = T.stages;
  int* s_tiles = reinterpret_cast<int*>(sm + S.tiles);    // [entries + 1] tiles of activation rows before an entry
  int* s_row0 = reinterpret_cast<int*>(sm + S.row0);      // [entries + 1] first activation row
  uint16_t* s_ent = reinterpret_cast<uint16_t*>(sm + S.ent);  // [entries] expert
  Mx4Item* s_items = reinterpret_cast<Mx4Item*>(sm + S.items);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S.bars);  // [NST] codes landed, scales in TMEM
  uint64_t* empty = full + 8;                                 // [NST] the stage's products are done
  uint64_t* sc_full = empty + 8;                              // [NST] scale bytes landed
  uint64_t* item_full = sc_full + 8;                          // [GIR]
  uint64_t* item_empty = item_full + GIR;                     // [GIR]
  uint64_t* acc_full = item_empty + GIR;                      // [2]
  uint64_t* acc_empty = acc_full + 2;                         // [2]
  uint64_t* fin = acc_empty + 2;
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(fin + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_taddr + 1);
  volatile uint32_t* s_issued = reinterpret_cast<volatile uint32_t*>(s_taddr + 2);  // stages whose weights are requested
  uint32_t* status = reinterpret_cast<uint32_t*>(A.ws);
  uint32_t* ready = reinterpret_cast<uint32_t*>(A.ws + A.L.ready);
  uint32_t* claim = reinterpret_cast<uint32_t*>(A.ws + A.L.claim);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 4 + 4);
      mbar_init(&empty[i], 1);
      mbar_init(&sc_full[i], 128);
    }
    for (int i = 0; i < GIR; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], GROLES);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8);
    }
    mbar_init(fin, 1);
    *s_abort = 0;
    *s_issued = 0;
    fence_barrier_init();
  }
  if (warp == GW_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_taddr)), "n"(GTMEM) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  int first = blockIdx.x;
  if (LAYER && warp == GW_SCHED && lane == 0) first = (int)atomicAdd(claim, 1u);  // under way while the tables load
  const int n_ent = LAYER ? __ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.hdr) + MH_NENT) : A.G;
  const int n_uniq = LAYER ? __ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.hdr) + MH_NUNIQ) : n_ent;
  for (int u = tid; u <= T.entries; u += GTHREADS) {  // (beyond n_ent: not looked at)
    if (LAYER) {
      s_row0[u] = __ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.ent_offset) + u);
      if (u < T.entries) s_ent[u] = (uint16_t)__ldcg(reinterpret_cast<const int32_t*>(A.ws + A.L.ent_expert) + u);
    } else {
      s_row0[u] = A.offsets ? min(max(__ldcg(A.offsets + u), 0), A.P) : u * A.P;
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t taddr = *s_taddr;
  const uint32_t acc_cols = T.n < 32 ? 32 : T.n;
  const uint32_t sc_col0 = 2 * acc_cols;

  // The roles' view of the ring of items.  Warps that meet at named barriers
  // agree on its answer first, so that after an expired wait none of them
  // waits at a barrier for one that has given up.
  uint32_t n_item = 0;
  auto next_item = [&](Mx4Item& it) {  // waits for item n_item and reads it; false: no more
    if (!gwait(&item_full[n_item % GIR], (n_item / GIR) & 1u, status, s_abort)) return false;
    it = s_items[n_item % GIR];
    return it.nst > 0;
  };
  auto done_item = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[n_item % GIR]);
    ++n_item;
  };

  if (warp == GW_SCHED) {
    // -------------------------------------------------------------- schedule
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
      const int tiles = (next - a + T.n - 1) / T.n;
      int inc = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      __syncwarp();
      if (u <= n_ent) {
        s_tiles[u] = run + inc - tiles;
        s_row0[u] = a;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
      __syncwarp();
    }
    if (lane == 0) {
      const coli_moe_cfg& c = A.cfg;
      const int all = s_tiles[n_ent], routed = s_tiles[n_uniq];
      const int mt = LAYER ? c.inter / 64 : (A.N + GM - 1) / GM, mts = LAYER ? c.shared_inter / 64 : 0, mtd = LAYER ? c.hidden / GM : 0;
      const int n_gr = mt * routed, n_gu = n_gr + mts * (all - routed);  // gate/up items (or all items of a product)
      const int n_items = n_gu + mtd * all;
      int item = first;
      uint32_t stages = 0;  // of the items posted
      for (uint32_t n = 0;; ++n) {
        Mx4Item it;
        it.nst = 0;
        if (item < n_items) {
          // position among the row tiles x token tiles of its part, then its entry
          it.down = item >= n_gu;
          const bool gs = LAYER && !it.down && item >= n_gr;
          const int m_all = it.down ? mtd : gs ? mts : mt;
          const int local = it.down ? item - n_gu : gs ? item - n_gr : item;
          const int q = local / m_all + (gs ? routed : 0);
          int lo = gs ? n_uniq : 0, hi = n_ent - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_tiles[mid] <= q) lo = mid; else hi = mid - 1;
          }
          const int ntn = s_tiles[lo + 1] - s_tiles[lo];
          const int in = local - (s_tiles[lo] - (gs ? routed : 0)) * m_all, m = in / ntn, nt = in - m * ntn;
          it.row0 = s_row0[lo] + nt * T.n;
          it.ntok = min(T.n, s_row0[lo + 1] - it.row0);
          it.shared = LAYER && lo >= n_uniq;
          if (LAYER) {
            const int inter = it.shared ? c.shared_inter : c.inter;
            const int rec = it.shared ? lo - n_uniq : ep_local(c, s_ent[lo]);
            it.r0 = m * (it.down ? GM : 64);
            it.rows = it.down ? c.hidden : inter;
            it.K = it.down ? inter : c.hidden;
            // a record is gate, up, down: 3 * inter rows of pitch hidden, or 3 * hidden
            // rows of pitch inter of which the last third are the down rows
            it.wrow = rec * 3 * it.rows + (it.down ? 2 * it.rows : 0) + it.r0;
            it.ready = 2 * (inter / 64) * ntn;  // both epilogue sets of every item
          } else {
            it.r0 = m * GM;
            it.rows = A.N;
            it.K = A.K;
            it.wrow = lo * A.N + it.r0;
            it.ready = 0;
          }
          it.entry = lo;
          it.nst = (it.K + GK - 1) / GK;
        }
        if (!gwait(&item_empty[n % GIR], ((n / GIR) & 1u) ^ 1u, status, s_abort)) break;
        s_items[n % GIR] = it;
        mbar_arrive(&item_full[n % GIR]);  // (release)
        if (it.nst == 0) break;
        stages += (uint32_t)it.nst;
        if (LAYER) {
          // the next claim only when the weights of all but GAHEAD posted stages
          // are requested: a CTA that claimed several items at once would hold
          // gate/up items back that others' down items wait for
          for (uint32_t i = 0; i < SPIN_LIMIT && stages > *s_issued + GAHEAD && !*s_abort; ++i) __nanosleep(40);
          item = (int)atomicAdd(claim, 1u);
        } else {
          item += (int)gridDim.x;
        }
      }
    }
  } else if (warp < GW_EPI) {
    // ------------------------------------------------- scales into tensor memory
    const uint32_t slot = g_scale_slot(T.n);
    const int groups = T.n <= 32 ? 1 : T.n / 32;  // 32-row groups of the activations
    const uint32_t lane0 = taddr + ((uint32_t)(32 * warp) << 16) + sc_col0;
    uint32_t gs = 0;
    Mx4Item it;
    while (next_item(it)) {
      for (int st = 0; st < it.nst; ++st, ++gs) {
        const uint32_t s = gs % NST;
        gwait(&sc_full[s], (gs / NST) & 1u, status, s_abort);
        const uint4* src = reinterpret_cast<const uint4*>(sm + S.scales + s * slot);
        uint32_t a[16], b[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // rows 32 c + lane: word j is K / 128 of the stage
          const uint4 v = src[32 * c + lane];
          a[c] = v.x; a[4 + c] = v.y; a[8 + c] = v.z; a[12 + c] = v.w;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 v = c < groups ? src[GM + 32 * c + lane] : make_uint4(0, 0, 0, 0);
          b[c] = v.x; b[4 + c] = v.y; b[8 + c] = v.z; b[12 + c] = v.w;
        }
        // the copies waited for the stage, so its columns are free as well
        tmem_fence_after();
        __syncwarp();
        tmem_st16(lane0 + s * GSCOLS, a);
        tmem_st16(lane0 + s * GSCOLS + 16, b);
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
      done_item();
    }
  } else if (warp >= GW_COPY && warp < GW_EPI2) {
    // ------------------------------------------------------- copies of scale bytes
    const int t = tid - 32 * GW_COPY;
    const uint32_t slot = g_scale_slot(T.n);
    const bool has_row = t < (T.n <= 32 ? 32 : T.n);
    uint32_t gs = 0;
    Mx4Item it;
    while (next_item(it)) {
      const bool gate_up = LAYER && !it.down;
      if (LAYER && it.down) {
        // one lane looks (thousands of threads on one counter hold its additions up)
        if (lane == 0) wait_ready(ready + it.entry, it.ready, status, s_abort);
        __syncwarp();
      }
      const int pitch = it.K / MXB, xpitch = (LAYER && it.down ? A.L.imax : A.xpitch) / MXB;
      // gate/up: threads 64..127 hold the up rows of threads 0..63
      const int r = gate_up ? t & 63 : t;
      const bool wlive = it.r0 + r < it.rows, xlive = t < it.ntok;
      const uint8_t* wp = it.shared ? A.shs : A.wsc;
      if (wlive) wp += ((long long)it.wrow + r + (gate_up && t >= 64 ? it.rows : 0)) * pitch;
      const uint8_t* xp = LAYER && it.down ? A.ws + A.L.hs : A.xs;
      if (xlive) xp += (long long)(it.row0 + t) * xpitch;
      if (!LAYER && (pitch & 3)) {
        // two stages ahead in registers: 2048 x 4096 x 6080 took 81 us with
        // byte loads at their use, 44 this way (K = 6016, whose scale rows
        // are whole words: 37)
        const uint8_t* wend = A.wsc + (long long)A.G * A.N * pitch;
        const uint8_t* xend = A.xs + (long long)A.P * pitch;
        auto wload = [&](int st) { const int at = st * (GK / MXB); return load_scales(wp, at, wlive ? pitch - at : 0, wend); };
        auto xload = [&](int st) { const int at = st * (GK / MXB); return load_scales(xp, at, xlive && has_row ? pitch - at : 0, xend); };
        ScaleWords w0 = wload(0), x0 = xload(0), w1 = wload(1), x1 = xload(1);
        for (int st = 0; st < it.nst; ++st, ++gs) {
          const uint32_t s = gs % NST;
          const ScaleWords w2 = wload(st + 2), x2 = xload(st + 2);
          gwait(&empty[s], ((gs / NST) & 1u) ^ 1u, status, s_abort);
          uint8_t* dst = sm + S.scales + s * slot;
          const int at = st * (GK / MXB);
          put_scales(dst + t * 16, w0, wp, at, wlive ? pitch - at : 0);
          if (has_row) put_scales(dst + (GM + t) * 16, x0, xp, at, xlive ? pitch - at : 0);
          mbar_arrive(&sc_full[s]);
          w0 = w1; w1 = w2;
          x0 = x1; x1 = x2;
        }
        done_item();
        continue;
      }
      for (int st = 0; st < it.nst; ++st, ++gs) {
        const uint32_t s = gs % NST;
        gwait(&empty[s], ((gs / NST) & 1u) ^ 1u, status, s_abort);
        uint8_t* dst = sm + S.scales + s * slot;
        const int at = st * (GK / MXB);
        copy_scales(dst + t * 16, wp, at, wlive ? pitch - at : 0);
        if (has_row) copy_scales(dst + (GM + t) * 16, xp, at, xlive ? pitch - at : 0);
        cp_async_arrive(&sc_full[s]);
      }
      done_item();
    }
    cp_async_wait<0>();
  } else if (warp >= GW_TMA && warp < GW_SCHED) {
    // ------------------------------------------------------------ TMA producers
    const int h = (warp - GW_TMA) & 1;         // 128-byte half of the stage
    const bool weights = warp - GW_TMA < 2;
    const uint64_t stream = policy_evict_first();
    uint32_t gs = 0;
    bool go = true;
    Mx4Item it;
    while (next_item(it)) {
      if (lane == 0 && go) {
        const bool down = LAYER && it.down;
        const CUtensorMap* wm = &maps.w[LAYER ? it.shared : 0];
        if constexpr (LAYER)
          if (down) wm = &maps.wd[it.shared];
        const int n16 = (it.ntok + 15) / 16;
        if (down && !weights) {  // h was written by ordinary stores
          wait_ready(ready + it.entry, it.ready, status, s_abort);
          fence_proxy_async_global();
        }
        for (int st = 0; st < it.nst; ++st, ++gs) {
          const uint32_t s = gs % NST;
          if (!gwait(&empty[s], ((gs / NST) & 1u) ^ 1u, status, s_abort)) { go = false; break; }
          const int x = st * (GK / 2) + h * 128;
          if (x >= it.K / 2) {  // nothing of the row in this half: no products either
            mbar_arrive(&full[s]);
            continue;
          }
          uint8_t* dst = sm + (size_t)s * STAGE;
          if (weights) {
            dst += h * (GABYTES / 2);
            if (h == 0) *s_issued = gs + 1;
            mbar_arrive_expect_tx(&full[s], GABYTES / 2);
            if (!LAYER) {
              tma_load_2d(dst, wm, x, it.wrow, &full[s]);
            } else if (down) {
              tma_load_2d_hint(dst, wm, x, it.wrow, &full[s], stream);
            } else {
              tma_load_2d_hint(dst, wm, x, it.wrow, &full[s], stream);
              tma_load_2d_hint(dst + GABYTES / 4, wm, x, it.wrow + it.rows, &full[s], stream);
            }
          } else {
            const CUtensorMap* xm = maps.x;
            if constexpr (LAYER)
              if (down) xm = maps.h;
            dst += GABYTES + h * T.n * 128;
            mbar_arrive_expect_tx(&full[s], (uint32_t)n16 * 2048);
            int row = 0;
#pragma unroll
            for (int i = 3; i >= 0; --i)  // the rows in boxes of 128, 64, 32, 16
              if (n16 >> i & 1) {
                tma_load_2d(dst + row * 128, xm + i, x, it.row0 + row, &full[s]);
                row += 16 << i;
              }
          }
        }
      }
      done_item();
    }
    // every copy issued has landed before the CTA can exit; a stage's phase
    // also needs the other warps, so after an abort this wait is bounded
    if (lane == 0)
      for (uint32_t k = gs > (uint32_t)NST ? gs - NST : 0; k < gs; ++k)
        for (uint32_t i = 0; i < SPIN_LIMIT && !mbar_try_wait(&full[k % NST], (k / NST) & 1u); ++i) {
        }
  } else if (warp == GW_MMA) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop and one elected lane issues: with the loop
    // in one lane every operand of every instruction went through a register
    // copy of its own, 95 cycles an instruction.
    const uint32_t leader = elect_one();
    const uint32_t bh = (uint32_t)T.n * 8;  // second box of B, in descriptor units of 16 bytes
    uint32_t s = 0, phase = 0;
    Mx4Item it;
    while (next_item(it)) {
      const uint32_t idesc = mx4_idesc((it.ntok + 15) & ~15);
      const uint32_t buf = n_item & 1u, d = taddr + buf * acc_cols;
      bool ok = gwait(&acc_empty[buf], ((n_item >> 1) & 1u) ^ 1u, status, s_abort);
      for (int st = 0; st < it.nst; ++st) {
        ok = ok && gwait(&full[s], phase, status, s_abort);
        if (ok) {  // (aborted: the results are flagged invalid; issue nothing)
          tmem_fence_after();
          const uint32_t a0 = smem_u32(sm) + s * STAGE, b0 = a0 + GABYTES;
          const uint32_t sa = taddr + sc_col0 + s * GSCOLS, sb = sa + 16;
          const uint64_t da = umma_desc_sw128(a0), db = umma_desc_sw128(b0);
          const int steps = min(GK / 64, (it.K - st * GK + 63) / 64);
          if (steps == GK / 64) {
#pragma unroll
            for (int k = 0; k < GK / 64; ++k)
              umma_mx4(d, da + (k >> 2) * (GABYTES / 32) + (k & 3) * 2, db + (k >> 2) * bh + (k & 3) * 2,
                       idesc | ((k & 1) * ((2u << 4) | (2u << 29))), sa + 4 * (k >> 1), sb + 4 * (k >> 1), k ? 1u : (uint32_t)(st != 0), leader);
          } else if (LAYER && steps == GK / 128) {
            // half a stage unrolled too, as in the down items of inter = 256 or
            // the end of 768: this warp's way from one item to the next is what
            // short items take.  256 experts of 2048 x 256 at 64 positions:
            // 76.7 us looping, 69.6 this way; 4096 x 512 (128 experts) 99.7 and
            // 102.9 for the longer code.  Not in the grouped product, whose long
            // reductions would pay for the short: 8192 x 4096 x 6144 101.8 us
            // without and 103.0 with it, 256 groups of 4096 x 256 53.4 and 44.9
#pragma unroll
            for (int k = 0; k < GK / 128; ++k)
              umma_mx4(d, da + (k & 3) * 2, db + (k & 3) * 2,
                       idesc | ((k & 1) * ((2u << 4) | (2u << 29))), sa + 4 * (k >> 1), sb + 4 * (k >> 1), k ? 1u : (uint32_t)(st != 0), leader);
          } else {
            for (int k = 0; k < steps; ++k)
              umma_mx4(d, da + (k >> 2) * (GABYTES / 32) + (k & 3) * 2, db + (k >> 2) * bh + (k & 3) * 2,
                       idesc | ((k & 1) * ((2u << 4) | (2u << 29))), sa + 4 * (k >> 1), sb + 4 * (k >> 1), (st | k) != 0, leader);
          }
        }
        umma_commit_if(&empty[s], leader);
        if (++s == (uint32_t)NST) {
          s = 0;
          phase ^= 1u;
        }
      }
      umma_commit_if(&acc_full[buf], leader);
      done_item();
    }
    // every MMA issued has completed before the accumulators are freed
    umma_commit_if(fin, leader);
    for (uint32_t i = 0; i < SPIN_LIMIT && !mbar_try_wait(fin, 0u); ++i) {
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int set = warp >= GW_EPI2, bar = 2 + set;
    const int q = warp & 3, r = q * 32 + lane;  // lane quarter, lane of the tile
    const uint32_t lane0 = taddr + ((uint32_t)(32 * q) << 16);
    Mx4Item it;
    while (named_bar_and(bar, 128, next_item(it))) {
      const uint32_t buf = n_item & 1u, d = lane0 + buf * acc_cols;
      gwait(&acc_full[buf], (n_item >> 1) & 1u, status, s_abort);
      tmem_fence_after();
      __syncwarp();
      if (LAYER && !it.down) {
        float* ex = reinterpret_cast<float*>(sm + S.ex) + set * GM * (GEC + 1);
        const int pitch = A.L.imax;
        const long long at = (long long)it.row0 * pitch + it.r0 + (q & 1) * 32;
        uint8_t* hq = A.ws + A.L.hq + at / 2;
        uint8_t* hs = A.ws + A.L.hs + at / MXB;
        for (int c = set * GEC; c < it.ntok; c += 2 * GEC)
          swiglu_cols(ex, bar, d + c, r, it.ntok - c, hq + c * (pitch / 2), hs + c * (pitch / MXB), pitch, status);
        named_bar(bar, 128);  // (the down items' producers order h before their TMA reads)
        if (r == 0) red_release_add(ready + it.entry, 1u);
      } else {
        const bool live = it.r0 + r < it.rows;
        for (int c = set * 16; c < it.ntok; c += 32) {
          uint32_t v[16];
          tmem_ld16_nowait(d + c, v);
          tmem_wait_ld();
          const int nc = live ? it.ntok - c : 0;
          const long long at = (long long)(it.row0 + c) * A.ldy + it.r0 + r;
          if (LAYER || A.y_type == COLI_F32) store_cols(static_cast<float*>(A.y) + at, A.ldy, v, nc);
          else if (A.y_type == COLI_BF16) store_cols(static_cast<__nv_bfloat16*>(A.y) + at, A.ldy, v, nc);
          else store_cols(static_cast<__half*>(A.y) + at, A.ldy, v, nc);
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
      done_item();
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

// The tile for at most `most` activation rows per entry: the smallest that
// holds them, up to 128, with as many stages as fit.  Wide tiles read a weight
// once for more rows although entries may hold fewer on average: 2048
// positions over 256 experts (64 rows each) take 990 us with 128, 1143 with
// 64; 4096 rows over 32 groups 90 us with 128, 121 with 64.
Mx4Tile tile_for(int most, int entries) {
  Mx4Tile T;
  T.n = most <= 16 ? 16 : most <= 32 ? 32 : most <= 64 ? 64 : 128;
  T.entries = entries;
  T.stages = 6;
  while (T.stages > 1 && g_smem(T).total > (uint32_t)G_MAX_SMEM) --T.stages;
  return T;
}

template <bool LAYER>
cudaError_t launch(const Mx4Maps<LAYER>& maps, const Mx4Gemm& A, const Mx4Tile& T, long long items, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const Mx4Smem S = g_smem(T);
  if (S.total > (uint32_t)G_MAX_SMEM) return cudaErrorInvalidConfiguration;
  // the kernel's shared-memory limit is raised once per device, to the most any tile needs
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(raised.load(std::memory_order_acquire) >> dev & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(mx4_gemm<LAYER>, cudaFuncAttributeMaxDynamicSharedMemorySize, G_MAX_SMEM);
    if (e != cudaSuccess) return e;
    raised.fetch_or(1ull << dev, std::memory_order_release);
  }
  return launch_pdl(mx4_gemm<LAYER>, (unsigned)(items < sms ? items : sms), GTHREADS, S.total, st, maps, A, T);
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4Gemm& A, cudaStream_t st) {
  const Mx4Tile T = tile_for(A.P, A.G);
  Mx4Maps<false> maps;
  bool ok = encode_bytes(&maps.w[0], A.wc, A.K / 2, (size_t)A.G * A.N, GM);
  for (int i = 0; ok && 16 << i <= T.n; ++i) ok = encode_bytes(&maps.x[i], A.xc, A.xpitch / 2, A.P, 16u << i);
  // (at most: a partial tile per group that can have rows)
  const long long tiles = A.P / T.n + (A.G < A.P ? A.G : A.P);
  return ok ? launch<false>(maps, A, T, tiles * ((A.N + GM - 1) / GM), st) : cudaErrorInvalidValue;
}

cudaError_t launch_mx4_layer(const Mx4Gemm& A, cudaStream_t st) {
  const Mx4Tile T = tile_for(A.L.T, A.L.n_ent_max);  // an expert holds at most every position
  Mx4Maps<true> maps;
  const coli_moe_cfg& c = A.cfg;
  const size_t H = c.hidden, I = c.inter, Is = c.shared_inter, n = (size_t)ep_records(c) * 3, ns = (size_t)c.n_shared * 3;
  bool ok = encode_bytes(&maps.w[0], A.wc, H / 2, n * I, 64) && encode_bytes(&maps.wd[0], A.wc, I / 2, n * H, GM);
  maps.w[1] = maps.w[0];
  maps.wd[1] = maps.wd[0];
  if (ok && ns > 0) ok = encode_bytes(&maps.w[1], A.shc, H / 2, ns * Is, 64) && encode_bytes(&maps.wd[1], A.shc, Is / 2, ns * H, GM);
  for (int i = 0; ok && 16 << i <= T.n; ++i)
    ok = encode_bytes(&maps.x[i], A.xc, H / 2, A.P, 16u << i) && encode_bytes(&maps.h[i], A.ws + A.L.hq, A.L.imax / 2, A.P, 16u << i);
  // A CTA for each item of the larger pass, the most that work at once.  (At
  // most: a partial tile per entry.)  With the down items of one tile per entry
  // instead, 1792 positions over 8 experts of 256 x 2048 took 377 us on 16
  // CTAs, 67 this way; one over 8 of 4096 x 14336 57 on 64 CTAs, 48 this way.
  const long long tiles = A.P / T.n + A.L.n_ent_max;
  const long long rows = std::max<long long>(std::max(c.inter, c.n_shared > 0 ? c.shared_inter : 0) / 64, c.hidden / GM);
  return ok ? launch<true>(maps, A, T, tiles * rows, st) : cudaErrorInvalidValue;
}

}  // namespace colimoe
