// Products of 8-bit codes grouped by expert, on the tensor cores.
//
// Mathematics (i8_product.cu has the whole of it).  This target has no integer
// tensor instruction, but tcgen05.mma kind::f16 adds whole numbers exactly in
// fp32 up to 2^24.  A weight code w becomes the fp16 whose bits are w + 128, a
// subnormal of value (w + 128) 2^-24, for which three integer instructions a
// four codes do; an activation code x becomes the fp16 x.  So tensor memory
// holds 2^-24 sum x (w + 128), exact over any codes whose |x| add up to at most
// 2^24 / 255: over 512 of them always, over all of K for most activations.  Runs
// of such a length are added as 32-bit integers in registers, and 128 sum x, which
// i8_widen has at hand, is taken off at the end.
//
// Operands.  Weights are the M side (128 rows a tile), widened by converter warps
// on their way from shared to tensor memory, where the instruction reads them:
// they are read from HBM as single bytes, once for all activation rows of a tile.
// Activations are the N side, widened once a call in the workspace (i8_widen,
// which also gathers the rows of y and finds the runs' length) and fetched by TMA.
//
// One persistent CTA an SM, 20 warps meeting at mbarriers, every wait bounded
// (after 0.3 s at a barrier it ends, and with it the other waits of both CTAs of a pair):
//   warp 0       TMA of weight codes, slots of 128 rows x 128 codes;
//   warps 1, 3   TMA of activations, slots of up to NT rows x SUB codes;
//   warp 2       MMA issuer, blocks of 256 codes;
//   warps 4-11   converters, two sets of four (a warp for each lane quarter)
//                that take the weight slots in turn;
//   warps 12-19  epilogue: runs into integer registers, at the end the scales and y.
// One barrier says that a block's operands are there, one a slot that its products
// are complete, which frees the activations and the weights' columns alike.
// Tiles of 128 activation rows are taken by two CTAs (cta_group::2): 256 weight
// rows, each CTA with 128 of them and half of the activations, the first issuing for
// both.  Few tiles are split along K (splits_of), and join in the workspace.
//
// What bounds it (GB300; 6.79 TB/s copy, 1924 TFLOP/s bf16 measured; times of whole calls).
//   16384 rows over 160 of 256 groups, 4096 x 6144   860 us, 4.7 TB/s of weights
//   4096 rows over 32 groups, 4096 x 6144            218 us
//       Both: the operands' way from L2 and the MMA warp's from block to block.
//       One CTA for a tile moves 48 KB for 128 codes x 128 rows, which at the 64
//       bytes a cycle of an SM's port take 768 cycles, the instructions 512: 935 and
//       245 us.  Two CTAs move 32 KB each.
//   8192 rows, 4096 x 6144                           280 us, 1.5 PFLOP/s: of these 20 are
//       i8_widen; the others the instructions at the clock (1.45 GHz) that the power
//       limit leaves
//   16 rows, 4096 x 6144                             13 us: two launches, 12 slots a CTA
// Steps that brought most: instructions issued by one lane inside a branch (21
// cycles each, 57 behind a wait in a predicated warp); the next block's barrier
// looked at before a block's last instructions; conversions by integer instructions
// alone; copies of activations by two warps; blocks of 256 codes (from one to the next the
// MMA warp needs about 400 cycles beside its instructions' issue: with 64 codes that
// was all a block's time); tiles of two CTAs.
#include "i8_product.cuh"
#include "tcgen05.cuh"
#include "tensormap.cuh"

namespace colimoe {
namespace {

constexpr int IG_M = 128;                    // weight rows of a tile
constexpr int IG_WK = 128;                   // codes of a weight slot's row
constexpr uint32_t IG_WSLOT = IG_M * IG_WK;  // 16 KB
constexpr int IG_RUN = 512;                  // codes of a run that is exact whatever they are: 512 * 128 * 255 < 2^24
constexpr uint32_t IG_MOST = (1u << 24) / 255;  // sum of an activation row's magnitudes up to which any run is
constexpr int IG_LEVELS = 9;                 // runs of 512 << level codes; the last: all of K
constexpr int IG_MB = 8;                     // weight tiles that share activation tiles while they are in L2
constexpr int IG_THREADS = 640;
constexpr int IG_RCTL = 32, IG_RCONV = 64, IG_REPI = 160;
constexpr int IG_MAX_SMEM = 227 * 1024;
constexpr int IG_MAXW = 9, IG_MAXB = 6;

// NT: activation rows of a tile at most; PAIR: two CTAs take a tile of 256 weight
// rows together, each with 128 of them and half of the activations in its
// shared memory; BK: codes of a block, the unit in which operands pass to the MMA
// warp; SUB: codes of an activation slot, the unit in which space is freed.
// Slots fill 208 KB.
template <int NT>
struct IgShape {
  static constexpr bool PAIR = NT == 128;
  static constexpr int BK = 256, SUB = PAIR ? 128 : 256, SUBS = BK / SUB;
  static constexpr int NW = NT == 32 ? 9 : 7;
  static constexpr int NB = NT == 32 ? 4 : NT == 64 ? 3 : 6;
  static constexpr int NF = PAIR ? 4 : NB;                     // barriers of blocks
  static constexpr int BROWS = PAIR ? NT / 2 : NT;             // activation rows of a slot
  static constexpr uint32_t BSLOT = BROWS * SUB * 2;
  static constexpr uint32_t BARS = NW * IG_WSLOT + NB * BSLOT;
  static constexpr uint32_t TABLES = BARS + 512;
  static constexpr int COLS = NT / 2;                          // columns of an epilogue warp
  // tensor memory: two accumulators, then widened weights for AS activation slots
  static constexpr int AW = SUB / 2, AS = PAIR ? 4 : 2, OF = SUB / IG_WK;  // OF: weight slots to an activation slot
  static_assert(2 * NT <= 256 && AS * AW <= 256 && AS <= NB && AS * SUB >= BK && NB * SUB >= BK && NB < 2 * NF, "tensor memory");
  // A set of converters looks at every other slot, by the parity of its use, so
  // it must not get to a slot before that slot's last use (the other set's, with
  // NW odd) has landed: copies land in any order.  It gets to slot g once the
  // products of slot g - 2 - AS * SUB / 128 are complete.
  static_assert(NW >= AS * OF + 2, "a slot's parity must not be ambiguous");
};
constexpr int IG_ACOL = 256;                 // first column of the widened weights
template <int NT>
constexpr size_t ig_smem(int G) { return IgShape<NT>::TABLES + 8 * (size_t)(G + 1) + 1024; }

static_assert(ig_smem<32>(COLI_I8_MAX_GROUPS) <= IG_MAX_SMEM && ig_smem<64>(COLI_I8_MAX_GROUPS) <= IG_MAX_SMEM &&
              ig_smem<128>(COLI_I8_MAX_GROUPS) <= IG_MAX_SMEM, "shared memory");

struct IgMaps {
  CUtensorMap w;     // weight codes [G][N][K]
  CUtensorMap x[3];  // widened activations, boxes of 64 codes x 16, 32, 64 rows
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;"
      ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// 8 codes (two words) -> 8 fp16 of value (code + 128) 2^-24: the subnormal whose
// bits are the code with its sign bit flipped.  Integer instructions alone:
// with fp16 subtractions among them (which make the plain code) these warps take
// every issue slot, and the MMA warp beside them 780 cycles a block instead of 510.
__device__ __forceinline__ void biased8(uint32_t w0, uint32_t w1, uint32_t* o) {
  const uint32_t x0 = w0 ^ 0x80808080u, x1 = w1 ^ 0x80808080u;
  o[0] = prmt(x0, 0u, 0x4140u);
  o[1] = prmt(x0, 0u, 0x4342u);
  o[2] = prmt(x1, 0u, 0x4140u);
  o[3] = prmt(x1, 0u, 0x4342u);
}
// D[tmem] (+)= A[tmem] x B[smem]; PAIR: by both CTAs of a pair, each on its own
// 128 rows of A and D, with its half of B
template <bool PAIR>
__device__ __forceinline__ void umma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// An arrival at `bar` once the products issued so far are complete; PAIR: at
// that barrier of both CTAs
template <bool PAIR>
__device__ __forceinline__ void commit_to(uint64_t* bar) {
  if (PAIR)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
  else
    umma_commit(bar);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// An arrival at the barrier of the pair's first CTA that stands where `bar` does
// in this one.  It announces this CTA's stores to tensor memory, which the tcgen05
// fences before it and behind the other CTA's wait order, and shared memory filled by
// asynchronous copies, whose completion has been seen here before; both are read by
// the pair's instructions alone.  No ordinary store has to be seen by the other CTA, so
// the arrival names no scope: for the copies that rests on their completion, where the
// memory model would ask for a release to the cluster and a wait that acquires from
// it; the release took 2000 cycles a block.
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(bar)));
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
}

struct IgItem {
  int g, row0, ntok, n0;
};

template <int NT>
__global__ void __launch_bounds__(IG_THREADS, 1) i8_gemm(const __grid_constant__ IgMaps maps, const I8Params A, const uint32_t off_xs, const int wide,
                                                           const int n_splits, uint32_t* __restrict__ part) {
  using S = IgShape<NT>;
  constexpr bool PAIR = S::PAIR;
  constexpr int NW = S::NW, NB = S::NB, NF = S::NF, BK = S::BK, SUB = S::SUB, SUBS = S::SUBS;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<size_t>(sm_raw), 1024));
  uint8_t* sm_b = sm + NW * IG_WSLOT;
  uint64_t* full_w = reinterpret_cast<uint64_t*>(sm + S::BARS);  // [NW] weight codes landed
  uint64_t* empty_w = full_w + IG_MAXW;                          // [NW] the converters have read them
  uint64_t* full = empty_w + IG_MAXW;                            // [NF] a block: activations landed, weights in tensor memory
  uint64_t* done = full + IG_MAXB;                               // [NB] an activation slot's products are complete
  uint64_t* d_full = done + IG_MAXB;                             // [2] a run is complete
  uint64_t* d_empty = d_full + 2;                                // [2] it has been read
  uint64_t* full2 = d_empty + 2;                                 // [NF] PAIR, in the first CTA: the other one's operands are there
  uint64_t* fin = full2 + IG_MAXB;
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(fin + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_taddr + 1);
  uint32_t* s_level = s_taddr + 2;
  uint32_t* s_parts = s_taddr + 3;
  int* s_row0 = reinterpret_cast<int*>(sm + S::TABLES);          // [G + 1] first row of a group
  int* s_tiles = s_row0 + A.G + 1;                               // [G + 1] activation tiles before it
  uint32_t* status = reinterpret_cast<uint32_t*>(A.ws);
  // (broadcast, so that the compiler knows them to be the same in every lane of a warp)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // With splits, this CTA takes one part of K of one tile (the grid holds all parts of all tiles)
  const int splits = PAIR ? 1 : n_splits;
  const int kall = (A.K + BK - 1) / BK, kpart = (kall + splits - 1) / splits;
  const int k0 = splits > 1 ? (int)blockIdx.x % splits * kpart : 0, ksteps = splits > 1 ? min(kpart, kall - k0) : kall;
  const int nblk = ksteps, nw = nblk * (BK / IG_WK);
  constexpr int MROWS = PAIR ? 2 * IG_M : IG_M;  // weight rows of an item
  const int rank = PAIR ? (int)blockIdx.x & 1 : 0, mt = (A.N + MROWS - 1) / MROWS;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NW; ++i) {
      mbar_init(&full_w[i], 1);
      mbar_init(&empty_w[i], 4);
    }
    for (int i = 0; i < NF; ++i) {
      mbar_init(&full[i], 2 * SUBS + 4 * (BK / IG_WK));
      mbar_init(&full2[i], 1);
    }
    for (int i = 0; i < NB; ++i) mbar_init(&done[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], PAIR ? 16 : 8);
    }
    mbar_init(fin, 1);
    *s_abort = 0;
    *s_level = IG_LEVELS - 1;
    fence_barrier_init();
  }
  if (warp == 2) {
    if (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_taddr)), "n"(512) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_taddr)), "n"(512) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 3) {
    // first rows and tiles of the groups, in ascending order
    int run = 0, top = 0;
    for (int base = 0; base <= A.G; base += 32) {
      const int u = base + lane;
      int a = u <= A.G ? i8_offset(A, u) : 0, b = u < A.G ? i8_offset(A, u + 1) : 0;
      a = max(a, top);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, a, o);
        if (lane >= o) a = max(a, v);
      }
      top = __shfl_sync(0xffffffffu, a, 31);
      const int tiles = u < A.G ? (max(a, b) - a + NT - 1) / NT : 0;
      int inc = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (u <= A.G) {
        s_row0[u] = a;
        s_tiles[u] = run + inc - tiles;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  {
    // the longest runs that are exact for every activation row (a level from each CTA of i8_widen)
    const uint32_t* level = reinterpret_cast<const uint32_t*>(A.ws + WS_HEADER_BYTES);
    uint32_t m = IG_LEVELS - 1;
    for (int i = threadIdx.x; i < wide; i += IG_THREADS) m = min(m, __ldcg(level + i));
    m = __reduce_min_sync(0xffffffffu, m);
    __syncthreads();  // (s_level is set)
    if (lane == 0) atomicMin(s_level, m);
  }
  tmem_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // (the other CTA's barriers are there)
  tmem_fence_after();
  const int run = *s_level < IG_LEVELS - 1 ? IG_RUN << *s_level : 1 << 30;
  // (runs end at multiples of their length from the row's beginning)
  const int kbegin = k0 * BK % run;
  const uint32_t taddr = __shfl_sync(0xffffffffu, *s_taddr, 0);
  const int items = __shfl_sync(0xffffffffu, s_tiles[A.G] * mt, 0);
  const int first = (int)blockIdx.x / (PAIR ? 2 : splits);  // (splits > 1: the only item)
  const int step = splits > 1 ? 1 << 30 : (int)gridDim.x / (PAIR ? 2 : 1);

  // Items of a group: IG_MB weight tiles for each activation tile, so that the
  // CTAs at work together share both operands in L2.
  auto item_at = [&](int item) {
    const int q = item / mt;
    int lo = 0, hi = A.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_tiles[mid] <= q) lo = mid; else hi = mid - 1;
    }
    const int t0 = s_tiles[lo], ntn = s_tiles[lo + 1] - t0, local = item - t0 * mt;
    constexpr int MB = IG_MB / (PAIR ? 2 : 1);
    const int mb = local / (MB * ntn), in = local - mb * MB * ntn, width = min(MB, mt - mb * MB);
    const int nt = in / width;
    IgItem it;
    it.g = lo;
    it.row0 = s_row0[lo] + nt * NT;
    it.ntok = min(NT, s_row0[lo + 1] - it.row0);
    it.n0 = (mb * MB + in - nt * width) * MROWS + rank * IG_M;
    return it;
  };

  if (warp < 4) {
    setmaxnreg_dec<IG_RCTL>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- TMA of weights
      const uint64_t stream = policy_evict_first();
      uint32_t gs = 0;
      bool go = true;
      for (int item = first; item < items && go; item += step) {
        const IgItem it = item_at(item);
        const bool once = A.wgroup && s_tiles[it.g + 1] - s_tiles[it.g] == 1;  // read for one activation tile alone
        const int z = A.wgroup ? it.g : 0;  // (one matrix for all groups)
        for (int st = 0; st < nw; ++st, ++gs) {
          const uint32_t s = gs % NW;
          if (!gwait(&empty_w[s], ((gs / NW) & 1u) ^ 1u, status, s_abort)) { go = false; break; }
          mbar_arrive_expect_tx(&full_w[s], IG_WSLOT);
          if (once) tma_load_3d_hint(sm + s * IG_WSLOT, &maps.w, k0 * BK + st * IG_WK, it.n0, z, &full_w[s], stream);
          else tma_load_3d(sm + s * IG_WSLOT, &maps.w, k0 * BK + st * IG_WK, it.n0, z, &full_w[s]);
        }
      }
      // every copy issued has landed before the CTA can exit (after an abort a
      // phase may lack the other warps' arrivals: the wait is bounded)
      uint32_t tries = SPIN_LIMIT;
      for (uint32_t k = gs > (uint32_t)NW ? gs - NW : 0; k < gs; ++k) drain_wait(&full_w[k % NW], (k / NW) & 1u, tries);
    } else if ((warp == 1 || warp == 3) && lane == 0) {
      // ------------------------------------------------ TMA of activations
      // Each warp takes half of a slot, every other 64 codes (one thread issues
      // 16 KB every 380 cycles).
      fence_proxy_async_global();  // (the widened rows were written by ordinary stores of the kernel before)
      const int half = warp >> 1;
      uint32_t gs = 0;
      bool go = true;
      for (int item = first; item < items && go; item += step) {
        const IgItem it = item_at(item);
        // PAIR: the tile's rows up to a multiple of 32, half of them in each CTA
        const int n16 = PAIR ? (it.ntok + 31) / 32 : (it.ntok + 15) / 16, row0 = it.row0 + rank * 16 * n16;
        for (int j = 0; j < nblk * SUBS; ++j, ++gs) {
          const uint32_t s = gs % NB;
          uint64_t* bar = &full[gs / SUBS % NF];
          if (!gwait(&done[s], ((gs / NB) & 1u) ^ 1u, status, s_abort)) { go = false; break; }
          mbar_arrive_expect_tx(bar, (uint32_t)n16 * 2048 * (SUB / 128));
          int row = 0;
          for (int left = n16; left > 0;) {  // the rows in boxes of 64, 32, 16
            const int i = left >= 4 ? 2 : left >= 2 ? 1 : 0;
#pragma unroll
            for (int c = half; c < SUB / 64; c += 2)
              tma_load_2d(sm_b + s * S::BSLOT + c * (S::BROWS * 128) + row * 128, &maps.x[i], k0 * BK + j * SUB + 64 * c, row0 + row, bar);
            row += 16 << i;
            left -= 1 << i;
          }
        }
      }
      // (the last copies are of the last blocks whose operands were asked for)
      const uint32_t blocks = (gs + SUBS - 1) / SUBS;
      uint32_t tries = SPIN_LIMIT;
      for (uint32_t k = blocks > (uint32_t)NF ? blocks - NF : 0; k < blocks; ++k) drain_wait(&full[k % NF], (k / NF) & 1u, tries);
    } else if (warp == 2 && PAIR && rank == 1) {
      // ------------------- second CTA: tells the first that a block is there
      // (after an abort the lanes go on to the end: they meet here, and may learn of
      // it at different blocks)
      uint32_t gs = 0;
      for (int item = first; item < items; item += step)
        for (int j = 0; j < nblk; ++j, ++gs) {
          const bool there = gwait(&full[gs % NF], (gs / NF) & 1u, status, s_abort);
          tmem_fence_after();
          tmem_fence_before();
          __syncwarp();
          if (lane == 0 && there) arrive_first(&full2[gs % NF]);
        }
      // the first CTA's last arrivals here
      if (!*s_abort) {
        const uint32_t subs = gs * SUBS;
        uint32_t tries = SPIN_LIMIT;
        for (uint32_t k = subs > (uint32_t)NB ? subs - NB : 0; k < subs; ++k) drain_wait(&done[k % NB], (k / NB) & 1u, tries);
      }
    } else if (warp == 2) {
      // -------------------------------------------------------- MMA issuer
      // (one elected lane issues a block's instructions inside a branch: 21
      // cycles an instruction; issued by a predicated lane of the whole warp
      // behind a wait they took 57, with operands copied one by one.  A block
      // waits at one barrier, looked at while the block before is under way)
      const uint32_t leader = elect_one();
      const uint64_t db0 = umma_desc_sw128(smem_u32(sm_b));
      constexpr int TAIL = 2;
      uint32_t s = 0, f = 0, ph = 0, a = 0, d = 0, dph = 1;
      bool ready = false, ok = true;
      for (int item = first; item < items; item += step) {
        const int ntok = item_at(item).ntok;
        const uint32_t idesc = PAIR ? umma_idesc((ntok + 31) & ~31) + ((uint32_t)(IG_M >> 4) << 24) : umma_idesc((ntok + 15) & ~15);  // (PAIR: M = 256)
        uint32_t acc = 0;          // whether the run has begun
        int left = (run - kbegin) / BK;  // blocks to its end
        for (int j = nblk; j > 0; --j) {
          if (acc == 0) ok = gwait(&d_empty[d], dph, status, s_abort) && ok;
          if (!ready) {
            ok = gwait(&full[f], ph, status, s_abort) && ok;
            if (PAIR) ok = gwait(&full2[f], ph, status, s_abort) && ok;
          }
          const bool end = --left == 0 || j == 1;
          const uint32_t dc = taddr + d * NT;
          // instructions of the block's activation slots, and each slot's barrier behind its last
          auto issue = [&](int from, int to) {
#pragma unroll
            for (int k = from; k < to; ++k) {
              constexpr int EACH = SUB / 16;
              const int sub = k / EACH, in = k % EACH;
              const uint32_t at = s + sub < (uint32_t)NB ? s + sub : s + sub - NB, col = a + sub < (uint32_t)S::AS ? a + sub : a + sub - S::AS;
              if (ok)  // (aborted: the results are flagged invalid; nothing is issued)
                umma_f16<PAIR>(dc, taddr + IG_ACOL + col * S::AW + 8 * in, db0 + at * (S::BSLOT >> 4) + (in >> 2) * (S::BROWS * 128 / 16) + 2 * (in & 3), idesc,
                         k ? 1u : acc);
              if (in == EACH - 1) commit_to<PAIR>(&done[at]);
            }
          };
          tmem_fence_after();
          __syncwarp();
          if (leader) issue(0, BK / 16 - TAIL);
          // behind the last TAIL instructions, which are still under way then,
          // the next block follows without a gap
          if (++f == (uint32_t)NF) {
            f = 0;
            ph ^= 1u;
          }
          ready = mbar_test_wait(&full[f], ph);
          if (PAIR) ready = mbar_test_wait(&full2[f], ph) && ready;
          if (leader) {
            issue(BK / 16 - TAIL, BK / 16);
            if (end) commit_to<PAIR>(&d_full[d]);
          }
          __syncwarp();
          s += SUBS;
          if (s >= (uint32_t)NB) s -= NB;
          a += SUBS;
          if (a >= (uint32_t)S::AS) a -= S::AS;
          acc = 1;
          if (end) {
            acc = 0;
            left = run / BK;
            if (++d == 2u) {
              d = 0;
              dph ^= 1u;
            }
          }
        }
      }
      // every MMA issued has completed before the accumulators are freed
      if (leader) {
        if (PAIR) asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(fin)) : "memory");
        else umma_commit(fin);
      }
      __syncwarp();
      uint32_t tries = SPIN_LIMIT;
      drain_wait(fin, 0u, tries);
    }
  } else if (warp < 12) {
    setmaxnreg_dec<IG_RCONV>();
    // ---------------------------------------------------------- converters
    // One after the other the CTA's blocks of 128 rows x 128 codes, the sets in
    // turn: a row a lane, all its loads before the first conversion.
    const int set = (warp - 4) >> 2, q = warp & 3, r = 32 * q + lane;
    const uint32_t total = (uint32_t)(items > first ? (items - first - 1) / step + 1 : 0) * (uint32_t)nw;
    const uint32_t src = smem_u32(sm) + r * IG_WK, sw = (r & 7) * 16;  // 16-byte unit c of row r is at unit c ^ (r % 8)
    const uint32_t dst = taddr + ((uint32_t)(32 * q) << 16) + IG_ACOL;
    constexpr int OF = S::OF;
    uint32_t s = set, sph = 0;
    for (uint32_t g = set; g < total; g += 2) {
      gwait(&full_w[s], sph, status, s_abort);
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = lds128(src + s * IG_WSLOT + ((16 * i) ^ sw));
      // what held these columns is done (that phase cannot have been overtaken:
      // the next in its slot needs these weights first)
      const uint32_t b = g / OF;
      if (b >= (uint32_t)S::AS) {
        const uint32_t before = b - S::AS;
        gwait(&done[before % NB], (before / NB) & 1u, status, s_abort);
      }
      tmem_fence_after();
      __syncwarp();
      const uint32_t at = dst + (b % S::AS) * S::AW + (OF > 1 ? g % OF * (IG_WK / 2) : 0);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t o[16];
        biased8(w[2 * h].x, w[2 * h].y, o);
        biased8(w[2 * h].z, w[2 * h].w, o + 4);
        biased8(w[2 * h + 1].x, w[2 * h + 1].y, o + 8);
        biased8(w[2 * h + 1].z, w[2 * h + 1].w, o + 12);
        tmem_st16(at + 16 * h, o);
      }
      if (lane == 0) mbar_arrive(&empty_w[s]);  // (every lane's loads are complete: its stores used them)
      tmem_wait_st();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[g / (BK / IG_WK) % NF]);
      s += 2;
      if (s >= (uint32_t)NW) {
        s -= NW;
        sph ^= 1u;
      }
    }
  } else {
    setmaxnreg_inc<IG_REPI>();
    // ------------------------------------------------------------ epilogue
    constexpr int COLS = S::COLS;
    const int set = (warp - 12) >> 2, q = warp & 3, col0 = set * COLS;
    const float* xs = reinterpret_cast<const float*>(A.ws + off_xs);
    const uint32_t* xsum = reinterpret_cast<const uint32_t*>(xs) + A.P;
    uint32_t d = 0, dph = 0;
    for (int item = first; item < items; item += step) {
      const IgItem it = item_at(item);
      const int cols = min(max(it.ntok - col0, 0), COLS);
      const int n = it.n0 + 32 * q + lane;
      const bool live = n < A.N;
      const float sw = live ? __ldg(A.ws_ + it.g * A.wsgroup + n) : 0.f;
      // scales and sums of the tile's rows, loaded ahead of the sums: lane l has columns l, l + 32
      constexpr int HELD = (COLS + 31) / 32;
      float sx_[HELD];
      uint32_t bias_[HELD];
#pragma unroll
      for (int h = 0; h < HELD; ++h) {
        const int c = 32 * h + lane;
        sx_[h] = c < cols ? __ldcg(xs + it.row0 + col0 + c) : 0.f;
        bias_[h] = c < cols ? __ldcg(xsum + it.row0 + col0 + c) : 0u;
      }
      uint32_t acc[COLS];  // (modulo 2^32, in which the end result fits)
#pragma unroll
      for (int i = 0; i < COLS; ++i) acc[i] = 0;
      for (int c = -kbegin; c < nblk * BK; c += run) {
        pf_wait(&d_full[d], dph, status, s_abort);  // (long: suspended, out of the other warps' way)
        tmem_fence_after();
        __syncwarp();
        const uint32_t t = taddr + ((uint32_t)(32 * q) << 16) + d * NT + col0;
#pragma unroll
        for (int i = 0; i < COLS; i += 16)
          if (i < cols) {
            uint32_t v[16];
            tmem_ld16_nowait(t + i, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[i + k] += (uint32_t)__float2int_rn(__uint_as_float(v[k]) * 16777216.f);
          }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR && rank == 1) arrive_first(&d_empty[d]);
          else mbar_arrive(&d_empty[d]);
        }
        if (++d == 2u) {
          d = 0;
          dph ^= 1u;
        }
        if (run == 1 << 30) break;  // (no overflow of c)
      }
      if (splits > 1) {
        // the parts of a tile are added up in global memory (zeroed by i8_widen):
        // whole numbers, so their order is free; the last part goes on to y
        uint32_t* tile = part + (size_t)item * (NT * IG_M) + col0 * IG_M + 32 * q + lane;
#pragma unroll
        for (int c = 0; c < COLS; c += 16)  // (whole sixteens of columns, also behind the last)
          if (c < cols) {
#pragma unroll
            for (int i = 0; i < 16; ++i) atomicAdd(tile + (c + i) * IG_M, acc[c + i]);
          }
        __threadfence();
        named_bar(2, 256);
        if (warp == 12 && lane == 0) *s_parts = atomicAdd(reinterpret_cast<uint32_t*>(A.ws + I8_OFF_PARTS) + item, 1u);
        named_bar(2, 256);
        if (*s_parts != (uint32_t)splits - 1) break;
        __threadfence();
#pragma unroll
        for (int c = 0; c < COLS; c += 16)
          if (c < cols) {
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c + i] = __ldcg(tile + (c + i) * IG_M);
          }
      }
      const long long at = (long long)(it.row0 + col0) * A.ldy + n;
      auto store = [&](auto* y) {
        using TY = std::remove_pointer_t<decltype(y)>;
        y += at;
#pragma unroll
        for (int c = 0; c < COLS; c += 16)
          if (c < cols) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int from = c % 32 + i;
              const float v = i8_value((int)(acc[c + i] - __shfl_sync(0xffffffffu, bias_[c / 32], from)), __shfl_sync(0xffffffffu, sx_[c / 32], from), sw);
              if (live && c + i < cols) y[(c + i) * A.ldy] = from_f32<TY>(v);
            }
          }
      };
      if (A.y_type == COLI_F32) store(static_cast<float*>(A.y));
      else if (A.y_type == COLI_BF16) store(static_cast<__nv_bfloat16*>(A.y));
      else store(static_cast<__half*>(A.y));
    }
  }
  // A wait that has run out ends the other CTA's waits too (a warp gets here soon
  // after: waits fail at once then, and the results are flagged invalid)
  if (PAIR && lane == 0 && *s_abort) abort_other(s_abort);
  tmem_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // (neither CTA ends while the other may arrive at its barriers)
  if (warp == 2) {
    if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(512) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(512) : "memory");
  }
}

// sum + the magnitudes of four codes: with m = -1 in the bytes of negative
// codes, |c| = (c ^ m) + 1 there
__device__ __forceinline__ int magnitudes(uint32_t w, int sum) {
  const uint32_t m = prmt(w, 0u, 0xba98u);  // the bytes' signs
  return dp4a_ss(w ^ m, 0x01010101u, dp4a_ss(m, 0xffffffffu, sum));
}

// The rows of y: fp16 copies of their activation codes, zero up to kp, and
// their scales, 128 times their sums; and for each CTA the level of its runs.  A row out of range gets scale NaN.
constexpr int WD_T = 256;
// ROW: threads of a row, a warp or four
template <int ROW>
__global__ void __launch_bounds__(WD_T) i8_widen(const I8Params A, int kp, float* __restrict__ xs, uint4* __restrict__ xb, uint4* __restrict__ zero, int zeros) {
  __shared__ int s_lo, s_hi;
  constexpr int ROWS = WD_T / ROW, WARPS = ROW / 32, WINDOWS = ROW > 32 ? 256 : 4;
  __shared__ uint32_t s_level, s_plain[WD_T / 32], s_win[ROWS][WINDOWS];  // sums of magnitudes over 512 codes
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in = threadIdx.x % ROW;
  pdl_wait();
  pdl_trigger();
  // split sums: the parts of a tile that are done, and their sums
  if (blockIdx.x == 0 && threadIdx.x < I8_SPLIT_TILES) reinterpret_cast<uint32_t*>(A.ws + I8_OFF_PARTS)[threadIdx.x] = 0u;
  for (int i = blockIdx.x * WD_T + threadIdx.x; i < zeros; i += gridDim.x * WD_T) zero[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) {
    s_lo = A.offsets ? i8_offset(A, 0) : 0;
    s_hi = A.offsets ? 0 : A.P;
    s_level = IG_LEVELS - 1;
  }
  __syncthreads();
  if (A.offsets) {  // rows of any group: up to the largest offset
    int hi = 0;
    for (int g = threadIdx.x; g <= A.G; g += WD_T) hi = max(hi, i8_offset(A, g));
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) atomicMax(&s_hi, hi);
    __syncthreads();
  }
  const int hi = s_hi;
  uint32_t level = IG_LEVELS - 1;
  uint32_t* win = s_win[threadIdx.x / ROW];
  const int windows = (kp + 511) / 512;
  for (long long p = s_lo + (long long)blockIdx.x * ROWS + threadIdx.x / ROW; p < hi; p += (long long)gridDim.x * ROWS) {
    const int row = A.rows ? __ldcg(A.rows + p) : (int)p;
    const bool ok = row >= 0 && row < A.X;
    const int8_t* src = A.x + (ok ? row : 0) * A.ldx;
    uint4* dst = xb + p * (kp / 8);
    int plain = 0;
    auto put = [&](int u, const uint4& c) {  // (32 units of a warp are a window)
      plain = dp4a_ss(c.x, 0x01010101u, dp4a_ss(c.y, 0x01010101u, dp4a_ss(c.z, 0x01010101u, dp4a_ss(c.w, 0x01010101u, plain))));
      uint32_t o[8];
      cvt_int8x8(c.x, c.y, o);
      cvt_int8x8(c.z, c.w, o + 4);
      dst[2 * u] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[2 * u + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    };
    auto add = [&](int u, const uint4& c) {  // by whole warps
      const uint32_t sum = (uint32_t)__reduce_add_sync(0xffffffffu, magnitudes(c.x, magnitudes(c.y, magnitudes(c.z, magnitudes(c.w, 0)))));
      if (lane == 0 && u / 32 < windows) win[u / 32] = sum;
    };
    const int whole = ok ? A.K / 16 : 0;
    constexpr int U = 4;  // loads under way together
    for (int u = in; (u & ~31) < kp / 16; u += U * ROW) {  // (the same for a whole warp)
      uint4 c[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int v = u + i * ROW;
        c[i] = v < whole ? __ldcg(reinterpret_cast<const uint4*>(src) + v) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int v = u + i * ROW, n = ok && v == whole ? A.K & 15 : 0;
        if ((v & ~31) >= kp / 16) break;
        if (n > 0) {  // the row's last codes
          uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (k < n) w[k >> 2] |= (uint32_t)(uint8_t)src[16 * v + k] << (8 * (k & 3));
          c[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (v < kp / 16) put(v, c[i]);
        add(v, c[i]);
      }
    }
    plain = __reduce_add_sync(0xffffffffu, plain);
    if (ROW > 32) {
      if (lane == 0) s_plain[warp] = (uint32_t)plain;
      named_bar(1 + warp / WARPS, ROW);
      if (in == 0) {
        plain = 0;
        for (int w = 0; w < WARPS; ++w) plain += (int)s_plain[warp + w];
      }
    }
    __syncwarp();
    if (in < 32 && ok) {
      // the level of this row: whole windows of 512 << level codes, each with
      // magnitudes of at most IG_MOST in all (level 0 always)
      uint32_t all = 0;
      for (int w = lane; w < windows; w += 32) all += win[w];
      if (__reduce_add_sync(0xffffffffu, all) > IG_MOST) {
        uint32_t mine = 0;
        for (int j = 1; j < IG_LEVELS - 1; ++j) {
          uint32_t most = 0;
          for (int w0 = lane << j; w0 < windows; w0 += 32 << j) {
            uint32_t sum = 0;
            for (int w = w0; w < min(w0 + (1 << j), windows); ++w) sum += win[w];
            most = max(most, sum);
          }
          if (__reduce_max_sync(0xffffffffu, most) > IG_MOST) break;
          mine = j;
        }
        level = min(level, mine);
      }
    }
    if (ROW > 32) named_bar(1 + warp / WARPS, ROW);
    __syncwarp();
    if (in == 0) {
      reinterpret_cast<uint32_t*>(xs)[A.P + p] = 128u * (uint32_t)plain;
      xs[p] = ok ? __ldcg(A.xs + row) : __uint_as_float(0x7fc00000u);
      if (!ok) atomicOr(reinterpret_cast<uint32_t*>(A.ws), COLI_STATUS_BADIDX);
    }
  }
  if (in == 0) atomicMin(&s_level, level);
  __syncthreads();
  if (threadIdx.x == 0) reinterpret_cast<uint32_t*>(A.ws + WS_HEADER_BYTES)[blockIdx.x] = s_level;
}

bool encode_weights(CUtensorMap* m, const I8Params& A) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)A.K, (cuuint64_t)A.N, (cuuint64_t)(A.wgroup ? A.G : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)A.ldw, (cuuint64_t)(A.wgroup ? A.wgroup : A.ldw)};
  const cuuint32_t box[3] = {IG_WK, IG_M, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(A.w), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_rows_f16(CUtensorMap* m, const void* base, int kp, int rows, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kp, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kp * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Once a device: the shared-memory limit, and that the warps' register split
// fits in what a CTA is launched with (setmaxnreg.inc would otherwise wait for
// registers that never come).
template <int NT>
cudaError_t check_kernel(int* pairs) {
  static std::atomic<uint64_t> checked{0};
  static std::atomic<int> fit[64];  // pairs of CTAs that run together
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(checked.load(std::memory_order_acquire) >> dev & 1)) {
    const auto kernel = i8_gemm<NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, IG_MAX_SMEM);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa{};
    if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
    const int need = 128 * IG_RCTL + 256 * IG_RCONV + 256 * IG_REPI;
    if (fa.numRegs * IG_THREADS < need || fa.numRegs < IG_RCONV || fa.numRegs > IG_REPI || fa.maxThreadsPerBlock < IG_THREADS)
      return cudaErrorInvalidConfiguration;
    if (IgShape<NT>::PAIR) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      cfg.gridDim = dim3(2);
      cfg.blockDim = dim3(IG_THREADS);
      cfg.dynamicSmemBytes = ig_smem<NT>(COLI_I8_MAX_GROUPS);
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
      if (n < 1) return cudaErrorInvalidConfiguration;
      fit[dev].store(n, std::memory_order_relaxed);
    }
    checked.fetch_or(1ull << dev, std::memory_order_release);
  }
  *pairs = fit[dev].load(std::memory_order_relaxed);
  return cudaSuccess;
}

// K in parts: where the tiles fill less than half of the SMs, a part of at least
// 512 codes for every SM (4096 x 6144 against 16 rows 22 us whole, 13 in four
// parts; parts of 256 codes gain nothing, and 500 x 496 against 30 rows takes 9.9 us
// in two of them, 8.4 whole).  None is empty.
template <int NT>
int splits_of(const I8Params& A, long long items, int sms) {
  constexpr int KSTEP = IgShape<NT>::BK;
  const int kall = (A.K + KSTEP - 1) / KSTEP, ctas = sms < 2 * I8_SPLIT_TILES ? sms : 2 * I8_SPLIT_TILES;
  if (IgShape<NT>::PAIR || items < 1 || 2 * items > ctas) return 1;
  const int most = kall / (512 / KSTEP), n = (int)(ctas / items) < most ? (int)(ctas / items) : most;
  if (n <= 1) return 1;
  const int per = (kall + n - 1) / n;
  return (kall + per - 1) / per;
}

// Cycles a call is expected to take with tiles of NT rows, fitted to measured
// times: a code of a full tile's rows takes PER of them (2.4 for its 128 weights, the
// rest falls with the rows), a call START more with pairs, JOIN where its sums
// are split.  (Groups: a tile and a half a group on average, at least one.)  Measured, tiles
// of 64 and of 128 rows, us: 8192 rows of 4096 x 6144 406, 280; 512 rows of 4096 x
// 4096 29, 26; 128 rows of 4096 x 6144 21, 23; in 32 groups of 4096 x 6144 10 rows a
// group 113, 115, 96 rows 231, 188, 1000 rows 1631, 1077; 16384 rows in 256 groups 1091, 860.
// Of 21 sizes (128 to 16000 rows, N 512 to 20000, K 1000 to 8200, 1 to 256 groups), most
// of which the fit has not seen, 15 got the faster tiles; the others lost 1 to 7 %, one 14 %
// (2000 rows in 8 groups of 1024 x 4096: 41, 36).
template <int NT>
double cycles_of(const I8Params& A, int sms) {
  constexpr bool PAIR = IgShape<NT>::PAIR;
  constexpr double WEIGHTS = 2.4, PER = PAIR ? 5.3 : 4.4, START = PAIR ? 10000 : 0, JOIN = 5700;
  constexpr int MROWS = (PAIR ? 2 : 1) * IG_M;
  const int mt = (A.N + MROWS - 1) / MROWS, at_once = PAIR ? sms / 2 : sms;
  if (A.G == 1) {
    const long long items = (long long)((A.P + NT - 1) / NT) * mt;
    const int splits = splits_of<NT>(A, items, sms);
    return START + (splits > 1 ? PER * A.K / splits + JOIN : PER * A.K * (double)((items + at_once - 1) / at_once));
  }
  const int groups = A.G < A.P ? A.G : A.P;
  const double each = (double)A.P / groups / NT + 0.5, tiles = groups * (each > 1.0 ? each : 1.0) * mt, share = 1.0 / (tiles > at_once ? at_once : tiles);
  return START + (WEIGHTS * A.K * tiles + (PER - WEIGHTS) / NT * A.K * (double)A.P * mt) * share;
}

template <int NT>
cudaError_t launch_nt(const I8Params& A, int sms, cudaStream_t st) {
  constexpr bool PAIR = IgShape<NT>::PAIR;
  int pairs = 0;
  cudaError_t e = check_kernel<NT>(&pairs);
  if (e != cudaSuccess) return e;
  const int kp = (int)i8_kp(A.K);
  float* xs = reinterpret_cast<float*>(A.ws + i8_off_xs());
  uint8_t *xb = A.ws + i8_off_xb(A.P), *part = A.ws + i8_off_part(A.P, A.K);
  IgMaps maps;
  bool ok = encode_weights(&maps.w, A);
  for (int i = 0; ok && i < 3; ++i) ok = encode_rows_f16(&maps.x[i], xb, kp, A.P, 16 << i);
  if (!ok) return cudaErrorInvalidValue;
  // (at most: a partial tile per group that can have rows)
  const long long items = (A.G == 1 ? (A.P + NT - 1) / NT : A.P / NT + (A.G < A.P ? A.G : A.P)) * (long long)((A.N + (PAIR ? 2 : 1) * IG_M - 1) / ((PAIR ? 2 : 1) * IG_M));
  if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int splits = splits_of<NT>(A, items, sms), zeros = splits > 1 ? (int)items * NT * IG_M / 4 : 0;
  // four warps a row where rows are long enough to fill them (8192 rows of 1536:
  // the call took 43.6 us with a warp a row, 48.0 with four; a warp sums 4 windows at most)
  const bool four = A.K >= 2048;
  const int rows = WD_T / (four ? 128 : 32), most = 8 * sms < I8_WIDEN_CTAS ? 8 * sms : I8_WIDEN_CTAS;
  int wide = (A.P + rows - 1) / rows;
  if (wide < zeros / (4 * WD_T)) wide = zeros / (4 * WD_T);
  if (wide > most) wide = most;
  e = launch_pdl(four ? i8_widen<128> : i8_widen<32>, (unsigned)wide, WD_T, 0, st, A, kp, xs, reinterpret_cast<uint4*>(xb), reinterpret_cast<uint4*>(part), zeros);
  if (e != cudaSuccess) return e;
  if (PAIR) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)(2 * (items < pairs ? items : pairs)));
    cfg.blockDim = dim3(IG_THREADS);
    cfg.dynamicSmemBytes = ig_smem<NT>(A.G);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, i8_gemm<NT>, maps, A, (uint32_t)i8_off_xs(), wide, 1, reinterpret_cast<uint32_t*>(part));
  }
  const long long grid = splits > 1 ? items * splits : items < sms ? items : sms;
  return launch_pdl(i8_gemm<NT>, (unsigned)grid, IG_THREADS, ig_smem<NT>(A.G), st, maps, A, (uint32_t)i8_off_xs(), wide, splits, reinterpret_cast<uint32_t*>(part));
}

}  // namespace

cudaError_t launch_i8_gemm(const I8Params& A, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (A.P <= 32) return launch_nt<32>(A, sms, st);
  return A.P <= 64 || cycles_of<64>(A, sms) <= cycles_of<128>(A, sms) ? launch_nt<64>(A, sms, st) : launch_nt<128>(A, sms, st);
}

}  // namespace colimoe
