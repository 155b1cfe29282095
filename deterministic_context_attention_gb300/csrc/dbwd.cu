// dbwd.cu -- backward of differential attention for sm_103a: dQ, dK, dV (the
// preprocess is in bwd.cu), and dlambda.
//
// With P_m = exp(scale q_m k_m^T - lse_m), dP = dO V^T and Delta_m = dO . O_m:
//   dV   = (P_1 - lambda P_2)^T dO
//   dS_1 = P_1 (dP - Delta_1),  dS_2 = P_2 (lambda Delta_2 - lambda dP)
//   dQ_m = scale dS_m K_m,      dK_m = scale dS_m^T Q_m
// Both maps share dP, and their P's meet in one product for dV: per 128 x 128
// tile pair the tensor core takes 48 units of a 128 x 128 x 16 product for
// dK/dV and 32 for dQ (map by map, with dP and dV of each, it is 72 and 40: that
// form, the plain kernels run over both maps, took 1000 + 700 us for 2 x 4096
// tokens of 32 heads over 8, this one 740 to 770 + 445).  P and dS enter as two BF16
// parts, as in the plain backward.
//
// Accumulation.  The tensor core truncates its FP32 sums: 5e-8 of the value a
// product on the average, all to one side, 1.1e-4 of dV after the 4096 products
// of a long sequence's group.  So an accumulator takes 128 products at most
// (kFlush tiles); then four warps of their own add it to the output in global
// memory, rounded to nearest, while the other accumulator's products go on: the
// gradients are then 4e-6 off.  A thread adds (red.add, so that nothing waits
// for the old value) to addresses that no other thread writes, in order, so the
// sums are the same in every run.
//
// Work of a step u: 64 streamed rows (half a tile) against 128 resident ones.
//   KIND 0 (dK/dV): resident K_j, V_j; streamed Q_i, dO_i of every head of the
//     group, query tiles ascending from the diagonal, heads inside.  TMEM rows
//     are keys, columns queries; four 64-column areas rotate:
//       a: S_1 -> P'    b: S_2 -> dS_2    c: dP -> dS_1    d: S_1 of u + 1
//     (P' = P_1 - lambda P_2).  S_2 of u + 1 follows dV(u) into a, dP of u + 1
//     follows dK_2(u) into b, S_1 of u + 2 follows dK_1(u) into c, so that P of
//     u + 1 is formed while dK(u) and dP(u + 1) run.  Each waits for the commit
//     of the product whose operand it overwrites: the tensor core orders the
//     products of one accumulator only.
//   KIND 1 (dQ): resident Q_i, dO_i; streamed K_j, V_j, ascending.  TMEM rows
//     are queries, columns keys; two sets of three areas, S_1, S_2 (dS_m over
//     them) and dP, one computed while the other is used.
//
// What bounds it: P and dS between the products.  A step's products take the
// tensor core 1792 cycles (dQ 1280), its 64 columns of exponentials, splits and
// TMEM traffic 1650 on their own and 3000 beside products with both operands in
// shared memory, whose bandwidth those take whole; 3160 a step are measured
// (dQ 1900).  So statistics are in registers before each wait, and the warps
// that form P and dS keep out of local memory (dK/dV's 128 bytes of spills are the
// accumulator warps': 4 are left in a build without those, all in one without P and
// dS).  At 2 x 4096 tokens (687 GFLOP by the formulas) the two take 1190 to 1215 us
// one after the other, 570 TFLOP/s.  Batches of few or uneven items are bounded by
// the longest dK/dV item instead, which one SM walks alone: one sequence of 1201
// tokens, 5 query heads over one KV head, 10 items, takes 166 us, 40 over 8 take 198.
//
// The two launches overlap: dK/dV's CTAs, all resident, let dQ's be scheduled at
// once, and one of those starts on each SM that the former leave (the shared
// memory holds one).  dQ reads nothing of dK/dV's and waits for it before its end.
// A dQ CTA's first item is the one of its number, whenever it starts; further ones
// it takes longest first from a counter as it gets done.  7 sequences of 5 to 1201
// tokens, 40 heads over 8: 343 -> 313 us for the whole call, 2 x 4096: 1265 -> 1230
// (one kernel with both roles' code: 335 and 1290, its dQ loop 10 % slower).
//
// Warp roles (512 threads):
//   warps 0-7    P and dS: warp w takes TMEM lane quadrant w mod 4 and 32 of the
//                64 columns
//   warp  8      TMA producer
//   warp  9      TMEM allocator, issuer of S and dP; warp 11 of dV, dK, dQ (one
//                warp for all: dK/dV 859 us and dQ 536; two, with dV and dK leaving
//                half a period apart: 876 and 474)
//   warp  10     dK/dV: the column statistics; dQ: dlambda, a head at a time (a kernel
//                of its own before dK/dV: 4 us a call)
//   warps 12-15  accumulators to global memory
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <type_traits>

#include "bwd_internal.h"
#include "numerics.cuh"
#include "ptx.cuh"

namespace rlk {
namespace {

constexpr int kDBThreads = 512;
constexpr int kDBRegsLaunch = 128;
// P/dS warps 160, producer / MMA 48, accumulators 144
static_assert(2 * 160 + 48 + 144 <= 4 * kDBRegsLaunch, "register split");
// tiles (of 16 products) between flushes of an accumulator, dV and dK half a
// period apart
constexpr int kFlush = 8;

template <int KIND>
struct DBwdLayout {
  static constexpr int kTile = 128 * kHeadDim * 2;  // one 128 x 128 BF16 tile, two 64-column halves
  static constexpr int kHalf = 128 * 128;
  // streamed tiles: dK/dV (Q_i, dO_i) in two slots each; dQ K_j in three, V_j,
  // which dP alone reads, in two (two and two with staging for the flush: 475 us)
  static constexpr int kSlots = KIND == 0 ? 2 : 3, kSlots2 = 2;
  static constexpr int kResOff = 0;  // (K_j, V_j) or (Q_i, dO_i)
  static constexpr int kStreamOff = 2 * kTile;
  static constexpr int kStream2Off = kStreamOff + kSlots * kTile;
  static constexpr int kStageOff = kStream2Off + kSlots2 * kTile;  // dK/dV: the flush's staging, 4 warps x 32 rows x 128 B
  static constexpr int kVecOff = kStageOff + (KIND == 0 ? 4 * 32 * 128 : 0);
  static constexpr int kVecFloats = 4 * 128 + 4;  // lse_1, lse_2 (log2), Delta_1, lambda Delta_2 of 128 queries; -lambda
  static constexpr int kBarOff = kVecOff + (KIND == 0 ? 2 * kVecFloats * 4 : 0);
  static constexpr int kResFull = 0, kResEmpty = 1, kStFull = 2, kStEmpty = 5, kSt2Empty = 8, kSFull = 10, kDPFull = 12,
                       kPFull = 14, kDSFull = 16, kAccFull = 18, kAccEmpty = 20, kVecFull = 22, kVecEmpty = 24, kVDone = 26,
                       kK2Done = 28, kK1Done = 30, kItemFull = 32, kItemEmpty = 36, kNumBars = 40;
  static constexpr int kItems = 4;  // dQ: items published, not yet taken by every warp
  static constexpr int kItemOff = kBarOff + kNumBars * 8;
  static constexpr int kMiscOff = kItemOff + kItems * 4;
  static constexpr int kTotal = kMiscOff + 16;
  static constexpr int kAlloc = kTotal + 1024;
  static_assert(kAlloc <= 232448, "backward shared memory");
  static_assert(kBarOff % 16 == 0, "alignment");
};

// KIND 0: area a of step n; b, c and d follow it mod 4, and d(n) = a(n + 1)
__device__ __forceinline__ uint32_t area_a(uint32_t n) { return (0u - n) & 3u; }

// A warp's bounded wait, and one arrival for a whole warp.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, ErrWord* err,
                                         unsigned int site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err, site));
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Streamed tiles of an item.  KIND 0: (query tile from j to the last) x (heads
// of the group); KIND 1: KV blocks 0 .. the last its rows see.
template <int KIND>
__device__ __forceinline__ int item_tiles(const BwdParams& p, const BwdItem& it) {
  const int len = p.cu[it.seq + 1] - p.cu[it.seq];
  return KIND == 0 ? ((len + 127) / 128 - it.block) * p.group : (it.block + it.rows - 1) / 128 + 1;
}

// A load from shared memory that stays where it is written.
__device__ __forceinline__ float4 lds4(const float* p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(smem_u32(p)) : "memory");
  return v;
}

__device__ __forceinline__ void red_add4(float* p, const float4& v) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}

template <int KIND>
__global__ void __launch_bounds__(kDBThreads, 1)
    rlk_dbwd_kernel(const __grid_constant__ BwdParams p, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_do) {
  using L = DBwdLayout<KIND>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  volatile int* items = reinterpret_cast<volatile int*>(smem + L::kItemOff);
  float* vecs = reinterpret_cast<float*>(smem + L::kVecOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&bars[L::kResFull], 1);
    mbar_init(&bars[L::kResEmpty], 1);
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(&bars[L::kStFull + s], 1);
      mbar_init(&bars[L::kStEmpty + s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[L::kSt2Empty + s], 1);
      mbar_init(&bars[L::kSFull + s], 1);
      mbar_init(&bars[L::kDPFull + s], 1);
      mbar_init(&bars[L::kPFull + s], 8);
      mbar_init(&bars[L::kDSFull + s], 8);
      mbar_init(&bars[L::kAccFull + s], 1);
      mbar_init(&bars[L::kAccEmpty + s], 4);
      mbar_init(&bars[L::kVecFull + s], 1);
      mbar_init(&bars[L::kVecEmpty + s], 8);
      mbar_init(&bars[L::kVDone + s], 1);
      mbar_init(&bars[L::kK2Done + s], 1);
      mbar_init(&bars[L::kK1Done + s], 1);
    }
    for (int s = 0; s < L::kItems; ++s) {
      mbar_init(&bars[L::kItemFull + s], 1);
      mbar_init(&bars[L::kItemEmpty + s], kDBThreads / 32 - 2);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (KIND == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // dQ may start on SMs left over
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // KIND 0: areas 0 .. 3, dV in 256 .. 383, dK in 384 .. 511; KIND 1: areas 0 .. 5, dQ in 384 .. 511
  auto area = [&](uint32_t i) { return tmem + 64 * i; };
  const uint32_t res_addr = smem_u32(smem + L::kResOff);
  auto slot_addr = [&](uint32_t t) { return smem_u32(smem + L::kStreamOff + (t % L::kSlots) * L::kTile); };
  auto slot2_addr = [&](uint32_t t) { return smem_u32(smem + L::kStream2Off + (t % L::kSlots2) * L::kTile); };

  // The CTA's items, in step for all its warps: the first is the CTA's number.
  // dK/dV: snake order over the longest-first list.  dQ: whatever the producer
  // took from the counter.
  const int first_item = blockIdx.x;
  bool fail = false;
  auto next_item = [&](uint32_t& n) -> int {
    if constexpr (KIND == 0) {
      const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x), k = static_cast<int>(++n);
      return k * g + ((k & 1) ? g - 1 - c : c);
    } else {
      const uint32_t s = n % L::kItems;
      fail = fail || !wait_all(&bars[L::kItemFull + s], (n / L::kItems) & 1, abort, p.err, 0xd51);
      const int item = items[s];
      arrive_warp(&bars[L::kItemEmpty + s], lane);
      ++n;
      return item;
    }
  };

  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;" ::: "memory");
    if (warp == 8) {
      // ---------------------------------------------------------- producer
      uint32_t res_it = 0, st_it = 0;
      uint32_t taken = 0;
      for (int item = first_item, next = 0; !fail && item < p.num_items; item = next) {
        const BwdItem it = bwd_item(p, item);
        const int tiles = item_tiles<KIND>(p, it);
        const int tok0 = p.cu[it.seq];
        if (!wait_all(&bars[L::kResEmpty], (res_it & 1) ^ 1, abort, p.err, 0xd01)) { fail = true; break; }
        ++res_it;
        if (lane == 0) {
          uint8_t* a = smem + L::kResOff;
          uint64_t* bar = &bars[L::kResFull];
          mbar_arrive_expect_tx(bar, 2 * L::kTile);
          const CUtensorMap* m0 = KIND == 0 ? &tm_k : &tm_q;
          const CUtensorMap* m1 = KIND == 0 ? &tm_v : &tm_do;
          const int r = tok0 + (KIND == 0 ? it.block * 128 : it.block);
          tma_load_3d(a, m0, bar, 0, it.head, r);
          tma_load_3d(a + L::kHalf, m0, bar, 64, it.head, r);
          tma_load_3d(a + L::kTile, m1, bar, 0, it.head, r);
          tma_load_3d(a + L::kTile + L::kHalf, m1, bar, 64, it.head, r);
        }
        int row = KIND == 0 ? tok0 + it.block * 128 : tok0, h = KIND == 0 ? it.head * p.group : it.head / p.group;
        for (int t = 0; t < tiles; ++t, ++st_it) {
          // both tiles land on the first one's barrier
          const uint32_t slot = st_it % L::kSlots, slot2 = st_it % L::kSlots2;
          bool ok = wait_all(&bars[L::kStEmpty + slot], ((st_it / L::kSlots) & 1) ^ 1, abort, p.err, 0xd02);
          ok = ok && (KIND == 0 || wait_all(&bars[L::kSt2Empty + slot2], ((st_it / L::kSlots2) & 1) ^ 1, abort, p.err, 0xd03));
          if (!ok) { fail = true; break; }
          // the next item is taken as late as hides the trip: the CTA that is
          // done first gets it
          if (KIND == 1 && lane == 0 && t + 1 == tiles) next = static_cast<int>(gridDim.x + atomicAdd(p.counter, 1u));
          if (lane == 0) {
            uint8_t* d = smem + L::kStreamOff + slot * L::kTile;
            uint8_t* d2 = smem + L::kStream2Off + slot2 * L::kTile;
            uint64_t* bar = &bars[L::kStFull + slot];
            mbar_arrive_expect_tx(bar, 2 * L::kTile);
            const CUtensorMap* m0 = KIND == 0 ? &tm_q : &tm_k;
            const CUtensorMap* m1 = KIND == 0 ? &tm_do : &tm_v;
            tma_load_3d(d, m0, bar, 0, h, row);
            tma_load_3d(d + L::kHalf, m0, bar, 64, h, row);
            tma_load_3d(d2, m1, bar, 0, h, row);
            tma_load_3d(d2 + L::kHalf, m1, bar, 64, h, row);
          }
          if (KIND == 1 || ++h == (it.head + 1) * p.group) {  // (KIND 0: the next query tile after the group's heads)
            if (KIND == 0) h -= p.group;
            row += 128;
          }
        }
        if constexpr (KIND == 0) {
          next = next_item(taken);
        } else {
          const uint32_t s = taken % L::kItems;
          fail = fail || !wait_all(&bars[L::kItemEmpty + s], ((taken / L::kItems) & 1) ^ 1, abort, p.err, 0xd04);
          ++taken;
          if (lane == 0) {
            items[s] = next;
            mbar_arrive(&bars[L::kItemFull + s]);
          }
          next = __shfl_sync(0xffffffffu, next, 0);
        }
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- S / dP issuer
      constexpr uint32_t kIdK = idesc_bf16(128, 64, false, false);  // both operands K-major
      const uint32_t leader = elect_one_sync();
      // S_m of half c of the streamed tile at st: the map's four K-steps
      auto issue_s = [&](uint32_t d, uint32_t st, int c, int m) {
        const Desc a = make_desc(res_addr + m * L::kHalf, 16, 1024), b = make_desc(st + m * L::kHalf + c * 64 * 128, 16, 1024);
        if (leader) {
          mma_ss<0>(d, a, 0, b, 0, kIdK);
#pragma unroll
          for (int k = 1; k < 4; ++k) mma_ss<1>(d, a, 2 * k, b, 2 * k, kIdK);
        }
      };
      auto issue_dp = [&](uint32_t d, uint32_t st, int c) {
        const Desc a = make_desc(res_addr + L::kTile, 16, 1024), b = make_desc(st + c * 64 * 128, 16, 1024);
        if (leader) {
          mma_ss<0>(d, a, 0, b, 0, kIdK);
#pragma unroll
          for (int k = 1; k < 8; ++k)
            mma_ss<1>(d, a, (k >> 2) * (L::kHalf >> 4) + (k & 3) * 2, b, (k >> 2) * (L::kHalf >> 4) + (k & 3) * 2, kIdK);
        }
      };
      auto commit = [&](int bar) {
        if (leader) umma_commit(&bars[bar]);
      };
      auto wait = [&](int bar, uint32_t parity, unsigned int site) {
        const bool ok = wait_all(&bars[bar], parity, abort, p.err, site);
        tc_fence_after();
        return ok;
      };
      uint32_t res_it = 0, st_it = 0, n = 0;
      uint32_t taken = 0;
      for (int item = first_item; !fail && item < p.num_items; item = next_item(taken)) {
        const BwdItem it = bwd_item(p, item);
        const int tiles = item_tiles<KIND>(p, it), steps = 2 * tiles;
        // of the streamed tiles only those of the last 128 rows can be short
        const int len = p.cu[it.seq + 1] - p.cu[it.seq];
        const int short_from = KIND == 0 ? tiles - p.group : (len & ~127) / 128, short_rows = len & 127;
        // the item's streamed tile t has landed; its rows past the sequence's
        // end (another sequence's, whose Inf or NaN times a weight of 0 would
        // be NaN) become zeros
        auto landed = [&](int t) {
          const uint32_t si = st_it + t;
          if (!wait(L::kStFull + si % L::kSlots, (si / L::kSlots) & 1, 0xd12)) return false;
          if (short_rows && t >= short_from) {
            uint8_t* d = smem + L::kStreamOff + (si % L::kSlots) * L::kTile;
            uint8_t* d2 = smem + L::kStream2Off + (si % L::kSlots2) * L::kTile;
            for (int i = lane; i < (128 - short_rows) * 16; i += 32) {
              const int row = short_rows + (i >> 4), piece = i & 15;  // 16-byte pieces: 8 per half row
              const int at = (piece >> 3) * L::kHalf + row * 128 + (piece & 7) * 16;
              *reinterpret_cast<uint4*>(d + at) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(d2 + at) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          return true;
        };
        if (!wait(L::kResFull, res_it & 1, 0xd11) || !landed(0)) { fail = true; break; }
        ++res_it;
        for (int u = 0; u < steps; ++u, ++n) {
          const int c = u & 1;
          const uint32_t st = slot_addr(st_it + (u >> 1)), st2 = slot2_addr(st_it + (u >> 1)), x = n & 1;
          if constexpr (KIND == 0) {
            // an area is free once the product that read it last is done: that
            // of a(n), dK_1 of n - 2; of b(n), dV of n - 1; of c(n), dK_2 of n - 1
            auto issue_s1 = [&](uint32_t k, uint32_t at, int cc) {
              if (!wait(L::kK1Done + (k & 1), ((k >> 1) & 1) ^ 1, 0xd13)) return false;
              issue_s(area(area_a(k)), at, cc, 0);
              return true;
            };
            if (u == 0 && !issue_s1(n, st, 0)) { fail = true; break; }
            if (n > 0 && !wait(L::kVDone + (x ^ 1), ((n - 1) >> 1) & 1, 0xd14)) { fail = true; break; }
            issue_s(area((area_a(n) + 1) & 3), st, c, 1);
            commit(L::kSFull + x);
            if (n > 0 && !wait(L::kK2Done + (x ^ 1), ((n - 1) >> 1) & 1, 0xd15)) { fail = true; break; }
            issue_dp(area((area_a(n) + 2) & 3), st2, c);
            commit(L::kDPFull + x);
            if (u + 1 == steps) commit(L::kResEmpty);  // the item's last S/dP
            if (u + 1 < steps) {
              if (c == 1 && !landed((u + 1) >> 1)) { fail = true; break; }
              if (!issue_s1(n + 1, slot_addr(st_it + ((u + 1) >> 1)), c ^ 1)) { fail = true; break; }
            }
          } else {
            if (c == 0 && u > 0 && !landed(u >> 1)) { fail = true; break; }
            if (!wait(L::kK2Done + x, ((n >> 1) & 1) ^ 1, 0xd13)) { fail = true; break; }  // the set's last products
            issue_s(area(3 * x), st, c, 0);
            issue_s(area(3 * x + 1), st, c, 1);
            issue_dp(area(3 * x + 2), st2, c);
            commit(L::kSFull + x);
            if (c == 1) commit(L::kSt2Empty + ((st_it + (u >> 1)) & 1));  // V_j: dP alone reads it
            if (u + 1 == steps) commit(L::kResEmpty);
          }
          __syncwarp();
        }
        st_it += tiles;
      }
    } else if (warp == 11) {
      // ---------------------------------------------------------- accumulation issuer
      // (a warp of its own: the tensor core's queue holds a few products, and
      // one warp's barrier checks between its bursts let it run dry)
      constexpr uint32_t kIdV = idesc_bf16(128, 128, false, true);   // dV: A in TMEM, B MN-major
      constexpr uint32_t kIdMap = idesc_bf16(128, 64, false, true);  // dK_m, dQ_m
      const uint32_t leader = elect_one_sync();
      // acc (+)= the 64-column area a (hi, then lo, of four K-steps) times rows 64 c .. of the tile at b
      auto issue_acc = [&](uint32_t acc, uint32_t a, uint32_t b, int c, uint32_t id, bool first) {
        const Desc bd = make_desc(b + c * 64 * 128, L::kHalf, 1024);
        if (leader) {
          if (first) mma_ts<0>(acc, a, bd, 0, id);
          else mma_ts<1>(acc, a, bd, 0, id);
#pragma unroll
          for (int k = 1; k < 4; ++k) mma_ts<1>(acc, a + 16 * k, bd, 128 * k, id);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ts<1>(acc, a + 16 * k + 8, bd, 128 * k, id);
        }
      };
      auto commit = [&](int bar) {
        if (leader) umma_commit(&bars[bar]);
      };
      auto wait = [&](int bar, uint32_t parity, unsigned int site) {
        const bool ok = wait_all(&bars[bar], parity, abort, p.err, site);
        tc_fence_after();
        return ok;
      };
      uint32_t st_it = 0, n = 0, fl_v = 0, fl_k = 0;
      uint32_t taken = 0;
      for (int item = first_item; !fail && item < p.num_items; item = next_item(taken)) {
        const BwdItem it = bwd_item(p, item);
        const int tiles = item_tiles<KIND>(p, it), steps = 2 * tiles;
        for (int u = 0; u < steps; ++u, ++n) {
          const int t = u >> 1, c = u & 1;
          const bool first = c == 0 && t % kFlush == 0;  // of dV (dQ)
          const bool last = c == 1 && (t % kFlush == kFlush - 1 || t + 1 == tiles);
          const uint32_t st = slot_addr(st_it + t), x = n & 1, par = (n >> 1) & 1;
          if constexpr (KIND == 0) {
            const uint32_t a = area_a(n);
            const bool first_k = c == 0 && (t == 0 || t % kFlush == kFlush / 2);
            const bool last_k = c == 1 && (t % kFlush == kFlush / 2 - 1 || t + 1 == tiles);
            if (first && !wait(L::kAccEmpty, (fl_v & 1) ^ 1, 0xd21)) { fail = true; break; }
            if (!wait(L::kPFull + x, par, 0xd22)) { fail = true; break; }
            issue_acc(tmem + 256, area(a), slot2_addr(st_it + t), c, kIdV, first);
            commit(L::kVDone + x);
            if (last) commit(L::kAccFull);
            __syncwarp();
            if (first_k && !wait(L::kAccEmpty + 1, (fl_k & 1) ^ 1, 0xd23)) { fail = true; break; }
            if (!wait(L::kDSFull + x, par, 0xd24)) { fail = true; break; }
            issue_acc(tmem + 448, area((a + 1) & 3), st + L::kHalf, c, kIdMap, first_k);
            commit(L::kK2Done + x);
            issue_acc(tmem + 384, area((a + 2) & 3), st, c, kIdMap, first_k);
            commit(L::kK1Done + x);
            if (last_k) {
              commit(L::kAccFull + 1);
              ++fl_k;
            }
          } else {
            if (first && !wait(L::kAccEmpty, (fl_v & 1) ^ 1, 0xd21)) { fail = true; break; }
            if (!wait(L::kDSFull + x, par, 0xd24)) { fail = true; break; }
            issue_acc(tmem + 384, area(3 * x), st, c, kIdMap, first);
            issue_acc(tmem + 448, area(3 * x + 1), st + L::kHalf, c, kIdMap, first);
            commit(L::kK2Done + x);
            if (last) commit(L::kAccFull);
          }
          if (last) ++fl_v;
          if (c == 1) commit(L::kStEmpty + (st_it + t) % L::kSlots);
          __syncwarp();
        }
        st_it += tiles;
      }
    } else if (warp == 10 && KIND == 1) {
      // ---------------------------------------------------------- dlambda
      if (p.dlam.out)
        for (int h = blockIdx.x; h < p.hq; h += gridDim.x) dlambda_head(p.dlam, h, lane);
    } else if (warp == 10) {
      // ---------------------------------------------------------- column statistics
      // of each streamed tile's queries: lse_m log2 e, Delta_1 and lambda Delta_2, 0
      // past the sequence's end, and -lambda of the tile's head
      uint32_t v_it = 0;
      uint32_t taken = 0;
      for (int item = first_item; !fail && item < p.num_items; item = next_item(taken)) {
        const BwdItem it = bwd_item(p, item);
        const int tiles = item_tiles<KIND>(p, it);
        const int tok0 = p.cu[it.seq], len = p.cu[it.seq + 1] - tok0;
        int q0 = it.block * 128, h = it.head * p.group - 1;
        for (int t = 0; t < tiles; ++t, ++v_it) {
          if (++h == (it.head + 1) * p.group) {
            h -= p.group;
            q0 += 128;
          }
          const int64_t at = 2 * static_cast<int64_t>(h) * p.t_pad + tok0 + q0;
          float x[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = q0 + 32 * i + lane < len;
            const int64_t k = at + 32 * i + lane;
            x[0][i] = in ? __ldg(p.lse_t + k) : 0.f;
            x[1][i] = in ? __ldg(p.lse_t + k + p.t_pad) : 0.f;
            x[2][i] = in ? __ldg(p.delta_t + k) : 0.f;
            x[3][i] = in ? __ldg(p.delta_t + k + p.t_pad) : 0.f;
          }
          const float nl = -__ldg(p.lambda + h);
          if (!wait_all(&bars[L::kVecEmpty + (v_it & 1)], ((v_it >> 1) & 1) ^ 1, abort, p.err, 0xd25)) { fail = true; break; }
          float* v = vecs + (v_it & 1) * L::kVecFloats;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[32 * i + lane] = __fmul_rn(x[0][i], kLog2e);
            v[128 + 32 * i + lane] = __fmul_rn(x[1][i], kLog2e);
            v[256 + 32 * i + lane] = x[2][i];
            v[384 + 32 * i + lane] = __fmul_rn(-nl, x[3][i]);
          }
          if (lane == 0) v[512] = nl;
          arrive_warp(&bars[L::kVecFull + (v_it & 1)], lane);
        }
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ P / dS
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;" ::: "memory");
    const int wh = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // tile row = TMEM lane
    const uint32_t off = (static_cast<uint32_t>((warp & 3) * 32) << 16) + 32 * wh;  // the warp's lanes and columns of an area
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t s_it = 0, v_it = 0;
    auto f2 = [](uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); };
    auto bar_wait = [&](int bar, uint32_t parity, unsigned int site) {
      const bool ok = wait_all(&bars[bar], parity, abort, p.err, site);
      tc_fence_after();
      return ok;
    };
    auto stored = [&](int bar) {
      tmem_st_wait();
      tc_fence_before();
      arrive_warp(&bars[bar], lane);
    };
    uint32_t taken = 0;
    for (int item = first_item; !fail && item < p.num_items; item = next_item(taken)) {
      const BwdItem it = bwd_item(p, item);
      const int tiles = item_tiles<KIND>(p, it);
      const int tok0 = p.cu[it.seq], len = p.cu[it.seq + 1] - tok0;
      if constexpr (KIND == 0) {
        const int key_pos = it.block * 128 + r;
        int q0 = it.block * 128 + 32 * wh, hh = 0;  // position of the warp's first column
        for (int u = 0; u < 2 * tiles; ++u, ++s_it) {
          const int c = u & 1;
          const uint32_t a = area_a(s_it), vb = v_it & 1, x = s_it & 1, par = (s_it >> 1) & 1;
          const uint32_t ta = area(a) + off, tb = area((a + 1) & 3) + off, td = area((a + 2) & 3) + off;
          const float* v = vecs + vb * L::kVecFloats + 64 * c + 32 * wh;
          if (c == 0 && !bar_wait(L::kVecFull + vb, (v_it >> 1) & 1, 0xd31)) { fail = true; break; }
          // the columns' statistics go into registers before the waits: S and dP
          // take the whole of shared memory's bandwidth, and a load beside them
          // takes hundreds of cycles
          float4 l1[8], l2[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            l1[i] = lds4(v + 4 * i);
            l2[i] = lds4(v + 128 + 4 * i);
          }
          const float nl = *reinterpret_cast<const volatile float*>(vecs + vb * L::kVecFloats + 512);
          if (!bar_wait(L::kSFull + x, par, 0xd32)) { fail = true; break; }
          // P_1 and P_2 of the warp's elements, kept for dS
          uint32_t p1[32], p2[32];
          tmem_ld32(ta, p1);
          tmem_ld32(tb, p2);
          const float2 nl2 = make_float2(nl, nl);
          const bool full = __all_sync(0xffffffffu, key_pos < len && q0 + 31 < len && q0 >= key_pos);
          tmem_ld_wait(p1);
          tmem_ld_wait(p2);
          auto weights = [&](auto masked) {
#pragma unroll
            for (int k = 0; k < 32; k += 16) {
              uint32_t w[16];  // a K-step of the product: 8 words hi, then 8 lo
#pragma unroll
              for (int e = k; e < k + 16; e += 4) {
                const float la[4] = {l1[e / 4].x, l1[e / 4].y, l1[e / 4].z, l1[e / 4].w};
                const float lb[4] = {l2[e / 4].x, l2[e / 4].y, l2[e / 4].z, l2[e / 4].w};
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                  const float2 y = ffma2(f2(p1[e + i], p1[e + i + 1]), sl2, make_float2(-la[i], -la[i + 1]));
                  const float2 z = ffma2(f2(p2[e + i], p2[e + i + 1]), sl2, make_float2(-lb[i], -lb[i + 1]));
                  float2 q = make_float2(ex2_hw(y.x), ex2_hw(y.y)), s = make_float2(ex2_hw(z.x), ex2_hw(z.y));
                  if constexpr (decltype(masked)::value) {
                    const int qa = q0 + e + i, qb = qa + 1;
                    const bool oka = key_pos < len && qa < len && qa >= key_pos;
                    const bool okb = key_pos < len && qb < len && qb >= key_pos;
                    q = make_float2(oka ? q.x : 0.0f, okb ? q.y : 0.0f);
                    s = make_float2(oka ? s.x : 0.0f, okb ? s.y : 0.0f);
                  }
                  p1[e + i] = __float_as_uint(q.x);
                  p1[e + i + 1] = __float_as_uint(q.y);
                  p2[e + i] = __float_as_uint(s.x);
                  p2[e + i + 1] = __float_as_uint(s.y);
                  const int slot = (e - k + i) >> 1;
                  split_pair2(ffma2(s, nl2, q), w[slot], w[8 + slot]);
                }
              }
              tmem_st16(ta + k, w);
            }
          };
          if (full) weights(std::false_type{});
          else weights(std::true_type{});
          stored(L::kPFull + x);
          float4 e1[4], e2[4];
          auto deltas = [&](int k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e1[i] = lds4(v + 256 + k + 4 * i);
              e2[i] = lds4(v + 384 + k + 4 * i);
            }
          };
          deltas(0);
          if (!bar_wait(L::kDPFull + x, par, 0xd33)) { fail = true; break; }
          uint32_t dp[32];
          tmem_ld32(td, dp);
          tmem_ld_wait(dp);
#pragma unroll
          for (int k = 0; k < 32; k += 16) {
            uint32_t w1[16], w2[16];
#pragma unroll
            for (int e = k; e < k + 16; e += 4) {
              const float4 d1 = e1[(e - k) / 4], d2 = e2[(e - k) / 4];
              const float da[4] = {d1.x, d1.y, d1.z, d1.w}, db[4] = {d2.x, d2.y, d2.z, d2.w};
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                const float2 g = f2(dp[e + i], dp[e + i + 1]);
                const int slot = (e - k + i) >> 1;
                split_pair2(fmul2(f2(p2[e + i], p2[e + i + 1]), ffma2(g, nl2, make_float2(db[i], db[i + 1]))), w2[slot],
                            w2[8 + slot]);
                split_pair2(fmul2(f2(p1[e + i], p1[e + i + 1]), fsub2(g, make_float2(da[i], da[i + 1]))), w1[slot], w1[8 + slot]);
              }
            }
            if (k == 0) deltas(16);
            tmem_st16(tb + k, w2);
            tmem_st16(td + k, w1);
          }
          stored(L::kDSFull + x);
          if (c == 0) {
            q0 += 64;
          } else {
            arrive_warp(&bars[L::kVecEmpty + vb], lane);
            ++v_it;
            q0 -= 64;
            if (++hh == p.group) {
              hh = 0;
              q0 += 128;
            }
          }
        }
      } else {
        // the row's statistics are fixed for the item
        const int row_pos = it.block + r;
        const bool row_ok = r < it.rows && row_pos < len;
        float lse1 = 0.f, lse2 = 0.f, dl1 = 0.f, dl2 = 0.f;
        if (row_ok) {
          const int64_t at = 2 * static_cast<int64_t>(it.head) * p.t_pad + tok0 + row_pos;
          lse1 = __fmul_rn(__ldg(p.lse_t + at), kLog2e);
          lse2 = __fmul_rn(__ldg(p.lse_t + at + p.t_pad), kLog2e);
          dl1 = __ldg(p.delta_t + at);
          dl2 = __ldg(p.delta_t + at + p.t_pad);
        }
        const float nl = -__ldg(p.lambda + it.head);
        const float2 nl2 = make_float2(nl, nl), n1 = make_float2(-lse1, -lse1), n2 = make_float2(-lse2, -lse2),
                     d1 = make_float2(dl1, dl1), d2 = make_float2(__fmul_rn(-nl, dl2), __fmul_rn(-nl, dl2));
        int k0 = 32 * wh;  // position of the warp's first column
        for (int u = 0; u < 2 * tiles; ++u, ++s_it, k0 += 64) {
          const uint32_t x = s_it & 1;
          const uint32_t t1 = area(3 * x) + off, t2 = t1 + 64, td = t1 + 128;
          if (!bar_wait(L::kSFull + x, (s_it >> 1) & 1, 0xd32)) { fail = true; break; }
          uint32_t s1[32], s2[32], dp[32];
          tmem_ld32(t1, s1);
          tmem_ld32(td, dp);
          tmem_ld32(t2, s2);
          const bool full = __all_sync(0xffffffffu, row_ok && k0 + 31 <= row_pos);
          tmem_ld_wait(s1);
          tmem_ld_wait(dp);
          tmem_ld_wait(s2);
          auto grads = [&](auto masked) {
#pragma unroll
            for (int k = 0; k < 32; k += 16) {
              uint32_t w1[16], w2[16];
#pragma unroll
              for (int e = k; e < k + 16; e += 2) {
                const float2 y = ffma2(f2(s1[e], s1[e + 1]), sl2, n1), z = ffma2(f2(s2[e], s2[e + 1]), sl2, n2);
                float2 q = make_float2(ex2_hw(y.x), ex2_hw(y.y)), s = make_float2(ex2_hw(z.x), ex2_hw(z.y));
                if constexpr (decltype(masked)::value) {
                  const bool oka = row_ok && k0 + e <= row_pos, okb = row_ok && k0 + e + 1 <= row_pos;
                  q = make_float2(oka ? q.x : 0.0f, okb ? q.y : 0.0f);
                  s = make_float2(oka ? s.x : 0.0f, okb ? s.y : 0.0f);
                }
                const float2 g = f2(dp[e], dp[e + 1]);
                const int slot = (e - k) >> 1;
                split_pair2(fmul2(q, fsub2(g, d1)), w1[slot], w1[8 + slot]);
                split_pair2(fmul2(s, ffma2(g, nl2, d2)), w2[slot], w2[8 + slot]);
              }
              tmem_st16(t1 + k, w1);
              tmem_st16(t2 + k, w2);
            }
          };
          if (full) grads(std::false_type{});
          else grads(std::true_type{});
          stored(L::kDSFull + x);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ accumulators to global memory
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;" ::: "memory");
    const int wq = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    float4* stg = reinterpret_cast<float4*>(smem + L::kStageOff + wq * (32 * 128));
    uint32_t fl[2] = {0, 0};
    uint32_t taken = 0;
    for (int item = first_item; !fail && item < p.num_items; item = next_item(taken)) {
      const BwdItem it = bwd_item(p, item);
      const int tiles = item_tiles<KIND>(p, it);
      const int tok0 = p.cu[it.seq], len = p.cu[it.seq + 1] - tok0;
      // rows 32 wq .. of the tile: keys of the block, or query rows
      const int row0 = (KIND == 0 ? it.block * 128 : it.block) + 32 * wq;
      const int rows = KIND == 0 ? min(32, len - row0) : min(32, min(it.rows - 32 * wq, len - row0));
      const int heads = KIND == 0 ? p.hkv : p.hq;
      const int64_t base = (static_cast<int64_t>(tok0 + row0) * heads + it.head) * kHeadDim;
      // dV (dQ) and dK half a period apart, so that one leaves while the other is summed
      for (int t = 0; t < tiles && !fail; t += kFlush / 2) {
        const bool end = t + kFlush / 2 >= tiles;
        const int v_now = t % kFlush != 0 || end, k_now = KIND == 0 && (t % kFlush == 0 || end);
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
          if (!(which ? k_now : v_now)) continue;
          if (!wait_all(&bars[L::kAccFull + which], fl[which] & 1, abort, p.err, 0xd41)) { fail = true; break; }
          ++fl[which];
          tc_fence_after();
          // the whole accumulator into registers: the next products wait for
          // this alone
          const uint32_t src = tmem + (KIND == 0 && which == 0 ? 256 : 384) + lane_off;
          uint32_t x[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(src + 32 * i, x[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld_wait(x[i]);
          tc_fence_before();
          arrive_warp(&bars[L::kAccEmpty + which], lane);
          float* dst = (KIND == 1 ? p.dq : which == 0 ? p.dv : p.dk) + base;
          const float mul = KIND == 0 && which == 0 ? 1.0f : p.scale;
          const bool fresh = which ? t == 0 || tiles <= kFlush / 2 : t < kFlush;  // nothing in the output yet
          if constexpr (KIND == 1) {
            // no room for staging beside the third slot: each thread its own
            // row (dK/dV: 775 us so, 740 staged)
            if (lane < rows) {
              float* to = dst + static_cast<int64_t>(lane) * heads * kHeadDim;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float4 val =
                      make_float4(__fmul_rn(__uint_as_float(x[i][4 * j]), mul), __fmul_rn(__uint_as_float(x[i][4 * j + 1]), mul),
                                  __fmul_rn(__uint_as_float(x[i][4 * j + 2]), mul),
                                  __fmul_rn(__uint_as_float(x[i][4 * j + 3]), mul));
                  if (fresh) *reinterpret_cast<float4*>(to + 32 * i + 4 * j) = val;
                  else red_add4(to + 32 * i + 4 * j, val);
                }
              }
            }
          } else {
            // each 32-column chunk through shared memory (piece j of a row in
            // slot j ^ (row & 7)), so that four rows leave as whole 128-byte lines
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                stg[lane * 8 + (j ^ (lane & 7))] =
                    make_float4(__fmul_rn(__uint_as_float(x[i][4 * j]), mul), __fmul_rn(__uint_as_float(x[i][4 * j + 1]), mul),
                                __fmul_rn(__uint_as_float(x[i][4 * j + 2]), mul),
                                __fmul_rn(__uint_as_float(x[i][4 * j + 3]), mul));
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int rr = 4 * k + (lane >> 3), jj = lane & 7;
                if (rr < rows) {
                  float* to = dst + static_cast<int64_t>(rr) * heads * kHeadDim + 32 * i + 4 * jj;
                  const float4 val = stg[rr * 8 + (jj ^ (rr & 7))];
                  if (fresh) *reinterpret_cast<float4*>(to) = val;
                  else red_add4(to, val);
                }
              }
              __syncwarp();
            }
          }
        }
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  // (dQ, launched while dK/dV may still run, ends after it)
  if (KIND == 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    if (*abort) {
      // let copies already in flight land before the CTA's memory is released
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int KIND>
cudaError_t configure_t() {
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, rlk_dbwd_kernel<KIND>);
  if (e != cudaSuccess) return e;
  // setmaxnreg.inc draws on what the launch was given
  if (a.numRegs < kDBRegsLaunch) {
    fprintf(stderr, "rlk_dbwd_kernel<%d>: %d registers at launch, the split needs %d\n", KIND, a.numRegs, kDBRegsLaunch);
    return cudaErrorInvalidConfiguration;
  }
  return cudaFuncSetAttribute(rlk_dbwd_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              DBwdLayout<KIND>::kAlloc);
}

}  // namespace

cudaError_t configure_dbwd_kernels() {
  cudaError_t e = configure_t<0>();
  return e != cudaSuccess ? e : configure_t<1>();
}

template <int KIND>
cudaError_t launch_dbwd(const BwdParams& p, int grid, const CUtensorMap& mq, const CUtensorMap& mk,
                        const CUtensorMap& mv, const CUtensorMap& mdo, bool overlap, cudaStream_t stream) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(kDBThreads);
  c.dynamicSmemBytes = DBwdLayout<KIND>::kAlloc;
  c.stream = stream;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = overlap ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&c, rlk_dbwd_kernel<KIND>, p, mq, mk, mv, mdo);
  if (e != cudaSuccess) (void)cudaGetLastError();  // it is returned, not left for the next launch to read
  return e;
}
template cudaError_t launch_dbwd<0>(const BwdParams&, int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                    const CUtensorMap&, bool, cudaStream_t);
template cudaError_t launch_dbwd<1>(const BwdParams&, int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                    const CUtensorMap&, bool, cudaStream_t);

}  // namespace rlk
