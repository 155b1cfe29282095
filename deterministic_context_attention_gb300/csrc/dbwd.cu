// dbwd.cu -- backward of differential attention for sm_103a: dQ, dK, dV (the
// preprocess and dlambda are in bwd.cu).
//
// With P_m = exp(scale q_m k_m^T - lse_m), dP = dO V^T and Delta_m = dO . O_m:
//   dV   = (P_1 - lambda P_2)^T dO
//   dS_1 = P_1 (dP - Delta_1),  dS_2 = -lambda P_2 (dP - Delta_2)
//   dQ_m = scale dS_m K_m,      dK_m = scale dS_m^T Q_m
// Both maps share dP, and their P's meet in one product for dV: per 128 x 128
// tile pair the tensor core takes 48 units of a 128 x 128 x 16 product for
// dK/dV and 32 for dQ (map by map, with dP and dV of each, it is 72 and 40:
// 1000 + 700 us for 2 x 4096 tokens of 32 heads where this form takes less than
// half).  P and dS enter as two BF16 parts, as in the plain backward.
//
// Accumulation.  The tensor core truncates its FP32 sums: 5e-8 of the value a
// product on the average, all to one side, 1.1e-4 of dV after the 4096 products
// of a long sequence's group.  So an accumulator takes 128 products at most
// (kFlush tiles); then four warps of their own add it to the output in global
// memory, rounded to nearest, while the other accumulator's products go on.  A
// thread adds to addresses that no other thread writes, in order, so the sums
// are the same in every run.
//
// Work of a step u: 64 streamed rows (half a tile) against 128 resident ones.
//   KIND 0 (dK/dV): resident K_j, V_j; streamed Q_i, dO_i of every head of the
//     group, query tiles ascending from the diagonal, heads inside.  TMEM rows
//     are keys, columns queries; four 64-column areas rotate:
//       a: S_1 -> P'    b: S_2 -> dS_2    c: dP -> dS_1    d: S_1 of u + 1
//     in the tensor core's order  dV(u) S_2(u+1)>a | dK_2(u) dP(u+1)>b dK_1(u)
//     S_1(u+2)>c, each product into an area that the one issued before it has
//     read, so that P of u + 1 is formed while dK(u) and dP(u + 1) run.
//   KIND 1 (dQ): resident Q_i, dO_i; streamed K_j, V_j, ascending.  TMEM rows
//     are queries, columns keys; two sets of three areas, S_1, S_2 (dS_m over
//     them) and dP:  S/dP(u+1) | dQ_1(u) dQ_2(u).
//
// Warp roles (512 threads):
//   warps 0-7    P and dS: warp w takes TMEM lane quadrant w mod 4 and 32 of the
//                64 columns
//   warp  8      TMA producer, warp 9 TMEM allocator and MMA issuer, warp 10 the
//                column statistics of dK/dV
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
// P/dS warps 168, producer / MMA 48, accumulators 128
static_assert(2 * 168 + 48 + 128 <= 4 * kDBRegsLaunch, "register split");
constexpr int kFlush = 8;  // tiles (of 16 products) between flushes of an accumulator

struct DBwdLayout {
  static constexpr int kTile = 128 * kHeadDim * 2;  // one 128 x 128 BF16 tile, two 64-column halves
  static constexpr int kHalf = 128 * 128;
  static constexpr int kStages = 2;
  static constexpr int kResOff = 0;  // (K_j, V_j) or (Q_i, dO_i)
  static constexpr int kStreamOff = 2 * kTile;
  static constexpr int kStageOff = kStreamOff + kStages * 2 * kTile;  // the flush's staging: 4 warps x 32 rows x 128 B
  static constexpr int kVecOff = kStageOff + 4 * 32 * 128;
  static constexpr int kVecFloats = 4 * 128 + 4;  // lse_1, lse_2 (log2), Delta_1, Delta_2 of 128 queries; -lambda
  static constexpr int kBarOff = kVecOff + 2 * kVecFloats * 4;
  static constexpr int kResFull = 0, kResEmpty = 1, kStFull = 2, kStEmpty = 4, kSFull = 6, kDPFull = 8, kPFull = 10,
                       kDSFull = 12, kAccFull = 14, kAccEmpty = 16, kVecFull = 18, kVecEmpty = 20, kNumBars = 22;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kTotal = kMiscOff + 16;
  static constexpr int kAlloc = kTotal + 1024;
};
static_assert(DBwdLayout::kAlloc <= 232448, "backward shared memory");
static_assert(DBwdLayout::kBarOff % 16 == 0, "alignment");
using L = DBwdLayout;

__device__ __forceinline__ uint64_t kdesc(uint32_t tile, int k) {  // K-major operand, K-step k (16 elements)
  return sdesc_sw128(tile + (k >> 2) * L::kHalf + (k & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t mndesc(uint32_t tile, int k) {  // MN-major operand, K-step k (16 rows)
  return sdesc_sw128(tile + k * 16 * 128, L::kHalf, 1024);
}

// A warp's bounded wait, and one arrival for a whole warp.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, ErrWord* err,
                                         unsigned int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err, site));
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ int item_of_round(const BwdParams& p, int round) {  // snake order, -1: none
  const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  const int item = round * g + ((round & 1) ? g - 1 - c : c);
  return item < p.num_items ? item : -1;
}

// Streamed tiles of an item.  KIND 0: (query tile from j to the last) x (heads
// of the group); KIND 1: KV blocks 0 .. the last its rows see.
template <int KIND>
__device__ __forceinline__ int item_tiles(const BwdParams& p, const BwdItem& it) {
  const int len = p.cu[it.seq + 1] - p.cu[it.seq];
  return KIND == 0 ? ((len + 127) / 128 - it.block) * p.group : (it.block + it.rows - 1) / 128 + 1;
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  float* vecs = reinterpret_cast<float*>(smem + L::kVecOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&bars[L::kResFull], 1);
    mbar_init(&bars[L::kResEmpty], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[L::kStFull + s], 1);
      mbar_init(&bars[L::kStEmpty + s], 1);
      mbar_init(&bars[L::kSFull + s], 1);
      mbar_init(&bars[L::kDPFull + s], 1);
      mbar_init(&bars[L::kPFull + s], 8);
      mbar_init(&bars[L::kDSFull + s], 8);
      mbar_init(&bars[L::kAccFull + s], 1);
      mbar_init(&bars[L::kAccEmpty + s], 4);
      mbar_init(&bars[L::kVecFull + s], 1);
      mbar_init(&bars[L::kVecEmpty + s], 8);
    }
    *abort = 0;
    fence_mbar_init();
  }
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
  uint8_t* st_base = smem + L::kStreamOff;
  auto stage_addr = [&](uint32_t t) { return smem_u32(st_base + (t & 1) * 2 * L::kTile); };

  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;" ::: "memory");
    if (warp == 8) {
      // ---------------------------------------------------------- producer
      uint32_t res_it = 0, st_it = 0;
      bool fail = false;
      for (int round = 0; !fail && round * static_cast<int>(gridDim.x) < p.num_items; ++round) {
        const int item = item_of_round(p, round);
        if (item < 0) continue;
        const BwdItem it = bwd_item(p, item);
        const int tiles = item_tiles<KIND>(p, it);
        const int tok0 = p.cu[it.seq];
        if (!wait_all(&bars[L::kResEmpty], (res_it & 1) ^ 1, abort, p.err, 0xd01)) break;
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
        for (int t = 0; t < tiles; ++t, ++st_it) {
          const uint32_t stage = st_it & 1;
          if (!wait_all(&bars[L::kStEmpty + stage], ((st_it >> 1) & 1) ^ 1, abort, p.err, 0xd02)) { fail = true; break; }
          if (lane == 0) {
            uint8_t* d = st_base + stage * 2 * L::kTile;
            uint64_t* bar = &bars[L::kStFull + stage];
            mbar_arrive_expect_tx(bar, 2 * L::kTile);
            const CUtensorMap* m0 = KIND == 0 ? &tm_q : &tm_k;
            const CUtensorMap* m1 = KIND == 0 ? &tm_do : &tm_v;
            const int h = KIND == 0 ? it.head * p.group + t % p.group : it.head / p.group;
            const int r = tok0 + (KIND == 0 ? it.block + t / p.group : t) * 128;
            tma_load_3d(d, m0, bar, 0, h, r);
            tma_load_3d(d + L::kHalf, m0, bar, 64, h, r);
            tma_load_3d(d + L::kTile, m1, bar, 0, h, r);
            tma_load_3d(d + L::kTile + L::kHalf, m1, bar, 64, h, r);
          }
        }
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdK = idesc_bf16(128, 64, false, false);    // S, dP: both operands K-major
      constexpr uint32_t kIdV = idesc_bf16(128, 128, false, true);    // dV: A in TMEM, B MN-major
      constexpr uint32_t kIdMap = idesc_bf16(128, 64, false, true);   // dK_m, dQ_m
      const uint32_t leader = elect_one_sync();
      // S_m of half c of the streamed tile at st: the map's four K-steps
      auto issue_s = [&](uint32_t d, uint32_t st, int c, int m) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (leader)
            umma_ss(d, kdesc(res_addr + m * L::kHalf, k), kdesc(st + m * L::kHalf + c * 64 * 128, k), kIdK, k > 0);
      };
      auto issue_dp = [&](uint32_t d, uint32_t st, int c) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (leader) umma_ss(d, kdesc(res_addr + L::kTile, k), kdesc(st + L::kTile + c * 64 * 128, k), kIdK, k > 0);
      };
      // acc (+)= the 64-column area a (hi, then lo, of four K-steps) times rows 64 c .. of the tile at b
      auto issue_acc = [&](uint32_t acc, uint32_t a, uint32_t b, int c, uint32_t id, bool first) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (leader) umma_ts(acc, a + 16 * k, mndesc(b, 4 * c + k), id, (first && k == 0) ? 0u : 1u);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (leader) umma_ts(acc, a + 16 * k + 8, mndesc(b, 4 * c + k), id, 1u);
      };
      auto commit = [&](int bar) {
        if (leader) umma_commit(&bars[bar]);
      };
      uint32_t res_it = 0, st_it = 0, u_it = 0, fl_it = 0;
      bool fail = false;
      for (int round = 0; !fail && round * static_cast<int>(gridDim.x) < p.num_items; ++round) {
        const int item = item_of_round(p, round);
        if (item < 0) continue;
        const BwdItem it = bwd_item(p, item);
        const int tiles = item_tiles<KIND>(p, it), steps = 2 * tiles;
        auto wait = [&](int bar, uint32_t parity, unsigned int site) {
          const bool ok = wait_all(&bars[bar], parity, abort, p.err, site);
          tc_fence_after();
          return ok;
        };
        // the item's streamed tile t has landed; its rows past the sequence's
        // end (another sequence's, whose Inf or NaN times a weight of 0 would
        // be NaN) become zeros
        const int len = p.cu[it.seq + 1] - p.cu[it.seq];
        auto landed = [&](int t) {
          const uint32_t si = st_it + t;
          if (!wait(L::kStFull + (si & 1), (si >> 1) & 1, 0xd12)) return false;
          const int valid = len - (KIND == 0 ? it.block + t / p.group : t) * 128;
          if (valid < 128) {
            uint8_t* d = st_base + (si & 1) * 2 * L::kTile;
            for (int i = lane; i < (128 - valid) * 32; i += 32) {
              const int row = valid + (i >> 5), piece = i & 31;  // 16-byte pieces: 8 per half row, two tiles
              *reinterpret_cast<uint4*>(d + (piece >> 3) * L::kHalf + row * 128 + (piece & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          return true;
        };
        if (!wait(L::kResFull, res_it & 1, 0xd11) || !landed(0)) break;
        ++res_it;
        if constexpr (KIND == 0) {
          uint32_t a = area(0), b = area(1), c3 = area(2), d = area(3);
          const uint32_t acc_v = tmem + 256, acc_k = tmem + 384;
          issue_s(a, stage_addr(st_it), 0, 0);
          issue_s(b, stage_addr(st_it), 0, 1);
          commit(L::kSFull + (u_it & 1));
          issue_dp(c3, stage_addr(st_it), 0);
          commit(L::kDPFull + (u_it & 1));
          issue_s(d, stage_addr(st_it), 1, 0);
          __syncwarp();
          for (int u = 0; u < steps; ++u, ++u_it) {
            const int t = u >> 1, c = u & 1;
            const bool first = c == 0 && t % kFlush == 0;  // of an accumulator
            const bool last = c == 1 && (t % kFlush == kFlush - 1 || t + 1 == tiles);
            const uint32_t cur = stage_addr(st_it + t), nxt = stage_addr(st_it + ((u + 1) >> 1));
            const uint32_t par = (u_it >> 1) & 1, npar = (u_it + 1) & 1;
            if (!wait(L::kPFull + (u_it & 1), par, 0xd13)) { fail = true; break; }
            if (first && !wait(L::kAccEmpty, (fl_it & 1) ^ 1, 0xd14)) { fail = true; break; }
            issue_acc(acc_v, a, cur + L::kTile, c, kIdV, first);
            if (last) commit(L::kAccFull);
            if (u + 1 < steps) {
              issue_s(a, nxt, c ^ 1, 1);
              commit(L::kSFull + npar);
            }
            __syncwarp();
            if (!wait(L::kDSFull + (u_it & 1), par, 0xd15)) { fail = true; break; }
            if (first && !wait(L::kAccEmpty + 1, (fl_it & 1) ^ 1, 0xd16)) { fail = true; break; }
            issue_acc(acc_k + 64, b, cur + L::kHalf, c, kIdMap, first);
            if (u + 1 < steps) {
              issue_dp(b, nxt, c ^ 1);
              commit(L::kDPFull + npar);
              if (u + 2 == steps) commit(L::kResEmpty);  // the item's last S/dP
            }
            issue_acc(acc_k, c3, cur, c, kIdMap, first);
            if (last) {
              commit(L::kAccFull + 1);
              ++fl_it;
            }
            if (c == 1) commit(L::kStEmpty + ((st_it + t) & 1));
            if (u + 2 < steps) {
              if (c == 0 && !landed((u + 2) >> 1)) { fail = true; break; }
              issue_s(c3, stage_addr(st_it + ((u + 2) >> 1)), c, 0);
            }
            __syncwarp();
            const uint32_t x = d;
            d = c3;
            c3 = b;
            b = a;
            a = x;
          }
        } else {
          const uint32_t acc = tmem + 384;
          auto issue_set = [&](uint32_t set, uint32_t st, int c) {
            issue_s(area(3 * set), st, c, 0);
            issue_s(area(3 * set + 1), st, c, 1);
            issue_dp(area(3 * set + 2), st, c);
            commit(L::kSFull + set);
          };
          issue_set(u_it & 1, stage_addr(st_it), 0);
          __syncwarp();
          for (int u = 0; u < steps; ++u, ++u_it) {
            const int t = u >> 1, c = u & 1;
            const bool first = c == 0 && t % kFlush == 0;
            const bool last = c == 1 && (t % kFlush == kFlush - 1 || t + 1 == tiles);
            const uint32_t set = u_it & 1, cur = stage_addr(st_it + t);
            if (u + 1 < steps) {
              if (c == 1 && !landed((u + 1) >> 1)) { fail = true; break; }
              issue_set(set ^ 1, stage_addr(st_it + ((u + 1) >> 1)), c ^ 1);
              if (u + 2 == steps) commit(L::kResEmpty);  // the item's last S/dP
            }
            __syncwarp();
            if (!wait(L::kDSFull + set, (u_it >> 1) & 1, 0xd15)) { fail = true; break; }
            if (first && !wait(L::kAccEmpty, (fl_it & 1) ^ 1, 0xd14)) { fail = true; break; }
            issue_acc(acc, area(3 * set), cur, c, kIdMap, first);
            issue_acc(acc + 64, area(3 * set + 1), cur + L::kHalf, c, kIdMap, first);
            if (last) {
              commit(L::kAccFull);
              ++fl_it;
            }
            if (c == 1) commit(L::kStEmpty + ((st_it + t) & 1));
            __syncwarp();
          }
        }
        st_it += tiles;
      }
    } else if (warp == 10 && KIND == 0) {
      // ---------------------------------------------------------- column statistics
      // of each streamed tile's queries: lse_m log2 e and Delta_m, 0 past the
      // sequence's end, and -lambda of the tile's head
      uint32_t v_it = 0;
      bool fail = false;
      for (int round = 0; !fail && round * static_cast<int>(gridDim.x) < p.num_items; ++round) {
        const int item = item_of_round(p, round);
        if (item < 0) continue;
        const BwdItem it = bwd_item(p, item);
        const int tiles = item_tiles<KIND>(p, it);
        const int tok0 = p.cu[it.seq], len = p.cu[it.seq + 1] - tok0;
        for (int t = 0; t < tiles; ++t, ++v_it) {
          const int q0 = (it.block + t / p.group) * 128, h = it.head * p.group + t % p.group;
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
          if (!wait_all(&bars[L::kVecEmpty + (v_it & 1)], ((v_it >> 1) & 1) ^ 1, abort, p.err, 0xd21)) { fail = true; break; }
          float* v = vecs + (v_it & 1) * L::kVecFloats;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[32 * i + lane] = __fmul_rn(x[0][i], kLog2e);
            v[128 + 32 * i + lane] = __fmul_rn(x[1][i], kLog2e);
            v[256 + 32 * i + lane] = x[2][i];
            v[384 + 32 * i + lane] = x[3][i];
          }
          if (lane == 0) v[512] = nl;
          arrive_warp(&bars[L::kVecFull + (v_it & 1)], lane);
        }
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ P / dS
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;" ::: "memory");
    const int wq = warp & 3, wh = warp >> 2;
    const int r = wq * 32 + lane;  // tile row = TMEM lane
    const uint32_t off = (static_cast<uint32_t>(wq * 32) << 16) + 32 * wh;  // the warp's lanes and columns of an area
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t u_it = 0, v_it = 0;
    bool fail = false;
    // stores a 32-column group's parts: per 16 columns 8 words hi, then 8 lo
    auto put = [&](uint32_t ta, const uint32_t (&w)[32]) { tmem_st32(ta + off, w); };
    for (int round = 0; !fail && round * static_cast<int>(gridDim.x) < p.num_items; ++round) {
      const int item = item_of_round(p, round);
      if (item < 0) continue;
      const BwdItem it = bwd_item(p, item);
      const int tiles = item_tiles<KIND>(p, it), steps = 2 * tiles;
      const int tok0 = p.cu[it.seq], len = p.cu[it.seq + 1] - tok0;
      if constexpr (KIND == 0) {
        const int key_pos = it.block * 128 + r;
        uint32_t a = 0, b = 1, c3 = 2, d = 3;
        for (int u = 0; u < steps; ++u, ++u_it) {
          const int t = u >> 1, c = u & 1;
          const uint32_t vb = (v_it + t) & 1, par = (u_it >> 1) & 1;
          const float* v = vecs + vb * L::kVecFloats + 64 * c + 32 * wh;
          const int q0 = (it.block + t / p.group) * 128 + 64 * c + 32 * wh;  // position of the warp's first column
          bool ok = c == 1 || wait_all(&bars[L::kVecFull + vb], ((v_it + t) >> 1) & 1, abort, p.err, 0xd31);
          ok = ok && wait_all(&bars[L::kSFull + (u_it & 1)], par, abort, p.err, 0xd32);
          if (!ok) { fail = true; break; }
          tc_fence_after();
          // P_1 and -lambda P_2 of the warp's elements, kept for dS
          uint32_t p1[32], p2[32];
          tmem_ld32(area(a) + off, p1);
          tmem_ld32(area(b) + off, p2);
          tmem_ld_wait(p1);
          tmem_ld_wait(p2);
          const float nl = vecs[vb * L::kVecFloats + 512];
          const float2 nl2 = make_float2(nl, nl);
          const bool full = __all_sync(0xffffffffu, key_pos < len && q0 + 31 < len && q0 >= key_pos);
          {
            uint32_t w[32];
            auto probs = [&](auto masked) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 l1 = *reinterpret_cast<const float4*>(v + e);
                const float4 l2 = *reinterpret_cast<const float4*>(v + 128 + e);
                const float la[4] = {l1.x, l1.y, l1.z, l1.w}, lb[4] = {l2.x, l2.y, l2.z, l2.w};
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                  const float2 x = ffma2(make_float2(__uint_as_float(p1[e + i]), __uint_as_float(p1[e + i + 1])), sl2,
                                         make_float2(-la[i], -la[i + 1]));
                  const float2 y = ffma2(make_float2(__uint_as_float(p2[e + i]), __uint_as_float(p2[e + i + 1])), sl2,
                                         make_float2(-lb[i], -lb[i + 1]));
                  float2 q = make_float2(ex2_hw(x.x), ex2_hw(x.y)), s = make_float2(ex2_hw(y.x), ex2_hw(y.y));
                  if constexpr (decltype(masked)::value) {
                    const int qa = q0 + e + i, qb = qa + 1;
                    const bool oka = key_pos < len && qa < len && qa >= key_pos;
                    const bool okb = key_pos < len && qb < len && qb >= key_pos;
                    q = make_float2(oka ? q.x : 0.0f, okb ? q.y : 0.0f);
                    s = make_float2(oka ? s.x : 0.0f, okb ? s.y : 0.0f);
                  }
                  s = fmul2(s, nl2);
                  p1[e + i] = __float_as_uint(q.x);
                  p1[e + i + 1] = __float_as_uint(q.y);
                  p2[e + i] = __float_as_uint(s.x);
                  p2[e + i + 1] = __float_as_uint(s.y);
                  const int slot = ((e + i) >> 4) * 16 + (((e + i) & 15) >> 1);
                  split_pair2(fadd2(q, s), w[slot], w[slot + 8]);
                }
              }
            };
            if (full) probs(std::false_type{});
            else probs(std::true_type{});
            put(area(a), w);
          }
          tmem_st_wait();
          tc_fence_before();
          arrive_warp(&bars[L::kPFull + (u_it & 1)], lane);
          if (!wait_all(&bars[L::kDPFull + (u_it & 1)], par, abort, p.err, 0xd33)) { fail = true; break; }
          tc_fence_after();
          uint32_t dp[32], w[32];
          tmem_ld32(area(c3) + off, dp);
          tmem_ld_wait(dp);
#pragma unroll
          for (int m = 1; m >= 0; --m) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 dl = *reinterpret_cast<const float4*>(v + 256 + 128 * m + e);
              const float da[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                const float2 q = m ? make_float2(__uint_as_float(p2[e + i]), __uint_as_float(p2[e + i + 1]))
                                   : make_float2(__uint_as_float(p1[e + i]), __uint_as_float(p1[e + i + 1]));
                const float2 ds = fmul2(q, fsub2(make_float2(__uint_as_float(dp[e + i]), __uint_as_float(dp[e + i + 1])),
                                                 make_float2(da[i], da[i + 1])));
                const int slot = ((e + i) >> 4) * 16 + (((e + i) & 15) >> 1);
                split_pair2(ds, w[slot], w[slot + 8]);
              }
            }
            put(area(m ? b : c3), w);
          }
          tmem_st_wait();
          tc_fence_before();
          arrive_warp(&bars[L::kDSFull + (u_it & 1)], lane);
          if (c == 1) arrive_warp(&bars[L::kVecEmpty + vb], lane);
          const uint32_t x = d;
          d = c3;
          c3 = b;
          b = a;
          a = x;
        }
        v_it += tiles;
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
        for (int u = 0; u < steps; ++u, ++u_it) {
          const uint32_t set = u_it & 1;
          const int k0 = (u >> 1) * 128 + 64 * (u & 1) + 32 * wh;  // position of the warp's first column
          if (!wait_all(&bars[L::kSFull + set], (u_it >> 1) & 1, abort, p.err, 0xd32)) { fail = true; break; }
          tc_fence_after();
          uint32_t dp[32], s1[32], s2[32];
          tmem_ld32(area(3 * set) + off, s1);
          tmem_ld32(area(3 * set + 2) + off, dp);
          tmem_ld32(area(3 * set + 1) + off, s2);
          tmem_ld_wait(s1);
          tmem_ld_wait(dp);
          tmem_ld_wait(s2);
          const bool full = __all_sync(0xffffffffu, row_ok && k0 + 31 <= row_pos);
          auto one = [&](uint32_t (&s)[32], uint32_t ta, float lse, float dl, float coef, auto second, auto masked) {
            const float2 nlse = make_float2(-lse, -lse), d2 = make_float2(dl, dl), c2 = make_float2(coef, coef);
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = ffma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sl2, nlse);
              float2 q = make_float2(ex2_hw(x.x), ex2_hw(x.y));
              if constexpr (decltype(masked)::value) {
                q.x = row_ok && k0 + e <= row_pos ? q.x : 0.0f;
                q.y = row_ok && k0 + e + 1 <= row_pos ? q.y : 0.0f;
              }
              if constexpr (decltype(second)::value) q = fmul2(q, c2);
              const float2 ds = fmul2(q, fsub2(make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), d2));
              const int slot = (e >> 4) * 16 + ((e & 15) >> 1);
              split_pair2(ds, w[slot], w[slot + 8]);
            }
            put(ta, w);
          };
          if (full) {
            one(s1, area(3 * set), lse1, dl1, 1.0f, std::false_type{}, std::false_type{});
            one(s2, area(3 * set + 1), lse2, dl2, nl, std::true_type{}, std::false_type{});
          } else {
            one(s1, area(3 * set), lse1, dl1, 1.0f, std::false_type{}, std::true_type{});
            one(s2, area(3 * set + 1), lse2, dl2, nl, std::true_type{}, std::true_type{});
          }
          tmem_st_wait();
          tc_fence_before();
          arrive_warp(&bars[L::kDSFull + set], lane);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ accumulators to global memory
    const int wq = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    float4* stg = reinterpret_cast<float4*>(smem + L::kStageOff + wq * (32 * 128));
    uint32_t fl_it = 0;
    bool fail = false;
    for (int round = 0; !fail && round * static_cast<int>(gridDim.x) < p.num_items; ++round) {
      const int item = item_of_round(p, round);
      if (item < 0) continue;
      const BwdItem it = bwd_item(p, item);
      const int tiles = item_tiles<KIND>(p, it);
      const int tok0 = p.cu[it.seq], len = p.cu[it.seq + 1] - tok0;
      // rows 32 wq .. of the tile: keys of the block, or query rows
      const int row0 = (KIND == 0 ? it.block * 128 : it.block) + 32 * wq;
      const int rows = KIND == 0 ? min(32, len - row0) : min(32, min(it.rows - 32 * wq, len - row0));
      const int heads = KIND == 0 ? p.hkv : p.hq;
      const int64_t base = (static_cast<int64_t>(tok0 + row0) * heads + it.head) * kHeadDim;
      for (int t0 = 0; t0 < tiles && !fail; t0 += kFlush, ++fl_it) {
#pragma unroll 1
        for (int which = 0; which < (KIND == 0 ? 2 : 1); ++which) {
          if (!wait_all(&bars[L::kAccFull + which], fl_it & 1, abort, p.err, 0xd41)) { fail = true; break; }
          tc_fence_after();
          const uint32_t src = tmem + (KIND == 0 && which == 0 ? 256 : 384) + lane_off;
          float* dst = (KIND == 1 ? p.dq : which == 0 ? p.dv : p.dk) + base;
          const float mul = KIND == 0 && which == 0 ? 1.0f : p.scale;
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            uint32_t x[2][32];
            tmem_ld32(src + 32 * c, x[0]);
            tmem_ld32(src + 32 * c + 32, x[1]);
            tmem_ld_wait(x[0]);
            tmem_ld_wait(x[1]);
            if (c == 2) {  // read: free for the next products
              tc_fence_before();
              arrive_warp(&bars[L::kAccEmpty + which], lane);
            }
            // each 32-column chunk through shared memory (piece j of a row in
            // slot j ^ (row & 7)), so that four rows leave as whole 128-byte lines
#pragma unroll
            for (int i = 0; i < 2; ++i) {
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
                  float* to = dst + static_cast<int64_t>(rr) * heads * kHeadDim + 32 * (c + i) + 4 * jj;
                  const float4 val = stg[rr * 8 + (jj ^ (rr & 7))];
                  if (t0 == 0) *reinterpret_cast<float4*>(to) = val;
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
  return cudaFuncSetAttribute(rlk_dbwd_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
}

}  // namespace

cudaError_t configure_dbwd_kernels() {
  cudaError_t e = configure_t<0>();
  return e != cudaSuccess ? e : configure_t<1>();
}

template <int KIND>
cudaError_t launch_dbwd(const BwdParams& p, int grid, const CUtensorMap& mq, const CUtensorMap& mk,
                        const CUtensorMap& mv, const CUtensorMap& mdo, cudaStream_t stream) {
  rlk_dbwd_kernel<KIND><<<grid, kDBThreads, L::kAlloc, stream>>>(p, mq, mk, mv, mdo);
  return cudaGetLastError();
}
template cudaError_t launch_dbwd<0>(const BwdParams&, int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                    const CUtensorMap&, cudaStream_t);
template cudaError_t launch_dbwd<1>(const BwdParams&, int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                    const CUtensorMap&, cudaStream_t);

}  // namespace rlk
