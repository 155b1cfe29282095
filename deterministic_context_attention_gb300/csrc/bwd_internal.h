// bwd_internal.h -- work items and launch parameters of the backward kernels
// (bwd.cu, dbwd.cu).  Not part of the public interface.
#pragma once
#include <cuda.h>

#include "rlk_internal.h"

namespace rlk {

constexpr float kLog2e = 1.44269504088896340736f;

struct alignas(16) BwdItem {
  int32_t seq;
  int32_t head;   // dK/dV: KV head g; dQ: query head h
  int32_t block;  // dK/dV: KV block j; dQ: first row of the query tile
  int32_t rows;   // dQ: rows of the tile written; dK/dV: unused
};

constexpr int kMaxBwdTiles = 1800;

// dlambda[h] = -(sum of Delta_2 over the rows of head h); add: to what an earlier
// range of the batch's sequences left.
struct DLambda {
  float* out;            // [hq], or null: not this launch's
  const float* delta_t;  // [hq][2 maps][t_pad]
  int64_t t_pad, rows;
  bool add;
};

// One warp a head: lane l adds rows l + 32 i, eight sums side by side (i mod 8) in
// ascending order, which meet in fixed trees.
__device__ __forceinline__ void dlambda_head(const DLambda& p, int h, int lane) {
  const float* x = p.delta_t + (2 * static_cast<int64_t>(h) + 1) * p.t_pad;
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.f;
  for (int64_t r = lane; r < p.rows; r += 256) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r + 32 * i < p.rows ? __ldg(x + r + 32 * i) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = __fadd_rn(s[i], v[i]);
  }
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) {
#pragma unroll
    for (int i = 0; i < off; ++i) s[i] = __fadd_rn(s[i], s[i + off]);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) s[0] = __fadd_rn(s[0], __shfl_xor_sync(0xffffffffu, s[0], off));
  if (lane == 0) p.out[h] = p.add ? __fsub_rn(p.out[h], s[0]) : -s[0];
}

// The item list holds tiles; item i is head i mod item_heads of tile
// i / item_heads (the heads of a tile are adjacent in the longest-first
// order), so a launch takes kMaxBwdTiles * heads items.
struct BwdParams {
  ErrWord* err;
  int32_t hq, hkv, group, num_items;
  int32_t item_heads, pad0;
  int64_t t_pad;        // row stride of the transposed lse / Delta
  float scale, scale_log2;
  const float* lse_t;   // [hq][t_pad] (differential: [hq][2 maps][t_pad])
  const float* delta_t; // [hq][t_pad] (the same)
  const float* lambda;  // differential: [hq]
  unsigned int* counter;  // differential dQ: items taken beyond each CTA's first, 0 at the launch
  DLambda dlam;         // differential dQ
  float* dq;
  float* dk;
  float* dv;
  int32_t cu[kMaxSeqs + 1];
  BwdItem items[kMaxBwdTiles];
};

__device__ __forceinline__ BwdItem bwd_item(const BwdParams& p, int item) {
  const int t = item / p.item_heads;
  BwdItem it = p.items[t];
  it.head = item - t * p.item_heads;
  return it;
}

// One launch of the differential kernels: KIND 0 dK/dV, 1 dQ (dbwd.cu).
// overlap: dQ may start on SMs that the launch before it, dK/dV's, leaves.
template <int KIND>
cudaError_t launch_dbwd(const BwdParams& p, int grid, const CUtensorMap& mq, const CUtensorMap& mk,
                        const CUtensorMap& mv, const CUtensorMap& mdo, bool overlap, cudaStream_t stream);
cudaError_t configure_dbwd_kernels();

}  // namespace rlk
