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
