// decode_common.cuh -- what the decode kernels (BF16 pools and the 8-bit
// cache) share: their work items, the state-table fill and the fold on chip.
#pragma once
#include <cuda_runtime.h>

#include <cmath>

#include "numerics.cuh"
#include "ptx.cuh"
#include "rlk_internal.h"

namespace rlk {

constexpr int kDecBlock = 128;  // keys of a global KV block in the transposed decode kernels

__device__ __forceinline__ int dec_snake_item(int round) {
  const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  return round * g + ((round & 1) ? g - 1 - c : c);
}

__device__ __forceinline__ float bf16_bits_as_f32(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }

// One item: the query heads of KV head g of sequence seq against the global
// blocks b0, b0 + stride, ... (nb of them).  Plain decode: all of the
// sequence's blocks (stride 1), folded on chip.  Split decode (state_o set):
// a fixed range of them (stride 1), or with the fold on chip the blocks
// b = r (mod split_stride) of item r; their block states are written to the
// state table at pair (cu_q[seq] + b) * hq + head, for the merge kernel or
// the fold CTAs to fold.
struct DecItem {
  int seq, g, kv_len, b0, nb, stride;
};
__device__ __forceinline__ DecItem dec_item(const FwdParams& p, int item) {
  const FwdTile& t = p.tiles[item];
  DecItem d;
  d.seq = t.seq;
  d.g = t.row_begin;
  d.kv_len = p.cu_k[t.seq];
  d.stride = 1;
  if (p.state_o) {
    d.b0 = t.block;
    d.nb = t.slab_row_count;
    if (p.split_stride > 0) {
      d.stride = p.split_stride;
    }
  } else {
    d.b0 = 0;
    d.nb = (d.kv_len + kDecBlock - 1) / kDecBlock;
  }
  return d;
}

// Split decode with the fold on chip: thread t of the 384 correction and
// softmax threads writes its share of the item's state-table slots with
// kUnwritten (o_b as 16-byte pieces, then lse_b) before any of the item's
// states can land.
constexpr int kFillThreads = 384;
__device__ __forceinline__ void fill_item_slots(const FwdParams& p, const DecItem& di, int G, int t) {
  const int64_t blk0 = p.cu_q[di.seq] + di.b0;
  const int per = G * (kHeadDim / 4);  // 16-byte pieces of one block's states
  const float u = __uint_as_float(kUnwritten);
  const float4 u4 = make_float4(u, u, u, u);
  for (int i = t; i < di.nb * per; i += kFillThreads) {
    const int j = i / per;
    reinterpret_cast<float4*>(p.state_o + ((blk0 + static_cast<int64_t>(j) * di.stride) * p.hq + di.g * G) *
                                              kHeadDim)[i - j * per] = u4;
  }
  for (int i = t; i < di.nb * G; i += kFillThreads) {
    const int j = i / G;
    p.state_lse[(blk0 + static_cast<int64_t>(j) * di.stride) * p.hq + di.g * G + (i - j * G)] = u;
  }
}

// Row maximum of the 32 lanes of a warp (exact; every lane receives it).
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// Split decode with the fold on chip, the fold side: one warp folds query
// head q of the pair (seq, g) over the pair's block states in ascending block
// order as the producer CTAs write them -- the fold the correction role
// applies in the single pass, operation for operation, so the result is the
// same bit for bit.  Lane l folds head dimensions 4 l .. 4 l + 3 and every
// lane runs the head's lse chain (the same inputs, so no lane waits on
// another).
//
// C blocks at a time, the next chunk's reads in flight while the current one
// folds.  The table holds the all-ones NaN until a state lands (arithmetic
// never produces that pattern, and a 32-bit store lands whole, so a value
// that differs from it is the final one).  Reads are weak first (they overlap
// one another); values still unwritten, or stale, are read again with strong
// (device-scope relaxed) loads, which the memory model guarantees to see
// other SMs' stores eventually (a thread's strong loads complete one after
// another).  When the producers fill the table themselves (fill_flag set),
// the chain first waits until every item of the pair has published its
// flag: before that, an item's slots may still hold an earlier call's
// states.  Returns false on a timeout (reported) or an abort.
static __device__ __noinline__ bool fold_chain_on_chip(const FwdParams& p, int seq, int g, int q, int lane,
                                                volatile int* abort) {
  constexpr int C = 8;
  const int G = p.group;
  const int nbp = (p.cu_k[seq] + kDecBlock - 1) / kDecBlock;
  const int64_t base = p.cu_q[seq];
  // lane i: the lse of block c0 + i; every lane: dimensions 4 lane .. of the
  // chunk's blocks (past the chunk: its last block, a valid value)
  auto lse_src = [&](int c0, int nc) { return p.state_lse + (base + c0 + min(lane, nc - 1)) * p.hq + g * G + q; };
  auto o_src = [&](int c0, int nc, int i) {
    return p.state_o + ((base + c0 + min(i, nc - 1)) * p.hq + g * G + q) * kHeadDim + 4 * lane;
  };
  auto issue = [&](int c0, float& lsl, float4 (&v)[C]) {
    const int nc = min(C, nbp - c0);
    lsl = ld_l2_weak(lse_src(c0, nc));
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = ld_l2_weak4(o_src(c0, nc, i));
  };
  auto unwritten4 = [](const float4& a) {
    return __float_as_uint(a.x) == kUnwritten || __float_as_uint(a.y) == kUnwritten ||
           __float_as_uint(a.z) == kUnwritten || __float_as_uint(a.w) == kUnwritten;
  };
  // until every value of the chunk has landed: strong re-reads of what is missing
  auto settle = [&](int c0, float& lsl, float4 (&v)[C]) -> bool {
    const int nc = min(C, nbp - c0);
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
      uint32_t miss = static_cast<uint32_t>(__float_as_uint(lsl) == kUnwritten);
#pragma unroll
      for (int i = 0; i < C; ++i) miss |= static_cast<uint32_t>(unwritten4(v[i]));
      if (__all_sync(0xffffffffu, miss == 0)) return true;
      const bool late = __shfl_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitTimeoutNs, 0);
      if (late || *abort) {
        if (late && lane == 0) {
          *abort = 1;
          report_error(p.err, kErrDeviceTimeout, 0x901);
        }
        return false;
      }
      if (__float_as_uint(lsl) == kUnwritten) lsl = ld_l2_poll(lse_src(c0, nc));
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (unwritten4(v[i])) v[i] = ld_l2_poll4(o_src(c0, nc, i));
    }
  };
  if (p.fill_flag) {
    // lane r (and r + 32): item r's flag; the warp barrier then orders every
    // lane's table reads after the acquiring loads
    const int nr = min(p.split_stride, nbp);
    const uint64_t* flag = p.fill_flag + (static_cast<int64_t>(seq) * p.hkv + g) * kMaxSplitK;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
      bool filled = true;
      for (int r = lane; r < nr; r += 32) filled = ld_acquire_u64(flag + r) == p.fill_nonce && filled;
      if (__all_sync(0xffffffffu, filled)) break;
      const bool late = __shfl_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitTimeoutNs, 0);
      if (late || *abort) {
        if (late && lane == 0) {
          *abort = 1;
          report_error(p.err, kErrDeviceTimeout, 0x903);
        }
        return false;
      }
    }
    __syncwarp();
  }
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  float Lrun = -INFINITY;
  float lsl, lsn = 0.f;
  float4 v[C], vn[C];
  issue(0, lsl, v);
  for (int c0 = 0; c0 < nbp; c0 += C) {
    const int nc = min(C, nbp - c0);
    if (!settle(c0, lsl, v)) return false;
    if (c0 + C < nbp) issue(c0 + C, lsn, vn);  // lands while this chunk folds
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (i < nc) {
        const float lb = __shfl_sync(0xffffffffu, lsl, i);
        if (c0 + i == 0) {
          O = v[i];
          Lrun = lb;
        } else {
          float Lp, al, be;
          fold_coeffs(Lrun, lb, Lp, al, be);
          O.x = __fmaf_rn(v[i].x, be, __fmul_rn(O.x, al));
          O.y = __fmaf_rn(v[i].y, be, __fmul_rn(O.y, al));
          O.z = __fmaf_rn(v[i].z, be, __fmul_rn(O.z, al));
          O.w = __fmaf_rn(v[i].w, be, __fmul_rn(O.w, al));
          Lrun = Lp;
        }
      }
    }
    lsl = lsn;
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = vn[i];
  }
  const int64_t row = static_cast<int64_t>(seq) * p.hq + g * G + q;
  if (p.out_f32) *reinterpret_cast<float4*>(p.out_f32 + row * kHeadDim + 4 * lane) = O;
  if (p.out_bf16) {
    const uint32_t w0 = pack_bf16x2(O.x, O.y), w1 = pack_bf16x2(O.z, O.w);
    *reinterpret_cast<uint2*>(p.out_bf16 + row * kHeadDim + 4 * lane) = make_uint2(w0, w1);
  }
  if (lane == 0 && p.lse) p.lse[row] = Lrun;
  return true;
}

}  // namespace rlk
