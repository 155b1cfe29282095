// append.cu -- appending K and V rows to the paged BF16 cache, K rotated by
// its positions on the way, with the queries of the same tokens and a packed
// copy of the rotated keys where asked.
//
// The rotation is the one of rope.cu on pairs (i, i + w/2) of every w-wide
// group of a row: w = 128 turns whole rows, w = 64 each half on its own (the
// maps of differential attention).  Pair i of a 64-wide group has frequency
// theta^(-2i/64) = theta^(-2(2i)/128): entry 2i of the 128-wide table, which
// therefore serves both widths.
//
// HBM-bound: a row is 256 bytes read and 256 written (twice for a key that is
// also kept packed); the table's rows come from L2.  A warp takes 16
// consecutive rows of one packed tensor (Q, K or V): four at a time, eight
// lanes a row, 16 bytes of either half of each pair a lane, all of the warp's
// loads in flight before the first use.  Lane i meanwhile works out row i's
// sequence, position and page (a binary search and one table read, once per
// row instead of once per lane), and the rows' places go round by shuffles.
// Prompts of 105,000 tokens (8 KV heads, no queries: 865 MB) take 126 us,
// 6.8 TB/s; chunks with 32 query heads rotated beside the keys (160 MB) 25.5 us,
// 6.3 TB/s; a step of 64 tokens 3.1 us, one chain of page table, rotation
// table and rows.
#include <cuda_runtime.h>

#include "numerics.cuh"
#include "ptx.cuh"
#include "rlk_internal.h"

namespace rlk {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendRows = 16;  // rows of a warp

// W: the width of a rotated group (64, 128), or 0 (no rotation).
template <int W>
__global__ void __launch_bounds__(kAppendThreads) rlk_append_kernel(const __grid_constant__ AppendParams p) {
  const int lane = threadIdx.x & 31, sub = lane >> 3, j = lane & 7;
  int64_t w = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
  // warps of Q, then of K, then of V
  const int64_t tokens = p.cu[p.num_seqs];
  const int64_t wq = p.q ? (tokens * p.hq + kAppendRows - 1) / kAppendRows : 0;
  const int64_t wk = (tokens * p.hkv + kAppendRows - 1) / kAppendRows;
  if (w >= wq + 2 * wk) return;
  const bool is_q = w < wq, is_v = w >= wq + wk;
  if (!is_q) w -= is_v ? wq + wk : wq;
  const int heads = is_q ? p.hq : p.hkv;
  const int64_t rows = tokens * heads, row0 = w * kAppendRows;
  const uint16_t* src = is_q ? p.q : is_v ? p.v : p.k;
  // 16-byte pieces of the lane's pairs: element i of a pair in piece ca, its
  // partner in piece cb
  const int ca = W == 64 ? (j >> 2) * 8 + (j & 3) : j, cb = W == 64 ? ca + 4 : ca + 8;
  uint4 a[4], b[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t row = row0 + 4 * t + sub;
    a[t] = b[t] = make_uint4(0u, 0u, 0u, 0u);
    if (row < rows) {
      const uint4* x = reinterpret_cast<const uint4*>(src + row * kHeadDim);
      a[t] = x[ca];
      b[t] = x[cb];
    }
  }
  // row `lane` (of the first 16): its position, and its row of the pool (-1: none)
  int my_pos = 0;
  int64_t my_at = -1;
  {
    const int64_t row = row0 + (lane & 15);
    if (row < rows) {
      const int tok = static_cast<int>(row / heads);
      const int head = static_cast<int>(row - static_cast<int64_t>(tok) * heads);
      // the sequence holding tok: the last s with cu[s] <= tok (empty
      // sequences share their start with the next one)
      int lo = 0, hi = p.num_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu[mid] <= tok) lo = mid;
        else hi = mid - 1;
      }
      my_pos = p.pos0[lo] + (tok - p.cu[lo]);
      if (!is_q) {
        const int page = __ldg(p.page_table + static_cast<int64_t>(lo) * p.max_pages + (my_pos >> p.page_shift));
        if (page >= 0 && page < p.n_pages) {
          const int slot = my_pos & ((1 << p.page_shift) - 1);
          my_at = ((static_cast<int64_t>(page) << p.page_shift) + slot) * p.hkv + head;
        } else {
          report_error(p.err, kErrBadPage, 0xb01);
        }
      }
    }
  }
  uint16_t* pool = is_v ? p.v_pool : p.k_pool;
  uint16_t* packed = is_q ? p.q_out : is_v ? nullptr : p.k_out;
  float c[8], s[8];
  int at_pos = -1;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t row = row0 + 4 * t + sub;
    const int pos = __shfl_sync(0xffffffffu, my_pos, 4 * t + sub);
    const int64_t at = __shfl_sync(0xffffffffu, my_at, 4 * t + sub);
    if (row >= rows) continue;
    if (W != 0 && !is_v) {
      if (pos != at_pos) {  // the next row of the lane is mostly of the same token
        const float4* tr = reinterpret_cast<const float4*>(p.rope_table + static_cast<int64_t>(pos) * kHeadDim);
        if (W == 128) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 x = __ldg(tr + 2 * j + i), y = __ldg(tr + 16 + 2 * j + i);
            c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
            s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // every second entry
            const float4 x = __ldg(tr + 4 * (j & 3) + i), y = __ldg(tr + 16 + 4 * (j & 3) + i);
            c[2 * i] = x.x, c[2 * i + 1] = x.z;
            s[2 * i] = y.x, s[2 * i + 1] = y.z;
          }
        }
        at_pos = pos;
      }
      rope_words8(a[t], b[t], c, s);
    }
    if (at >= 0) {
      uint4* y = reinterpret_cast<uint4*>(pool + at * kHeadDim);
      y[ca] = a[t];
      y[cb] = b[t];
    }
    if (packed) {
      uint4* y = reinterpret_cast<uint4*>(packed + row * kHeadDim);
      y[ca] = a[t];
      y[cb] = b[t];
    }
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t stream) {
  const int64_t tokens = p.cu[p.num_seqs];
  const int64_t warps = (p.q ? (tokens * p.hq + kAppendRows - 1) / kAppendRows : 0) +
                        2 * ((tokens * p.hkv + kAppendRows - 1) / kAppendRows);
  const int grid = static_cast<int>((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
  if (!p.rope_table)
    rlk_append_kernel<0><<<grid, kAppendThreads, 0, stream>>>(p);
  else if (p.rope_width == 64)
    rlk_append_kernel<64><<<grid, kAppendThreads, 0, stream>>>(p);
  else
    rlk_append_kernel<128><<<grid, kAppendThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace rlk
