// qcache.cu -- the 8-bit paged KV cache: quantising K and V rows as they
// enter it, and reading token ranges of it back as BF16.
//
// Pages hold E4M3 codes [n_pages][hkv][page][128] (one head's page is one
// contiguous run of page x 128 bytes) with one FP32 scale 2^e per (page, KV
// head).  A value becomes a code in two steps:
//   q4   = the value rounded to 4 significant bits (nearest, ties to even)
//   code = q4 / 2^e, or +0 where |q4 / 2^e| < 2^-6 (E4M3's smallest normal)
// with e = max(-120, floor(log2 max |q4|) - 7) over the page's tokens so far.
// The largest code lies in [128, 240]; E4M3's top binade and its subnormals
// stay unused, so that
//   - q4 does not depend on e, and a flush at 2^e followed by one at a larger
//     scale is the flush at the larger scale alone.  When a later token
//     raises e by d, the page's earlier codes lose d in their exponent field
//     (or become 0) and hold exactly what writing all tokens at once would
//     have given: a page's bytes are a function of its tokens, whatever calls
//     wrote them, with no BF16 copy of the page being filled;
//   - code * 2^e is a BF16 number, so reading back is exact.
// What it costs: values below max * 2^-13 become 0, against a rounding error
// of up to max * 2^-5 of the largest ones.
//
// Both passes move 3 bytes per element (2 BF16, 1 code) and are bound by
// HBM; the arithmetic is kept to packed 16-bit integer steps on the BF16
// words (write) and one multiply per element (read).  A unit of work is one
// (page, head) of K or of V: a warp takes up to 16 of its rows, 16 bytes of
// BF16 a lane, all loads in flight before the first use; neighbouring warps
// take neighbouring heads, whose rows are contiguous in the packed tensors.
#include <cuda_runtime.h>

#include <algorithm>

#include "numerics.cuh"
#include "ptx.cuh"
#include "qcache_internal.h"

namespace rlk {
namespace {

constexpr int kQThreads = 256;
constexpr int kQWarps = kQThreads / 32;
constexpr int kQEsMin = 14;  // the biased exponent of the smallest block maximum that sets a scale (e = -120)

// One unit: head h of page `page` (of K or V) and its slots [slot0, slot1),
// which hold the packed rows row0 + slot - slot0.
struct QUnit {
  bool valid;
  bool is_v;
  int head, slot0, slot1;
  int64_t row0;   // packed row of slot slot0
  int64_t entry;  // page-table entry
  int pos_slot0;  // position of slot 0's token
};
__device__ __forceinline__ QUnit q_unit(const QCacheParams& p, int64_t u) {
  QUnit r;
  const int hkv = p.c.hkv, ps = p.c.page_size;
  const int64_t pk = u / hkv;
  r.head = static_cast<int>(u - pk * hkv);
  r.is_v = pk & 1;
  const int64_t pg = pk >> 1;
  r.valid = pg < p.page0[p.num_seqs];
  // the sequence of the touched page: the last s with page0[s] <= pg
  int lo = 0, hi = p.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.page0[mid] <= pg) lo = mid;
    else hi = mid - 1;
  }
  const int pos0 = p.pos0[lo], n = p.cu[lo + 1] - p.cu[lo];
  const int logical = pos0 / ps + static_cast<int>(pg - p.page0[lo]);
  r.pos_slot0 = logical * ps;
  r.slot0 = max(pos0 - r.pos_slot0, 0);
  r.slot1 = static_cast<int>(min(static_cast<int64_t>(ps), static_cast<int64_t>(pos0) + n - r.pos_slot0));
  r.row0 = static_cast<int64_t>(p.cu[lo]) + (r.pos_slot0 + r.slot0 - pos0);
  r.entry = static_cast<int64_t>(lo) * p.c.max_pages + logical;
  return r;
}

__device__ __forceinline__ uint32_t umax2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Two BF16 magnitudes (sign bits cleared) rounded to 3 mantissa bits; a half
// at or past 0x7F80 (overflow, Inf or NaN) is settled by fix_pair.
__device__ __forceinline__ uint32_t round4_pair(uint32_t w) {
  const uint32_t m = w & 0x7FFF7FFFu;
  return (m + 0x00070007u + ((m >> 4) & 0x00010001u)) & 0xFFF0FFF0u;
}
// Non-finite inputs become 0x7FF0 (the NaN code, which sets no scale);
// finite ones that rounded past the largest value are held at it; BF16
// subnormals (which only count where they rounded to a normal) become 0.
__device__ __forceinline__ uint32_t fix_half(uint32_t m, uint32_t r) {
  if (m >= 0x7F80u) return 0x7FF0u;
  if (r >= 0x7F80u) return 0x7F70u;
  return m < 0x0080u ? 0u : r;
}
__device__ __forceinline__ uint32_t fix_pair(uint32_t w, uint32_t r) {
  const uint32_t m = w & 0x7FFF7FFFu;
  return fix_half(m & 0xFFFFu, r & 0xFFFFu) | (fix_half(m >> 16, r >> 16) << 16);
}

// Codes of a rounded pair (one in each half's low byte) under the anchor
// `floor2` = ((es - 14) << 3) + 7 in both halves: exponent field E - es + 14,
// 0 where that is below 1.
__device__ __forceinline__ uint32_t encode_pair(uint32_t w, uint32_t r, uint32_t floor2) {
  const uint32_t t = umax2(r >> 4, floor2) - floor2;  // 0: flushed; otherwise code - 7
  const uint32_t one = __vminu2(t, 0x00010001u);
  return (t + one * 7u) | ((w >> 8) & (one << 7));
}

// An existing code under a scale 2^d times larger (d >= 0).
__device__ __forceinline__ uint32_t rescale_byte(uint32_t c, int d) {
  const int m = static_cast<int>(c & 0x7Fu);
  if (m == 0x7F) return c;
  const int f = m - 8 * d;
  return f >= 8 ? ((c & 0x80u) | static_cast<uint32_t>(f)) : 0u;
}

// R: rows a warp takes (8 for 8-token pages, else 16).  Lane l holds elements
// 8 (l mod 16) .. + 7 of rows 2 i + l / 16.
template <int R, bool ROPE>
__global__ void __launch_bounds__(kQThreads) rlk_qcache_write_kernel(const __grid_constant__ QCacheParams p) {
  __shared__ uint32_t s_max[kQWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ps = p.c.page_size, hkv = p.c.hkv;
  const int wpu = ps / R;  // warps per unit: a power of two up to 8
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kQWarps + warp;
  const QUnit un = q_unit(p, gw / wpu);
  const int part = static_cast<int>(gw % wpu);
  const int c8 = lane & 15, sub = lane >> 4;
  const uint16_t* in = un.is_v ? p.v_in : p.k_in;
  uint4 x[R / 2];
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    const int slot = part * R + 2 * i + sub;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (un.valid && slot >= un.slot0 && slot < un.slot1)
      x[i] = __ldcs(reinterpret_cast<const uint4*>(in + ((un.row0 + slot - un.slot0) * hkv + un.head) * kHeadDim) + c8);
  }
  int page = -1;
  if (un.valid) page = __ldg(p.c.page_table + un.entry);
  const bool page_ok = page >= 0 && page < p.c.n_pages;
  float* scale_at = (un.is_v ? p.c.v_scale : p.c.k_scale) + (static_cast<int64_t>(page) * hkv + un.head);
  const bool had = page_ok && un.slot0 > 0;  // tokens an earlier call wrote
  uint32_t old_bits = 0;
  if (had) old_bits = __float_as_uint(*scale_at);
  if (ROPE && !un.is_v) {
    // the canonical rotation of the rows at their positions; the pair of
    // element 8 c + e is held by lane l xor 8
#pragma unroll
    for (int i = 0; i < R / 2; ++i) {
      const int slot = part * R + 2 * i + sub;
      uint4 o;
      o.x = __shfl_xor_sync(0xffffffffu, x[i].x, 8);
      o.y = __shfl_xor_sync(0xffffffffu, x[i].y, 8);
      o.z = __shfl_xor_sync(0xffffffffu, x[i].z, 8);
      o.w = __shfl_xor_sync(0xffffffffu, x[i].w, 8);
      if (un.valid && slot >= un.slot0 && slot < un.slot1) {
        const float4* t =
            reinterpret_cast<const float4*>(p.rope_table + static_cast<int64_t>(un.pos_slot0 + slot) * kHeadDim);
        const int j = c8 & 7;
        const float4 ca = __ldg(t + 2 * j), cb = __ldg(t + 2 * j + 1);
        const float4 sa = __ldg(t + 16 + 2 * j), sb = __ldg(t + 16 + 2 * j + 1);
        const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
        const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
        uint4 a = c8 < 8 ? x[i] : o, b = c8 < 8 ? o : x[i];
        rope_words8(a, b, c, s);
        x[i] = c8 < 8 ? a : b;
      }
    }
  }
  // 4 significant bits, and the largest magnitude (bit patterns order as the
  // magnitudes do)
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    mx = umax2(mx, umax2(umax2(round4_pair(x[i].x), round4_pair(x[i].y)),
                         umax2(round4_pair(x[i].z), round4_pair(x[i].w))));
  }
  mx = max(mx & 0xFFFFu, mx >> 16);
  // rare: a non-finite or overflowing value, or (where e may be at its lower
  // bound) values next to the smallest normal: settle each element
  const bool rare = mx >= 0x7F80u || mx < static_cast<uint32_t>((kQEsMin + 1) << 7);
  if (rare) {
    mx = 0;
#pragma unroll
    for (int i = 0; i < R / 2; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t r = fix_pair(w[k], round4_pair(w[k]));
        const uint32_t lo = r & 0xFFFFu, hi = r >> 16;
        if (lo < 0x7F80u) mx = max(mx, lo);
        if (hi < 0x7F80u) mx = max(mx, hi);
      }
    }
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (wpu > 1) {
    if (lane == 0) s_max[warp] = mx;
    __syncthreads();
    for (int i = 0; i < wpu; ++i) mx = max(mx, s_max[(warp / wpu) * wpu + i]);
  }
  if (!un.valid) return;
  if (!page_ok) {
    if (lane == 0 && part == 0) report_error(p.err, kErrBadPage, 0xa01);
    return;
  }
  int es = max(static_cast<int>(mx >> 7), kQEsMin);
  const int es_old = static_cast<int>((old_bits >> 23) & 0xFFu) + 7;
  if (had) es = max(es, min(es_old, 254));
  uint8_t* codes = (un.is_v ? p.c.v : p.c.k) + (static_cast<int64_t>(page) * hkv + un.head) * ps * kHeadDim;
  if (had && es > es_old) {
    // earlier tokens of the page: their codes under the larger scale
    for (int slot = part * R + sub; slot < min((part + 1) * R, un.slot0); slot += 2) {
      uint2* at = reinterpret_cast<uint2*>(codes + slot * kHeadDim) + c8;
      uint2 v = *at;
      uint32_t w[2] = {v.x, v.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t r = 0;
#pragma unroll
        for (int b = 0; b < 32; b += 8) r |= rescale_byte((w[k] >> b) & 0xFFu, es - es_old) << b;
        w[k] = r;
      }
      *at = make_uint2(w[0], w[1]);
    }
  }
  const uint32_t floor1 = static_cast<uint32_t>((es - 14) << 3) + 7u;
  const uint32_t floor2 = floor1 | (floor1 << 16);
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    const int slot = part * R + 2 * i + sub;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t e[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t r = round4_pair(w[k]);
      if (rare) r = fix_pair(w[k], r);
      e[k] = encode_pair(w[k], r, floor2);
      if (rare) {
        // non-finite: the NaN code
        if ((r & 0xFFFFu) == 0x7FF0u) e[k] = (e[k] & 0xFFFF0000u) | 0x7Fu;
        if ((r >> 16) == 0x7FF0u) e[k] = (e[k] & 0xFFFFu) | 0x7F0000u;
      }
    }
    if (slot >= un.slot0 && slot < un.slot1)
      reinterpret_cast<uint2*>(codes + slot * kHeadDim)[c8] =
          make_uint2(__byte_perm(e[0], e[1], 0x6420), __byte_perm(e[2], e[3], 0x6420));
  }
  if (lane == 0 && part == 0) *scale_at = __uint_as_float(static_cast<uint32_t>(es - 7) << 23);
}

// The BF16 value of code byte b of word w under scale: the byte's magnitude
// placed as the exponent and mantissa of an FP32 number is the E4M3 value
// times 2^-120 (E4M3 subnormals land on FP32 normals and subnormals alike).
__device__ __forceinline__ float code_value(uint32_t w, int b, float scale) {
  const uint32_t m = b >= 3 ? (w >> 4) : (b == 2 ? w << 4 : (b == 1 ? w << 12 : w << 20));
  const uint32_t sg = b >= 3 ? w : (b == 2 ? w << 8 : (b == 1 ? w << 16 : w << 24));
  const float f = __uint_as_float((m & 0x07F00000u) | (sg & 0x80000000u));
  return __fmul_rn(__fmul_rn(f, 0x1p120f), scale);
}
__device__ __forceinline__ float nan_if(uint32_t w, int b, float v) {
  return ((w >> (8 * b)) & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : v;
}

template <int R>
__global__ void __launch_bounds__(kQThreads) rlk_qcache_read_kernel(const __grid_constant__ QCacheParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ps = p.c.page_size, hkv = p.c.hkv;
  const int wpu = ps / R;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kQWarps + warp;
  const QUnit un = q_unit(p, gw / wpu);
  if (!un.valid) return;
  const int part = static_cast<int>(gw % wpu);
  const int c8 = lane & 15, sub = lane >> 4;
  const int page = __ldg(p.c.page_table + un.entry);
  const bool page_ok = page >= 0 && page < p.c.n_pages;
  if (!page_ok && lane == 0 && part == 0) report_error(p.err, kErrBadPage, 0xa02);
  const int64_t ph = static_cast<int64_t>(page) * hkv + un.head;
  const uint8_t* codes = (un.is_v ? p.c.v : p.c.k) + ph * ps * kHeadDim;
  uint2 x[R / 2];
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    const int slot = part * R + 2 * i + sub;
    x[i] = make_uint2(0u, 0u);
    if (page_ok && slot >= un.slot0 && slot < un.slot1)
      x[i] = __ldcs(reinterpret_cast<const uint2*>(codes + slot * kHeadDim) + c8);
  }
  const float scale = page_ok ? __ldg((un.is_v ? p.c.v_scale : p.c.k_scale) + ph) : 1.0f;
  uint16_t* out = un.is_v ? p.v_out : p.k_out;
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    const int slot = part * R + 2 * i + sub;
    const uint32_t w[2] = {x[i].x, x[i].y};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float f[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) f[b] = code_value(w[k], b, scale);
      if (((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) {
#pragma unroll
        for (int b = 0; b < 4; ++b) f[b] = nan_if(w[k], b, f[b]);
      }
      o[2 * k] = pack_bf16x2(f[0], f[1]);
      o[2 * k + 1] = pack_bf16x2(f[2], f[3]);
    }
    if (slot >= un.slot0 && slot < un.slot1)
      __stcs(reinterpret_cast<uint4*>(out + ((un.row0 + slot - un.slot0) * hkv + un.head) * kHeadDim) + c8,
             make_uint4(o[0], o[1], o[2], o[3]));
  }
}

// blocks of kQWarps warps over every (page, K or V, head, part) of the call
int64_t q_blocks(const QCacheParams& p, int rows) {
  const int64_t warps = static_cast<int64_t>(p.page0[p.num_seqs]) * 2 * p.c.hkv * (p.c.page_size / rows);
  return (warps + kQWarps - 1) / kQWarps;
}

}  // namespace

cudaError_t launch_qcache_write(const QCacheParams& p, cudaStream_t stream) {
  const int rows = std::min(p.c.page_size, 16);
  const unsigned blocks = static_cast<unsigned>(q_blocks(p, rows));
  if (p.rope_table) {
    if (rows == 8) rlk_qcache_write_kernel<8, true><<<blocks, kQThreads, 0, stream>>>(p);
    else rlk_qcache_write_kernel<16, true><<<blocks, kQThreads, 0, stream>>>(p);
  } else {
    if (rows == 8) rlk_qcache_write_kernel<8, false><<<blocks, kQThreads, 0, stream>>>(p);
    else rlk_qcache_write_kernel<16, false><<<blocks, kQThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_qcache_read(const QCacheParams& p, cudaStream_t stream) {
  const int rows = std::min(p.c.page_size, 16);
  const unsigned blocks = static_cast<unsigned>(q_blocks(p, rows));
  if (rows == 8) rlk_qcache_read_kernel<8><<<blocks, kQThreads, 0, stream>>>(p);
  else rlk_qcache_read_kernel<16><<<blocks, kQThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace rlk
