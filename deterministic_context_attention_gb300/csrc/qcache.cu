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
// What it costs: values below max * 2^-13 become 0, where the largest ones are
// off by up to 2^-4 of themselves.
//
// Both passes move 3 bytes per element (2 BF16, 1 code) and are bound by
// HBM; what could bind the write instead is the integer pipe (half the rate of
// the FP32 one), so its steps are packed: a maximum per pair of elements, three
// integer steps per pair for the flush, a multiply per element and the
// hardware's conversion.  A unit of work is one
// (page, head) of K or of V: a warp takes up to 16 of its rows, 16 bytes of
// BF16 a lane, all loads in flight before the first use; neighbouring warps
// take neighbouring heads, whose rows are contiguous in the packed tensors.
// Measured (GB300, 6.79 TB/s copy rate): 158,491 tokens of 8 heads, 16-token
// pages, written or read in 145 us, 0.99 of that rate; 125,558 of 4 heads,
// 64-token pages, written in 61.7 us (0.92); one token each of 64 sequences 4 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "numerics.cuh"
#include "ptx.cuh"
#include "qcache_internal.h"

namespace rlk {
namespace {

// A CTA: 8 warps for 128-token pages, whose (page, head)s take them all, else 4
// (writing 64-token pages: 63.4 us with 8, of which a unit waits for the unit
// beside it too, 61.7 with 4).
constexpr int kQThreads = 256;
constexpr int kQWarps = kQThreads / 32;
int q_warps(int page_size) { return page_size > 64 ? 8 : 4; }
constexpr int kQEsMin = 14;  // the biased exponent of the smallest block maximum that sets a scale (e = -120)

// One unit: head `head` of a page (of K or V) and its slots [slot0, slot1),
// which hold the packed rows row0 + slot - slot0; `part` is the warp's run of
// R slots of it.
struct QUnit {
  bool valid;
  bool is_v;
  int head, slot0, slot1, part;
  int64_t row0;   // packed row of slot slot0
  int64_t entry;  // page-table entry
  int pos_slot0;  // position of slot 0's token
};
template <int R>
__device__ __forceinline__ QUnit q_unit(const QCacheParams& p, int warp) {
  QUnit r;
  const int hkv = p.c.hkv, ps = p.c.page_size;
  const int lw = __clz(R) - __clz(ps);  // log2 of the warps of a unit (1 .. 8)
  const unsigned u = blockIdx.x * (blockDim.x >> 5 >> lw) + (warp >> lw);
  r.part = warp & ((1 << lw) - 1);
  const unsigned pk = u / hkv;
  r.head = static_cast<int>(u - pk * hkv);
  r.is_v = pk & 1;
  const int pg = static_cast<int>(pk >> 1);
  r.valid = pg < p.page0[p.num_seqs];
  // the sequence of the touched page: the last s with page0[s] <= pg
  int lo = 0, hi = p.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.page0[mid] <= pg) lo = mid;
    else hi = mid - 1;
  }
  const int lps = 31 - __clz(ps);
  const int pos0 = p.pos0[lo], n = p.cu[lo + 1] - p.cu[lo];
  const int logical = (pos0 >> lps) + (pg - p.page0[lo]);
  r.pos_slot0 = logical << lps;
  r.slot0 = max(pos0 - r.pos_slot0, 0);
  r.slot1 = min(ps, pos0 + n - r.pos_slot0);
  r.row0 = static_cast<int64_t>(p.cu[lo]) + (r.pos_slot0 + r.slot0 - pos0);
  r.entry = static_cast<int64_t>(lo) * p.c.max_pages + logical;
  return r;
}

// The larger magnitude of each half of two packed BF16 words, NaN if either
// is one (the sign bits are of no use).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A BF16 magnitude rounded to 3 mantissa bits (nearest, ties to even).
__device__ __forceinline__ uint32_t round4(uint32_t m) { return (m + 7u + ((m >> 4) & 1u)) & 0xFFF0u; }

// Eight elements among which there may be what the packed steps do not take:
// Inf and NaN (which become 0 here, a bit of `nan` each, and set no scale),
// magnitudes that would round past the largest one (held at 1.875 * 2^127)
// and subnormals (0).  mx: the largest magnitude of the result.  Out of line:
// hardly any warp runs it.
struct Settled {
  uint4 x;
  uint32_t mx, nan;
};
__device__ __noinline__ Settled settle(uint4 x) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  Settled r;
  r.mx = r.nan = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int sh = 16 * (k & 1);
    uint32_t h = (w[k >> 1] >> sh) & 0xFFFFu;
    const uint32_t m = h & 0x7FFFu;
    if (m >= 0x7F80u) {
      r.nan |= 1u << k;
      h = 0;
    } else if (m >= 0x7F78u) {
      h = (h & 0x8000u) | 0x7F70u;
    } else if (m < 0x0080u) {
      h = 0;
    }
    r.mx = max(r.mx, h & 0x7FFFu);
    w[k >> 1] = (w[k >> 1] & (0xFFFF0000u >> sh)) | (h << sh);
  }
  r.x = make_uint4(w[0], w[1], w[2], w[3]);
  return r;
}

// Codes of four elements (two packed BF16 words).  above2: 0x8000 less the
// smallest magnitude that does not become 0, in both halves -- that is 31/32 of
// the smallest normal code's value, which 4 significant bits round up to it.
// Past the flush the hardware's rounding to E4M3 is the one to 4 bits (it
// rounds [31/32, 1) of the smallest normal number to that number too).
__device__ __forceinline__ uint32_t encode4(uint32_t w0, uint32_t w1, uint32_t above2, float inv_scale) {
  const uint32_t w[2] = {w0, w1};
  uint32_t c[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t keep;  // each half's bit 15 of the sum, 16 times
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(keep) : "r"((w[k] & 0x7FFF7FFFu) + above2));
    const uint32_t v = w[k] & keep;
    const float lo = __fmul_rn(bf16_lo_as_f32(v), inv_scale), hi = __fmul_rn(bf16_hi_as_f32(v), inv_scale);
    uint16_t e;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e) : "f"(hi), "f"(lo));
    c[k] = e;
  }
  return c[0] | (c[1] << 16);
}

// An existing code under a scale 2^d times larger (d >= 0).
__device__ __forceinline__ uint32_t rescale_byte(uint32_t c, int d) {
  const int m = static_cast<int>(c & 0x7Fu);
  if (m == 0x7F) return c;
  const int f = m - 8 * d;
  return f >= 8 ? ((c & 0x80u) | static_cast<uint32_t>(f)) : 0u;
}

// R: rows a warp takes (8 for 8-token pages, else 16).  Lane l holds elements
// 8 j .. 8 j + 7 and 64 + 8 j .. (j = l mod 8; the RoPE pairs of one another) of
// rows 4 i + l / 8.
// Registers are held to 64 (R = 16), 48 and 40 (R = 8 with and without RoPE):
// the fewer, the more loads in flight, and the 16 to 32 bytes a thread that spill
// at these counts cost less than that gives.  104,000 tokens of 8 heads: with
// RoPE 113.9 us (120.0 with 80 registers, 127 with 89), 8-token pages 106.5 (114.7
// with 60, 146.7 with 32) and with RoPE 124.6 (137 with 71).
// With RoPE a warp waits for its rows and then, row group by row group, for its
// rows of the table: chunks of 333 to 2048 tokens of 5 sequences take 11 to 12 us
// for 39 MB, with 48 % of the issue slots used, 28 % of DRAM and 1.24 waves.
template <int R, bool ROPE>
__global__ void __launch_bounds__(kQThreads, R == 16 ? 4 : (ROPE ? 5 : 6))
    rlk_qcache_write_kernel(const __grid_constant__ QCacheParams p) {
  __shared__ uint32_t s_max[kQWarps];
  constexpr int I = R / 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ps = p.c.page_size, hkv = p.c.hkv;
  const QUnit un = q_unit<R>(p, warp);
  const int j = lane & 7, sub = lane >> 3;
  // the warp's slots that are written, this lane's first (i = 0), and the i
  // that have any (the same for the whole warp)
  const int s_lo = un.valid ? max(un.slot0, un.part * R) : 0;
  const int s_hi = un.valid ? min(un.slot1, un.part * R + R) : 0;
  const int slot_a = un.part * R + sub;
  const int i_lo = (s_lo - un.part * R) >> 2, i_hi = (s_hi - un.part * R + 3) >> 2;
  const uint16_t* in = (un.is_v ? p.v_in : p.k_in) + ((un.row0 + slot_a - un.slot0) * hkv + un.head) * kHeadDim;
  uint4 xa[I], xb[I];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int slot = slot_a + 4 * i;
    xa[i] = xb[i] = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= s_lo && slot < s_hi) {
      const uint4* row = reinterpret_cast<const uint4*>(in + static_cast<int64_t>(4 * i) * hkv * kHeadDim) + j;
      xa[i] = __ldcs(row);
      xb[i] = __ldcs(row + 8);
    }
  }
  int page = -1;
  if (un.valid) page = __ldg(p.c.page_table + un.entry);
  const bool page_ok = page >= 0 && page < p.c.n_pages;
  float* scale_at = (un.is_v ? p.c.v_scale : p.c.k_scale) + (static_cast<int64_t>(page) * hkv + un.head);
  const bool had = page_ok && un.slot0 > 0;  // tokens an earlier call wrote
  uint32_t old_bits = 0;
  if (had) old_bits = __float_as_uint(*scale_at);
  if (ROPE && !un.is_v) {
    // the canonical rotation of the rows at their positions
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int slot = slot_a + 4 * i;
      if (slot >= s_lo && slot < s_hi) {
        const float4* t =
            reinterpret_cast<const float4*>(p.rope_table + static_cast<int64_t>(un.pos_slot0 + slot) * kHeadDim);
        const float4 ca = __ldg(t + 2 * j), cb = __ldg(t + 2 * j + 1);
        const float4 sa = __ldg(t + 16 + 2 * j), sb = __ldg(t + 16 + 2 * j + 1);
        const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
        const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
        rope_words8(xa[i], xb[i], c, s);
      }
    }
  }
  // the largest magnitude (bit patterns order as the magnitudes do, and
  // rounding keeps their order, so it is rounded alone)
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    mx = max_abs2(mx, max_abs2(max_abs2(xa[i].x, xa[i].y), max_abs2(xa[i].z, xa[i].w)));
    mx = max_abs2(mx, max_abs2(max_abs2(xb[i].x, xb[i].y), max_abs2(xb[i].z, xb[i].w)));
  }
  mx &= 0x7FFF7FFFu;
  mx = max(mx & 0xFFFFu, mx >> 16);
  uint64_t nan = 0;  // bit 16 i + e: element e (of xa, then xb) of row i is Inf or NaN
  if (mx >= 0x7F78u || (mx > 0 && round4(mx) < static_cast<uint32_t>((kQEsMin + 1) << 7))) {
    mx = 0;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const Settled ra = settle(xa[i]), rb = settle(xb[i]);
      xa[i] = ra.x;
      xb[i] = rb.x;
      mx = max(mx, max(ra.mx, rb.mx));
      nan |= static_cast<uint64_t>(ra.nan | (rb.nan << 8)) << (16 * i);
    }
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (ps > R) {
    if (lane == 0) s_max[warp] = mx;
    __syncthreads();
    const int wpu = ps / R;
    for (int i = 0; i < wpu; ++i) mx = max(mx, s_max[(warp & ~(wpu - 1)) + i]);
  }
  if (!un.valid) return;
  if (!page_ok) {
    if (lane == 0 && un.part == 0) report_error(p.err, kErrBadPage, 0xa01);
    return;
  }
  int es = max(static_cast<int>(round4(mx) >> 7), kQEsMin);
  const int es_old = static_cast<int>((old_bits >> 23) & 0xFFu) + 7;
  if (had) es = max(es, min(es_old, 254));
  uint8_t* codes = (un.is_v ? p.c.v : p.c.k) + (static_cast<int64_t>(page) * hkv + un.head) * ps * kHeadDim + j * 8;
  if (had && es > es_old) {
    // earlier tokens of the page: their codes under the larger scale
#pragma unroll 1
    for (int at = 2 * slot_a; at < 2 * min((un.part + 1) * R, un.slot0); at += (at & 1) ? 7 : 1) {
      uint2* half = reinterpret_cast<uint2*>(codes + (at >> 1) * kHeadDim + (at & 1) * 64);
      const uint2 v = *half;
      uint32_t w[2] = {v.x, v.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t r = 0;
#pragma unroll
        for (int b = 0; b < 32; b += 8) r |= rescale_byte((w[k] >> b) & 0xFFu, es - es_old) << b;
        w[k] = r;
      }
      *half = make_uint2(w[0], w[1]);
    }
  }
  const uint32_t above1 = 0x8000u - ((static_cast<uint32_t>(es - 14) << 7) | 0x78u);
  const uint32_t above2 = above1 | (above1 << 16);
  const float inv_scale = __uint_as_float(static_cast<uint32_t>(261 - es) << 23);  // 2^(134 - es)
#pragma unroll
  for (int i = 0; i < I; ++i) {
    if (i < i_lo || i >= i_hi) continue;
    const int slot = slot_a + 4 * i;
    const uint2 ea = make_uint2(encode4(xa[i].x, xa[i].y, above2, inv_scale),
                                encode4(xa[i].z, xa[i].w, above2, inv_scale));
    const uint2 eb = make_uint2(encode4(xb[i].x, xb[i].y, above2, inv_scale),
                                encode4(xb[i].z, xb[i].w, above2, inv_scale));
    if (slot >= s_lo && slot < s_hi) {
      uint2* row = reinterpret_cast<uint2*>(codes + slot * kHeadDim);
      row[0] = ea;
      row[8] = eb;
    }
  }
  while (nan) {
    const int b = __ffsll(static_cast<long long>(nan)) - 1;
    nan &= nan - 1;
    codes[(slot_a + 4 * (b >> 4)) * kHeadDim + ((b >> 3) & 1) * 64 + (b & 7)] = 0x7F;
  }
  if (lane == 0 && un.part == 0) *scale_at = __uint_as_float(static_cast<uint32_t>(es - 7) << 23);
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
  const QUnit un = q_unit<R>(p, warp);
  if (!un.valid) return;
  const int part = un.part;
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

// CTAs over every (page, K or V, head, part) of the call
unsigned q_blocks(const QCacheParams& p, int rows) {
  const int64_t warps = static_cast<int64_t>(p.page0[p.num_seqs]) * 2 * p.c.hkv * (p.c.page_size / rows);
  const int per = q_warps(p.c.page_size);
  return static_cast<unsigned>((warps + per - 1) / per);
}

}  // namespace

cudaError_t launch_qcache_write(const QCacheParams& p, cudaStream_t stream) {
  const int rows = std::min(p.c.page_size, 16);
  const unsigned blocks = q_blocks(p, rows), threads = 32 * q_warps(p.c.page_size);
  if (p.rope_table) {
    if (rows == 8) rlk_qcache_write_kernel<8, true><<<blocks, threads, 0, stream>>>(p);
    else rlk_qcache_write_kernel<16, true><<<blocks, threads, 0, stream>>>(p);
  } else {
    if (rows == 8) rlk_qcache_write_kernel<8, false><<<blocks, threads, 0, stream>>>(p);
    else rlk_qcache_write_kernel<16, false><<<blocks, threads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_qcache_read(const QCacheParams& p, cudaStream_t stream) {
  const int rows = std::min(p.c.page_size, 16);
  const unsigned blocks = q_blocks(p, rows), threads = 32 * q_warps(p.c.page_size);
  if (rows == 8) rlk_qcache_read_kernel<8><<<blocks, threads, 0, stream>>>(p);
  else rlk_qcache_read_kernel<16><<<blocks, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace rlk
