// qdecode.cu -- paged decode over the 8-bit KV cache for sm_103a.
//
// A transposed decode (keys, then head dimensions, on the MMA's M side) over
// the pages' E4M3 codes as they are: TMA brings them to shared memory and
// tcgen05.mma kind::f8f6f4 reads them there, so no code is ever converted.
// The other operand is split into E4M3 pieces, each 2^5 below the one before
// (a rounding to 4 bits of a value in [2^E, 2^(E+1)) leaves at most 2^(E-4),
// which times 32 fills the same range again), which ride in the N columns the
// few query heads leave free:
//   S^T = K_b [q0 | q1 | q2]^T        q 2^x = q0 + q1 / 32 + q2 / 1024
//   O^T = V_b^T [p0 | p1 | p2 | p3]^T  w 2^8 = p0 + p1 / 32 + p2 / 1024 + p3 / 32768
// q 2^x has its row maximum in [128, 256): a BF16 query's 8 significant bits
// are q0 + q1 / 32 exactly, q2 serves elements 2^13 and more below the row's
// maximum.  w_c = p_c sv_c / A, with sv_c the V scale of key c's page and A
// (a power of two) the largest p sv of the block and query head, so that w <= 1
// and a page that a head does not attend to takes no bits from the others.
// What the pieces leave: 2^-19 of w_c down to w = 2^-14, from there (the last
// piece's smallest step) at most 2^-33 of A, 2^-32 of the largest p sv (2^-31
// where scales are no powers of two).  The K scale multiplies the FP32 score of
// its key,
//   s_c = (q . code_c) sk_c.
//
// Softmax, all in FP32.  A block b of 128 keys gives m_b = max s, p = 2^((s -
// m_b) c), l_b = sum p and O_b = sum p v, with c = scale log2(e).  Blocks are
// folded left to right into the segment (kSegBlocks blocks, a fixed cut of the
// sequence) they lie in, and segments left to right into the sequence, both by
//   M = max(m, m'),  O = O' 2^((m' - M) c) + O 2^((m - M) c),  l likewise.
// Maxima stay unscaled and scores are subtracted before they are scaled: the
// largest key's p is exactly 1 and no p is above it, however large the scores
// (p = 2^(s c - rn(m c)) is off by half a last place of m c, a factor of 2 and
// more from 2^24 on, which the sums below do not hold).  The arithmetic is the
// same whichever CTAs take which segments: a result depends on the cached codes,
// scales and the query alone, not on the batch, the order of the pages or the
// split.  (Two levels, because the fold is a
// chain: one over every block of a 32768-token sequence, on states written
// out per block, took 125 us for 4 sequences where the pages take 40.)
//
// Work split.  Neighbouring CTAs take neighbouring KV heads of the same keys
// side by side (a group: all 8 heads of 8, as many as divide the SMs), because
// the heads' pages lie next to each other: 64 sequences of 512 .. 32768 tokens
// in 16-token pages took 341 us with one head's line of pages a CTA, 333 with
// the groups.  The blocks of all (sequence, head group) pairs in order form one
// line; each group takes an equal part of it by cost (a pair counts 1.5 blocks
// more than it has), cut at segment ends, so that with split_k = 0 the SMs'
// loads differ by about a segment, or by up to a pair where pairs are of one or
// two segments (which are not cut: counting and folding the parts costs more
// than it evens out).  A CTA that holds a whole pair writes its output;
// otherwise a pair's first piece leaves what it has folded as one state, the
// others the state of each segment, in the workspace, and the CTA that counts
// the last segment of a pair (which one changes nothing in the result) folds
// them.  (With a state per segment from the first piece too, 64 sequences of
// 512 .. 32768 tokens took 348 us instead of 342.)
//
// What bounds it: HBM, 32 KB of codes per (KV head, 128-key block), 0.73 us a
// block and SM at the measured copy rate; long sequences in 16-token pages and
// larger run at that (0.69 .. 0.73 us), 8-token pages at 0.9 (32 TMA copies a
// block: their issue).  Fed from L2 the pipeline takes 0.57 us a block with 4
// query heads in 64-token pages, 0.66 in 16-token ones, 0.75 with 8 heads (0.19
// more while the warp that issues the O products also fetched the scales).  Per
// block the tensor core issues 4 + 4 MMAs of K = 32 codes (the BF16 decode needs
// 8 + 16), and the softmax's 8 warps run two blocks at a time.  A call costs
// about 5 us before its first block is folded and, where pairs are cut, 3 to 6 us
// for counting and folding: 64 sequences of 512 .. 32768 tokens take 331 .. 336 us
// (0.96 .. 0.98 of the copy rate), 4 of 32768 tokens 56 (0.71).
//
// Warp roles (512 threads):
//   warps 0-3   correction / epilogue: thread d owns head dimension d
//   warps 4-7   softmax of the even blocks, warps 8-11 of the odd ones:
//               thread t owns key t of the block
//   warp  12    producer of the K pages (TMA) and of both scales (cp.async: it
//               runs ahead of the softmax, the V ring follows it)
//   warp  13    producer of the V pages; loads the query rows, rotates them
//               where asked and splits them, a piece of work ahead
//   warp  14    the S^T products, warp 15 the O^T products
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "numerics.cuh"
#include "ptx.cuh"
#include "qcache_internal.h"
#include "segments.cuh"

namespace rlk {
namespace {

constexpr int kQDThreads = 512;
constexpr int kQPieces = 3, kPPieces = 4;

// MG: query heads per KV head.  N: MMA columns, their pieces (of Q at column
// piece * MG + head, of P at p_col)
template <int MG>
struct QDecLayout {
  static constexpr int B = 128;           // keys per block
  static constexpr int N = MG <= 4 ? 16 : 32;
  static_assert(kPPieces * MG <= N && kQPieces * MG <= N, "the pieces fit the MMA's columns");
  static constexpr int kSK = 6, kSV = 5;  // K and V rings
  static constexpr int kPS = 2;           // P^T operand slots
  static constexpr int kQS = 2;           // query slots (the next item's rows are prepared ahead)
  static constexpr int kSS = 4, kOS = 4;  // TMEM rings of S^T and O^T
  // statistics ring: block s is written once P slot s - 2 is free, so O slot
  // s - 6 and the statistics beside it have been read; 8 where memory allows
  // (a power of two)
  static constexpr int kSR = MG < 8 ? 8 : 6;
  static_assert(kSR >= kPS + kOS, "statistics ring");
  // scales ring: fetched with the K codes, in groups of up to 4 blocks; the
  // softmax reads a block's scales before it frees the block's S slot
  static constexpr int kScRing = 16;
  static_assert(kScRing >= kSK + kSS + 4, "scales ring");
  static constexpr int kKVBytes = B * 128;
  static constexpr int kTBytes = N * 128;  // an operand tile: N x 128 codes
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + kQS * kTBytes;
  static constexpr int kKOff = (kPOff + kPS * kTBytes + 1023) / 1024 * 1024;
  static constexpr int kVOff = kKOff + kSK * kKVBytes;
  // per softmax group, double-buffered by block: float [s, log2 of p sv][MG
  // heads][4 warps] maxima
  static constexpr int kRedBytes = 2 * 2 * MG * 16;
  static constexpr int kRedOff = kVOff + kSV * kKVBytes;
  // per block: uint32 l[MG][4 warps], then float m[MG] and the V factors [MG]
  static constexpr int kStatWords = (6 * MG + 3) / 4 * 4;
  static constexpr int kStatsOff = kRedOff + 2 * kRedBytes;
  static constexpr int kQsOff = kStatsOff + kSR * kStatWords * 4;  // float [kQS][MG]
  static constexpr int kBarOff = (kQsOff + kQS * MG * 4 + 7) / 8 * 8;
  static constexpr int kQFull = 0, kQEmpty = kQFull + kQS, kKFull = kQEmpty + kQS, kKEmpty = kKFull + kSK,
                       kVFull = kKEmpty + kSK, kVEmpty = kVFull + kSV, kSFull = kVEmpty + kSV,
                       kSEmpty = kSFull + kSS, kPFull = kSEmpty + kSS, kPEmpty = kPFull + kPS,
                       kOFull = kPEmpty + kPS, kOEmpty = kOFull + kOS, kStatsFull = kOEmpty + kOS,
                       kSyncMax = kStatsFull + kSR, kStored = kSyncMax + 4, kCounted = kStored + 1,
                       kEndCounted = kCounted + 1, kScales = kEndCounted + 1, kNumBars = kScales + kScRing;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // tmem base (u32), abort (i32)
  // pairs to fold: int4 {seq, g, first state, states} [2]
  static constexpr int kCutOff = (kMiscOff + 16 + 15) / 16 * 16;
  static constexpr int kScOff = kCutOff + 2 * 16;  // float [K, V][kScRing][16 pages]
  static constexpr int kRowOff = kScOff + 2 * kScRing * 16 * 4;  // staged query rows and RoPE table row
  static constexpr int kRowBytes = MG * 256 + 512;
  static constexpr int kFoldGroups = N == 16 ? 4 : 3;  // per correction warp: segment states being folded
  static constexpr int kEndGroups = 7;  // per correction and softmax warp, in the K and V rings
  static_assert(12 * kEndGroups * 4 * 512 <= (kSK + kSV) * kKVBytes, "the rings hold them");
  static constexpr int kFoldOff = kRowOff + kQS * kRowBytes;
  static constexpr int kTotal = kFoldOff + 4 * kFoldGroups * 4 * 512;
  static constexpr int kAlloc = kTotal + 1024;
  static constexpr int kTmemCols = N * (kSS + kOS);
  static_assert(kAlloc <= 232448, "decode shared memory");
  static_assert(kTmemCols == 128 || kTmemCols == 256, "TMEM columns are allocated in powers of two");
};

// Byte offset of (row, code column) of a K-major operand tile of 128-byte rows
// in the 128-byte swizzle (what a TMA load with that swizzle produces).
__device__ __forceinline__ uint32_t tile8_off(int row, int col) {
  return static_cast<uint32_t>(row * 128) + ((static_cast<uint32_t>(col >> 4) ^ static_cast<uint32_t>(row & 7)) << 4) +
         static_cast<uint32_t>(col & 15);
}

// P^T is stored N-major: the N pieces of key t are one run of bytes, which
// the key's thread writes whole, 16 bytes a store.  N = 16: runs of 16 bytes,
// no swizzle; N = 32: runs of 32 bytes in the 32-byte swizzle (its two halves
// swapped for keys with bit 2 set).  The piece k of head q is column
// 8 (q / 2) + 2 k + q mod 2, so that the pairs next_piece makes pack as they
// are.
__host__ __device__ constexpr int p_col(int q, int k) { return 8 * (q >> 1) + 2 * k + (q & 1); }
template <int N>
__device__ __forceinline__ Desc p_desc(uint32_t saddr) {
  // 8 keys are N * 8 bytes apart; no second group along N
  const uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(N * 8 >> 4) << 16) |
                     (static_cast<uint64_t>(N * 8 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
                     (static_cast<uint64_t>(N == 32 ? 6 : 0) << 61);
  return Desc{static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)};
}
template <int N>
__device__ __forceinline__ void p_store(uint8_t* tile, int t, const uint32_t (&w)[N / 4]) {
#pragma unroll
  for (int h = 0; h < N / 16; ++h) {
    const int at = N == 32 ? t * 32 + ((h ^ ((t >> 2) & 1)) << 4) : t * 16;
    *reinterpret_cast<uint4*>(tile + at) = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
  }
}

// Instruction descriptor, kind::f8f6f4 with E4M3 A and B and FP32 accumulation.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// One K = 32 step of D[tmem] (+)= A B^T, both from shared memory.
template <int ACC>
__device__ __forceinline__ void mma8_ss(uint32_t d_tmem, Desc a, uint32_t a_off, Desc b, uint32_t b_off,
                                        uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t.reg .b32 la, lb;\n\t"
      "add.u32 la, %1, %3;\n\tadd.u32 lb, %4, %6;\n\t"
      "mov.b64 da, {la, %2};\n\tmov.b64 db, {lb, %5};\n\t"
      "setp.ne.b32 p, %8, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %7, p;\n\t}" ::"r"(d_tmem),
      "r"(a.lo), "r"(a.hi), "r"(a_off), "r"(b.lo), "r"(b.hi), "r"(b_off), "r"(idesc), "n"(ACC)
      : "memory");
}

__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {  // a in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 e4m3_pair_value(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  float2 f;
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// The next piece of a and b (packed, a low), which keep what it leaves times
// 32 (both steps exact: the residual of a rounding to 4 bits is a multiple of
// the value's last place).
__device__ __forceinline__ uint32_t next_piece(float& a, float& b) {
  const uint32_t c = e4m3_pair(a, b);
  const float2 f = e4m3_pair_value(c);
  a = __fmul_rn(__fsub_rn(a, f.x), 32.0f);
  b = __fmul_rn(__fsub_rn(b, f.y), 32.0f);
  return c;
}

__device__ __forceinline__ float pow2_bits(int biased) { return __uint_as_float(static_cast<uint32_t>(biased) << 23); }

template <int N>
struct TmemRow;
template <>
struct TmemRow<16> {
  static __device__ __forceinline__ void ld(uint32_t a, uint32_t (&r)[16]) { tmem_ld16(a, r); }
};
template <>
struct TmemRow<32> {
  static __device__ __forceinline__ void ld(uint32_t a, uint32_t (&r)[32]) { tmem_ld32(a, r); }
};

__device__ const float g_unit_scale = 1.0f;  // the scale of a page id out of range

// Arrives on bar once this thread's earlier cp.async copies have landed (the
// arrival is one of the barrier's count).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The fold of a cut pair's ns states (the first piece's, then its other
// segments', from segment `seg` of the workspace on), one warp a query head: lane
// l takes head dimensions 4 l .. 4 l + 3.  Groups of 4 segments are copied ahead
// into the warp's ring (a lane reads what it copied itself).  One warp a
// scheduler, so what costs is the chain of dependent steps: for 32 segments at
// a time the running maxima are a scan over the lanes and the factors come out
// side by side (the same values as one after another: a maximum rounds
// nothing), which leaves a multiply and an fma a segment on the chain.
template <int GROUPS>
__device__ __noinline__ void fold_pair(const QDecodeParams& p, int seq, int seg, int ns, int h, int lane,
                                       float4* ring) {
  constexpr int C = 4;
  const int64_t base = static_cast<int64_t>(seg) * p.hq + h;
  const int64_t pitch = static_cast<int64_t>(p.hq) * kHeadDim;
  const float* src = p.state_o + base * kHeadDim + 4 * lane;
  const float2* sml = reinterpret_cast<const float2*>(p.state_ml) + base;
  // past the last segment: m = -inf, a factor of 0
  auto load_ml = [&](int c0) {
    return c0 + lane < ns ? __ldcg(sml + static_cast<int64_t>(c0 + lane) * p.hq) : make_float2(-INFINITY, 0.f);
  };
  int next = 0;  // the next segment to copy
  float4* to = ring + lane;
  auto copy = [&]() {
    if (next < ns) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        if (next + i < ns) cp_async16(to + i * 32, src + i * pitch);
        else to[i * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    cp_async_commit();  // empty groups keep the count uniform
    next += C;
    src += C * pitch;
    to = to + C * 32 == ring + lane + GROUPS * C * 32 ? ring + lane : to + C * 32;
  };
  float2 ml = load_ml(0);
#pragma unroll 1
  for (int c = 0; c < GROUPS; ++c) copy();
  float4 O = make_float4(-0.f, -0.f, -0.f, -0.f);  // the first state as it is, its sign of zero too
  float m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int s0 = 0; s0 < ns; s0 += 32) {
    const float2 ml_next = load_ml(s0 + 32);
    float run = fmaxf(m, ml.x);  // lane i: the maximum up to segment s0 + i
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float o = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run = fmaxf(run, o);
    }
    float before = __shfl_up_sync(0xffffffffu, run, 1);
    if (lane == 0) before = m;
    const float fa = weight(before, run, p.scale_log2), fb = weight(ml.x, run, p.scale_log2);
    m = __shfl_sync(0xffffffffu, run, 31);
#pragma unroll 1
    for (int s = s0; s < min(s0 + 32, ns); s += C) {
      cp_async_wait<GROUPS - 1>();
      float4 v[C];
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = to[i * 32];  // the slot the next copy fills is the oldest one
      copy();
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float a = __shfl_sync(0xffffffffu, fa, s - s0 + i), b = __shfl_sync(0xffffffffu, fb, s - s0 + i);
        const float lb = __shfl_sync(0xffffffffu, ml.y, s - s0 + i);
        O.x = __fmaf_rn(v[i].x, b, __fmul_rn(O.x, a));
        O.y = __fmaf_rn(v[i].y, b, __fmul_rn(O.y, a));
        O.z = __fmaf_rn(v[i].z, b, __fmul_rn(O.z, a));
        O.w = __fmaf_rn(v[i].w, b, __fmul_rn(O.w, a));
        l = __fmaf_rn(lb, b, __fmul_rn(l, a));
      }
    }
    ml = ml_next;
  }
  cp_async_wait<0>();
  const float r = __frcp_rn(l);
  O = make_float4(__fmul_rn(O.x, r), __fmul_rn(O.y, r), __fmul_rn(O.z, r), __fmul_rn(O.w, r));
  const int64_t row = static_cast<int64_t>(seq) * p.hq + h;
  if (p.out_f32) *(reinterpret_cast<float4*>(p.out_f32 + row * kHeadDim) + lane) = O;
  if (p.out_bf16)
    *(reinterpret_cast<uint2*>(p.out_bf16 + row * kHeadDim) + lane) =
        make_uint2(pack_bf16x2(O.x, O.y), pack_bf16x2(O.z, O.w));
  if (p.lse && lane == 0) p.lse[row] = log_sum(m, l, p.scale_log2);
}

template <int MG>
__global__ void __launch_bounds__(kQDThreads, 1)
    rlk_qdecode_kernel(const __grid_constant__ QDecodeParams p, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v) {
  using L = QDecLayout<MG>;
  constexpr int B = L::B, N = L::N, SK = L::kSK, SV = L::kSV, PS = L::kPS, QS = L::kQS, SS = L::kSS, OS = L::kOS,
                SR = L::kSR;
  static_assert(MG <= kDecodeMaxGroup && PS == 2 && QS == 2, "decode layout");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  int4* to_fold = reinterpret_cast<int4*>(smem + L::kCutOff);
  uint32_t* stats = reinterpret_cast<uint32_t*>(smem + L::kStatsOff);
  float* qscale = reinterpret_cast<float*>(smem + L::kQsOff);
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  // query rows of no head's piece are never written: they must read as zero
  for (int i = tid; i < QS * L::kTBytes / 16; i += kQDThreads)
    reinterpret_cast<uint4*>(smem + L::kQOff)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (tid == 0) {
    for (int s = 0; s < QS; ++s) {
      mbar_init(&bars[L::kQFull + s], 1);
      mbar_init(&bars[L::kQEmpty + s], 1 + 8);  // the S products' commit and the softmax warps
    }
    for (int s = 0; s < SK; ++s) {
      mbar_init(&bars[L::kKFull + s], 1);
      mbar_init(&bars[L::kKEmpty + s], 1);
    }
    for (int s = 0; s < SV; ++s) {
      mbar_init(&bars[L::kVFull + s], 1);
      mbar_init(&bars[L::kVEmpty + s], 1);
    }
    for (int s = 0; s < SS; ++s) {
      mbar_init(&bars[L::kSFull + s], 1);
      mbar_init(&bars[L::kSEmpty + s], 4);
    }
    for (int s = 0; s < PS; ++s) {
      mbar_init(&bars[L::kPFull + s], 4);
      mbar_init(&bars[L::kPEmpty + s], 1);
    }
    for (int s = 0; s < OS; ++s) {
      mbar_init(&bars[L::kOFull + s], 1);
      mbar_init(&bars[L::kOEmpty + s], 4);
    }
    for (int s = 0; s < SR; ++s) mbar_init(&bars[L::kStatsFull + s], 4);
    for (int s = 0; s < 4; ++s) mbar_init(&bars[L::kSyncMax + s], 4);
    for (int s = 0; s < L::kScRing; ++s) mbar_init(&bars[L::kScales + s], 32);
    mbar_init(&bars[L::kStored], 4);
    mbar_init(&bars[L::kCounted], 1);
    mbar_init(&bars[L::kEndCounted], 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 14) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm_s = *tmem_slot;       // S^T slots: + N * slot
  const uint32_t tm_o = tm_s + N * SS;    // O^T slots: + N * slot
  uint8_t* q_base = smem + L::kQOff;
  uint8_t* p_base = smem + L::kPOff;
  uint8_t* k_base = smem + L::kKOff;
  uint8_t* v_base = smem + L::kVOff;

  // Folds the pairs whose last segment this CTA has counted.  Once all blocks
  // are done (end), the softmax warps help the correction ones and the K and V
  // rings are free for the copies.
  auto fold_pairs = [&](bool end) {
    __threadfence();
    const int4 c0 = to_fold[0], c1 = to_fold[1];
    const int n0 = c0.w ? MG : 0, n = n0 + (c1.w ? MG : 0);
    for (int i = warp; i < n; i += end ? 12 : 4) {
      const int4 c = i < n0 ? c0 : c1;
      const int h = c.y * MG + (i < n0 ? i : i - n0);
      if (end)
        fold_pair<L::kEndGroups>(p, c.x, c.z, c.w, h, lane,
                                 reinterpret_cast<float4*>(k_base) + warp * L::kEndGroups * 4 * 32);
      else
        fold_pair<L::kFoldGroups>(p, c.x, c.z, c.w, h, lane,
                                  reinterpret_cast<float4*>(smem + L::kFoldOff) + warp * L::kFoldGroups * 4 * 32);
    }
  };

  if (warp == 12 || warp == 13) {
    // ------------------------------------------------------------ producers
    const bool is_v = warp == 13;
    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
    if (lane == 0) tma_prefetch_desc(map);
    const uint32_t leader = elect_one_sync();
    const int S = is_v ? SV : SK;
    uint64_t* full_b = &bars[is_v ? L::kVFull : L::kKFull];
    uint64_t* empty_b = &bars[is_v ? L::kVEmpty : L::kKEmpty];
    uint8_t* ring = is_v ? v_base : k_base;
    const int lps = 31 - __clz(p.page_size), lg = 7 - lps;  // log2 of a page's tokens, of a block's pages
    const int lbox = min(lps, 31 - __clz(kQBoxRows));       // and of a copy's tokens
    // page ids: two groups of blocks ahead, across pieces
    QGroups<QDecodeParams> cur(p, lg), ahead(p, lg);
    int id = ahead.page_id(p, lg, lane);
    ahead.step(p, lg);
    int id1 = ahead.page_id(p, lg, lane);
    ahead.step(p, lg);
    float* scales = reinterpret_cast<float*>(smem + L::kScOff);
    uint32_t stage = 0, par = 1, n = 0;
    bool fail = false;
    // The query rows, by the V warp (whose ring is the slower one to free): of
    // the first piece before its first page, of each later one once the first
    // pages of the piece before it are on their way; the rows and the RoPE
    // table's row land in shared memory a piece earlier still.  Rolled loops: a
    // piece runs this code once, and unrolled it took 3 us, most of it fetching
    // instructions.
    uint8_t* row_stage = smem + L::kRowOff;
    QWalk<QDecodeParams> qwalk(p);
    uint32_t q_it = 0;
    bool q_more = false;
    auto fetch_rows = [&]() {
      QPiece q;
      q_more = qwalk.next(p, &q);
      if (q_more) {
        uint8_t* to = row_stage + (q_it & 1) * L::kRowBytes;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(
            p.q + (static_cast<int64_t>(q.seq) * p.hq + q.g * MG) * kHeadDim);
        for (int i = lane; i < MG * 16; i += 32) cp_async16(to + i * 16, src + i * 16);
        if (p.rope_table)
          cp_async16(to + MG * 256 + lane * 16,
                     p.rope_table + static_cast<int64_t>(q.kv_len - 1) * kHeadDim + lane * 4);
      }
      cp_async_commit();
    };
    auto split_rows = [&]() -> bool {  // of the piece fetch_rows took
      if (!q_more) return true;
      const uint32_t qslot = q_it & 1;
      cp_async_wait<0>();
      __syncwarp();
      if (!wait_warp(&bars[L::kQEmpty + qslot], ((q_it >> 1) & 1) ^ 1, abort, p.err, 0xb31)) return false;
      const uint8_t* rows = row_stage + qslot * L::kRowBytes;
      uint8_t* tile = q_base + qslot * L::kTBytes;
#pragma unroll 1
      for (int i = 0; i < MG; ++i) {
        // lane l: elements 4 l .. 4 l + 3
        const uint2 x = *reinterpret_cast<const uint2*>(rows + i * 256 + lane * 8);
        float v[4] = {bf16_lo_as_f32(x.x), bf16_hi_as_f32(x.x), bf16_lo_as_f32(x.y), bf16_hi_as_f32(x.y)};
        if (p.rope_table) {
          // the pair of element e is e +- 64, 16 lanes away
          const uint2 o = *reinterpret_cast<const uint2*>(rows + i * 256 + (lane ^ 16) * 8);
          const float4 c = *reinterpret_cast<const float4*>(rows + MG * 256 + (lane & 15) * 16);
          const float4 s = *reinterpret_cast<const float4*>(rows + MG * 256 + 256 + (lane & 15) * 16);
          const float w[4] = {bf16_lo_as_f32(o.x), bf16_hi_as_f32(o.x), bf16_lo_as_f32(o.y), bf16_hi_as_f32(o.y)};
          const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y0, y1;
            rope_pair(lane < 16 ? v[e] : w[e], lane < 16 ? w[e] : v[e], cc[e], ss[e], y0, y1);
            v[e] = __uint_as_float(static_cast<uint32_t>(f32_to_bf16_rn(lane < 16 ? y0 : y1)) << 16);
          }
        }
        // the row's largest finite magnitude to [128, 256)
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = fabsf(v[e]);
          if (a <= 3.4028234e38f) m = fmaxf(m, a);
          else v[e] = __uint_as_float(0x7FC00000u);  // Inf and NaN queries give NaN rows
        }
        m = warp_max(m);
        const int up = min(261 - static_cast<int>(__float_as_uint(m) >> 23), 253);
        const float f = pow2_bits(up);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __fmul_rn(v[e], f);
#pragma unroll
        for (int k = 0; k < kQPieces; ++k) {
          const uint32_t lo = next_piece(v[0], v[1]);
          const uint32_t hi = next_piece(v[2], v[3]);
          *reinterpret_cast<uint32_t*>(tile + tile8_off(k * MG + i, 4 * lane)) = lo | (hi << 16);
        }
        if (lane == 0) qscale[qslot * MG + i] = pow2_bits(254 - up);
      }
      fence_proxy_async_smem();
      warp_arrive(&bars[L::kQFull + qslot], lane);
      ++q_it;
      fetch_rows();
      return true;
    };
    if (is_v) {
      fetch_rows();
      fail = !split_rows();
    }
    while (cur.ok && !fail) {
      const int id2 = ahead.page_id(p, lg, lane);
      ahead.step(p, lg);
      // the (page, head) row of the codes; out of range: past the last one,
      // where the copy reads the zero fill
      int row = id * p.hkv + cur.pc.g;
      const bool bad = static_cast<unsigned>(id) >= static_cast<unsigned>(p.n_pages);
      const bool real = lane < cur.n << lg && ((cur.b << lg) + lane) << lps < cur.pc.kv_len;  // a page of the group
      if (bad) row = p.n_pages * p.hkv;
      if (bad && real) report_error(p.err, kErrBadPage, 0xb04);
      for (int i = 0; i < cur.n; ++i) {
        const bool ok = wait_warp(empty_b + stage, par, abort, p.err, is_v ? 0xb03 : 0xb02);
        if (!ok) { fail = true; break; }
        if (!is_v && i == 0) {
          // the group's scales, with its first block's codes: by now the
          // softmax has read those of block n - kSK - kSS, so the ring has room
          if (real) {
            float* to = scales + ((n + (lane >> lg)) % L::kScRing) * 16 + (lane & ((1 << lg) - 1));
            cp_async4(to, bad ? &g_unit_scale : p.k_scale + row);
            cp_async4(to + L::kScRing * 16, bad ? &g_unit_scale : p.v_scale + row);
          }
          for (int k = 0; k < cur.n; ++k) cp_async_arrive(&bars[L::kScales + (n + k) % L::kScRing]);
          n += cur.n;
        }
        uint8_t* dst = ring + stage * L::kKVBytes;
        const int n_box = (min(B, cur.pc.kv_len - (cur.b + i) * B) + (1 << lbox) - 1) >> lbox;
        if (lane == 0) mbar_arrive_expect_tx(full_b + stage, (n_box << lbox) * 128);
        __syncwarp();
        // copies of a page's boxes of up to kQBoxRows tokens (a context's last
        // page is not read past the box it ends in), issued by one lane in a
        // loop the whole warp walks (issued by the lanes that hold the page ids,
        // one lane after another, they took more than a block's time at HBM rate)
#pragma unroll 4
        for (int k = 0; k < n_box; ++k) {
          const int r = __shfl_sync(0xffffffffu, row, (i << lg) + (k << lbox >> lps));
          if (leader)
            tma_load_3d(dst + ((k << lbox) * 128), map, full_b + stage, 0, (k << lbox) & (p.page_size - 1), r);
        }
        if (++stage == static_cast<uint32_t>(S)) {
          stage = 0;
          par ^= 1;
        }
      }
      if (is_v && !fail && cur.b == cur.pc.block0()) fail = !split_rows();
      cur.step(p, lg);
      id = id1;
      id1 = id2;
    }
    cp_async_wait<0>();
  } else if (warp == 14) {
    // ------------------------------------------------------------ S issuer
    constexpr uint32_t kIdS = idesc_e4m3(128, N, false, false);  // A = K (K-major), B = Q pieces (K-major)
    const uint32_t leader = elect_one_sync();
    uint32_t stage = 0, kpar = 0, s_it = 0, q_it = 0;
    QWalk<QDecodeParams> walk(p);
    QPiece pc;
    while (walk.next(p, &pc)) {
      const uint32_t qslot = q_it & 1;
      const bool ok = wait_warp(&bars[L::kQFull + qslot], (q_it >> 1) & 1, abort, p.err, 0xb11);
      if (!ok) break;
      ++q_it;
      const Desc qd = make_desc(smem_u32(q_base + qslot * L::kTBytes), 16, 1024);
      bool fail = false;
      const int b1 = pc.block1();
      for (int b = pc.block0(); b < b1; ++b, ++s_it) {
        const uint32_t slot = s_it % SS;
        bool w = wait_warp(&bars[L::kKFull + stage], kpar, abort, p.err, 0xb12);
        w = w && wait_warp(&bars[L::kSEmpty + slot], ((s_it / SS) & 1) ^ 1, abort, p.err, 0xb13);
        if (!w) { fail = true; break; }
        tc_fence_after();
        const Desc kd = make_desc(smem_u32(k_base + stage * L::kKVBytes), 16, 1024);
        const uint32_t d = tm_s + slot * N;
        if (leader) {
          mma8_ss<0>(d, kd, 0, qd, 0, kIdS);
#pragma unroll
          for (int s = 1; s < kHeadDim / 32; ++s) mma8_ss<1>(d, kd, s * 2, qd, s * 2, kIdS);
          umma_commit(&bars[L::kSFull + slot]);
          umma_commit(&bars[L::kKEmpty + stage]);
          if (b + 1 == b1) umma_commit(&bars[L::kQEmpty + qslot]);
        }
        __syncwarp();
        if (++stage == SK) {
          stage = 0;
          kpar ^= 1;
        }
      }
      if (fail) break;
    }
  } else if (warp == 15) {
    // ------------------------------------------------------------ PV issuer
    constexpr uint32_t kIdO = idesc_e4m3(128, N, true, true);  // A = V^T (dims contiguous), B = P^T (pieces contiguous)
    const uint32_t leader = elect_one_sync();
    uint32_t stage = 0, vpar = 0, o_it = 0;
    QWalk<QDecodeParams> walk(p);
    QPiece pc;
    while (walk.next(p, &pc)) {
      bool fail = false;
      const int b1 = pc.block1();
      for (int b = pc.block0(); b < b1; ++b, ++o_it) {
        const uint32_t oslot = o_it % OS, pslot = o_it % PS;
        bool w = wait_warp(&bars[L::kVFull + stage], vpar, abort, p.err, 0xb22);
        if (!w) { fail = true; break; }
        uint8_t* vd = v_base + stage * L::kKVBytes;
        // V rows past the context may hold anything, NaN codes among it; P is
        // exactly 0 there, so zero them (0 * NaN = NaN)
        const int valid = min(B, pc.kv_len - b * B);
        if (valid < B) {
          for (int i = lane; i < (B - valid) * 8; i += 32)
            *reinterpret_cast<uint4*>(vd + valid * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        w = wait_warp(&bars[L::kPFull + pslot], (o_it / PS) & 1, abort, p.err, 0xb21);
        w = w && wait_warp(&bars[L::kOEmpty + oslot], ((o_it / OS) & 1) ^ 1, abort, p.err, 0xb23);
        if (!w) { fail = true; break; }
        tc_fence_after();
        // K-step s covers keys 32 s .. 32 s + 31: V rows 4096 B a step, P^T
        // 32 N B a step
        const Desc vdd = make_desc(smem_u32(vd), 16, 1024);
        const Desc pd = p_desc<N>(smem_u32(p_base + pslot * L::kTBytes));
        const uint32_t d = tm_o + oslot * N;
        if (leader) {
          mma8_ss<0>(d, vdd, 0, pd, 0, kIdO);
#pragma unroll
          for (int s = 1; s < B / 32; ++s) mma8_ss<1>(d, vdd, s * 256, pd, s * 2 * N, kIdO);
          umma_commit(&bars[L::kOFull + oslot]);
          umma_commit(&bars[L::kVEmpty + stage]);
          umma_commit(&bars[L::kPEmpty + pslot]);
        }
        __syncwarp();
        if (++stage == SV) {
          stage = 0;
          vpar ^= 1;
        }
      }
      if (fail) break;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int grp = warp >= 8 ? 1 : 0;
    const int t = tid - (grp ? 256 : 128);  // key lane
    const int w = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(w * 32) << 16;
    float* red = reinterpret_cast<float*>(smem + L::kRedOff + grp * L::kRedBytes);
    const float sl = p.scale_log2;
    const int lps = 31 - __clz(p.page_size);
    uint32_t s_base = 0, sy_it = 0, q_it = 0;
    bool after_cut = false, end_fold = false;
    const float* k_scales = reinterpret_cast<const float*>(smem + L::kScOff) + (t >> lps);
    const float* v_scales = k_scales + L::kScRing * 16;
    QWalk<QDecodeParams> walk(p);
    QPiece pc;
    while (walk.next(p, &pc)) {
      const int kv_len = pc.kv_len, b0 = pc.block0(), nb = pc.block1() - b0;
      const int j0 = static_cast<int>(s_base & 1) == grp ? 0 : 1;
      // whether the correction warps will count, and fold, after their last
      // piece: when that is cut, or follows a cut piece
      const bool cut = !pc.whole();
      end_fold = walk.left <= 0 && (cut || after_cut);
      after_cut = cut && !after_cut;
      const uint32_t qslot = q_it & 1;
      bool ok = wait_warp(&bars[L::kQFull + qslot], (q_it >> 1) & 1, abort, p.err, 0xb41);
      if (!ok) break;
      ++q_it;
      float qs[MG];
#pragma unroll
      for (int q = 0; q < MG; ++q) qs[q] = qscale[qslot * MG + q];
      warp_arrive(&bars[L::kQEmpty + qslot], lane);
      bool fail = false;
      for (int j = j0; j < nb; j += 2) {
        const uint32_t s_it = s_base + j;
        const uint32_t slot = s_it % SS;
        // the scales of this thread's key
        const uint32_t isl = s_it % L::kScRing;
        ok = wait_warp(&bars[L::kScales + isl], (s_it / L::kScRing) & 1, abort, p.err, 0xb46);
        const float sk = k_scales[isl * 16], sv = v_scales[isl * 16];
        ok = ok && wait_warp(&bars[L::kSFull + slot], (s_it / SS) & 1, abort, p.err, 0xb42);
        if (!ok) { fail = true; break; }
        tc_fence_after();
        uint32_t raw[N];
        TmemRow<N>::ld(tm_s + lane_off + slot * N, raw);
        tmem_ld_wait(raw);
        tc_fence_before();
        warp_arrive(&bars[L::kSEmpty + slot], lane);
        const bool vis = (b0 + j) * B + t < kv_len;
        float* rd = red + static_cast<int>(sy_it & 1) * (2 * MG * 4);
        // the V scale is at most 2^up
        const float up = static_cast<float>(static_cast<int>((__float_as_uint(sv) + 0x7FFFFFu) >> 23) - 127);
        // scores, and the warp's maxima over its visible keys: of s (exact), and
        // of the exponent of p sv, p relative to the warp's own maximum
        float sc[MG];
#pragma unroll
        for (int q = 0; q < MG; ++q) {
          const float a = __fmaf_rn(__uint_as_float(raw[2 * MG + q]), 0x1p-10f,
                                    __fmaf_rn(__uint_as_float(raw[MG + q]), 0x1p-5f, __uint_as_float(raw[q])));
          // the two scales first: a row near the type's largest over small keys
          // would leave FP32's range on the way.  Where they leave it together, a
          // may still be small, or 0: then one after the other (neither below 1,
          // so what overflows here is past FP32 anyway).  With the scales that
          // writing sets, powers of two as the query's are, neither order rounds
          const float f = __fmul_rn(qs[q], sk);
          const float s = f <= 3.4028234e38f ? __fmul_rn(a, f) : __fmul_rn(__fmul_rn(a, sk), qs[q]);
          sc[q] = vis ? s : -INFINITY;
          const float m = warp_max_nan(sc[q]);
          const float x = warp_max(vis ? __fmaf_rn(__fsub_rn(sc[q], m), sl, up) : -INFINITY);
          if (lane == 0) {
            rd[q * 4 + w] = m;
            rd[(MG + q) * 4 + w] = x;
          }
        }
        uint64_t* sync = &bars[L::kSyncMax + grp * 2 + (sy_it & 1)];
        warp_arrive(sync, lane);
        ok = wait_warp(sync, (sy_it >> 1) & 1, abort, p.err, 0xb43);
        ++sy_it;
        if (!ok) { fail = true; break; }
        // lane q: the block's maximum of query head q, and the exponent ae of
        // its A = 2^ae (rounded up, so that w <= 1 but for the exponent's last
        // places: 2^8 w stays far below E4M3's 448)
        float m_mine;
        int ae;
        {
          const int q = min(lane, MG - 1);
          const float4 r = *reinterpret_cast<const float4*>(rd + q * 4);
          const float4 a = *reinterpret_cast<const float4*>(rd + (MG + q) * 4);
          m_mine = max_nan(max_nan(r.x, r.y), max_nan(r.z, r.w));
          auto rel = [&](float m, float x) { return __fmaf_rn(__fsub_rn(m, m_mine), sl, x); };
          ae = __float2int_ru(fmaxf(fmaxf(rel(r.x, a.x), rel(r.y, a.y)), fmaxf(rel(r.z, a.z), rel(r.w, a.w))));
          ae = min(max(ae, -118), 128);
        }
        const float wf_mine = pow2_bits(127 + 8 - ae);
        const float sv_vis = vis ? sv : 0.0f;  // stale behind the context
        float pr[MG];
#pragma unroll
        for (int q = 0; q < MG; ++q) {
          const float m = __shfl_sync(0xffffffffu, m_mine, q);  // (every lane: vis differs between them)
          pr[q] = vis ? weight(sc[q], m, sl) : 0.0f;
        }
        ok = wait_warp(&bars[L::kPEmpty + grp], ((s_it / PS) & 1) ^ 1, abort, p.err, 0xb44);
        if (!ok) { fail = true; break; }
        uint32_t pw[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) pw[i] = 0u;
#pragma unroll
        for (int q = 0; q < MG; q += 2) {
          // w 2^8 = (p sv) 2^(8 - ae): p sv stays in range, sv / A need not
          auto w8 = [&](int h) {
            return __fmul_rn(__fmul_rn(pr[h], sv_vis), __shfl_sync(0xffffffffu, wf_mine, h));
          };
          float a = w8(q), b = q + 1 < MG ? w8(q + 1 < MG ? q + 1 : q) : 0.0f;
          static_assert(kPPieces == 4 && p_col(2, 0) == 8 && p_col(1, 3) == 7, "a pair's pieces are two words");
          const uint32_t c0 = next_piece(a, b), c1 = next_piece(a, b), c2 = next_piece(a, b);
          pw[q] = __byte_perm(c0, c1, 0x5410);
          pw[q + 1] = __byte_perm(c2, e4m3_pair(a, b), 0x5410);
        }
        p_store<N>(p_base + grp * L::kTBytes, t, pw);
        fence_proxy_async_smem();
        warp_arrive(&bars[L::kPFull + grp], lane);
        // the warp's part of the block sums: p <= 1 (and a block's largest is
        // 1), so a warp's sum fits 32 bits with 26 fraction bits.  Each p is
        // off by at most 2^-27, a block's sum by 128 * 2^-27 of at least 1 (128
        // FP32 numbers in a tree: 7 * 2^-24), in one instruction and in no order
        uint32_t* st = stats + (s_it % SR) * L::kStatWords;
        uint32_t l_mine = 0;  // lane q: query head q's
#pragma unroll
        for (int q = 0; q < MG; ++q) {
          const uint32_t l = __reduce_add_sync(0xffffffffu, __float2uint_rn(__fmul_rn(pr[q], kLUnit)));
          l_mine = lane == q ? l : l_mine;
        }
        if (lane < MG) {
          st[lane * 4 + w] = l_mine;
          if (w == 0) {
            st[4 * MG + lane] = __float_as_uint(m_mine);
            st[5 * MG + lane] = __float_as_uint(pow2_bits(127 - 8 + ae));  // PV carries 2^8 / A
          }
        }
        warp_arrive(&bars[L::kStatsFull + (s_it % SR)], lane);
      }
      if (fail) break;
      s_base += nb;
    }
    if (end_fold && wait_warp(&bars[L::kEndCounted], 0, abort, p.err, 0xb47)) fold_pairs(true);
  } else {
    // ------------------------------------------------------------ correction / epilogue
    const int d = tid;  // head dimension lane
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    uint32_t o_it = 0, cut_it = 0;
    struct Cut {
      int seq, g, n, ns, first;
    } cut0 = {}, cut1 = {};
    int n_cut = 0;
    bool fail = false;
    // Counts the cut pieces and folds the pairs they complete: every thread's
    // states are in device memory before the count, and the CTA that counts a
    // pair's last segment reads them after it.
    auto flush = [&](bool end) -> bool {
      __threadfence();
      warp_arrive(&bars[L::kStored], lane);
      if (warp == 0) {
        const bool ok = wait_warp(&bars[L::kStored], cut_it & 1, abort, p.err, 0xb54);
        if (!ok) return false;
        if (lane < 2) {
          const Cut q = lane == 0 ? cut0 : cut1;
          int last = 0;
          if (lane < n_cut) {
            last = count_segments(p.counts + static_cast<int64_t>(q.seq) * p.hkv + q.g, q.n, q.ns);
            __threadfence();
          }
          to_fold[lane] = make_int4(q.seq, q.g, p.seg0[q.seq] + q.first - 1, last ? q.ns - q.first + 1 : 0);
        }
        warp_arrive(&bars[end ? L::kEndCounted : L::kCounted], lane);
      }
      const bool ok = end ? wait_warp(&bars[L::kEndCounted], 0, abort, p.err, 0xb56)
                          : wait_warp(&bars[L::kCounted], cut_it & 1, abort, p.err, 0xb55);
      if (!ok) return false;
      ++cut_it;
      fold_pairs(end);
      n_cut = 0;
      return true;
    };
    QWalk<QDecodeParams> walk(p);
    QPiece pc;
    while (walk.next(p, &pc)) {
      const bool whole = pc.whole();
      if (!whole && tid == 0) begin_count(p.counts + static_cast<int64_t>(pc.seq) * p.hkv + pc.g, p.nonce);
      // O: the segment's, T: the sequence's (of a pair's first or only piece);
      // lane q holds m and l of query head q
      float O[MG], T[MG];
#pragma unroll
      for (int q = 0; q < MG; ++q) O[q] = T[q] = 0.0f;
      float m = 0.0f, l = 0.0f, mt = -INFINITY, lt = 0.0f;
      const int b1 = pc.block1();
      for (int b = pc.block0(); b < b1; ++b) {
        const uint32_t sslot = o_it % SR, oslot = o_it % OS;
        bool ok = wait_warp(&bars[L::kStatsFull + sslot], (o_it / SR) & 1, abort, p.err, 0xb51);
        ok = ok && wait_warp(&bars[L::kOFull + oslot], (o_it / OS) & 1, abort, p.err, 0xb52);
        if (!ok) { fail = true; break; }
        tc_fence_after();
        uint32_t raw[N];
        TmemRow<N>::ld(tm_o + lane_off + oslot * N, raw);
        // fold factors of query head `lane` (overlap the TMEM load)
        const uint32_t* st = stats + sslot * L::kStatWords;
        const bool first = b % kSegBlocks == 0;
        float vf[MG];
#pragma unroll
        for (int q = 0; q < MG; ++q) vf[q] = __uint_as_float(st[5 * MG + q]);
        float fa = 0.0f, fb = 1.0f;
        if (lane < MG) {
          const float mb = __uint_as_float(st[4 * MG + lane]);
          const uint4 ls = *reinterpret_cast<const uint4*>(st + 4 * lane);
          const float lb = __fmul_rn(__fadd_rn(__fadd_rn(__uint2float_rn(ls.x), __uint2float_rn(ls.y)),
                                               __fadd_rn(__uint2float_rn(ls.z), __uint2float_rn(ls.w))),
                                     1.0f / kLUnit);
          if (first) {
            m = mb;
            l = lb;
          } else {
            float mn;
            fold_factors(m, mb, p.scale_log2, mn, fa, fb);
            l = __fmaf_rn(lb, fb, __fmul_rn(l, fa));
            m = mn;
          }
        }
        tmem_ld_wait(raw);
        tc_fence_before();
        warp_arrive(&bars[L::kOEmpty + oslot], lane);
#pragma unroll
        for (int q = 0; q < MG; ++q) {
          const float aq = __shfl_sync(0xffffffffu, fa, q);
          const float bq = __shfl_sync(0xffffffffu, fb, q);
          float pv = __uint_as_float(raw[p_col(q, kPPieces - 1)]);
#pragma unroll
          for (int k = kPPieces - 2; k >= 0; --k) pv = __fmaf_rn(pv, 0x1p-5f, __uint_as_float(raw[p_col(q, k)]));
          pv = __fmul_rn(pv, vf[q]);
          O[q] = first ? pv : __fmaf_rn(pv, bq, __fmul_rn(O[q], aq));
        }
        ++o_it;
        if ((b + 1) % kSegBlocks != 0 && b + 1 != pc.nb) continue;
        // the segment is complete
        if (pc.s0 == 0) {
          float mn, ta, tb;
          fold_factors(mt, m, p.scale_log2, mn, ta, tb);
          lt = __fmaf_rn(l, tb, __fmul_rn(lt, ta));
          mt = mn;
#pragma unroll
          for (int q = 0; q < MG; ++q) {
            const float aq = __shfl_sync(0xffffffffu, ta, q);
            const float bq = __shfl_sync(0xffffffffu, tb, q);
            T[q] = __fmaf_rn(O[q], bq, __fmul_rn(T[q], aq));
          }
          if (whole || b + 1 < b1) continue;
          m = mt;  // the pair's first piece leaves as one state, its last segment's
          l = lt;
        }
        const int64_t r = static_cast<int64_t>(p.seg0[pc.seq] + b / kSegBlocks) * p.hq + pc.g * MG;
#pragma unroll
        for (int q = 0; q < MG; ++q) p.state_o[(r + q) * kHeadDim + d] = pc.s0 == 0 ? T[q] : O[q];
        if (warp == 0 && lane < MG) reinterpret_cast<float2*>(p.state_ml)[r + lane] = make_float2(m, l);
      }
      if (fail) break;
      if (whole) {
        const float rl = __frcp_rn(lt);
#pragma unroll
        for (int q = 0; q < MG; ++q) {
          const float rq = __shfl_sync(0xffffffffu, rl, q);
          const int64_t row = static_cast<int64_t>(pc.seq) * p.hq + pc.g * MG + q;
          const float o = __fmul_rn(T[q], rq);
          if (p.out_f32) p.out_f32[row * kHeadDim + d] = o;
          if (p.out_bf16) p.out_bf16[row * kHeadDim + d] = f32_to_bf16_rn(o);
        }
        if (warp == 0 && lane < MG && p.lse)
          p.lse[static_cast<int64_t>(pc.seq) * p.hq + pc.g * MG + lane] = log_sum(mt, lt, p.scale_log2);
        if (n_cut > 0 && !flush(walk.left <= 0)) break;
        continue;
      }
      // a part of a pair: counted once the next piece is done too (waiting
      // here for the stores and the count would hold up the blocks behind)
      cut1 = cut0;
      cut0 = {pc.seq, pc.g, pc.s1 - pc.s0, pc.ns, pc.first};
      if (++n_cut == 2 && !flush(walk.left <= 0)) break;
    }
    if (!fail && n_cut > 0) flush(true);
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 14) {
    if (*abort) {
      // let copies already in flight land before the CTA's memory is released
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
    tc_fence_after();
    tmem_dealloc(tm_s, L::kTmemCols);
  }
}

template <int MG>
cudaError_t launch_qdecode_t(const QDecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                             cudaStream_t stream) {
  rlk_qdecode_kernel<MG><<<grid, kQDThreads, QDecLayout<MG>::kAlloc, stream>>>(p, tk, tv);
  return cudaGetLastError();
}

template <int MG>
cudaError_t configure_qdecode_mg() {
  return cudaFuncSetAttribute(rlk_qdecode_kernel<MG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              QDecLayout<MG>::kAlloc);
}

}  // namespace

cudaError_t configure_qdecode_kernels() {
  cudaError_t e;
  if ((e = configure_qdecode_mg<1>()) || (e = configure_qdecode_mg<2>()) || (e = configure_qdecode_mg<3>()) ||
      (e = configure_qdecode_mg<4>()) || (e = configure_qdecode_mg<5>()) || (e = configure_qdecode_mg<6>()) ||
      (e = configure_qdecode_mg<7>()))
    return e;
  return configure_qdecode_mg<8>();
}

cudaError_t launch_qdecode(const QDecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                           cudaStream_t stream) {
  switch (p.hq / p.hkv) {
    case 1: return launch_qdecode_t<1>(p, tk, tv, grid, stream);
    case 2: return launch_qdecode_t<2>(p, tk, tv, grid, stream);
    case 3: return launch_qdecode_t<3>(p, tk, tv, grid, stream);
    case 4: return launch_qdecode_t<4>(p, tk, tv, grid, stream);
    case 5: return launch_qdecode_t<5>(p, tk, tv, grid, stream);
    case 6: return launch_qdecode_t<6>(p, tk, tv, grid, stream);
    case 7: return launch_qdecode_t<7>(p, tk, tv, grid, stream);
    default: return launch_qdecode_t<8>(p, tk, tv, grid, stream);
  }
}

}  // namespace rlk
