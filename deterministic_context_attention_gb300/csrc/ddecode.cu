// ddecode.cu -- differential attention of one new token a sequence over the
// paged BF16 cache, for sm_103a.
//
// A head's 128 columns of Q and K are two 64-wide maps; the query rows of a KV
// head are then R = 2 G rows, row 2 i + m map m of query head i, its columns as
// they are and zeros in the other map's.  So one transposed product (keys, then
// head dimensions, on the MMA's M side) serves both maps and the cache is read
// once:
//   S^T = K_b Q^T                (M = 128 keys, N = 16 rows, K = 128)
//   O^T = V_b^T [P_hi | P_lo]^T  (M = 128 dims, N = 16 or 32, K = 128)
// with P in two BF16 pieces (2^-18 of itself) side by side in the columns, so
// that the low pieces' products are summed on their own and the two sums meet
// in one FP32 addition.
//
// Softmax in FP32, per row: a block b of 128 keys gives m_b = max s, p =
// 2^((s - m_b) c), l_b = sum p, O_b = sum p v, c = scale log2(e); blocks are
// folded left to right into segments of 512 keys (a fixed cut of the sequence),
// segments left to right into the row, with a running maximum (segments.cuh).
// l_b alone is summed in fixed point, each p to 2^-27 and p below that not at all:
// at the worst 2^-20 of l_b, where a tree of FP32 sums has 2^-21.
// out = O_1 / l_1 - lambda O_2 / l_2.  The result depends on the cached rows and
// the query alone, not on the batch, the order of the pages or the split.  (Not
// the log-sum-exp fold of the plain decode: a log sum of 40 and more, as keys of
// uneven channels give, holds 2^-19 at best, which a fold of 256 blocks drifts
// by; that difference of maps was 1.8e-4 off at 32768 keys, this one is 1e-6.)
//
// Work split, pieces, counts and folds as in the decode over the 8-bit cache:
// neighbouring CTAs take neighbouring KV heads of the same keys, each group of
// them an equal part of the line of all blocks, cut at segment ends; a cut
// pair's states meet in the workspace and the CTA that counts the last folds
// them.
//
// What bounds it: HBM, 64 KB of K and V per (KV head, 128-key block).  64
// contexts of 512 to 32768 (8 KV heads, 4.4 GB) take 640 us, 6.8 TB/s; 4 of 32768
// (537 MB) 96 us, 5.6 TB/s: a part's 13 or 14 segments are a step of 4 %, the
// rest is the launch, the first pages and the last fold, which are the 10 us of a
// single context of 700.  (Through the plain decode's kernel, a pass a map over
// the whole page, these were 671, 108 and 12.)
//
// Warp roles (512 threads):
//   warps 0-3   correction / epilogue: thread d owns head dimension d
//   warps 4-7   softmax of the even blocks, warps 8-11 of the odd ones:
//               thread t owns key t of the block
//   warp  12    producer of the query rows and the K pages, warp 13 of the V
//               pages (TMA)
//   warp  14    the S^T products, warp 15 the O^T products
#include <cuda.h>
#include <cuda_runtime.h>

#include "numerics.cuh"
#include "ptx.cuh"
#include "segments.cuh"

namespace rlk {
namespace {

constexpr int kDDThreads = 512;

// R: rows (2 per query head of the group), NQ: columns of S^T, NO: of O^T
// (the high pieces' R8, then the low ones').
template <int R>
struct DDecLayout {
  static constexpr int B = 128;
  static constexpr int NQ = 16;
  static constexpr int R8 = R <= 8 ? 8 : 16;
  static constexpr int NO = 2 * R8;
  static constexpr int kSK = 3, kSV = 2;  // K and V rings
  static constexpr int kPS = 2, kQS = 2;  // P^T and query slots
  static constexpr int kSS = 4, kOS = 4;  // TMEM rings of S^T and O^T
  // statistics ring: block s is written once P slot s - 2 is free, so O slot
  // s - 6 and the statistics beside it have been read
  static constexpr int kSR = 8;
  static_assert(kSR >= kPS + kOS, "statistics ring");
  static constexpr int kKVHalf = B * 128;
  static constexpr int kKVBytes = 2 * kKVHalf;
  static constexpr int kQHalf = NQ * 128;  // one 64-column half of the query rows
  static constexpr int kQBytes = 2 * kQHalf;
  static constexpr int kPBytes = B * NO * 2;  // a key's NO weights are one run of bytes
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + kQS * kQBytes;
  static constexpr int kKOff = (kPOff + kPS * kPBytes + 1023) / 1024 * 1024;
  static constexpr int kVOff = kKOff + kSK * kKVBytes;
  static constexpr int kRedOff = kVOff + kSV * kKVBytes;  // per softmax group, double-buffered: float [R][4 warps]
  static constexpr int kRedBytes = 2 * R * 16;
  static constexpr int kStatWords = (5 * R + 3) / 4 * 4;  // per block: uint32 l[R][4 warps], then float m[R]
  static constexpr int kStatsOff = kRedOff + 2 * kRedBytes;
  static constexpr int kBarOff = (kStatsOff + kSR * kStatWords * 4 + 7) / 8 * 8;
  static constexpr int kQFull = 0, kQEmpty = kQFull + kQS, kKFull = kQEmpty + kQS, kKEmpty = kKFull + kSK,
                       kVFull = kKEmpty + kSK, kVEmpty = kVFull + kSV, kSFull = kVEmpty + kSV,
                       kSEmpty = kSFull + kSS, kPFull = kSEmpty + kSS, kPEmpty = kPFull + kPS,
                       kOFull = kPEmpty + kPS, kOEmpty = kOFull + kOS, kStatsFull = kOEmpty + kOS,
                       kSyncMax = kStatsFull + kSR, kStored = kSyncMax + 4, kCounted = kStored + 1,
                       kEndCounted = kCounted + 1, kNumBars = kEndCounted + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // tmem base (u32), abort (i32)
  static constexpr int kCutOff = (kMiscOff + 16 + 15) / 16 * 16;  // pairs to fold: int4 {seq, g, first state, states} [2]
  // segment states being folded, groups of 4 of a head's two rows: per
  // correction warp, and at the end per correction and softmax warp in the rings
  static constexpr int kFoldGroups = 2, kEndGroups = 3;
  static_assert(12 * kEndGroups * 8 * 512 <= (kSK + kSV) * kKVBytes, "the rings hold them");
  static constexpr int kFoldOff = kCutOff + 2 * 16;
  static constexpr int kTotal = kFoldOff + 4 * kFoldGroups * 8 * 512;
  static constexpr int kAlloc = kTotal + 1024;
  static constexpr int kTmemCols = NQ * kSS + NO * kOS <= 128 ? 128 : 256;
  static_assert(kAlloc <= 232448, "decode shared memory");
};

// P^T is stored N-major: key t's NO weights are one run of 32 or 64 bytes in
// the 32- or 64-byte swizzle, which the key's thread writes whole.
template <int NO>
__device__ __forceinline__ Desc pt_desc(uint32_t saddr) {
  constexpr uint64_t kGroup = NO * 2 * 8 >> 4;  // 8 keys; no second group along N
  const uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (kGroup << 16) | (kGroup << 32) |
                     (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(NO == 16 ? 6 : 4) << 61);
  return Desc{static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)};
}
template <int NO>
__device__ __forceinline__ void pt_store(uint8_t* tile, int t, const uint32_t (&w)[NO / 2]) {
#pragma unroll
  for (int i = 0; i < NO / 8; ++i) {
    const int at = t * NO * 2 + ((i ^ (NO == 16 ? (t >> 2) & 1 : (t >> 1) & 3)) << 4);
    *reinterpret_cast<uint4*>(tile + at) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

template <int NO>
struct TmemCols;
template <>
struct TmemCols<16> {
  static __device__ __forceinline__ void ld(uint32_t a, uint32_t (&r)[16]) { tmem_ld16(a, r); }
};
template <>
struct TmemCols<32> {
  static __device__ __forceinline__ void ld(uint32_t a, uint32_t (&r)[32]) { tmem_ld32(a, r); }
};

// The fold of a cut pair's ns states (the first piece's, then its other
// segments', from segment `seg` of the workspace on) for both maps of query
// head h, one warp a head: lane l takes head dimensions 4 l .. 4 l + 3 of
// either.  Groups of 4 segments are copied ahead into the warp's ring (a lane
// reads what it copied itself); for 32 segments at a time the running maxima
// are a scan over the lanes and the factors come out side by side, which
// leaves a multiply and an fma a segment and map on the chain.
template <int GROUPS>
__device__ __noinline__ void fold_head(const DDecodeParams& p, int seq, int seg, int ns, int h, int lane,
                                       float4* ring) {
  constexpr int C = 4;
  const int rows = 2 * p.hq;
  const int64_t base = static_cast<int64_t>(seg) * rows + 2 * h;
  const int64_t pitch = static_cast<int64_t>(rows) * kHeadDim;
  const float* src = p.state_o + base * kHeadDim + 4 * lane;
  const float2* sml = reinterpret_cast<const float2*>(p.state_ml) + base;
  // past the last segment: m = -inf, a factor of 0
  auto load_ml = [&](int c0, int mp) {
    return c0 + lane < ns ? __ldcg(sml + static_cast<int64_t>(c0 + lane) * rows + mp) : make_float2(-INFINITY, 0.f);
  };
  int next = 0;  // the next segment to copy
  float4* to = ring + lane;
  auto copy = [&]() {
    if (next < ns) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
#pragma unroll
        for (int mp = 0; mp < 2; ++mp) {
          if (next + i < ns) cp_async16(to + (2 * i + mp) * 32, src + i * pitch + mp * kHeadDim);
          else to[(2 * i + mp) * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
    cp_async_commit();  // empty groups keep the count uniform
    next += C;
    src += C * pitch;
    to = to + C * 64 == ring + lane + GROUPS * C * 64 ? ring + lane : to + C * 64;
  };
  float2 ml[2] = {load_ml(0, 0), load_ml(0, 1)};
#pragma unroll 1
  for (int c = 0; c < GROUPS; ++c) copy();
  float4 O[2];
  float m[2], l[2];
#pragma unroll
  for (int mp = 0; mp < 2; ++mp) {
    O[mp] = make_float4(-0.f, -0.f, -0.f, -0.f);  // the first state as it is, its sign of zero too
    m[mp] = -INFINITY;
    l[mp] = 0.f;
  }
#pragma unroll 1
  for (int s0 = 0; s0 < ns; s0 += 32) {
    const float2 ml_next[2] = {load_ml(s0 + 32, 0), load_ml(s0 + 32, 1)};
    float fa[2], fb[2];
#pragma unroll
    for (int mp = 0; mp < 2; ++mp) {
      float run = fmaxf(m[mp], ml[mp].x);  // lane i: the maximum up to segment s0 + i
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const float o = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run = fmaxf(run, o);
      }
      float before = __shfl_up_sync(0xffffffffu, run, 1);
      if (lane == 0) before = m[mp];
      fa[mp] = weight(before, run, p.scale_log2);
      fb[mp] = weight(ml[mp].x, run, p.scale_log2);
      m[mp] = __shfl_sync(0xffffffffu, run, 31);
    }
#pragma unroll 1
    for (int s = s0; s < min(s0 + 32, ns); s += C) {
      cp_async_wait<GROUPS - 1>();
      float4 v[2 * C];
#pragma unroll
      for (int i = 0; i < 2 * C; ++i) v[i] = to[i * 32];  // the slot the next copy fills is the oldest one
      copy();
#pragma unroll
      for (int i = 0; i < C; ++i) {
#pragma unroll
        for (int mp = 0; mp < 2; ++mp) {
          const float a = __shfl_sync(0xffffffffu, fa[mp], s - s0 + i), b = __shfl_sync(0xffffffffu, fb[mp], s - s0 + i);
          const float lb = __shfl_sync(0xffffffffu, ml[mp].y, s - s0 + i);
          const float4 x = v[2 * i + mp];
          O[mp].x = __fmaf_rn(x.x, b, __fmul_rn(O[mp].x, a));
          O[mp].y = __fmaf_rn(x.y, b, __fmul_rn(O[mp].y, a));
          O[mp].z = __fmaf_rn(x.z, b, __fmul_rn(O[mp].z, a));
          O[mp].w = __fmaf_rn(x.w, b, __fmul_rn(O[mp].w, a));
          l[mp] = __fmaf_rn(lb, b, __fmul_rn(l[mp], a));
        }
      }
    }
    ml[0] = ml_next[0];
    ml[1] = ml_next[1];
  }
  cp_async_wait<0>();
  const float r1 = __frcp_rn(l[0]), r2 = __frcp_rn(l[1]), nl = -__ldg(p.lambda + h);
  auto diff = [&](float a, float b) { return __fmaf_rn(nl, __fmul_rn(b, r2), __fmul_rn(a, r1)); };
  const float4 o =
      make_float4(diff(O[0].x, O[1].x), diff(O[0].y, O[1].y), diff(O[0].z, O[1].z), diff(O[0].w, O[1].w));
  const int64_t row = static_cast<int64_t>(seq) * p.hq + h;
  if (p.out_f32) *(reinterpret_cast<float4*>(p.out_f32 + row * kHeadDim) + lane) = o;
  if (p.out_bf16)
    *(reinterpret_cast<uint2*>(p.out_bf16 + row * kHeadDim) + lane) =
        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  if (p.lse && lane < 2)
    p.lse[2 * row + lane] = log_sum(lane ? m[1] : m[0], lane ? l[1] : l[0], p.scale_log2);
}

template <int R>
__global__ void __launch_bounds__(kDDThreads, 1)
    rlk_ddecode_kernel(const __grid_constant__ DDecodeParams p, const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using L = DDecLayout<R>;
  constexpr int B = L::B, NQ = L::NQ, NO = L::NO, R8 = L::R8, SK = L::kSK, SV = L::kSV, PS = L::kPS, QS = L::kQS,
                SS = L::kSS, OS = L::kOS, SR = L::kSR, G = R / 2;
  static_assert(R % 2 == 0 && R <= 16 && PS == 2 && QS == 2, "decode layout");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  int4* to_fold = reinterpret_cast<int4*>(smem + L::kCutOff);
  uint32_t* stats = reinterpret_cast<uint32_t*>(smem + L::kStatsOff);
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  // the query tiles' other map of each row, and rows of no head, are never
  // written: they must read as zero
  for (int i = tid; i < QS * L::kQBytes / 16; i += kDDThreads)
    reinterpret_cast<uint4*>(smem + L::kQOff)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (tid == 0) {
    for (int s = 0; s < QS; ++s) {
      mbar_init(&bars[L::kQFull + s], 1);
      mbar_init(&bars[L::kQEmpty + s], 1);
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
  const uint32_t tm_s = *tmem_slot;      // S^T slots: + NQ * slot
  const uint32_t tm_o = tm_s + NQ * SS;  // O^T slots: + NO * slot
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
    const int n0 = c0.w ? G : 0, n = n0 + (c1.w ? G : 0);
    for (int i = warp; i < n; i += end ? 12 : 4) {
      const int4 c = i < n0 ? c0 : c1;
      const int h = c.y * G + (i < n0 ? i : i - n0);
      if (end)
        fold_head<L::kEndGroups>(p, c.x, c.z, c.w, h, lane,
                                 reinterpret_cast<float4*>(k_base) + warp * L::kEndGroups * 8 * 32);
      else
        fold_head<L::kFoldGroups>(p, c.x, c.z, c.w, h, lane,
                                  reinterpret_cast<float4*>(smem + L::kFoldOff) + warp * L::kFoldGroups * 8 * 32);
    }
  };

  if (warp == 12 || warp == 13) {
    // ------------------------------------------------------------ producers
    const bool is_v = warp == 13;
    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
    if (lane == 0) {
      if (!is_v) tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(map);
    }
    const uint32_t leader = elect_one_sync();
    const int S = is_v ? SV : SK;
    uint64_t* full_b = &bars[is_v ? L::kVFull : L::kKFull];
    uint64_t* empty_b = &bars[is_v ? L::kVEmpty : L::kKEmpty];
    uint8_t* ring = is_v ? v_base : k_base;
    const int lps = 31 - __clz(p.page_size), lg = 7 - lps;  // log2 of a page's tokens, of a block's pages
    const int lbox = min(lps, 31 - __clz(kQBoxRows));       // and of a copy's tokens
    // page ids: two groups of blocks ahead, across pieces
    QGroups<DDecodeParams> cur(p, lg), ahead(p, lg);
    int id = ahead.page_id(p, lg, lane);
    ahead.step(p, lg);
    int id1 = ahead.page_id(p, lg, lane);
    ahead.step(p, lg);
    uint32_t stage = 0, par = 1, q_it = 0;
    bool fail = false;
    while (cur.ok && !fail) {
      const int id2 = ahead.page_id(p, lg, lane);
      ahead.step(p, lg);
      if (!is_v && cur.b == cur.pc.block0()) {
        // the piece's query rows: map 1 of head i into row 2 i, map 2 into row 2 i + 1
        const uint32_t qslot = q_it & 1;
        if (!wait_warp(&bars[L::kQEmpty + qslot], ((q_it >> 1) & 1) ^ 1, abort, p.err, 0xc01)) break;
        ++q_it;
        if (leader) {
          uint8_t* tile = q_base + qslot * L::kQBytes;
          mbar_arrive_expect_tx(&bars[L::kQFull + qslot], G * kHeadDim * 2);
#pragma unroll 1
          for (int i = 0; i < G; ++i) {
            tma_load_3d(tile + 2 * i * 128, &tm_q, &bars[L::kQFull + qslot], 0, cur.pc.g * G + i, cur.pc.seq);
            tma_load_3d(tile + L::kQHalf + (2 * i + 1) * 128, &tm_q, &bars[L::kQFull + qslot], 64, cur.pc.g * G + i,
                        cur.pc.seq);
          }
        }
        __syncwarp();
      }
      // the first token of the page; out of range: past the last one, where
      // the copy reads the zero fill
      const bool bad = static_cast<unsigned>(id) >= static_cast<unsigned>(p.n_pages);
      const bool real = lane < cur.n << lg && ((cur.b << lg) + lane) << lps < cur.pc.kv_len;  // a page of the group
      const int tok = (bad ? p.n_pages : id) << lps;
      if (bad && real) report_error(p.err, kErrBadPage, 0xc04);
      for (int i = 0; i < cur.n; ++i) {
        if (!wait_warp(empty_b + stage, par, abort, p.err, is_v ? 0xc03 : 0xc02)) { fail = true; break; }
        uint8_t* dst = ring + stage * L::kKVBytes;
        const int n_box = (min(B, cur.pc.kv_len - (cur.b + i) * B) + (1 << lbox) - 1) >> lbox;
        if (lane == 0) mbar_arrive_expect_tx(full_b + stage, (n_box << lbox) * 256);
        __syncwarp();
        // copies of a page's boxes of up to kQBoxRows tokens (a context's last
        // page is not read past the box it ends in), issued by one lane in a
        // loop the whole warp walks
#pragma unroll 4
        for (int k = 0; k < n_box; ++k) {
          const int r = __shfl_sync(0xffffffffu, tok, (i << lg) + (k << lbox >> lps)) + ((k << lbox) & (p.page_size - 1));
          if (leader) {
            uint8_t* to = dst + ((k << lbox) * 128);
            tma_load_3d(to, map, full_b + stage, 0, cur.pc.g, r);
            tma_load_3d(to + L::kKVHalf, map, full_b + stage, 64, cur.pc.g, r);
          }
        }
        if (++stage == static_cast<uint32_t>(S)) {
          stage = 0;
          par ^= 1;
        }
      }
      cur.step(p, lg);
      id = id1;
      id1 = id2;
    }
  } else if (warp == 14) {
    // ------------------------------------------------------------ S issuer
    constexpr uint32_t kIdS = idesc_bf16(128, NQ, false, false);  // A = K (K-major), B = Q (K-major)
    const uint32_t leader = elect_one_sync();
    uint32_t stage = 0, kpar = 0, s_it = 0, q_it = 0;
    QWalk<DDecodeParams> walk(p);
    QPiece pc;
    while (walk.next(p, &pc)) {
      const uint32_t qslot = q_it & 1;
      if (!wait_warp(&bars[L::kQFull + qslot], (q_it >> 1) & 1, abort, p.err, 0xc11)) break;
      ++q_it;
      const Desc qd = make_desc(smem_u32(q_base + qslot * L::kQBytes), 16, 1024);
      bool fail = false;
      const int b1 = pc.block1();
      for (int b = pc.block0(); b < b1; ++b, ++s_it) {
        const uint32_t slot = s_it % SS;
        bool w = wait_warp(&bars[L::kKFull + stage], kpar, abort, p.err, 0xc12);
        w = w && wait_warp(&bars[L::kSEmpty + slot], ((s_it / SS) & 1) ^ 1, abort, p.err, 0xc13);
        if (!w) { fail = true; break; }
        tc_fence_after();
        const Desc kd = make_desc(smem_u32(k_base + stage * L::kKVBytes), 16, 1024);
        const uint32_t d = tm_s + slot * NQ;
        if (leader) {
          // K-steps over the head's columns: 0-3 map 1's, 4-7 map 2's
          mma_ss<0>(d, kd, 0, qd, 0, kIdS);
#pragma unroll
          for (int s = 1; s < kHeadDim / 16; ++s)
            mma_ss<1>(d, kd, (s >> 2) * (L::kKVHalf >> 4) + (s & 3) * 2, qd, (s >> 2) * (L::kQHalf >> 4) + (s & 3) * 2,
                      kIdS);
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
    constexpr uint32_t kIdO = idesc_bf16(128, NO, true, true);  // A = V^T (dims contiguous), B = P^T (rows contiguous)
    const uint32_t leader = elect_one_sync();
    uint32_t stage = 0, vpar = 0, o_it = 0;
    QWalk<DDecodeParams> walk(p);
    QPiece pc;
    while (walk.next(p, &pc)) {
      bool fail = false;
      const int b1 = pc.block1();
      for (int b = pc.block0(); b < b1; ++b, ++o_it) {
        const uint32_t oslot = o_it % OS, pslot = o_it % PS;
        bool w = wait_warp(&bars[L::kVFull + stage], vpar, abort, p.err, 0xc22);
        if (!w) { fail = true; break; }
        uint8_t* vd = v_base + stage * L::kKVBytes;
        // V rows past the context may hold anything; P is exactly 0 there, so
        // zero them (0 * NaN = NaN)
        const int valid = min(B, pc.kv_len - b * B);
        if (valid < B) {
          for (int i = lane; i < (B - valid) * 16; i += 32) {
            const int row = valid + (i >> 4), piece = i & 15;  // 16-byte pieces: 8 per half row
            *reinterpret_cast<uint4*>(vd + (piece >> 3) * L::kKVHalf + row * 128 + (piece & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        w = wait_warp(&bars[L::kPFull + pslot], (o_it / PS) & 1, abort, p.err, 0xc21);
        w = w && wait_warp(&bars[L::kOEmpty + oslot], ((o_it / OS) & 1) ^ 1, abort, p.err, 0xc23);
        if (!w) { fail = true; break; }
        tc_fence_after();
        // K-step s covers keys 16 s .. 16 s + 15: V rows 2048 B a step, P^T 32 NO B a step
        const Desc vdd = make_desc(smem_u32(vd), L::kKVHalf, 1024);
        const Desc pd = pt_desc<NO>(smem_u32(p_base + pslot * L::kPBytes));
        const uint32_t d = tm_o + oslot * NO;
        if (leader) {
          mma_ss<0>(d, vdd, 0, pd, 0, kIdO);
#pragma unroll
          for (int s = 1; s < B / 16; ++s) mma_ss<1>(d, vdd, s * 128, pd, s * 2 * NO, kIdO);
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
    uint32_t s_base = 0, sy_it = 0;
    bool after_cut = false, end_fold = false;
    QWalk<DDecodeParams> walk(p);
    QPiece pc;
    while (walk.next(p, &pc)) {
      const int kv_len = pc.kv_len, b0 = pc.block0(), nb = pc.block1() - b0;
      const int j0 = static_cast<int>(s_base & 1) == grp ? 0 : 1;
      // whether the correction warps will count, and fold, after their last
      // piece: when that is cut, or follows a cut piece
      const bool cut = !pc.whole();
      end_fold = walk.left <= 0 && (cut || after_cut);
      after_cut = cut && !after_cut;
      bool fail = false;
      for (int j = j0; j < nb; j += 2) {
        const uint32_t s_it = s_base + j;
        const uint32_t slot = s_it % SS;
        bool ok = wait_warp(&bars[L::kSFull + slot], (s_it / SS) & 1, abort, p.err, 0xc42);
        if (!ok) { fail = true; break; }
        tc_fence_after();
        uint32_t raw[16];
        tmem_ld16(tm_s + lane_off + slot * NQ, raw);
        tmem_ld_wait(raw);
        tc_fence_before();
        warp_arrive(&bars[L::kSEmpty + slot], lane);
        const bool vis = (b0 + j) * B + t < kv_len;
        // the warp's maxima over its visible keys (exact), row q's in lane q
        float* rd = red + static_cast<int>(sy_it & 1) * (R * 4);
        float sc[R], m_mine = 0.0f;
#pragma unroll
        for (int q = 0; q < R; ++q) {
          sc[q] = vis ? __uint_as_float(raw[q]) : -INFINITY;
          const float m = warp_max_nan(sc[q]);
          m_mine = lane == q ? m : m_mine;
        }
        if (lane < R) rd[lane * 4 + w] = m_mine;
        uint64_t* sync = &bars[L::kSyncMax + grp * 2 + (sy_it & 1)];
        warp_arrive(sync, lane);
        ok = wait_warp(sync, (sy_it >> 1) & 1, abort, p.err, 0xc43);
        ++sy_it;
        if (!ok) { fail = true; break; }
        {
          const float4 r = *reinterpret_cast<const float4*>(rd + min(lane, R - 1) * 4);
          m_mine = max_nan(max_nan(r.x, r.y), max_nan(r.z, r.w));
        }
        float pr[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
          const float m = __shfl_sync(0xffffffffu, m_mine, q);
          pr[q] = vis ? weight(sc[q], m, sl) : 0.0f;
        }
        uint32_t pw[NO / 2];  // rows 2 i, 2 i + 1 in word i; the low pieces after the high ones
#pragma unroll
        for (int i = 0; i < R8 / 2; ++i) {
          pw[i] = pw[R8 / 2 + i] = 0u;
          if (2 * i < R) split_pair2(make_float2(pr[2 * i], pr[2 * i + 1]), pw[i], pw[R8 / 2 + i]);
        }
        ok = wait_warp(&bars[L::kPEmpty + grp], ((s_it / PS) & 1) ^ 1, abort, p.err, 0xc44);
        if (!ok) { fail = true; break; }
        pt_store<NO>(p_base + grp * L::kPBytes, t, pw);
        fence_proxy_async_smem();
        warp_arrive(&bars[L::kPFull + grp], lane);
        // the warp's part of the block sums: p <= 1 (and a block's largest is
        // 1), so a warp's sum fits 32 bits with 26 fraction bits; each p is off
        // by at most 2^-27 (128 FP32 numbers in a tree: 7 * 2^-24 of the sum),
        // in one instruction and in no order
        uint32_t* st = stats + (s_it % SR) * L::kStatWords;
        uint32_t l_mine = 0;  // lane q: row q's
#pragma unroll
        for (int q = 0; q < R; ++q) {
          const uint32_t l = __reduce_add_sync(0xffffffffu, __float2uint_rn(__fmul_rn(pr[q], kLUnit)));
          l_mine = lane == q ? l : l_mine;
        }
        if (lane < R) {
          st[lane * 4 + w] = l_mine;
          if (w == 0) st[4 * R + lane] = __float_as_uint(m_mine);
        }
        warp_arrive(&bars[L::kStatsFull + (s_it % SR)], lane);
      }
      if (fail) break;
      s_base += nb;
    }
    if (end_fold && wait_warp(&bars[L::kEndCounted], 0, abort, p.err, 0xc47)) fold_pairs(true);
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
        const bool ok = wait_warp(&bars[L::kStored], cut_it & 1, abort, p.err, 0xc54);
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
      const bool ok = end ? wait_warp(&bars[L::kEndCounted], 0, abort, p.err, 0xc56)
                          : wait_warp(&bars[L::kCounted], cut_it & 1, abort, p.err, 0xc55);
      if (!ok) return false;
      ++cut_it;
      fold_pairs(end);
      n_cut = 0;
      return true;
    };
    QWalk<DDecodeParams> walk(p);
    QPiece pc;
    while (walk.next(p, &pc)) {
      const bool whole = pc.whole();
      if (!whole && tid == 0) begin_count(p.counts + static_cast<int64_t>(pc.seq) * p.hkv + pc.g, p.nonce);
      // O: the segment's, T: the sequence's (of a pair's first or only piece);
      // lane q holds m and l of row q
      float O[R], T[R];
#pragma unroll
      for (int q = 0; q < R; ++q) O[q] = T[q] = 0.0f;
      float m = 0.0f, l = 0.0f, mt = -INFINITY, lt = 0.0f;
      const int b1 = pc.block1();
      for (int b = pc.block0(); b < b1; ++b) {
        const uint32_t sslot = o_it % SR, oslot = o_it % OS;
        bool ok = wait_warp(&bars[L::kStatsFull + sslot], (o_it / SR) & 1, abort, p.err, 0xc51);
        ok = ok && wait_warp(&bars[L::kOFull + oslot], (o_it / OS) & 1, abort, p.err, 0xc52);
        if (!ok) { fail = true; break; }
        tc_fence_after();
        uint32_t raw[NO];
        TmemCols<NO>::ld(tm_o + lane_off + oslot * NO, raw);
        // fold factors of row `lane` (overlap the TMEM load)
        const uint32_t* st = stats + sslot * L::kStatWords;
        const bool first = b % kSegBlocks == 0;
        float fa = 0.0f, fb = 1.0f;
        if (lane < R) {
          const float mb = __uint_as_float(st[4 * R + lane]);
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
        for (int q = 0; q < R; ++q) {
          const float aq = __shfl_sync(0xffffffffu, fa, q);
          const float bq = __shfl_sync(0xffffffffu, fb, q);
          const float pv = __fadd_rn(__uint_as_float(raw[q]), __uint_as_float(raw[R8 + q]));
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
          for (int q = 0; q < R; ++q) {
            const float aq = __shfl_sync(0xffffffffu, ta, q);
            const float bq = __shfl_sync(0xffffffffu, tb, q);
            T[q] = __fmaf_rn(O[q], bq, __fmul_rn(T[q], aq));
          }
          if (whole || b + 1 < b1) continue;
          m = mt;  // the pair's first piece leaves as one state, its last segment's
          l = lt;
        }
        const int64_t r = static_cast<int64_t>(p.seg0[pc.seq] + b / kSegBlocks) * (2 * p.hq) + pc.g * R;
#pragma unroll
        for (int q = 0; q < R; ++q) p.state_o[(r + q) * kHeadDim + d] = pc.s0 == 0 ? T[q] : O[q];
        if (warp == 0 && lane < R) reinterpret_cast<float2*>(p.state_ml)[r + lane] = make_float2(m, l);
      }
      if (fail) break;
      if (whole) {
        const float rl = __frcp_rn(lt);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const float r1 = __shfl_sync(0xffffffffu, rl, 2 * i), r2 = __shfl_sync(0xffffffffu, rl, 2 * i + 1);
          const int64_t row = static_cast<int64_t>(pc.seq) * p.hq + pc.g * G + i;
          const float o = __fmaf_rn(-__ldg(p.lambda + pc.g * G + i), __fmul_rn(T[2 * i + 1], r2), __fmul_rn(T[2 * i], r1));
          if (p.out_f32) p.out_f32[row * kHeadDim + d] = o;
          if (p.out_bf16) p.out_bf16[row * kHeadDim + d] = f32_to_bf16_rn(o);
        }
        if (warp == 0 && lane < R && p.lse)
          p.lse[(static_cast<int64_t>(pc.seq) * p.hkv + pc.g) * R + lane] = log_sum(mt, lt, p.scale_log2);
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

template <int R>
cudaError_t launch_t(const DDecodeParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     int grid, cudaStream_t stream) {
  rlk_ddecode_kernel<R><<<grid, kDDThreads, DDecLayout<R>::kAlloc, stream>>>(p, tq, tk, tv);
  return cudaGetLastError();
}

template <int R>
cudaError_t configure_t() {
  return cudaFuncSetAttribute(rlk_ddecode_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              DDecLayout<R>::kAlloc);
}

}  // namespace

cudaError_t configure_ddecode_kernels() {
  cudaError_t e;
  if ((e = configure_t<2>()) || (e = configure_t<4>()) || (e = configure_t<6>()) || (e = configure_t<8>()) ||
      (e = configure_t<10>()) || (e = configure_t<12>()) || (e = configure_t<14>()))
    return e;
  return configure_t<16>();
}

cudaError_t launch_ddecode(const DDecodeParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           int grid, cudaStream_t stream) {
  switch (p.hq / p.hkv) {
    case 1: return launch_t<2>(p, tq, tk, tv, grid, stream);
    case 2: return launch_t<4>(p, tq, tk, tv, grid, stream);
    case 3: return launch_t<6>(p, tq, tk, tv, grid, stream);
    case 4: return launch_t<8>(p, tq, tk, tv, grid, stream);
    case 5: return launch_t<10>(p, tq, tk, tv, grid, stream);
    case 6: return launch_t<12>(p, tq, tk, tv, grid, stream);
    case 7: return launch_t<14>(p, tq, tk, tv, grid, stream);
    default: return launch_t<16>(p, tq, tk, tv, grid, stream);
  }
}

}  // namespace rlk
