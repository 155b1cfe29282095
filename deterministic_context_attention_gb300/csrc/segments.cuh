// segments.cuh -- what the decodes that cut a sequence's keys into segments of
// kQSegKeys share: the pieces of work of a CTA and their pages, the running
// maximum and sum of a softmax and their folds, the count of a cut pair's
// segments.  P: the kernel's parameters (ctx, start, group, hkv, page_table,
// max_pages).
#pragma once
#include "numerics.cuh"
#include "ptx.cuh"
#include "qcache_internal.h"

namespace rlk {

constexpr int kSegBlocks = kQSegKeys / 128;
constexpr float kLUnit = 0x1p26f;  // block sums of p: fixed point, 26 fraction bits

// A warp's wait on a barrier (bounded, mbar_wait): one test and one vote when
// the phase is complete already, the rest out of line (the roles' code
// competes for the instruction cache).
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, ErrWord* err,
                                       unsigned int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err, site));
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, ErrWord* err,
                                          unsigned int site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_slow(bar, parity, abort, err, site);
}

// One arrival for the whole warp, after every lane's earlier writes.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Row maximum of the 32 lanes of a warp (exact; every lane receives it).
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// The same, NaN where any lane holds one, and the maximum of two like it: a NaN
// score makes its row's maximum, and from there the whole row, NaN.
__device__ __forceinline__ float warp_max_nan(float v) {
  float m;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// A piece of work: segments [s0, s1) of the ns of (sequence, KV head g).
struct QPiece {
  int seq, g, kv_len, nb, s0, s1, ns;
  int first;  // the segments that the pair's first piece has
  __device__ int block0() const { return s0 * kSegBlocks; }
  __device__ int block1() const { return min(s1 * kSegBlocks, nb); }
  __device__ bool whole() const { return s0 == 0 && s1 == ns; }
};

// The pieces of this CTA, in order; every role walks them on its own from the
// CTA's start, which the host worked out (found here, by searching the tables
// in the parameters, it was the first 4 us of every CTA: each probe of a table
// missed the constant cache).
template <class P>
struct QWalk {
  int seq, g, b;  // where the next piece starts (g: the first KV head of the group's)
  int left;       // blocks still to take
  int cut;        // b > 0: where that pair is first cut
  __device__ explicit QWalk(const P& p) {
    const QStart s = p.start[blockIdx.x / p.group];
    seq = s.seq;
    g = s.g * p.group + blockIdx.x % p.group;
    b = s.b;
    left = s.left;
    cut = s.cut;
  }
  __device__ bool next(const P& p, QPiece* q) {
    if (left <= 0) return false;
    q->seq = seq;
    q->g = g;
    q->kv_len = p.ctx[seq];
    q->nb = (q->kv_len + 127) / 128;
    q->ns = (q->nb + kSegBlocks - 1) / kSegBlocks;
    const int stop = min(left, q->nb - b);
    q->s0 = b / kSegBlocks;
    q->s1 = (b + stop + kSegBlocks - 1) / kSegBlocks;
    q->first = b > 0 ? cut / kSegBlocks : q->s1;
    left -= stop;
    b = 0;
    g += p.group;
    if (g >= p.hkv) {
      g -= p.hkv;
      ++seq;
    }
    return true;
  }
};

// The blocks of those pieces in groups of up to 4 consecutive ones of a piece
// whose page ids fill a warp (32 pages: 2 blocks of 8-token pages, 4 of larger).
template <class P>
struct QGroups {
  QWalk<P> walk;
  QPiece pc;
  int b, n;  // first block, blocks
  bool ok;
  __device__ QGroups(const P& p, int lg) : walk(p) {
    b = n = 0;
    ok = walk.next(p, &pc);
    if (ok) begin(pc.block0(), lg);
  }
  __device__ void begin(int first, int lg) {
    b = first;
    n = min(1 << min(5 - lg, 2), pc.block1() - b);
  }
  __device__ void step(const P& p, int lg) {
    if (!ok) return;
    if (b + n >= pc.block1()) {
      ok = walk.next(p, &pc);
      if (ok) begin(pc.block0(), lg);
    } else {
      begin(b + n, lg);
    }
  }
  // lane l: the id of page l of the group (-1: none)
  __device__ int page_id(const P& p, int lg, int lane) const {
    const int gp = (b << lg) + lane;
    if (!ok || lane >= (n << lg) || gp * (128 >> lg) >= pc.kv_len) return -1;
    return __ldg(p.page_table + static_cast<int64_t>(pc.seq) * p.max_pages + gp);
  }
};

// 2^((s - m) c), exactly 1 for s = m.
__device__ __forceinline__ float weight(float s, float m, float c) { return ex2_hw(__fmul_rn(__fsub_rn(s, m), c)); }

// (O, m, l) folded with a later state: the factors of the two, and m.
__device__ __forceinline__ void fold_factors(float m, float mb, float c, float& mn, float& a, float& b) {
  mn = fmaxf(m, mb);
  a = weight(m, mn, c);
  b = weight(mb, mn, c);
}

// ln of the sum of e^(s scale): m the maximum of s, l the sum relative to it.
__device__ __forceinline__ float log_sum(float m, float l, float c) {
  return __fmaf_rn(__fmul_rn(m, c), kLn2f, logf(l));
}

// The count of a cut pair's finished segments: a word that holds the call's
// nonce (40 bits) over the count (24).  Another nonce means that no segment of
// this call has been counted yet; every CTA with a part of the pair sees to it
// early (begin_count) that the word holds its nonce, so that counting is one
// addition.  The CTA that counts the last segment clears the word.
__device__ __forceinline__ void begin_count(unsigned long long* word, uint64_t nonce) {
  const unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(word);
  // where this fails, another CTA of the call has done it
  if ((old >> 24) != nonce) atomicCAS(word, old, static_cast<unsigned long long>(nonce << 24));
}
__device__ __forceinline__ bool count_segments(unsigned long long* word, int n, int ns) {
  const bool last = (atomicAdd(word, static_cast<unsigned long long>(n)) & 0xFFFFFFu) + n == static_cast<unsigned>(ns);
  if (last) *reinterpret_cast<volatile unsigned long long*>(word) = 0ull;
  return last;
}

}  // namespace rlk
