// qcache_internal.h -- launch parameter blocks of the 8-bit paged KV cache
// (write, read, decode).  Not part of the public interface.
#pragma once
#include <cuda.h>

#include "rlk_internal.h"

namespace rlk {

constexpr int kQMaxSeqs = 256;  // sequences per launch

// The pages: E4M3 codes [n_pages][hkv][page_size][128] and FP32 scales
// [n_pages][hkv], for K and for V, under one page table.
struct QCachePools {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;  // device [num_seqs][max_pages]
  int32_t n_pages, page_size, max_pages, hkv;
};

// Write and read: tokens pos0[s] .. pos0[s] + n - 1 of sequence s, packed
// rows cu[s] .. cu[s + 1] - 1 of k / v [T, hkv, 128] BF16.
struct QCacheParams {
  ErrWord* err;
  QCachePools c;
  const uint16_t* k_in;  // write
  const uint16_t* v_in;
  uint16_t* k_out;  // read
  uint16_t* v_out;
  const float* rope_table;  // write: rotates K at its positions, or null
  int32_t num_seqs;
  int32_t cu[kQMaxSeqs + 1];
  int32_t pos0[kQMaxSeqs];
  int32_t page0[kQMaxSeqs + 1];  // prefix sum of the pages the sequences touch
};
cudaError_t launch_qcache_write(const QCacheParams& p, cudaStream_t stream);
cudaError_t launch_qcache_read(const QCacheParams& p, cudaStream_t stream);

// Decode over the 8-bit pages.  The keys of a sequence are cut into segments
// of kQSegKeys, whatever CTAs take them (qdecode.cu).
constexpr int kQSegKeys = 512;
// tokens of a page that one copy takes at the most: a context's last page is read
// to the end of its last box (200 short sequences in 128-token pages: 94.8 us,
// with whole pages 95.6)
constexpr int kQBoxRows = 32;
constexpr int kQMaxParts = 160;  // CTAs per launch
constexpr int kPairCost = 6;  // a (sequence, KV head)'s fixed cost in quarters of a 128-key block (1.2 us of 0.73)
struct QStart {  // where a group of CTAs starts (g: a group of KV heads), and how many blocks each has
  int32_t seq, g, b, left;
  int32_t cut;  // b > 0: the block at which that pair is first cut
};
struct QDecodeParams {
  ErrWord* err;
  int32_t num_seqs, hq, hkv;
  int32_t group;  // KV heads that consecutive CTAs take side by side
  float scale_log2;
  const uint16_t* q;  // [num_seqs, hq, 128] BF16
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  int32_t n_pages, page_size, max_pages;
  const float* rope_table;  // rotates the query at ctx - 1, or null
  float* out_f32;
  uint16_t* out_bf16;
  float* lse;
  // states of the pairs several CTAs share: row (seg0[s] + segment) * hq + head
  // of state_o [.., 128] and state_ml [.., 2] (m unscaled, l), the first piece's
  // at its last segment; and one count of finished segments per (sequence, KV
  // head)
  float* state_o;
  float* state_ml;
  unsigned long long* counts;
  uint64_t nonce;              // 40 bits, new to every call
  int32_t ctx[kQMaxSeqs];
  int32_t seg0[kQMaxSeqs + 1];  // prefix sums of the sequences' segments
  QStart start[kQMaxParts];
};
cudaError_t configure_qdecode_kernels();
cudaError_t launch_qdecode(const QDecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                           cudaStream_t stream);

// Differential decode over the BF16 pages, cut and folded like the 8-bit one.
// States: row (seg0[s] + segment) * 2 hq + 2 head + map of state_o [.., 128] and
// state_ml [.., 2].
struct DDecodeParams {
  ErrWord* err;
  int32_t num_seqs, hq, hkv;
  int32_t group;  // KV heads that consecutive CTAs take side by side
  float scale_log2;
  const float* lambda;  // [hq]
  const int32_t* page_table;
  int32_t n_pages, page_size, max_pages;
  float* out_f32;
  uint16_t* out_bf16;
  float* lse;  // [num_seqs, hq, 2]
  float* state_o;
  float* state_ml;
  unsigned long long* counts;
  uint64_t nonce;  // 40 bits, new to every call
  int32_t ctx[kQMaxSeqs];
  int32_t seg0[kQMaxSeqs + 1];
  QStart start[kQMaxParts];
};
cudaError_t configure_ddecode_kernels();
cudaError_t launch_ddecode(const DDecodeParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           int grid, cudaStream_t stream);

}  // namespace rlk
