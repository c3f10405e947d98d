// Launch boundary of the row-tiled decode-attention kernel (row_attn_kernel.cuh) and
// its merge: shared prefixes, capped and biased scores.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pda {
namespace row {

constexpr int kT = 128;             // tokens of a chunk, and query rows of a tile
constexpr int kMaxPrefixes = 128;   // prefix groups a call may have
constexpr int kMaxBatch = 16384;    // sequences a call may have
constexpr int kPlanInts = 8;        // plan entry of a sequence (SeqPlan)

struct Params {
  const int32_t* block_table;   // [B, max_blocks]
  const int32_t* context_lens;  // [B]
  const int32_t* cu_seqs;       // [P + 1], P = 0: none
  const int32_t* prefix_lens;   // [P]
  const float* slopes;          // [Hq] distance bias per token and head, or null
  void* out;                    // [B, Hq, D]
  float* ws_o;                  // partial rows (normalised outputs), D floats each
  float* ws_lse;                // and their log-sum-exps, base 2
  int* plan;                    // cost per CTA, 2^32 over it; from kPlanInts on SeqPlan of each sequence
  int* err;
  int B, P, Hq, Hkv, G, max_blocks, block_size;
  int bs_log;      // log2(block_size)
  int spt;         // sequences of a row tile: kT / G
  uint32_t tile_mul, group_mul;  // ceil(2^32 / (2 spt)), ceil(2^16 / G)
  int64_t num_blocks;
  int window;      // > 0: only the last `window` tokens
  float qscale;    // scale * log2(e)
  float cap;       // > 0: cap on the scores (natural units)
  float cap_in;    // scale / cap
};

// Rows of partials a call of `batch` sequences may need on `ctas` CTAs.
inline int64_t workspace_rows(int64_t batch, int num_q_heads, int group, int ctas) {
  const int64_t rows = batch * group < kT ? batch * group : kT;
  return 4 * batch * num_q_heads + 2 * rows * ctas;
}

// What the items of a call may cost at most, in the units that the kernel's plan adds up in 32
// bits (item_cost): 6 + 8 a chunk for a sequence's own part of `tokens`. Behind prefixes its
// chunks are one more (both parts end in a part of a chunk), and of a shared item's 14 + 14 a
// chunk a sequence bears half at most: a row tile of 2 kT / G rows is that of two sequences or more.
inline int64_t most_cost(int64_t batch, int num_kv_heads, int64_t tokens, bool prefixes) {
  const int64_t chunks = (tokens + kT - 1) / kT;
  return batch * num_kv_heads * (prefixes ? 6 + 7 + 8 * (chunks + 1) : 6 + 8 * chunks);
}
constexpr int64_t kMostCost = int64_t{1} << 30;  // half of what 32 bits hold: room for a CTA's range on top

// 16-bit K/V, head dim 64 or 128, any group size up to 16.
inline bool supported(int group, int head_dim) {
  return group >= 1 && group <= 16 && (head_dim == 64 || head_dim == 128);
}

cudaError_t prepare(int head_dim, int dtype);
// tmap_q: boxes of kT / G sequences' G rows; tmap_q1: of one sequence's.
cudaError_t launch(int head_dim, int dtype, const CUtensorMap& tmap_k, const CUtensorMap& tmap_v,
                   const CUtensorMap& tmap_q, const CUtensorMap& tmap_q1, const Params& p,
                   int num_sms, cudaStream_t stream);

}  // namespace row
}  // namespace pda
