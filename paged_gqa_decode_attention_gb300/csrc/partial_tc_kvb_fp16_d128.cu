// Instantiations of the tensor-core split-K partial kernel for block-scaled FP8 (E4M3)
// K/V caches with fp16 queries and head dim 128.
#include "partial_tc_kernel.cuh"

namespace pda {

cudaError_t launch_partial_tc_kvb_fp16_d128(int G, int BS, const CUtensorMap* tk,
                                            const CUtensorMap* tv, const CUtensorMap* tq,
                                            const PartialParams& p, cudaStream_t s) {
  return tc::Dispatch<128, true, true, 1, 8, true>::launch(G, BS, tk, tv, tq, p, s);
}

cudaError_t prepare_partial_tc_kvb_fp16_d128(int G, int BS) {
  return tc::Dispatch<128, true, true, 1, 8, true>::prepare(G, BS);
}

int occupancy_partial_tc_kvb_fp16_d128(int G, int BS) {
  return tc::Dispatch<128, true, true, 1, 8, true>::occupancy(G, BS);
}

int max_clusters_partial_tc_kvb_fp16_d128(int G, int BS, int cluster) {
  return tc::Dispatch<128, true, true, 1, 8, true>::max_clusters(G, BS, cluster);
}

}  // namespace pda
