// Launch of one (head dim, type) of the row-tiled kernel, in a translation unit of its own.
#pragma once

#include "row_attn_kernel.cuh"

namespace pda {
namespace row {

constexpr int64_t kSmallTokens = 1 << 18;  // tokens of the block table x kv heads

template <int D, bool FP16, bool MOD>
cudaError_t launch_one(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq,
                       const CUtensorMap& tq1, const Params& p, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<D>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // Not behind shared prefixes: started while the merge before it leaves the SMs, the CTAs
  // come to lie on them in any order, and a wide segment beside an own one on an SM pair
  // slowed some of both (128 sequences of 64/8 heads behind 16384 tokens: 112 us for 97 with
  // weights of one term). A small call, whose segments are a chunk or two, gains by it (8 sequences
  // of 32/8 heads behind 1504 tokens: 16.7 us for 17.4). Between them a limit of 2^20 or 2^22 in
  // place of 2^18 gains 2% at 16 sequences behind 4096 tokens and loses 7% at 64 of 64/8 heads
  // behind 1024. The host knows the table's width only, not the lengths: behind a table of
  // 65536 tokens the small call starts late (16.5 us in a graph for 16.4).
  const int64_t tokens = (int64_t)p.B * p.max_blocks * p.block_size;
  cfg.numAttrs = pdl_enabled() && (p.P == 0 || tokens * p.Hkv <= kSmallTokens) ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, row_attn_kernel<D, FP16, MOD>, tk, tv, tq, tq1, p);
}

template <int D, bool FP16>
cudaError_t prepare_one() {
  cudaError_t e = cudaFuncSetAttribute(row_attn_kernel<D, FP16, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(row_attn_kernel<D, FP16, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kBytes);
  return e;
}

}  // namespace row
}  // namespace pda

#define PDA_ROW_ATTN(dt, D, FP16)                                                                \
  namespace pda {                                                                                \
  namespace row {                                                                                \
  cudaError_t prepare_##dt##_d##D() { return prepare_one<D, FP16>(); }                           \
  cudaError_t launch_##dt##_d##D(const CUtensorMap& tk, const CUtensorMap& tv,                   \
                                 const CUtensorMap& tq, const CUtensorMap& tq1, const Params& p, \
                                 int ctas, cudaStream_t s) {                                     \
    return p.cap > 0.f || p.slopes != nullptr                                                    \
               ? launch_one<D, FP16, true>(tk, tv, tq, tq1, p, ctas, s)                          \
               : launch_one<D, FP16, false>(tk, tv, tq, tq1, p, ctas, s);                        \
  }                                                                                              \
  }                                                                                              \
  }
