// Row-tiled decode attention: dispatch over (head dim, type) and the merge of a row's
// partials.
//
// A row (sequence b, query head) has one partial for every segment and pipe that worked on
// the shared part and on its own part of the context: normalised outputs o_i and base-2
// log-sum-exps lse_i,
//   M = max_i lse_i,  out = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M)
// (an empty partial has lse_i = -inf and is not read). Which ones those are follows from
// the plan that the first kernel left (SeqPlan): a lane each works out where one is. One warp
// a row while there are many rows; four that take the partials in turns where a warp each
// would leave the GPU empty.
#include "row_attn_kernel.cuh"

namespace pda {
namespace row {
namespace {

constexpr int kMergeWarps = 4;
constexpr float kRoom = 10.f;  // weights carry a factor 2^-10: sums of large outputs stay finite
// One warp a row from this many rows an SM on: a block of four warps a row, as below, then takes
// more than a round or two of blocks. (Whole calls with one warp and with four, 64/8 heads: 768
// rows behind 4096 shared tokens 25.0 and 22.2 us, 1024 rows of own tokens 25.8 and 26.8, 1536
// rows 27.1 and 28.8 us, 1536 behind shared tokens 28.2 and 30.4, 6144 rows 40.0 and 50.3.)
constexpr int kManyRowsPerSm = 8;

// The workspace rows of one part of a row's context.
struct Part {
  int kind, n_chunks, x;  // the item, and where the first CTA's range begins in it (<= 0)
  int per;
  int64_t first;  // partial(s) of the segment that starts the item
  int64_t next;   // of the first CTA's slab, as if it held one
  int64_t slab;   // rows from one CTA's slab to the next one's
  int n, m, cap;  // partials, of which m a segment; rows from one pipe's to the next one's in a slab
  // Partial i's row, or -1: a CTA whose range holds no chunk's beginning.
  __device__ __forceinline__ int64_t at(int i) const {
    const int seg = m == 2 ? i >> 1 : i, pipe = m == 2 ? i & 1 : 0;
    if (seg == 0) return first + pipe;
    const int x0 = x + seg * per;
    if (chunk_at(kind, n_chunks, x0) >= chunk_at(kind, n_chunks, x0 + per)) return -1;
    return next + seg * slab + pipe * cap;
  }
};
// x / per by per_mul = floor((2^32 - 1) / per): the product falls short by at most one.
__device__ __forceinline__ int div_per(int x, int per, unsigned per_mul) {
  const int q = (int)__umulhi((unsigned)x, per_mul);
  return q + (x - q * per >= per);
}
__device__ __forceinline__ Part part_of(const Params& p, int64_t row, int kind, int start, int n,
                                        int per, unsigned per_mul, int tile, int r) {
  Part d = {};
  if (n == 0) return d;
  const int c0 = div_per(start, per, per_mul), c1 = div_per(start + item_cost(kind, n) - 1, per, per_mul);
  d.kind = kind;
  d.n_chunks = n;
  d.x = c0 * per - start;
  d.per = per;
  d.cap = ws_cap(p);
  d.m = kind == kWideItem ? 1 : 2;
  d.n = (c1 - c0 + 1) * d.m;
  d.first = ws_first(p, kind == kOwnItem, row, 0);
  d.next = ws_next(p, c0, d.cap, tile, r);
  d.slab = 2 * d.cap;
  return d;
}

template <int D, bool FP16, int WPR>
__global__ void __launch_bounds__(kMergeWarps * 32, WPR == 1 ? 8 : 1) row_merge_kernel(const Params p) {
  constexpr int V = D / 32;   // dims of a lane
  constexpr int U = WPR == 1 ? 4 : 8;  // partials in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.B * p.Hq;
  const int row = WPR == 1 ? blockIdx.x * kMergeWarps + warp : blockIdx.x;
  const int sub = WPR == 1 ? 0 : warp;
  griddep_launch_dependents();
  griddep_wait();
  if (row >= rows) return;
  const int b = row / p.Hq, hq = row - b * p.Hq, h = hq / p.G, g = hq - h * p.G;
  const int per = p.plan[0];
  const unsigned per_mul = (unsigned)p.plan[1];
  const SeqPlan s = reinterpret_cast<const SeqPlan*>(p.plan + kPlanInts)[b];
  const int pr = s.pre_row & (kWide - 1);
  const Part pre = part_of(p, row, s.pre_row >= kWide ? kWideItem : kTileItem,
                           s.pre_start + h * s.pre_stride, s.pre_n, per, per_mul, pr >= kT ? 1 : 0,
                           (pr & (kT - 1)) + g);
  const Part own = part_of(p, row, kOwnItem, s.own_start + h * item_cost(kOwnItem, s.own_n), s.own_n,
                           per, per_mul, 0, g);
  const int n = pre.n + own.n;
  float M = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  // 32 partials at a time, one a lane: where it is and what it weighs
  for (int i0 = sub; i0 < n; i0 += 32 * WPR) {
    const int i = i0 + lane * WPR;
    int64_t at = -1;
    if (i < n) at = i < pre.n ? pre.at(i) : own.at(i - pre.n);
    const float l = at >= 0 ? __ldcg(p.ws_lse + at) : -INFINITY;
    unsigned used = __ballot_sync(kFull, l != -INFINITY);
    if (used == 0) continue;
    float top = l;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    const float Mn = fmaxf(M, top);
    const float a = M == Mn ? 1.f : exp2f(M - Mn);
    sum *= a;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= a;
    M = Mn;
    const float w = l == -INFINITY ? 0.f : exp2f(l - M - kRoom);
    float ws = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ws += __shfl_xor_sync(kFull, ws, off);
    sum += ws;
    while (used) {
      float o[U][V], wu[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        wu[u] = 0.f;
        if (used) {
          const int j = __ffs(used) - 1;
          used &= used - 1;
          wu[u] = __shfl_sync(kFull, w, j);
          const float* src = p.ws_o + __shfl_sync(kFull, at, j) * D + lane * V;
          if constexpr (V == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
            o[u][0] = f.x, o[u][1] = f.y, o[u][2] = f.z, o[u][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
            o[u][0] = f.x, o[u][1] = f.y;
          }
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) o[u][v] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(wu[u], o[u][v], acc[v]);
    }
  }
  if constexpr (WPR > 1) {
    __shared__ float sm[kMergeWarps][D + 2];
    if (lane == 0) {
      sm[warp][D] = M;
      sm[warp][D + 1] = sum;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) sm[warp][lane * V + v] = acc[v];
    __syncthreads();
    if (warp != 0) return;
    float Mn = M;
#pragma unroll
    for (int w = 1; w < kMergeWarps; ++w) Mn = fmaxf(Mn, sm[w][D]);
    if (Mn == -INFINITY) Mn = 0.f;  // no tokens
    float a = exp2f(M - Mn);
    sum *= a;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= a;
#pragma unroll
    for (int w = 1; w < kMergeWarps; ++w) {
      a = exp2f(sm[w][D] - Mn);
      sum = fmaf(a, sm[w][D + 1], sum);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(a, sm[w][lane * V + v], acc[v]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no tokens: zeros
  uint32_t* dst = static_cast<uint32_t*>(p.out) + ((int64_t)row * D + lane * V) / 2;
#pragma unroll
  for (int v = 0; v < V; v += 2) dst[v / 2] = pack16<FP16>(acc[v] * inv, acc[v + 1] * inv);
}

template <int D, bool FP16>
cudaError_t launch_merge_rows(const Params& p, int num_sms, cudaStream_t stream) {
  const int rows = p.B * p.Hq;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  if (rows >= num_sms * kManyRowsPerSm) {
    cfg.gridDim = dim3((unsigned)((rows + kMergeWarps - 1) / kMergeWarps));
    return cudaLaunchKernelEx(&cfg, row_merge_kernel<D, FP16, 1>, p);
  }
  cfg.gridDim = dim3((unsigned)rows);
  return cudaLaunchKernelEx(&cfg, row_merge_kernel<D, FP16, kMergeWarps>, p);
}

}  // namespace

#define PDA_DECLARE_ROW(dt, D)                                                                  \
  cudaError_t prepare_##dt##_d##D();                                                            \
  cudaError_t launch_##dt##_d##D(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,    \
                                 const CUtensorMap&, const Params&, int, cudaStream_t);
PDA_DECLARE_ROW(bf16, 64)
PDA_DECLARE_ROW(bf16, 128)
PDA_DECLARE_ROW(fp16, 64)
PDA_DECLARE_ROW(fp16, 128)
#undef PDA_DECLARE_ROW

cudaError_t prepare(int head_dim, int dtype) {
  if (head_dim == 64) return dtype == 1 ? prepare_fp16_d64() : prepare_bf16_d64();
  return dtype == 1 ? prepare_fp16_d128() : prepare_bf16_d128();
}

cudaError_t launch(int head_dim, int dtype, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CUtensorMap& tq, const CUtensorMap& tq1, const Params& p, int num_sms,
                   cudaStream_t stream) {
  cudaError_t e;
  if (head_dim == 64) {
    e = (dtype == 1 ? launch_fp16_d64 : launch_bf16_d64)(tk, tv, tq, tq1, p, num_sms, stream);
    if (e == cudaSuccess) e = dtype == 1 ? launch_merge_rows<64, true>(p, num_sms, stream) : launch_merge_rows<64, false>(p, num_sms, stream);
  } else {
    e = (dtype == 1 ? launch_fp16_d128 : launch_bf16_d128)(tk, tv, tq, tq1, p, num_sms, stream);
    if (e == cudaSuccess) e = dtype == 1 ? launch_merge_rows<128, true>(p, num_sms, stream) : launch_merge_rows<128, false>(p, num_sms, stream);
  }
  return e;
}

}  // namespace row
}  // namespace pda
