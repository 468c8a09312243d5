// Block scores: the largest logit that a key of a block can have.
//
// With lo <= k <= hi in every channel, q.k <= sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d: a
// matrix product of the queries' positive and negative parts with the two bounds.  One
// warp takes one (sequence, key head, block): the lanes share the channels.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"

namespace pagedkv {
namespace {

constexpr int kWarps = 8;

struct ScoreParams {
  const void* q;
  const void* k_min;
  const void* k_max;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  float* scores;
  int32_t* err;
  int num_heads, num_kv_heads, block_size, max_blocks, num_blocks;
  float scale;
};

template <class Tag, int D>
__global__ void __launch_bounds__(kWarps * 32) paged_block_scores_kernel(const ScoreParams p) {
  using T = typename Tag::T;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int head = blockIdx.y, seq = blockIdx.z;
  int L = __ldg(p.seq_lens + seq);
  const int cap = p.max_blocks * p.block_size;
  if (L < 0 || L > cap) {
    if (blockIdx.x == 0 && head == 0 && threadIdx.x == 0)
      report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    L = min(max(L, 0), cap);
  }
  if (b >= p.max_blocks) return;
  float* out = p.scores + (static_cast<size_t>(seq) * p.num_kv_heads + head) * p.max_blocks + b;
  if (static_cast<long long>(b) * p.block_size >= L) {
    if (lane == 0) *out = -INFINITY;
    return;
  }
  int blk = __ldg(p.block_tables + static_cast<size_t>(seq) * p.max_blocks + b);
  if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
    if (head == 0 && lane == 0) report_error(p.err, PA_ERR_BAD_BLOCK, seq, blk);
    blk = 0;
  }
  const int group = p.num_heads / p.num_kv_heads;
  const size_t at = (static_cast<size_t>(blk) * p.num_kv_heads + head) * D;
  const T* lo = static_cast<const T*>(p.k_min) + at;
  const T* hi = static_cast<const T*>(p.k_max) + at;
  const T* q = static_cast<const T*>(p.q) +
               (static_cast<size_t>(seq) * p.num_heads + static_cast<size_t>(head) * group) * D;
  float best = -INFINITY;
  for (int g = 0; g < group; ++g) {
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < D; d += 32) {
      const float x = static_cast<float>(q[static_cast<size_t>(g) * D + d + lane]);
      s = fmaf(max_nan(x, 0.f), static_cast<float>(hi[d + lane]), s);
      s = fmaf(-max_nan(-x, 0.f), static_cast<float>(lo[d + lane]), s);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFullMask, s, off);
    best = max_nan(best, s);
  }
  if (lane == 0) *out = best * p.scale;
}

template <class Tag, int D>
int launch(const ScoreParams& p, int num_seqs, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((p.max_blocks + kWarps - 1) / kWarps, p.num_kv_heads, num_seqs);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_block_scores_kernel<Tag, D>, p) != cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int paged_block_scores(const void* q, const void* k_min, const void* k_max,
                                  const int32_t* block_tables, const int32_t* seq_lens,
                                  int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                  int block_size, int max_blocks_per_seq, int num_blocks,
                                  float scale, int dtype, float* scores, int32_t* error_record,
                                  void* stream) {
  NvtxRange range("paged_block_scores");
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || !(scale > 0.f)) return PA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size > (1ll << 30) || num_seqs > 65535 ||
      num_kv_heads > 65535)
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_min || !k_max || !block_tables || !seq_lens || !scores) return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_min) || !aligned16(k_max)) return PA_ERR_INVALID_ARG;
  const ScoreParams p{q, k_min, k_max, block_tables, seq_lens, scores, error_record, num_heads,
                      num_kv_heads, block_size, max_blocks_per_seq, num_blocks, scale};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == PA_BF16) {
    switch (head_dim) {
      case 64: return launch<BF16, 64>(p, num_seqs, st);
      case 128: return launch<BF16, 128>(p, num_seqs, st);
      default: return launch<BF16, 256>(p, num_seqs, st);
    }
  }
  switch (head_dim) {
    case 64: return launch<F16, 64>(p, num_seqs, st);
    case 128: return launch<F16, 128>(p, num_seqs, st);
    default: return launch<F16, 256>(p, num_seqs, st);
  }
}
