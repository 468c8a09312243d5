// Decode attention over listed blocks.
//
// One warp takes one (sequence, query head): the lanes share the channels, and the tokens
// of the listed blocks go by one at a time with a running maximum and sum.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"

namespace pagedkv {
namespace {

constexpr int kWarps = 4;

struct SparseParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* selected;
  void* out;
  int32_t* err;
  int num_selected, num_seqs, num_heads, num_kv_heads, block_size, max_blocks, num_blocks;
  int out_dtype;
  float scale;
};

template <class Tag, int D>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_sparse_kernel(const SparseParams p) {
  using T = typename Tag::T;
  constexpr int DPL = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.num_seqs) * p.num_heads) return;
  const int seq = static_cast<int>(row / p.num_heads), g = static_cast<int>(row % p.num_heads);
  const int group = p.num_heads / p.num_kv_heads, head = g / group;
  const bool reports = lane == 0 && g % group == 0;
  int L = __ldg(p.seq_lens + seq);
  const int cap = p.max_blocks * p.block_size;
  if (L < 0 || L > cap) {
    if (lane == 0 && g == 0) report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    L = min(max(L, 0), cap);
  }
  float q[DPL], acc[DPL];
#pragma unroll
  for (int j = 0; j < DPL; ++j) {
    q[j] = static_cast<float>(static_cast<const T*>(p.q)[row * D + lane * DPL + j]);
    acc[j] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  bool some = false;
  const size_t list = (static_cast<size_t>(seq) * p.num_kv_heads + head) * p.num_selected;
  for (int e = 0; e < p.num_selected; ++e) {
    const int b = __ldg(p.selected + list + e);
    if (b < -1 || b >= p.max_blocks) {
      if (reports) report_error(p.err, PA_ERR_BAD_BLOCK, static_cast<long long>(seq) * p.num_kv_heads + head, b);
      continue;
    }
    if (b < 0) continue;
    const long long t0 = static_cast<long long>(b) * p.block_size;
    const int rows = static_cast<int>(min(static_cast<long long>(p.block_size), L - t0));
    if (rows <= 0) continue;
    some = true;
    int blk = __ldg(p.block_tables + static_cast<size_t>(seq) * p.max_blocks + b);
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
      if (reports && head == 0) report_error(p.err, PA_ERR_BAD_BLOCK, seq, blk);
      blk = 0;
    }
    const size_t at = (static_cast<size_t>(blk) * p.num_kv_heads + head) * p.block_size * D + lane * DPL;
    for (int r = 0; r < rows; ++r) {
      const T* k = static_cast<const T*>(p.k_cache) + at + static_cast<size_t>(r) * D;
      const T* v = static_cast<const T*>(p.v_cache) + at + static_cast<size_t>(r) * D;
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < DPL; ++j) s = fmaf(q[j], static_cast<float>(k[j]), s);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFullMask, s, off);
      s *= p.scale;
      const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
      const float alpha = expf(m - base), w = expf(s - base);
      l = fmaf(l, alpha, w);
#pragma unroll
      for (int j = 0; j < DPL; ++j) acc[j] = fmaf(acc[j], alpha, w * static_cast<float>(v[j]));
      m = mn;
    }
  }
  const float inv = some ? 1.f / l : 0.f;
#pragma unroll
  for (int j = 0; j < DPL; ++j) acc[j] *= inv;
  store_out<DPL>(p.out, row * D + lane * DPL, acc, p.out_dtype);
}

template <class Tag, int D>
int launch(const SparseParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.num_seqs) * p.num_heads;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_attn_sparse_kernel<Tag, D>, p) != cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int paged_attn_sparse(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* block_tables, const int32_t* seq_lens,
                                 const int32_t* selected, int num_selected, int num_seqs,
                                 int num_heads, int num_kv_heads, int head_dim, int block_size,
                                 int max_blocks_per_seq, int num_blocks, float scale, int dtype,
                                 void* out, int out_dtype, int32_t* error_record, void* stream) {
  NvtxRange range("paged_attn_sparse");
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || num_selected < 0)
    return PA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (block_size % 16 != 0 && block_size != 8) return PA_ERR_UNSUPPORTED;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (out_dtype != PA_F16 && out_dtype != PA_BF16 && out_dtype != PA_F32)
    return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size > (1ll << 30) || num_seqs > 65535 ||
      num_heads > 65535)
    return PA_ERR_INVALID_ARG;
  if (static_cast<long long>(num_blocks) * num_kv_heads * block_size >= (1ll << 31))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !out ||
      (!selected && num_selected > 0))
    return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return PA_ERR_INVALID_ARG;
  const SparseParams p{q, k_cache, v_cache, block_tables, seq_lens, selected, out, error_record,
                       num_selected, num_seqs, num_heads, num_kv_heads, block_size,
                       max_blocks_per_seq, num_blocks, out_dtype, scale};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == PA_BF16) {
    switch (head_dim) {
      case 64: return launch<BF16, 64>(p, st);
      case 128: return launch<BF16, 128>(p, st);
      default: return launch<BF16, 256>(p, st);
    }
  }
  switch (head_dim) {
    case 64: return launch<F16, 64>(p, st);
    case 128: return launch<F16, 128>(p, st);
    default: return launch<F16, 256>(p, st);
  }
}
