// Block selection: the best num_selected of a row's scores, in increasing block order.
//
// One thread block per (sequence, key head).  A score becomes a 32-bit key that orders as
// the scores do; the key of the last block that is kept is found one 8-bit digit at a
// time from histograms of the keys that agree with it so far (four passes over the row);
// a last pass in block order writes the blocks above it, and of those equal to it the
// lowest.  The sums are of whole numbers, so the result is the same on every run.
#include <cuda_runtime.h>

#include "common.cuh"

namespace pagedkv {
namespace {

constexpr int kThreads = 256;

struct SelectParams {
  const float* scores;
  const int32_t* seq_lens;
  int32_t* selected;
  int32_t* err;
  int num_kv_heads, block_size, max_blocks, num_selected, sink, recent;
};

// Larger scores have larger keys; 0 and -0 the same one; NaN the largest.
__device__ __forceinline__ uint32_t key_of(float s) {
  if (s != s) return 0xffffffffu;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(kThreads) paged_block_select_kernel(const SelectParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int head = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x;
  const size_t row = static_cast<size_t>(seq) * p.num_kv_heads + head;
  int L = __ldg(p.seq_lens + seq);
  const int cap = p.max_blocks * p.block_size;
  if (L < 0 || L > cap) {
    if (head == 0 && tid == 0) report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    L = min(max(L, 0), cap);
  }
  const int nb = static_cast<int>((static_cast<long long>(L) + p.block_size - 1) / p.block_size);
  int32_t* out = p.selected + row * p.num_selected;
  if (nb <= p.num_selected) {
    for (int i = tid; i < p.num_selected; i += kThreads) out[i] = i < nb ? i : -1;
    return;
  }
  const float* s = p.scores + row * p.max_blocks;
  const int begin = p.sink, end = nb - p.recent;  // the blocks that compete
  int want = p.num_selected - p.sink - p.recent;  // how many of them are kept
  __shared__ int hist[256];
  __shared__ int digit_of, above_of;
  __shared__ int warp_sum[2][kThreads / 32];
  uint32_t prefix = 0;  // the last kept key's leading digits
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      hist[tid] = 0;
      __syncthreads();
      for (int i = begin + tid; i < end; i += kThreads) {
        const uint32_t k = key_of(s[i]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int above = 0, d = 255;
        for (; d > 0 && above + hist[d] < want; --d) above += hist[d];
        digit_of = d;
        above_of = above;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(digit_of) << shift;
      want -= above_of;  // now counted among the keys that agree so far
    }
  }
  // want: how many of the keys equal to prefix are kept (the lowest blocks)
  int written = 0, equal_seen = 0;
  const bool any = p.num_selected > p.sink + p.recent;
  for (int base = 0; base < nb; base += kThreads) {
    const int i = base + tid;
    bool above = false, equal = false;
    if (i < nb) {
      if (i < begin || i >= end) {
        above = true;
      } else if (any) {
        const uint32_t k = key_of(s[i]);
        above = k > prefix;
        equal = k == prefix;
      }
    }
    const int lane = tid & 31, warp = tid >> 5;
    const unsigned eq = __ballot_sync(kFullMask, equal);
    if (lane == 0) warp_sum[0][warp] = __popc(eq);
    __syncthreads();
    int before = equal_seen;
    for (int w = 0; w < warp; ++w) before += warp_sum[0][w];
    const bool keep = above || (equal && before + __popc(eq & ((1u << lane) - 1)) < want);
    const unsigned kp = __ballot_sync(kFullMask, keep);
    if (lane == 0) warp_sum[1][warp] = __popc(kp);
    __syncthreads();
    int at = written;
    for (int w = 0; w < warp; ++w) at += warp_sum[1][w];
    if (keep) out[at + __popc(kp & ((1u << lane) - 1))] = i;
    for (int w = 0; w < kThreads / 32; ++w) {
      equal_seen += warp_sum[0][w];
      written += warp_sum[1][w];
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int paged_block_select(const float* scores, const int32_t* seq_lens, int num_seqs,
                                  int num_kv_heads, int block_size, int max_blocks_per_seq,
                                  int num_selected, int sink_blocks, int recent_blocks,
                                  int32_t* selected, int32_t* error_record, void* stream) {
  NvtxRange range("paged_block_select");
  if (num_seqs < 0 || num_kv_heads <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
      num_selected <= 0 || sink_blocks < 0 || recent_blocks < 0 ||
      static_cast<long long>(sink_blocks) + recent_blocks > num_selected)
    return PA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size > (1ll << 30) || num_seqs > 65535 ||
      num_kv_heads > 65535)
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!scores || !seq_lens || !selected) return PA_ERR_INVALID_ARG;
  const SelectParams p{scores, seq_lens, selected, error_record, num_kv_heads, block_size,
                       max_blocks_per_seq, num_selected, sink_blocks, recent_blocks};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(num_kv_heads, num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_block_select_kernel, p) != cudaSuccess) return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
