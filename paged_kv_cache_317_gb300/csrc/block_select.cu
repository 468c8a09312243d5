// Block selection: the best num_selected of a row's scores, in increasing block order.
//
// One thread block per (sequence, key head).  A score becomes a 32-bit key that orders as
// the scores do.  The key of the last block that is kept is found 11 bits at a time from
// histograms of the keys that agree with it so far (the first digit holds sign, exponent and
// two bits of the fraction, so that ordinary scores spread over the bins), and no further than
// needed to tell the kept from the others.  Then each warp goes over a contiguous part of the
// row twice: it counts the blocks above that key and equal to it, and, knowing the counts of
// the parts before, writes them; of the equal ones the lowest.  The sums are of whole numbers,
// so the result is the same on every run.  The row is read once from memory and from the L1
// cache after that; bound by latency (of the launch and of a dozen barriers) for one sequence
// and by instructions for batches.
#include <cuda_runtime.h>

#include "common.cuh"

namespace pagedkv {
namespace {

constexpr int kBits = 11, kBins = 1 << kBits;

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

template <int kThreads>
__global__ void __launch_bounds__(kThreads) paged_block_select_kernel(const SelectParams p) {
  constexpr int kWarps = kThreads / 32, kPer = kBins / kThreads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int head = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const size_t row = static_cast<size_t>(seq) * p.num_kv_heads + head;
  int L = p.seq_lens[seq];
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
  __shared__ int hist[kBins];
  __shared__ int warp_sum[kWarps];
  __shared__ int found[3];  // the digit, the keys above it, the keys that have it
  uint32_t prefix = 0, known = 0;  // the last kept key's leading bits, and which they are
  int equal = 0;                   // keys that agree with it in those
  if (want > 0) {
    for (int top = 32; top > 0; top -= kBits) {
      const int shift = max(top - kBits, 0);
      const uint32_t digits = (1u << (top - shift)) - 1;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int i = begin + tid; i < end; i += kThreads) {
        const uint32_t k = key_of(s[i]);
        if ((k & known) == prefix) atomicAdd(&hist[(k >> shift) & digits], 1);
      }
      __syncthreads();
      // thread t sums the bins kBins - 1 - t kPer and the kPer - 1 below; then the sums of all
      // bins above, warp by warp
      int mine = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) mine += hist[kBins - 1 - tid * kPer - j];
      int upto = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(kFullMask, upto, off);
        if (lane >= off) upto += v;
      }
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      for (int w = 0; w < warp; ++w) upto += warp_sum[w];
      int above = upto - mine;
      if (above < want && upto >= want) {  // in one thread
        int bin = kBins - 1 - tid * kPer;
        while (above + hist[bin] < want) above += hist[bin--];
        found[0] = bin;
        found[1] = above;
        found[2] = hist[bin];
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(found[0]) << shift;
      known |= digits << shift;
      want -= found[1];
      equal = found[2];
      if (equal == want) break;  // every key that agrees so far is kept
    }
  } else {
    known = prefix = 0xffffffffu;  // none above it, and none of the equal ones is kept
  }
  // kept: the blocks that do not compete, the keys above, and `want` of the equal ones
  const int part = (nb + kWarps - 1) / kWarps, first = min(nb, warp * part);
  const int last = min(nb, first + part);
  auto classify = [&](int i, bool& over, bool& same) {
    over = same = false;
    if (i >= last) return;
    if (i < begin || i >= end) {
      over = true;
      return;
    }
    const uint32_t k = key_of(s[i]) & known;
    over = k > prefix;
    same = k == prefix;
  };
  int overs = 0, sames = 0;
#pragma unroll 4
  for (int i = first; i < last; i += 32) {
    bool over, same;
    classify(i + lane, over, same);
    overs += over;
    sames += same;
  }
  overs = __reduce_add_sync(kFullMask, overs);
  sames = __reduce_add_sync(kFullMask, sames);
  __syncthreads();
  if (lane == 0) {
    warp_sum[warp] = overs;
    hist[warp] = sames;
  }
  __syncthreads();
  int at = 0, seen = 0;  // kept and equal blocks before this warp's part
  for (int w = 0; w < warp; ++w) {
    at += warp_sum[w];
    seen += hist[w];
  }
  at += min(seen, want);
  const unsigned below = (1u << lane) - 1;
#pragma unroll 2
  for (int i = first; i < last; i += 32) {
    bool over, same;
    classify(i + lane, over, same);
    const unsigned eq = __ballot_sync(kFullMask, same);
    const bool keep = over || (same && seen + __popc(eq & below) < want);
    const unsigned kp = __ballot_sync(kFullMask, keep);
    if (keep) out[at + __popc(kp & below)] = i + lane;
    seen += __popc(eq);
    at += __popc(kp);
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
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool wide = max_blocks_per_seq > 16384;
  cfg.blockDim = dim3(wide ? 1024 : 512);
  if (cudaLaunchKernelEx(&cfg, wide ? paged_block_select_kernel<1024> : paged_block_select_kernel<512>,
                         p) != cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
