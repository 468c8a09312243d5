// Block selection: the best num_selected of a row's scores, in increasing block order.
//
// A cluster of thread blocks (one, but for few long rows) per (sequence, key head), each with
// a contiguous part of the row.  A score becomes a 32-bit key that orders as the scores do, and
// the keys stay in shared memory.  The key of the last block that is kept is found 11 bits at a
// time from histograms of the keys that agree with it so far (the first digit holds sign,
// exponent and two bits of the fraction, so that ordinary scores spread over the bins), and no
// further than needed to tell the kept from the others; the blocks of a cluster add up each
// other's histograms.  Then each thread counts the blocks above that key and equal to it in a
// run of its own, a scan of the counts says where its run goes, and it writes them; of the
// equal ones the lowest.  Runs of odd length keep the threads of a warp on different banks.
// The sums are of whole numbers, so the result is the same on every run.  The row is read once;
// bound by latency (the launch and some ten barriers) for one sequence and by instructions for
// batches.
#include <cuda_runtime.h>

#include "cluster.cuh"
#include "common.cuh"

namespace pagedkv {
namespace {

constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 49152;  // per thread block: 192 KB of shared memory
constexpr int kAhead = 8;        // loads in flight per thread

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

__device__ __forceinline__ uint32_t warp_scan(uint32_t x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t v = __shfl_up_sync(kFullMask, x, off);
    if (lane >= off) x += v;
  }
  return x;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) paged_block_select_kernel(const SelectParams p) {
  constexpr int kWarps = kThreads / 32, kPer = kBins / kThreads;
  static_assert(kThreads <= kBins, "a thread has a bin at least");
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) int hist[2][kBins];
  __shared__ uint32_t warp_sum[2][kWarps];
  __shared__ int found[3];       // the digit, the keys above it, the keys that have it
  __shared__ uint32_t block_sum;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int head = blockIdx.x / ranks, seq = blockIdx.y;
  for (int i = tid; i < kBins; i += kThreads) hist[0][i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const size_t row = static_cast<size_t>(seq) * p.num_kv_heads + head;
  int L = p.seq_lens[seq];
  const int cap = p.max_blocks * p.block_size;
  if (L < 0 || L > cap) {
    if (head == 0 && rank == 0 && tid == 0) report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    L = min(max(L, 0), cap);
  }
  const int nb = static_cast<int>((static_cast<long long>(L) + p.block_size - 1) / p.block_size);
  int32_t* out = p.selected + row * p.num_selected;
  if (nb <= p.num_selected) {  // alike for all blocks of the cluster
    for (int i = rank * kThreads + tid; i < p.num_selected; i += ranks * kThreads)
      out[i] = i < nb ? i : -1;
    return;
  }
  const int part = (nb + ranks - 1) / ranks;
  const int base = min(nb, rank * part), n = min(part, nb - base);
  const float* s = p.scores + row * p.max_blocks + base;
  // of this part, the blocks begin .. end - 1 compete; `want` of the row's are kept
  const int begin = p.sink - base, end = nb - p.recent - base;
  int want = p.num_selected - p.sink - p.recent;
  __syncthreads();
  for (int i0 = tid; i0 < n; i0 += kAhead * kThreads) {
    float x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kThreads;
      x[j] = i < n ? s[i] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kThreads;
      const uint32_t k = key_of(x[j]);
      if (i < n) keys[i] = k;
      if (i < n && i >= begin && i < end) atomicAdd(&hist[0][k >> (32 - kBits)], 1);
    }
  }
  const int run = ((n + kThreads - 1) / kThreads) | 1;
  const int first = min(n, tid * run), last = min(n, first + run);
  uint32_t prefix = 0xffffffffu, known = 0xffffffffu;  // want = 0: nothing above, none of the equal
  if (want > 0) {
    prefix = known = 0;  // the last kept key's leading bits, and which they are
    for (int top = 32, turn = 0; top > 0; top -= kBits, turn ^= 1) {
      const int shift = max(top - kBits, 0);
      const uint32_t digits = (1u << (top - shift)) - 1;
      if (top < 32) {
        const int from = max(first, begin), to = min(last, end);
        for (int i = from; i < to; ++i) {
          const uint32_t k = keys[i];
          if ((k & known) == prefix) atomicAdd(&hist[turn][(k >> shift) & digits], 1);
        }
      }
      if (ranks > 1) cluster_sync();
      else __syncthreads();
      // thread t has the bins kBins - 1 - t kPer and the kPer - 1 below
      const int bin0 = kBins - (tid + 1) * kPer;
      int bin[kPer];
      if (ranks == 1) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) bin[j] = hist[turn][bin0 + j];
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) bin[j] = 0;
        const uint32_t at = smem_addr(&hist[turn][bin0]);
        for (int r = 0; r < ranks; ++r) {
          const uint32_t peer = peer_addr(at, r);
#pragma unroll
          for (int j = 0; j < kPer; ++j) bin[j] += static_cast<int>(ld_peer_u32(peer + 4 * j));
        }
      }
      // the other histogram, for the next digit: its readers are past the barrier above
#pragma unroll
      for (int j = 0; j < kPer; ++j) hist[turn ^ 1][bin0 + j] = 0;
      int mine = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) mine += bin[j];
      uint32_t upto = warp_scan(mine, lane);
      if (lane == 31) warp_sum[turn][warp] = upto;
      __syncthreads();
      const uint32_t sums = warp_scan(lane < kWarps ? warp_sum[turn][lane] : 0u, lane);
      if (warp > 0) upto += __shfl_sync(kFullMask, sums, max(warp - 1, 0));
      int above = static_cast<int>(upto) - mine;
      if (above < want && static_cast<int>(upto) >= want) {  // in one thread
#pragma unroll
        for (int j = kPer - 1; j >= 0; --j) {
          if (above < want && above + bin[j] >= want) {
            found[0] = bin0 + j;
            found[1] = above;
            found[2] = bin[j];
          }
          above += bin[j];
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(found[0]) << shift;
      known |= digits << shift;
      want -= found[1];
      if (found[2] == want) break;  // every key that agrees so far is kept
    }
  } else {
    __syncthreads();
  }
  // kept: the blocks that do not compete, the keys above, and `want` of the equal ones
  uint32_t count = 0;  // above in the upper half, equal in the lower (n < 2^16)
  for (int i = first; i < last; ++i) {
    const uint32_t k = keys[i] & known;
    const bool in = i >= begin && i < end;
    count += !in || k > prefix ? 0x10000u : k == prefix ? 1u : 0u;
  }
  uint32_t upto = warp_scan(count, lane);
  if (lane == 31) warp_sum[0][warp] = upto;
  __syncthreads();
  const uint32_t sums = warp_scan(lane < kWarps ? warp_sum[0][lane] : 0u, lane);
  if (warp > 0) upto += __shfl_sync(kFullMask, sums, max(warp - 1, 0));
  upto -= count;  // before this thread's run, within the block
  int over = static_cast<int>(upto >> 16), same = static_cast<int>(upto & 0xffffu);
  if (ranks > 1) {
    if (tid == kThreads - 1) block_sum = upto + count;
    cluster_sync();
    const uint32_t at = smem_addr(&block_sum);
    for (int r = 0; r < rank; ++r) {
      const uint32_t v = ld_peer_u32(peer_addr(at, r));
      over += static_cast<int>(v >> 16);
      same += static_cast<int>(v & 0xffffu);
    }
  }
  int at = over + min(same, want);
  if (count != 0) {
    for (int i = first; i < last; ++i) {
      const uint32_t k = keys[i] & known;
      const bool in = i >= begin && i < end;
      bool keep = !in || k > prefix;
      if (in && k == prefix) keep = same++ < want;
      if (keep) out[at++] = base + i;
    }
  }
  if (ranks > 1) cluster_sync();  // no block leaves while another may read its memory
}

template <int kThreads>
int launch(const SelectParams& p, int num_seqs, int ranks, size_t smem, cudaStream_t stream) {
  // Always the same value, so that concurrent callers never lower it for one another, and on
  // every launch that needs it (it is lost with the context).
  if (smem > 24 * 1024 &&
      cudaFuncSetAttribute(paged_block_select_kernel<kThreads>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kMaxKeys * static_cast<int>(sizeof(uint32_t))) != cudaSuccess)
    return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_kv_heads) * ranks, num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, paged_block_select_kernel<kThreads>, p) != cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
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
  // Parts of at least 2048 keys while there are SMs to spare, and at most kMaxKeys.
  const long long rows = static_cast<long long>(num_seqs) * num_kv_heads;
  int ranks = 1;
  while (ranks < kMaxCluster &&
         ((rows * ranks < 152 && max_blocks_per_seq > 4096 * ranks) ||
          max_blocks_per_seq > kMaxKeys * ranks))
    ranks *= 2;
  const int part = (max_blocks_per_seq + ranks - 1) / ranks;
  if (part > kMaxKeys) return PA_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(part) * sizeof(uint32_t);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return part <= 8192 ? launch<256>(p, num_seqs, ranks, smem, st)
                      : launch<1024>(p, num_seqs, ranks, smem, st);
}
