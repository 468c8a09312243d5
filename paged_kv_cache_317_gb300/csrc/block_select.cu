// Block selection: the best num_selected of a row's scores, in increasing block order.
//
// A cluster of thread blocks (one, but for few long rows) per (sequence, key head), each with
// a contiguous part of the row, of which each warp has a contiguous part in turn: up to 32
// groups of 32 scores, one of each group per lane, read once and kept in registers.  A score
// becomes a 32-bit key that orders as the scores do.  The key of the last block that is kept
// is found 11 bits at a time from histograms of the keys that agree with it so far (the first
// digit holds sign, exponent and two bits of the fraction, so that ordinary scores spread over
// the bins), and no further than needed to tell the kept from the others; the blocks of a
// cluster add up each other's histograms.  Then two votes per group tell which of its blocks
// are above that key and which equal to it; lane j takes the votes of group j, a scan of
// their counts over lanes, warps and blocks says where its blocks go, and it writes them, of
// the equal ones the lowest.  The sums are of whole numbers, so the result is the same on every
// run.  Bound by latency (the launch and some ten barriers) for one sequence and by
// instructions for batches.
#include <cuda_runtime.h>

#include "cluster.cuh"
#include "common.cuh"

namespace pagedkv {
namespace {

constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kMaxCluster = 8;
constexpr int kGroups = 32;  // groups of 32 keys per warp: one vote per lane
constexpr int kStep = 8;     // of them between two looks at how many there are

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

// hist[bin] += 1 where bit j of `which` is set: predicated, for a branch per key costs more than
// the rest of a pass.
__device__ __forceinline__ void count_if(uint32_t which, int j, int* hist, uint32_t bin) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 b;\n\t"
      "and.b32 b, %0, %1;\n\t"
      "setp.ne.u32 p, b, 0;\n\t"
      "@p red.shared::cta.add.u32 [%2], 1;\n\t}" ::"r"(which),
      "r"(1u << j), "r"(smem_addr(hist + bin))
      : "memory");
}

// Bits 0 .. n - 1, for any n.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) paged_block_select_kernel(const SelectParams p) {
  constexpr int kWarps = kThreads / 32, kPer = kBins / kThreads;
  static_assert(kThreads <= kBins, "a thread has a bin at least");
  __shared__ __align__(16) int hist[2][kBins];
  __shared__ uint32_t warp_sum[2][kWarps];
  __shared__ int found[3];  // the digit, the keys above it, the keys that have it
  __shared__ uint32_t part_sum[kWarps], block_sum;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int head = blockIdx.x / ranks, seq = blockIdx.y;
  for (int i = tid; i < kBins; i += kThreads) hist[0][i] = 0;
  const size_t row = static_cast<size_t>(seq) * p.num_kv_heads + head;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  // Groups of 32 blocks per warp of the row, at most kGroups as the capacity is in range.
  const int groups = (nb + 32 * kWarps * ranks - 1) / (32 * kWarps * ranks);
  const int base = (rank * kWarps + warp) * groups * 32;  // the warp's first block
  const float* s = p.scores + row * p.max_blocks + base + lane;
  // Of this lane's groups, the ones that have a block, and those whose block competes; `want`
  // of the row's are kept.
  const int mine = nb - base - lane;  // group j has a block if 32 j < mine
  const uint32_t have = bits_below(min((mine + 31) >> 5, groups));
  const uint32_t in = bits_below(min((mine - p.recent + 31) >> 5, groups)) &
                      ~bits_below((p.sink - base - lane + 31) >> 5);
  int want = p.num_selected - p.sink - p.recent;
  uint32_t key[kGroups];
#pragma unroll
  for (int j0 = 0; j0 < kGroups; j0 += kStep) {
    if (j0 < groups) {
#pragma unroll
      for (int j = j0; j < j0 + kStep; ++j)
        key[j] = __float_as_uint(have >> j & 1 ? s[32 * j] : 0.f);
    }
  }
  __syncthreads();  // hist[0] is zero
#pragma unroll
  for (int j0 = 0; j0 < kGroups; j0 += kStep) {
    if (j0 < groups) {
#pragma unroll
      for (int j = j0; j < j0 + kStep; ++j) {
        key[j] = key_of(__uint_as_float(key[j]));
        count_if(in, j, hist[0], key[j] >> (32 - kBits));
      }
    }
  }
  uint32_t prefix = 0xffffffffu, known = 0xffffffffu;  // want = 0: nothing above, none of the equal
  if (want > 0) {
    prefix = known = 0;  // the last kept key's leading bits, and which they are
    for (int top = 32, turn = 0; top > 0; top -= kBits, turn ^= 1) {
      const int shift = max(top - kBits, 0);
      const uint32_t digits = (1u << (top - shift)) - 1;
      if (top < 32) {
#pragma unroll
        for (int j0 = 0; j0 < kGroups; j0 += kStep) {
          if (j0 < groups) {
#pragma unroll
            for (int j = j0; j < j0 + kStep; ++j)
              count_if((key[j] & known) == prefix ? in : 0u, j, hist[turn], (key[j] >> shift) & digits);
          }
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
      int sum = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) sum += bin[j];
      uint32_t upto = warp_scan(sum, lane);
      if (lane == 31) warp_sum[turn][warp] = upto;
      __syncthreads();
      upto += __reduce_add_sync(kFullMask, lane < warp ? warp_sum[turn][lane] : 0u);
      int above = static_cast<int>(upto) - sum;
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
  }
  // kept: the blocks that do not compete, the keys above, and `want` of the equal ones
  uint32_t over_here = 0, same_here = 0;  // of group `lane`
#pragma unroll
  for (int j0 = 0; j0 < kGroups; j0 += kStep) {
    if (j0 < groups) {
#pragma unroll
      for (int j = j0; j < j0 + kStep; ++j) {
        const uint32_t k = key[j] & known;
        const bool inside = in >> j & 1;
        const unsigned over = __ballot_sync(kFullMask, (have >> j & 1) && (!inside || k > prefix));
        const unsigned same = __ballot_sync(kFullMask, inside && k == prefix);
        if (lane == j) {
          over_here = over;
          same_here = same;
        }
      }
    }
  }
  // above in the upper half, equal in the lower (a thread block has at most 2^14 keys)
  const uint32_t count = static_cast<uint32_t>(__popc(over_here)) << 16 | __popc(same_here);
  uint32_t upto = warp_scan(count, lane);
  if (lane == 31) part_sum[warp] = upto;
  __syncthreads();
  upto += __reduce_add_sync(kFullMask, lane < warp ? part_sum[lane] : 0u);
  int at = 0, same = 0;
  if (ranks > 1) {
    if (tid == kThreads - 1) block_sum = upto;
    cluster_sync();
    const uint32_t sum_at = smem_addr(&block_sum);
    for (int r = 0; r < rank; ++r) {
      const uint32_t v = ld_peer_u32(peer_addr(sum_at, r));
      at += static_cast<int>(v >> 16);
      same += static_cast<int>(v & 0xffffu);
    }
  }
  upto -= count;
  at += static_cast<int>(upto >> 16);
  same += static_cast<int>(upto & 0xffffu);
  at += min(same, want);
  int left = max(want - same, 0);  // equal ones that are still kept
  for (uint32_t bits = over_here | same_here; bits != 0; bits &= bits - 1) {
    const int i = __ffs(bits) - 1;
    if (same_here >> i & 1) {
      if (left == 0) continue;
      --left;
    }
    out[at++] = base + 32 * lane + i;
  }
  if (ranks > 1) cluster_sync();  // no block leaves while another may read its memory
}

template <int kThreads>
int launch(const SelectParams& p, int num_seqs, int ranks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_kv_heads) * ranks, num_seqs);
  cfg.blockDim = dim3(kThreads);
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
  // Parts of at least 2048 keys while there are SMs to spare, and at most the 16384 of 16 warps.
  const long long rows = static_cast<long long>(num_seqs) * num_kv_heads;
  int ranks = 1;
  while (ranks < kMaxCluster && ((rows * ranks < 152 && max_blocks_per_seq > 4096 * ranks) ||
                                 max_blocks_per_seq > 16384 * ranks))
    ranks *= 2;
  if (max_blocks_per_seq > 16384 * ranks) return PA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return max_blocks_per_seq <= 8192 * ranks ? launch<256>(p, num_seqs, ranks, st)
                                            : launch<512>(p, num_seqs, ranks, st);
}
