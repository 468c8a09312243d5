// Block selection: the best num_selected of a row's scores, in increasing block order.
//
// A thread block (for rows of over 16384 blocks a cluster of them) per (sequence, key head), each
// with a contiguous part of the row, of which each warp has a contiguous part in turn: up to 32
// groups of 32 scores, one of each group per lane, read once and kept in registers.  Three
// steps find the last score that is kept:
//  1. The scores between the row's smallest and largest are spread evenly over the bins
//     (subtraction, product and rounding keep their order) and counted; the blocks of a cluster
//     add up each other's counts.  Every score above the bin in which the count reaches
//     num_selected is kept, and as a rule that bin holds a handful.  Skipped where a score is NaN
//     or infinite.
//  2. If the bin holds more than are wanted, its scores, listed in shared memory, are each
//     ranked among one another.  Where they are too many, or the row is a cluster's, or step 1
//     was skipped, a score becomes a 32-bit key that orders as the scores do, and the last kept
//     key is found 9 to 12 bits at a time from histograms of the keys that agree with it so far.
//  3. A vote per group (two, where equal scores are kept in part) tells which of its blocks are
//     kept; lane j takes the votes of group j, a scan of their counts over lanes, warps and
//     blocks says where its blocks go, and it writes them, of equal ones the lowest.
// Sums are of whole numbers, so the result is the same on every run.  Bound by latency (the
// launch and, as a rule, seven barriers) for one sequence (8 rows of 1876 blocks: 3.6 us) and by
// instructions for batches (1280 rows of up to 8192: 23 us): few warps with many groups each for many
// rows, many warps with few groups for few (6464 rows of up to 215: 21 us with 2 warps; before the
// cluster's code left the kernel of one block 22 us, and 45 us with 8 warps).
#include <cuda_runtime.h>

#include "cluster.cuh"
#include "common.cuh"

namespace pagedkv {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kStep = 8;  // groups of a sweep between two looks at how many the warp has

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

// The score of a key (any NaN for that of NaN).
__device__ __forceinline__ float score_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
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

// f(j) for the groups j < `groups`, and up to kStep - 1 more, which no mask names.  Unrolled, so
// that the scores stay in registers.
template <int kGroups, class F>
__device__ __forceinline__ void each_group(int groups, F f) {
#pragma unroll
  for (int j0 = 0; j0 < kGroups; j0 += kStep) {
    if (j0 < groups) {
#pragma unroll
      for (int j = j0; j < j0 + kStep; ++j) f(j);
    }
  }
}

// kGroups: groups of 32 scores per warp, at most 32, one vote for each lane.
// 64 registers a thread: four blocks of 256 threads an SM (1280 rows of up to 8192 blocks: 24.1 us,
// 25.1 us with the 80 registers and three blocks of the compiler's choice).
// kClustered: a row is a cluster's; without that code in it, the kernel of one block does not spill
// (the same case: 23.0 us, 24.0 us with it).
template <int kThreads, int kGroups, bool kClustered>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) paged_block_select_kernel(const SelectParams p) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kPer = 8, kBins = kPer * kThreads;  // bins per thread, and in all
  constexpr int kBits = kThreads == 64 ? 9 : kThreads == 128 ? 10 : kThreads == 256 ? 11 : 12;
  static_assert(kBins == 1 << kBits, "a bin for each digit");
  __shared__ __align__(16) int hist[2][kBins];
  __shared__ uint32_t warp_sum[2][kWarps], warp_range[2][kWarps];
  __shared__ int found[3];  // the bin, the scores above it, the scores in it
  __shared__ uint32_t part_sum[kWarps], block_sum, block_range[2];
  __shared__ int listed;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kClustered ? static_cast<int>(cluster_rank()) : 0;
  const int ranks = kClustered ? static_cast<int>(cluster_size()) : 1;
  const size_t row = blockIdx.x / ranks;
  const int seq = static_cast<int>(row / p.num_kv_heads), head = static_cast<int>(row % p.num_kv_heads);
  for (int i = tid; i < kBins; i += kThreads) hist[0][i] = 0;
  if (tid == 0) listed = 0;
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
    // (unsigned: num_selected may be the largest int, and a step goes past it)
    for (unsigned i = rank * kThreads + tid; i < static_cast<unsigned>(p.num_selected); i += ranks * kThreads)
      out[i] = i < static_cast<unsigned>(nb) ? static_cast<int>(i) : -1;
    return;
  }
  // Groups of 32 blocks per warp of the row, at most kGroups as the capacity is in range.
  const int groups = (nb + 32 * kWarps * ranks - 1) / (32 * kWarps * ranks);
  const int base = (rank * kWarps + warp) * groups * 32;  // the warp's first block
  const float* s = p.scores + row * p.max_blocks + base + lane;
  // Bit j of a mask is this lane's block of group j.  `kept` will be; of `open`, the blocks whose
  // scores compete, `want` of the row's are kept.
  const int mine = nb - base - lane;  // group j has a block if 32 j < mine
  const uint32_t have = bits_below(min((mine + 31) >> 5, groups));
  uint32_t open = bits_below(min((mine - p.recent + 31) >> 5, groups)) &
                  ~bits_below((p.sink - base - lane + 31) >> 5);
  uint32_t kept = have & ~open;
  int want = p.num_selected - p.sink - p.recent;
  float x[kGroups];
  each_group<kGroups>(groups, [&](int j) { x[j] = have >> j & 1 ? s[32 * j] : 0.f; });

  // The bin of hist[turn] in which the count from the top reaches `want`, into `found`.
  auto find = [&](int turn) {
    if constexpr (kClustered) cluster_sync();
    else __syncthreads();
    // thread t has the bins kBins - 1 - t kPer and the kPer - 1 below
    const int bin0 = kBins - (tid + 1) * kPer;
    int bin[kPer];
    if constexpr (!kClustered) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) bin[j] = hist[turn][bin0 + j];
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) bin[j] = 0;
      const uint32_t at = smem_addr(&hist[turn][bin0]);
#pragma unroll 2
      for (int r = 0; r < ranks; ++r) {
        const uint32_t peer = peer_addr(at, r);
#pragma unroll
        for (int j = 0; j < kPer; j += 4) {
          const uint4 v = ld_peer4_u32(peer + 4 * j);
          bin[j] += static_cast<int>(v.x);
          bin[j + 1] += static_cast<int>(v.y);
          bin[j + 2] += static_cast<int>(v.z);
          bin[j + 3] += static_cast<int>(v.w);
        }
      }
    }
    // the other histogram, for the next count: its readers are past the barrier above
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
    want -= found[1];
    return found[0];
  };

  bool ties = false;  // more open blocks than wanted, of the same score
  if (want > 0) {
    int turn = 0;
    bool ranked = false;  // `open` are the blocks with the last kept score
    ties = true;
    {
      float low = INFINITY, high = -INFINITY;  // high is NaN if a score is
      each_group<kGroups>(groups, [&](int j) {
        if (open >> j & 1) {
          low = fminf(low, x[j]);
          high = max_nan(high, x[j]);
        }
      });
      const uint32_t low_key = __reduce_min_sync(kFullMask, key_of(low));
      const uint32_t high_key = __reduce_max_sync(kFullMask, key_of(high));
      if (lane == 0) {
        warp_range[0][warp] = low_key;
        warp_range[1][warp] = high_key;
      }
      __syncthreads();
      uint32_t from = __reduce_min_sync(kFullMask, lane < kWarps ? warp_range[0][lane] : 0xffffffffu);
      uint32_t to = __reduce_max_sync(kFullMask, lane < kWarps ? warp_range[1][lane] : 0u);
      if constexpr (kClustered) {
        if (tid == 0) {
          block_range[0] = from;
          block_range[1] = to;
        }
        cluster_sync();
        const uint32_t at = smem_addr(block_range);
        const uint32_t peer = peer_addr(at, min(lane, ranks - 1));
        from = __reduce_min_sync(kFullMask, ld_peer_u32(peer));
        to = __reduce_max_sync(kFullMask, ld_peer_u32(peer + 4));
      }
      low = score_of(from);
      high = score_of(to);
      // (not so if a score is NaN or infinite, or if all are nearly equal)
      const float scale = (kBins - 1) / (high - low);
      if (low > -INFINITY && high < INFINITY && scale > 0.f && scale < 1e38f) {
        // (v - low) scale to the nearest whole number, in the low bits of a sum with 1.5 * 2^23
        constexpr float kMagic = 12582912.f;
        auto bin_of = [&](float v) { return __float_as_int(fmaf(v - low, scale, kMagic)) - 0x4b400000; };
        each_group<kGroups>(groups, [&](int j) { count_if(open, j, hist[0], bin_of(x[j])); });
        const int last = find(0);
        turn = 1;
        ties = found[2] != want;
        uint32_t same = 0;
        each_group<kGroups>(groups, [&](int j) {
          const int bin = bin_of(x[j]);
          if (bin > last) kept |= open & (1u << j);
          if (bin == last) same |= 1u << j;
        });
        open &= same;
        const int n = found[2];
        if (ties && !kClustered && n <= kThreads) {  // list the bin's scores (over hist[0]) and rank each
          const bool some = __any_sync(kFullMask, open != 0);
          if (some)
            each_group<kGroups>(groups, [&](int j) {
              if (open >> j & 1) hist[0][atomicAdd(&listed, 1)] = static_cast<int>(key_of(x[j]));
            });
          __syncthreads();
          if (tid < n) {
            const uint32_t k = static_cast<uint32_t>(hist[0][tid]);
            int above = 0, equal = 0;
            for (int i = 0; i < n; ++i) {
              const uint32_t v = static_cast<uint32_t>(hist[0][i]);
              above += v > k;
              equal += v == k;
            }
            if (above < want && above + equal >= want) {  // in one thread, or alike in several
              found[0] = static_cast<int>(k);
              found[1] = above;
              found[2] = equal;
            }
          }
          __syncthreads();
          const uint32_t k = static_cast<uint32_t>(found[0]);
          want -= found[1];
          ties = found[2] != want;
          ranked = true;
          if (some) {
            same = 0;
            each_group<kGroups>(groups, [&](int j) {
              const uint32_t v = key_of(x[j]);
              if (v > k) kept |= open & (1u << j);
              if (v == k) same |= 1u << j;
            });
            open &= same;
          }
        }
      }
    }
    uint32_t prefix = 0, known = 0;  // the last kept key's leading bits, and which they are
    for (int top = 32; ties && !ranked && top > 0; top -= kBits, turn ^= 1) {
      const int shift = max(top - kBits, 0);
      const uint32_t digits = (1u << (top - shift)) - 1;
      if (__any_sync(kFullMask, open != 0)) {
        each_group<kGroups>(groups, [&](int j) {
          const uint32_t k = key_of(x[j]);
          count_if((k & known) == prefix ? open : 0u, j, hist[turn], (k >> shift) & digits);
        });
      }
      prefix |= static_cast<uint32_t>(find(turn)) << shift;
      known |= digits << shift;
      ties = found[2] != want;
    }
    if (known != 0 && __any_sync(kFullMask, open != 0)) {
      uint32_t same = 0;
      each_group<kGroups>(groups, [&](int j) {
        const uint32_t k = key_of(x[j]) & known;
        if (k > prefix) kept |= open & (1u << j);
        if (k == prefix) same |= 1u << j;
      });
      open &= same;
    }
    if (!ties) kept |= open;
  }
  // kept: the blocks of `kept` and, with ties, `want` of the row's open ones
  uint32_t over_here = 0, same_here = 0;  // of group `lane`
  each_group<kGroups>(groups, [&](int j) {
    const unsigned over = __ballot_sync(kFullMask, kept >> j & 1);
    if (lane == j) over_here = over;
  });
  if (ties) {
    each_group<kGroups>(groups, [&](int j) {
      const unsigned same = __ballot_sync(kFullMask, open >> j & 1);
      if (lane == j) same_here = same;
    });
  }
  // above in the upper half, equal in the lower (a thread block has at most 2^14 keys)
  const uint32_t count = static_cast<uint32_t>(__popc(over_here)) << 16 | __popc(same_here);
  uint32_t upto = warp_scan(count, lane);
  if (lane == 31) part_sum[warp] = upto;
  __syncthreads();
  upto += __reduce_add_sync(kFullMask, lane < warp ? part_sum[lane] : 0u);
  int at = 0, same = 0;
  if constexpr (kClustered) {
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
  if constexpr (kClustered) cluster_sync();  // no block leaves while another may read its memory
}

int launch(void (*kernel)(SelectParams), const SelectParams& p, dim3 grid, int threads, int ranks,
           cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return PA_ERR_CUDA;
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
  const long long rows = static_cast<long long>(num_seqs) * num_kv_heads;
  const SelectParams p{scores, seq_lens, selected, error_record, num_kv_heads, block_size,
                       max_blocks_per_seq, num_selected, sink_blocks, recent_blocks};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // As many thread blocks a row as its length takes: up to 16384 scores for each.
  int ranks = 1;
  while (ranks < kMaxCluster && max_blocks_per_seq > 16384 * ranks) ranks *= 2;
  if (max_blocks_per_seq > 16384 * ranks) return PA_ERR_UNSUPPORTED;
  if (rows * ranks > 0x7fffffffll) return PA_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(rows * ranks));
  if (ranks > 1) return launch(paged_block_select_kernel<512, 32, true>, p, grid, 512, ranks, st);
  if (rows >= 152 * 4) {
    if (max_blocks_per_seq <= 1024) return launch(paged_block_select_kernel<64, 16, false>, p, grid, 64, 1, st);
    if (max_blocks_per_seq <= 4096)
      return launch(paged_block_select_kernel<128, 32, false>, p, grid, 128, 1, st);
  }
  if (max_blocks_per_seq <= 2048) return launch(paged_block_select_kernel<256, 8, false>, p, grid, 256, 1, st);
  if (max_blocks_per_seq <= 8192) return launch(paged_block_select_kernel<256, 32, false>, p, grid, 256, 1, st);
  return launch(paged_block_select_kernel<512, 32, false>, p, grid, 512, 1, st);
}
