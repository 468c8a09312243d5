// Block scores: the largest logit that a key of a block can have.
//
// With lo <= k <= hi in every channel, q.k <= sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d: a
// matrix product of the queries' positive and negative parts with the two bounds, of which
// the largest over the query heads of a key head is kept.
//  * One warp takes up to 64 blocks of one key head, 16 at a time, on mma.sync m16n8k16 with
//    the blocks as the rows, the channels of hi and then of lo as the inner dimension and the
//    query heads, 8 at a time, as the columns.  Consecutive warps take consecutive heads,
//    whose bounds lie side by side.
//  * A warp copies whole rows, asynchronously, into a ring of its own in shared memory: the next
//    16 blocks are on their way during the products (64-byte pieces of rows instead: 38.5 us).
//  * A product does not mind in which order the channels come, as long as both operands agree:
//    each lane takes 16 consecutive bytes of its rows and of its head's query and uses them as
//    fragments where they are.
//  * Products of two half-precision numbers are exact in fp32, sums are kept in fp32; the matrix
//    units cut sums off instead of rounding them: a score is off by up to 2.6e-7 of the terms'
//    magnitudes as measured (rms of the batch below relative to its scores: 1.3e-7, with plain fp32
//    sums 0.95e-7).
// 4 operations per bound and query head: bound by HBM for batches (48 contexts of up to 32768
// tokens, 8 key heads x 8, 225 MB: 37 us, 6.0 TB/s), by latency for one sequence (3.1 us).
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "mma.cuh"
#include "rope.cuh"

namespace pagedkv {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;    // blocks per matrix product
constexpr int kMaxTiles = 4; // of 16 blocks per warp

struct ScoreParams {
  const void* q;
  const void* k_min;
  const void* k_max;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  float* scores;
  int32_t* err;
  int num_heads, num_kv_heads, block_size, max_blocks, num_blocks;
  int tiles;  // of 16 blocks per warp
  float scale;
};

__device__ __forceinline__ void copy_async16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// kStages: 16-block tiles in the ring; 1 where a warp has one tile, else 2 (48 contexts, 225 MB:
// 37.0 us with 2, 40.6 us with 3: more warps on an SM count for more than deeper rings).
template <class Tag, int D, int kStages>
__global__ void __launch_bounds__(kWarps * 32) paged_block_scores_kernel(const ScoreParams p) {
  constexpr int kPieces = D / 8;         // 16-byte pieces of a row
  constexpr int kSteps = D / 32;         // pieces of a row that one lane takes
  constexpr int kAhead = kSteps < 4 ? kSteps : 4;  // of them at a time
  extern __shared__ uint4 ring[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seq = blockIdx.y;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int head = static_cast<int>(item % p.num_kv_heads);
  const long long b0 = item / p.num_kv_heads * (kRows * p.tiles);  // the warp's first block
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (b0 >= p.max_blocks) return;
  // Block numbers of blocks b0 + lane and b0 + 32 + lane, fetched along with the length,
  // before it says which ones count.
  const int32_t* table = p.block_tables + static_cast<size_t>(seq) * p.max_blocks;
  int blk[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    blk[e] = table[min(b0 + 32 * e + lane, static_cast<long long>(p.max_blocks - 1))];
  int L = p.seq_lens[seq];
  const int cap = p.max_blocks * p.block_size;
  if (L < 0 || L > cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    L = min(max(L, 0), cap);
  }
  const int nb = static_cast<int>((static_cast<long long>(L) + p.block_size - 1) / p.block_size);
  float* out = p.scores + (static_cast<size_t>(seq) * p.num_kv_heads + head) * p.max_blocks;
  const int end = static_cast<int>(min(b0 + kRows * p.tiles, static_cast<long long>(p.max_blocks)));
  for (int b = max(static_cast<int>(b0), nb) + lane; b < end; b += 32) out[b] = -INFINITY;
  if (b0 >= nb) return;
  const int first = static_cast<int>(b0), held = min(end, nb) - first;  // blocks with a score
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (32 * e + lane < held && static_cast<unsigned>(blk[e]) >= static_cast<unsigned>(p.num_blocks)) {
      if (head == 0) report_error(p.err, PA_ERR_BAD_BLOCK, seq, blk[e]);
      blk[e] = 0;
    }
  }
  const int g = lane >> 2, tq = lane & 3;
  // A stage is hi then lo, [16 rows][pieces], odd rows with their 64-byte halves exchanged, so that
  // the rows g and g + 1 that a quarter of a warp reads at the same pieces lie on other banks.
  uint4* mine = ring + static_cast<size_t>(warp) * kStages * kPieces * 32;
  // Copies tile t into stage t % kStages, whole rows at a time: kPieces lanes to a row.
  const int my_row = lane / kPieces, my_piece = lane % kPieces;
  auto issue = [&](int t) {
    if (16 * t < held) {
      uint4* dst = mine + (t % kStages) * kPieces * 32 + lane / kPieces * kPieces;
#pragma unroll
      for (int r0 = 0; r0 < kRows; r0 += 32 / kPieces) {
        const int r = r0 + my_row;
        const int b = __shfl_sync(kFullMask, t < 2 ? blk[0] : blk[1], (t & 1) * 16 + r);
        if (16 * t + r < held) {  // the other rows' products are not used
          const size_t at = (static_cast<size_t>(b) * p.num_kv_heads + head) * kPieces + my_piece;
          const int to = r0 * kPieces + (my_piece ^ ((r & 1) << 2));
          copy_async16(dst + to, static_cast<const uint4*>(p.k_max) + at);
          copy_async16(dst + kRows * kPieces + to, static_cast<const uint4*>(p.k_min) + at);
        }
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int t = 0; t < kStages - 1; ++t) issue(t);

  const int group = p.num_heads / p.num_kv_heads;
  const size_t q0 = static_cast<size_t>(seq) * p.num_heads + static_cast<size_t>(head) * group;
  const uint4* q = static_cast<const uint4*>(p.q) + q0 * kPieces + tq;
  for (int t = 0; 16 * t < held; ++t) {
    issue(t + kStages - 1);
    uint4 x[kAhead];
    auto fetch = [&](int h0, int i0) {  // columns past the last head repeat it
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        x[i] = q[static_cast<size_t>(min(h0 + g, group - 1)) * kPieces + 4 * (i0 + i)];
    };
    fetch(0, 0);
    copy_wait<kStages - 1>();
    __syncwarp();
    const uint4* src = mine + (t % kStages) * kPieces * 32 + g * kPieces;
    float best[2] = {-INFINITY, -INFINITY};
    for (int h0 = 0; h0 < group; h0 += 8) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int i0 = 0; i0 < kSteps; i0 += kAhead) {
        if (h0 + i0 > 0) fetch(h0, i0);
        // four products to a sum, then the sums: the tensor cores drop bits at every addition
        float up[kAhead / 2][4], down[kAhead / 2][4];
#pragma unroll
        for (int i = 0; i < kAhead / 2; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) up[i][e] = down[i][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          const uint4 qp = max8(x[i], zero, Tag{}), qn = min8(x[i], zero, Tag{});
          const int at = (4 * (i0 + i) + tq) ^ ((g & 1) << 2);
          const uint4 h_0 = src[at], h_1 = src[8 * kPieces + at];
          const uint4 l_0 = src[16 * kPieces + at], l_1 = src[24 * kPieces + at];
          const uint32_t u0[4] = {h_0.x, h_1.x, h_0.y, h_1.y}, u1[4] = {h_0.z, h_1.z, h_0.w, h_1.w};
          const uint32_t v0[4] = {l_0.x, l_1.x, l_0.y, l_1.y}, v1[4] = {l_0.z, l_1.z, l_0.w, l_1.w};
          mma(up[i / 2], u0, qp.x, qp.y, Tag{});
          mma(down[i / 2], v0, qn.x, qn.y, Tag{});
          mma(up[i / 2], u1, qp.z, qp.w, Tag{});
          mma(down[i / 2], v1, qn.z, qn.w, Tag{});
        }
#pragma unroll
        for (int i = 0; i < kAhead / 2; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] += up[i][e] + down[i][e];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) best[e] = max_nan(best[e], max_nan(sum[2 * e], sum[2 * e + 1]));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      best[e] = max_nan(best[e], __shfl_xor_sync(kFullMask, best[e], 1));
      best[e] = max_nan(best[e], __shfl_xor_sync(kFullMask, best[e], 2));
      if (tq == 0 && 16 * t + 8 * e + g < held) out[first + 16 * t + 8 * e + g] = best[e] * p.scale;
    }
    __syncwarp();  // the stage is read
  }
  copy_wait<0>();
}

template <class Tag, int D, int kStages>
int launch(const ScoreParams& p, long long blocks, int num_seqs, cudaStream_t stream) {
  constexpr int smem = kWarps * kStages * (D / 8) * 32 * 16;
  // on every launch that needs it (the attribute is lost with the context)
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(paged_block_scores_kernel<Tag, D, kStages>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), num_seqs);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_block_scores_kernel<Tag, D, kStages>, p) != cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <class Tag, int D>
int launch(ScoreParams p, int num_seqs, cudaStream_t stream) {
  // 64 blocks per warp, down to 16 while that leaves fewer than 8 warps for each SM
  const auto warps = [&](int tiles) {
    return (p.max_blocks + kRows * tiles - 1) / (kRows * tiles) * static_cast<long long>(p.num_kv_heads);
  };
  p.tiles = kMaxTiles;
  while (p.tiles > 1 && warps(p.tiles) * num_seqs < 152 * 8) p.tiles /= 2;
  const long long blocks = (warps(p.tiles) + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffll) return PA_ERR_INVALID_ARG;
  return p.tiles == 1 ? launch<Tag, D, 1>(p, blocks, num_seqs, stream)
                      : launch<Tag, D, 2>(p, blocks, num_seqs, stream);
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
                      num_kv_heads, block_size, max_blocks_per_seq, num_blocks, 0, scale};
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
