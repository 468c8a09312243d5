// Block scores: the largest logit that a key of a block can have.
//
// With lo <= k <= hi in every channel, q.k <= sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d: a
// matrix product of the queries' positive and negative parts with the two bounds, of which
// the largest over the query heads of a key head is kept.
//  * One warp takes 16 blocks of one key head, on mma.sync m16n8k16 with the blocks as the
//    rows, the channels of hi and then of lo as the inner dimension and the query heads, 8 at
//    a time, as the columns.  Consecutive warps take consecutive heads, whose bounds lie side
//    by side.
//  * A product does not mind in which order the channels come, as long as both operands agree:
//    each lane loads 16 consecutive bytes of its rows and of its head's query and uses them as
//    fragments where they are.  No shared memory, no shuffles on the way in.
//  * Products of two half-precision numbers are exact in fp32, sums are kept in fp32.
// 4 operations per bound and query head: bound by HBM for batches, by latency for one sequence.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "mma.cuh"
#include "rope.cuh"

namespace pagedkv {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;  // blocks per warp

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
  constexpr int kPieces = D / 8;             // 16-byte pieces of a row
  constexpr int kSteps = D / 32;             // pieces of a row that one lane loads
  constexpr int kBatch = kSteps < 4 ? kSteps : 4;  // of them at a time
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int seq = blockIdx.y;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int head = static_cast<int>(item % p.num_kv_heads);
  const long long b0 = item / p.num_kv_heads * kRows;
  int L = p.seq_lens[seq];
  const int cap = p.max_blocks * p.block_size;
  if (L < 0 || L > cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    L = min(max(L, 0), cap);
  }
  if (b0 >= p.max_blocks) return;
  const int nb = static_cast<int>((static_cast<long long>(L) + p.block_size - 1) / p.block_size);
  float* out = p.scores + (static_cast<size_t>(seq) * p.num_kv_heads + head) * p.max_blocks;
  if (b0 >= nb) {
    if (lane < kRows && b0 + lane < p.max_blocks) out[b0 + lane] = -INFINITY;
    return;
  }
  const int g = lane >> 2, tq = lane & 3;
  const int row0 = static_cast<int>(b0) + g;  // this lane's blocks: row0 and row0 + 8
  const uint4* lo[2];
  const uint4* hi[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = min(row0 + 8 * e, nb - 1);  // rows past the last block repeat it, unused
    int blk = p.block_tables[static_cast<size_t>(seq) * p.max_blocks + b];
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
      if (head == 0 && tq == 0 && b == row0 + 8 * e) report_error(p.err, PA_ERR_BAD_BLOCK, seq, blk);
      blk = 0;
    }
    const size_t at = (static_cast<size_t>(blk) * p.num_kv_heads + head) * kPieces + tq;
    lo[e] = static_cast<const uint4*>(p.k_min) + at;
    hi[e] = static_cast<const uint4*>(p.k_max) + at;
  }
  const int group = p.num_heads / p.num_kv_heads;
  const uint4* q = static_cast<const uint4*>(p.q) +
                   (static_cast<size_t>(seq) * p.num_heads + static_cast<size_t>(head) * group) * kPieces + tq;
  float best[2] = {-INFINITY, -INFINITY};
  for (int h0 = 0; h0 < group; h0 += 8) {
    // columns past the last head repeat it
    const uint4* qh = q + static_cast<size_t>(min(h0 + g, group - 1)) * kPieces;
    float up[4] = {0.f, 0.f, 0.f, 0.f}, down[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i0 = 0; i0 < kSteps; i0 += kBatch) {
      uint4 a[kBatch][4], x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        a[i][0] = hi[0][(i0 + i) * 4];
        a[i][1] = hi[1][(i0 + i) * 4];
        a[i][2] = lo[0][(i0 + i) * 4];
        a[i][3] = lo[1][(i0 + i) * 4];
        x[i] = qh[(i0 + i) * 4];
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        const uint4 qp = max8(x[i], zero, Tag{}), qn = min8(x[i], zero, Tag{});
        const uint32_t u0[4] = {a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y};
        const uint32_t u1[4] = {a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w};
        const uint32_t v0[4] = {a[i][2].x, a[i][3].x, a[i][2].y, a[i][3].y};
        const uint32_t v1[4] = {a[i][2].z, a[i][3].z, a[i][2].w, a[i][3].w};
        mma(up, u0, qp.x, qp.y, Tag{});
        mma(down, v0, qn.x, qn.y, Tag{});
        mma(up, u1, qp.z, qp.w, Tag{});
        mma(down, v1, qn.z, qn.w, Tag{});
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      best[e] = max_nan(best[e], max_nan(up[2 * e] + down[2 * e], up[2 * e + 1] + down[2 * e + 1]));
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    best[e] = max_nan(best[e], __shfl_xor_sync(kFullMask, best[e], 1));
    best[e] = max_nan(best[e], __shfl_xor_sync(kFullMask, best[e], 2));
    const int b = row0 + 8 * e;
    if (tq == 0 && b < p.max_blocks) out[b] = b < nb ? best[e] * p.scale : -INFINITY;
  }
}

template <class Tag, int D>
int launch(const ScoreParams& p, int num_seqs, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  const long long items = static_cast<long long>((p.max_blocks + kRows - 1) / kRows) * p.num_kv_heads;
  const long long blocks = (items + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffll) return PA_ERR_INVALID_ARG;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), num_seqs);
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
