// Append with rotary positions: one pass that rotates a step's queries and keys,
// writes keys and values into their slots and keeps the touched blocks' key bounds.
//
// The work is cut into tiles: the new tokens of one sequence that fall into one
// block.  A thread takes 16 dims (two 16-byte pieces, 8 rotary pairs) of one head of
// q, k or v and walks the tile's rows, so that a key thread sees every new key of its
// block and channel and holds their minimum and maximum in registers: the bounds need
// no atomics and no second pass, and come out the same on every run.
// The cosines and sines of a tile with several rows or axes are brought into shared
// memory once for all of the thread block's heads, while the first rows are loading.
// The rotation is 3 operations per element, the traffic one read and one write of
// each q, k and v element: the kernel is bound by HBM for prompts and by latency for
// decode steps.
#include <cuda_runtime.h>

#include "common.cuh"
#include "rope.cuh"

namespace pagedkv {
namespace {

constexpr int kThreads = 128;

struct AppendRopeParams {
  const void* q;  // null: keys and values only
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* query_start;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  void* k_cache;
  void* v_cache;
  void* k_min;  // null: no bounds
  void* k_max;
  void* q_out;
  int32_t* err;
  int total_tokens, max_query_len, num_seqs, num_heads, num_kv_heads, head_dim;
  int block_size, max_blocks, num_blocks;
  int tiles;  // tile slots of the grid; blocks past them check the sequences
  RopeParams rope;
};

// A sequence's new tokens are rows first .. first + count of q, k and v, and places
// len - count .. len - 1 of the sequence.
struct Range {
  int first, count, len;
};

__device__ __forceinline__ bool range_of(const AppendRopeParams& p, int seq, Range& r) {
  const int begin = p.query_start[seq], end = p.query_start[seq + 1];
  const int len = p.seq_lens[seq];
  r = {begin, end - begin, len};
  return begin >= 0 && end >= begin && end <= p.total_tokens && end - begin <= p.max_query_len &&
         len <= static_cast<long long>(p.max_blocks) * p.block_size && end - begin <= len;
}

// The first tile slot of a sequence.  n tokens touch at most (n - 1) / bs + 2 blocks,
// and query_start[i + 1] / bs - query_start[i] / bs + 2 is never less, so the slots of
// consecutive sequences do not overlap and are found from query_start alone.
__device__ __forceinline__ long long first_slot(const AppendRopeParams& p, int seq) {
  return static_cast<long long>(p.query_start[seq]) / p.block_size + 2ll * seq;
}

// kRows: rows of cosines and sines in shared memory; kBatch: rows that a thread loads at a time.
// A step of one token a sequence needs one row of each, and leaves the SM to more threads (256 x
// 40 heads: 7.0 us, against 8.5 us with the 16 and 4 of prompts).
template <class Tag, int kRows, int kBatch>
__global__ void __launch_bounds__(kThreads) kv_append_rope_kernel(const AppendRopeParams p) {
  using T = typename Tag::T;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int slot = blockIdx.x;
  int seq = slot, tile = 0;
  if constexpr (kRows > 1) {
    if (slot >= p.tiles) {  // check the sequences' ranges; tiles skip the bad ones silently
      const int i = (slot - p.tiles) * kThreads + threadIdx.x;
      Range r;
      if (blockIdx.y == 0 && i < p.num_seqs && !range_of(p, i, r))
        report_error(p.err, PA_ERR_BAD_SEQ_LEN, i, r.len);
      return;
    }
    int lo = 0, hi = p.num_seqs - 1;  // the last sequence whose slots begin at or before this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first_slot(p, mid) <= slot) lo = mid;
      else hi = mid - 1;
    }
    seq = lo;
    const long long t = slot - first_slot(p, seq);
    if (t < 0) return;
    tile = static_cast<int>(t);
  }
  Range rg;
  if (!range_of(p, seq, rg)) {
    if (kRows == 1 && threadIdx.x == 0 && blockIdx.y == 0)
      report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, rg.len);
    return;
  }
  if (rg.count == 0) return;
  const int place0 = rg.len - rg.count;  // place of the sequence's first new token
  const int block = place0 / p.block_size + tile;  // logical block of this tile
  const long long lo_place = max(static_cast<long long>(block) * p.block_size,
                                 static_cast<long long>(place0));
  const long long hi_place = min((static_cast<long long>(block) + 1) * p.block_size,
                                 static_cast<long long>(rg.len));
  if (lo_place >= hi_place) return;  // a slot without a tile
  const int rows = static_cast<int>(hi_place - lo_place);
  const int token0 = rg.first + static_cast<int>(lo_place - place0);
  const int row0 = static_cast<int>(lo_place - static_cast<long long>(block) * p.block_size);

  const bool staged = p.rope.cos_sin != nullptr && (rows > 1 || p.rope.num_axes > 1);
  if (p.rope.cos_sin != nullptr && blockIdx.y == 0)
    for (int r = threadIdx.x; r < rows; r += kThreads)
      check_positions(p.rope, token0 + r, static_cast<int>(lo_place) + r, p.err);

  const int per_head = p.head_dim / 16;
  const int task = blockIdx.y * kThreads + threadIdx.x;
  const int vhead = task / per_head, x = task - vhead * per_head;
  const bool idle = vhead >= p.num_heads + 2 * p.num_kv_heads;
  const int part = vhead < p.num_heads ? 0 : vhead < p.num_heads + p.num_kv_heads ? 1 : 2;
  const int head = vhead - (part == 0 ? 0 : part == 1 ? p.num_heads : p.num_heads + p.num_kv_heads);

  // dims of the two pieces (pairs >= R/2: not turned)
  const int half = p.rope.rotary_dim / 2;
  int da = 16 * x, db = 16 * x + 8;
  const bool turn = !idle && part < 2 && 8 * x < half;
  if (turn && !p.rope.interleaved) {
    da = 8 * x;
    db = 8 * x + half;
  }

  int blk = 0;
  bool store = !idle;
  if (part > 0) {
    blk = p.block_tables[static_cast<size_t>(seq) * p.max_blocks + block];
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
      if (part == 1 && head == 0 && x == 0) report_error(p.err, PA_ERR_BAD_BLOCK, seq, blk);
      store = false;
    }
  }

  const T* src;
  T* dst;
  size_t src_step, dst_step;
  if (part == 0) {
    src_step = p.q_stride;
    dst_step = static_cast<size_t>(p.num_heads) * p.head_dim;
    src = static_cast<const T*>(p.q) + token0 * src_step + static_cast<size_t>(head) * p.head_dim;
    dst = static_cast<T*>(p.q_out) + token0 * dst_step + static_cast<size_t>(head) * p.head_dim;
  } else {
    src_step = part == 1 ? p.k_stride : p.v_stride;
    dst_step = p.head_dim;
    src = static_cast<const T*>(part == 1 ? p.k : p.v) + token0 * src_step +
          static_cast<size_t>(head) * p.head_dim;
    dst = static_cast<T*>(part == 1 ? p.k_cache : p.v_cache) +
          ((static_cast<size_t>(blk) * p.num_kv_heads + head) * p.block_size + row0) * p.head_dim;
  }

  __shared__ __align__(16) float table[kRows * 256];
  const bool bounds = part == 1 && p.k_min != nullptr && store;
  uint4 lo[2], hi[2];
  for (int r0 = 0; r0 < rows; r0 += kBatch) {
    uint4 a[kBatch], b[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (store && r0 + e < rows) {
        a[e] = *reinterpret_cast<const uint4*>(src + (r0 + e) * src_step + da);
        b[e] = *reinterpret_cast<const uint4*>(src + (r0 + e) * src_step + db);
      }
    }
    if (staged && r0 % kRows == 0) {  // rows r0 .. r0 + kRows - 1
      if (r0 > 0) __syncthreads();
      for (int r = threadIdx.x >> 5; r < min(kRows, rows - r0); r += kThreads / 32)
        stage_row(p.rope, token0 + r0 + r, static_cast<int>(lo_place) + r0 + r,
                  table + r * p.rope.rotary_dim, threadIdx.x & 31);
      __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (store && r0 + e < rows) {
        if (turn) {
          const float* cs =
              staged ? table + (r0 % kRows + e) * p.rope.rotary_dim
                     : p.rope.cos_sin + static_cast<size_t>(position(p.rope, 0, token0, static_cast<int>(lo_place))) *
                                            p.rope.rotary_dim;
          rotate(p.rope, cs + 8 * x, a[e], b[e], Tag{});
        }
        *reinterpret_cast<uint4*>(dst + (r0 + e) * dst_step + da) = a[e];
        *reinterpret_cast<uint4*>(dst + (r0 + e) * dst_step + db) = b[e];
        if (bounds) {
          if (r0 + e == 0) {
            lo[0] = hi[0] = a[e];
            lo[1] = hi[1] = b[e];
          } else {
            lo[0] = min8(lo[0], a[e], Tag{});
            lo[1] = min8(lo[1], b[e], Tag{});
            hi[0] = max8(hi[0], a[e], Tag{});
            hi[1] = max8(hi[1], b[e], Tag{});
          }
        }
      }
    }
  }
  if (bounds) {
    const size_t at = (static_cast<size_t>(blk) * p.num_kv_heads + head) * p.head_dim;
    uint4* mn[2] = {reinterpret_cast<uint4*>(static_cast<T*>(p.k_min) + at + da),
                    reinterpret_cast<uint4*>(static_cast<T*>(p.k_min) + at + db)};
    uint4* mx[2] = {reinterpret_cast<uint4*>(static_cast<T*>(p.k_max) + at + da),
                    reinterpret_cast<uint4*>(static_cast<T*>(p.k_max) + at + db)};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (row0 > 0) {  // rows below are in the stored bounds
        lo[e] = min8(lo[e], *mn[e], Tag{});
        hi[e] = max8(hi[e], *mx[e], Tag{});
      }
      *mn[e] = lo[e];
      *mx[e] = hi[e];
    }
  }
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int kv_cache_append_rope(const void* q, int64_t q_stride, const void* k,
                                    int64_t k_stride, const void* v, int64_t v_stride,
                                    const int32_t* query_start, int total_tokens,
                                    int max_query_len, void* k_cache, void* v_cache, void* k_min,
                                    void* k_max, const int32_t* block_tables,
                                    const int32_t* seq_lens, int num_seqs, int num_heads,
                                    int num_kv_heads, int head_dim, int block_size,
                                    int max_blocks_per_seq, int num_blocks, const pa_rope* rope,
                                    int dtype, void* q_out, int32_t* error_record, void* stream) {
  NvtxRange range("kv_cache_append_rope");
  if (!q && !q_out) num_heads = 0;
  if (num_seqs < 0 || total_tokens < 0 || max_query_len < 0 || num_heads < 0 ||
      num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (head_dim % 16 != 0 || head_dim > 256) return PA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_blocks_per_seq) * block_size > (1ll << 30) || num_seqs > 65535 ||
      num_heads > 65535 || num_kv_heads > 65535 || total_tokens > (1 << 30))
    return PA_ERR_INVALID_ARG;
  AppendRopeParams p{};
  if (rope != nullptr) {
    const int st = rope_params(*rope, head_dim, p.rope);
    if (st != PA_OK) return st;
  }
  if (num_seqs == 0 || total_tokens == 0 || max_query_len == 0) return PA_OK;
  if (!k || !v || !k_cache || !v_cache || !query_start || !block_tables || !seq_lens ||
      (!q) != (!q_out) || (!k_min) != (!k_max) || (num_heads == 0 && q))
    return PA_ERR_INVALID_ARG;
  for (const void* a : {q, k, v, static_cast<const void*>(k_cache),
                        static_cast<const void*>(v_cache), static_cast<const void*>(k_min),
                        static_cast<const void*>(k_max), static_cast<const void*>(q_out)})
    if (!aligned16(a)) return PA_ERR_INVALID_ARG;
  const long long q_row = static_cast<long long>(num_heads) * head_dim;
  const long long kv_row = static_cast<long long>(num_kv_heads) * head_dim;
  if ((q && (q_stride < q_row || q_stride % 8)) || k_stride < kv_row || k_stride % 8 ||
      v_stride < kv_row || v_stride % 8 || (q && q == q_out && q_stride != q_row))
    return PA_ERR_INVALID_ARG;

  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.query_start = query_start;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_min = k_min;
  p.k_max = k_max;
  p.q_out = q_out;
  p.err = error_record;
  p.total_tokens = total_tokens;
  p.max_query_len = max_query_len;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.block_size = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.rope.total_tokens = total_tokens;
  // one token a sequence: a tile each; otherwise the slots of first_slot, and behind
  // them blocks that check the ranges
  p.tiles = max_query_len == 1 ? num_seqs : total_tokens / block_size + 2 * num_seqs;
  const int checkers = max_query_len == 1 ? 0 : (num_seqs + kThreads - 1) / kThreads;
  const long long tasks = (num_heads + 2ll * num_kv_heads) * (head_dim / 16);
  const long long groups = (tasks + kThreads - 1) / kThreads;
  if (groups > 65535) return PA_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles + checkers), static_cast<unsigned>(groups));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (max_query_len == 1)
    e = dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, kv_append_rope_kernel<BF16, 1, 1>, p)
                         : cudaLaunchKernelEx(&cfg, kv_append_rope_kernel<F16, 1, 1>, p);
  else
    e = dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, kv_append_rope_kernel<BF16, 16, 4>, p)
                         : cudaLaunchKernelEx(&cfg, kv_append_rope_kernel<F16, 16, 4>, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
