// Append with rotary positions: one pass that rotates a step's queries and keys,
// writes keys and values into their slots and keeps the touched blocks' key bounds.
//
// The work is cut into tiles, the new tokens of one sequence that fall into one block.
//
// Steps of one to a few tokens a sequence (kv_append_step_kernel): a thread takes 16 dims (two
// 16-byte pieces, 8 rotary pairs) of one head of q, k or v, and the tile's tokens one after the
// other.  Bound by latency, and by HBM for large batches.
//
// Prompts (kv_append_rope_kernel): a thread block takes up to 32 heads of q, k or v of a tile, 4 heads
// of k where a tile's rows need several passes; of q and v 16 tokens of a longer tile, or a 64th of
// the longest tile if that is more, of k the whole tile.  A thread keeps the cosines and sines of
// its row and 8 pairs in registers and goes over the heads, 4 at a time.  Rotated keys also go to
// shared memory, where each channel's minimum and maximum over the tile's rows are taken: as the
// tile holds every new key of its block, the bounds need no atomics and no second pass, and come
// out the same on every run.  One read and one write of each element, 3 operations: bound by HBM
// (24 prompts of up to 700 tokens, 32 + 2 x 8 heads of 128, 240 MB: 43 us, 5.6 TB/s), four blocks of
// 127 registers a thread on an SM.  With one head a thread block has 2 KB in flight and half its
// threads idle (63,000 tokens of one head of 64, 50 MB: 62 us).
#include <cuda_runtime.h>

#include "common.cuh"
#include "rope.cuh"

namespace pagedkv {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 4;  // heads that a thread loads at a time
constexpr int kFew = 4;    // tokens a sequence of a step

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
  int heads, key_heads;  // of q and v, and of k, of a thread block, for prompts
  int split;  // tokens of q and v of a thread block, for prompts
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

// What a thread block works on: `rows` new tokens of sequence `seq`, from row `token` of q, k
// and v and place `place` of the sequence, all in its logical block `block`.
struct Tile {
  int seq, rows, token, place, block;
};

__device__ __forceinline__ int table_entry(const AppendRopeParams& p, const Tile& t) {
  return p.block_tables[static_cast<size_t>(t.seq) * p.max_blocks + t.block];
}
// Whether a table entry names a block; if not it is recorded, by one thread of the tile.
__device__ __forceinline__ bool is_block(const AppendRopeParams& p, const Tile& t, int blk,
                                         bool reports) {
  if (static_cast<unsigned>(blk) < static_cast<unsigned>(p.num_blocks)) return true;
  if (reports) report_error(p.err, PA_ERR_BAD_BLOCK, t.seq, blk);
  return false;
}

// The two pieces of dims that slice x of a head covers, and whether it is rotated.
__device__ __forceinline__ bool dims_of(const RopeParams& r, int x, bool rotated, int& da, int& db) {
  const int half = r.rotary_dim / 2;
  da = 16 * x;
  db = 16 * x + 8;
  if (!rotated || 8 * x >= half) return false;
  if (!r.interleaved) {
    da = 8 * x;
    db = 8 * x + half;
  }
  return true;
}

// The tile of a slot; false for a slot without one.
__device__ __forceinline__ bool find_tile(const AppendRopeParams& p, int slot, Tile& t) {
  // the last sequence whose slots begin at or before this one: each warp looks at 32 at once
  int lo = 0, size = p.num_seqs;
  while (size > 1) {
    const int step = (size + 31) / 32, at = lo + static_cast<int>(threadIdx.x & 31) * step;
    const bool before = at < lo + size && first_slot(p, at) <= slot;
    const int n = max(__popc(__ballot_sync(kFullMask, before)), 1);
    size = min(step, lo + size - (lo + (n - 1) * step));
    lo += (n - 1) * step;
  }
  const long long nth = slot - first_slot(p, lo);
  Range rg;
  if (nth < 0 || !range_of(p, lo, rg) || rg.count == 0) return false;
  const int place0 = rg.len - rg.count;  // place of the sequence's first new token
  const long long block = place0 / p.block_size + nth;
  const long long from = max(block * p.block_size, static_cast<long long>(place0));
  const long long to = min((block + 1) * p.block_size, static_cast<long long>(rg.len));
  if (from >= to) return false;
  t = {lo, static_cast<int>(to - from), rg.first + static_cast<int>(from - place0), static_cast<int>(from),
       static_cast<int>(block)};
  return true;
}

// A block behind the tiles: the sequences' ranges, of which tiles skip the bad ones silently.
__device__ __forceinline__ void check_ranges(const AppendRopeParams& p, int nth) {
  const int i = nth * kThreads + threadIdx.x;
  Range r;
  if (blockIdx.y == 0 && blockIdx.z == 0 && i < p.num_seqs && !range_of(p, i, r))
    report_error(p.err, PA_ERR_BAD_SEQ_LEN, i, r.len);
}

template <class Tag>
__device__ __forceinline__ void merge_bounds(const AppendRopeParams& p, size_t at, uint4 lo, uint4 hi,
                                             bool stored, Tag) {
  using T = typename Tag::T;
  uint4* mn = reinterpret_cast<uint4*>(static_cast<T*>(p.k_min) + at);
  uint4* mx = reinterpret_cast<uint4*>(static_cast<T*>(p.k_max) + at);
  *mn = stored ? min8(lo, *mn, Tag{}) : lo;
  *mx = stored ? max8(hi, *mx, Tag{}) : hi;
}

// kOne: one token a sequence, whose tile needs no search (256 x 40 heads, 26 MB: 5.5 us in a graph).
template <class Tag, bool kOne>
__global__ void __launch_bounds__(kThreads) kv_append_step_kernel(const AppendRopeParams p) {
  using T = typename Tag::T;
  const int per_head = p.head_dim / 16;
  const int task = blockIdx.y * kThreads + threadIdx.x;
  const int vhead = task / per_head, x = task - vhead * per_head;
  const int part = vhead < p.num_heads ? 0 : vhead < p.num_heads + p.num_kv_heads ? 1 : 2;
  const int head = vhead - (part == 0 ? 0 : part == 1 ? p.num_heads : p.num_heads + p.num_kv_heads);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int slot = blockIdx.x;
  Tile t;
  if constexpr (kOne) {
    Range rg;
    if (!range_of(p, slot, rg)) {
      if (threadIdx.x == 0 && blockIdx.y == 0) report_error(p.err, PA_ERR_BAD_SEQ_LEN, slot, rg.len);
      return;
    }
    if (rg.count == 0) return;
    t = {slot, 1, rg.first, rg.len - 1, (rg.len - 1) / p.block_size};
  } else {
    if (slot >= p.tiles) {
      check_ranges(p, slot - p.tiles);
      return;
    }
    if (!find_tile(p, slot, t)) return;
  }
  if (vhead >= p.num_heads + 2 * p.num_kv_heads) return;
  if (task == 0 && p.rope.cos_sin != nullptr)
    for (int r = 0; r < t.rows; ++r) check_positions(p.rope, t.token + r, t.place + r, p.err);
  int da, db;
  const bool turn = dims_of(p.rope, x, part < 2, da, db);
  const int blk = part > 0 ? table_entry(p, t) : 0;
  const int row = t.place - t.block * p.block_size;

  const size_t step = part == 0 ? p.q_stride : part == 1 ? p.k_stride : p.v_stride;
  const T* src = static_cast<const T*>(part == 0 ? p.q : part == 1 ? p.k : p.v) + t.token * step +
                 static_cast<size_t>(head) * p.head_dim;
  uint4 lo[2], hi[2];
  const size_t bh = static_cast<size_t>(blk) * p.num_kv_heads + head;
  for (int r = 0; r < t.rows; ++r) {
    uint4 a = *reinterpret_cast<const uint4*>(src + r * step + da);
    uint4 b = *reinterpret_cast<const uint4*>(src + r * step + db);
    if (turn) {
      float c[8], s[8];
      load_cos_sin(p.rope, t.token + r, t.place + r, 8 * x, c, s);
      rotate(p.rope, c, s, a, b, Tag{});
    }
    if (part > 0 && !is_block(p, t, blk, part == 1 && head == 0 && x == 0)) return;
    T* dst = part == 0 ? static_cast<T*>(p.q_out) +
                             (static_cast<size_t>(t.token + r) * p.num_heads + head) * p.head_dim
                       : static_cast<T*>(part == 1 ? p.k_cache : p.v_cache) +
                             (bh * p.block_size + row + r) * p.head_dim;
    *reinterpret_cast<uint4*>(dst + da) = a;
    *reinterpret_cast<uint4*>(dst + db) = b;
    lo[0] = r == 0 ? a : min8(lo[0], a, Tag{});
    lo[1] = r == 0 ? b : min8(lo[1], b, Tag{});
    hi[0] = r == 0 ? a : max8(hi[0], a, Tag{});
    hi[1] = r == 0 ? b : max8(hi[1], b, Tag{});
    if constexpr (kOne) break;
  }
  if (part == 1 && p.k_min != nullptr) {  // rows below are in the stored bounds
    merge_bounds(p, bh * p.head_dim + da, lo[0], hi[0], row > 0, Tag{});
    merge_bounds(p, bh * p.head_dim + db, lo[1], hi[1], row > 0, Tag{});
  }
}

template <class Tag>
__global__ void __launch_bounds__(kThreads) kv_append_rope_kernel(const AppendRopeParams p) {
  using T = typename Tag::T;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int slot = blockIdx.x;
  if (slot >= p.tiles) {
    check_ranges(p, slot - p.tiles);
    return;
  }
  Tile t;
  if (!find_tile(p, slot, t)) return;
  if (p.rope.cos_sin != nullptr && blockIdx.y == 0 && blockIdx.z == 0)
    for (int r = threadIdx.x; r < t.rows; r += kThreads)
      check_positions(p.rope, t.token + r, t.place + r, p.err);

  // this block's heads
  const int q_chunks = (p.num_heads + p.heads - 1) / p.heads;
  const int k_chunks = (p.num_kv_heads + p.key_heads - 1) / p.key_heads;
  const int chunk = blockIdx.y;
  const int part = chunk < q_chunks ? 0 : chunk < q_chunks + k_chunks ? 1 : 2;
  const int size = part == 1 ? p.key_heads : p.heads;
  const int h0 = (chunk - (part == 0 ? 0 : part == 1 ? q_chunks : q_chunks + k_chunks)) * size;
  const int h1 = min(h0 + size, part == 0 ? p.num_heads : p.num_kv_heads);
  const int skip = blockIdx.z * p.split;
  if (part == 1 ? skip > 0 : skip >= t.rows) return;
  if (part != 1) {  // keys take the whole tile, for their bounds
    t.rows = min(p.split, t.rows - skip);
    t.token += skip;
    t.place += skip;
  }
  const int row0 = t.place - t.block * p.block_size;
  const int blk = part > 0 ? table_entry(p, t) : 0;

  // Thread (x, r, h): slice x of the head, row r of `span` at a time, and of the heads every
  // `lanes`-th from h on.
  const int per_head = p.head_dim / 16;
  int span = 1;
  while (2 * span * per_head <= kThreads && span < t.rows) span *= 2;
  const int lanes = kThreads / (span * per_head);
  const int x = threadIdx.x % per_head, r = threadIdx.x / per_head % span;
  const int h = threadIdx.x / (per_head * span);
  int da, db;
  const bool turn = dims_of(p.rope, x, part < 2, da, db);
  const bool bounds = part == 1 && p.k_min != nullptr;
  const int pieces = p.head_dim / 8;
  __shared__ uint4 keys[kThreads * kBatch * 2];  // [head of the batch][row][piece]

  const size_t step = part == 0 ? p.q_stride : part == 1 ? p.k_stride : p.v_stride;
  const T* src = static_cast<const T*>(part == 0 ? p.q : part == 1 ? p.k : p.v) +
                 static_cast<size_t>(h0 + h) * p.head_dim;
  // elements from head to head of the output
  const size_t head_step = part == 0 ? p.head_dim : static_cast<size_t>(p.block_size) * p.head_dim;
  const bool many = t.rows > span;  // passes over the rows; then a thread has at most one reduction
  float c[8], s[8];
  for (int hb = h0; hb < h1; hb += kBatch * lanes) {
    const int tasks = min(kBatch * lanes, h1 - hb) * pieces;
    uint4 mn, mx;
    for (int pass = 0; pass < t.rows; pass += span) {
      const bool active = pass + r < t.rows && h < lanes;
      const int token = t.token + pass + r;
      const T* from = src + token * step;
      uint4 a[kBatch], b[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (active && hb + h + lanes * i < h1) {
          const T* at = from + (hb - h0 + lanes * i) * p.head_dim;
          a[i] = *reinterpret_cast<const uint4*>(at + da);
          b[i] = *reinterpret_cast<const uint4*>(at + db);
        }
      }
      // with the loads on their way
      if ((many || hb == h0) && turn && active)
        load_cos_sin(p.rope, token, t.place + pass + r, 8 * x, c, s);
      if (hb == h0 && pass == 0 && part > 0 &&
          !is_block(p, t, blk, part == 1 && h0 == 0 && threadIdx.x == 0))
        return;
      const size_t row =
          part == 0 ? static_cast<size_t>(token) * p.num_heads
                    : static_cast<size_t>(blk) * p.num_kv_heads * p.block_size + row0 + pass + r;
      T* to = static_cast<T*>(part == 0 ? p.q_out : part == 1 ? p.k_cache : p.v_cache) +
              row * p.head_dim + (hb + h) * head_step;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (active && hb + h + lanes * i < h1) {
          if (turn) rotate(p.rope, c, s, a[i], b[i], Tag{});
          *reinterpret_cast<uint4*>(to + da) = a[i];
          *reinterpret_cast<uint4*>(to + db) = b[i];
          to += lanes * head_step;
          if (bounds) {
            uint4* k = keys + ((h + lanes * i) * span + r) * pieces;
            k[da / 8] = a[i];
            k[db / 8] = b[i];
          }
        }
      }
      if (bounds) {
        __syncthreads();
        const int n = min(span, t.rows - pass);
        for (int j = threadIdx.x; j < tasks; j += kThreads) {
          const int slot_head = j / pieces, piece = j % pieces;
          const uint4* k = keys + slot_head * span * pieces + piece;
          if (!many || pass == 0) mn = mx = k[0];
          for (int i = 0; i < n; ++i) {
            mn = min8(mn, k[i * pieces], Tag{});
            mx = max8(mx, k[i * pieces], Tag{});
          }
          if (pass + span >= t.rows) {  // rows below the tile are in the stored bounds
            const size_t bh = static_cast<size_t>(blk) * p.num_kv_heads + hb + slot_head;
            merge_bounds(p, bh * p.head_dim + 8 * piece, mn, mx, row0 > 0, Tag{});
          }
        }
        __syncthreads();
      }
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
  // Up to kFew tokens a sequence: a thread for 16 dims of each head of a tile, otherwise by chunks of
  // heads (217 sequences of 2, 3, 4 tokens, 48 + 2 x 3 heads of 64: 5.6, 6.6, 7.3 us, by chunks of
  // heads 13.3, 13.9, 14.4 us; 64 of 3, 4, 6 tokens, 32 + 2 x 8 heads of 128: 5.3, 6.0, 7.5 us, by
  // chunks 5.9, 5.9, 6.6 us).  A tile for each sequence, or the tile slots of first_slot with behind them blocks that
  // check the ranges.
  const bool one = max_query_len == 1, few = max_query_len <= kFew;
  p.tiles = one ? num_seqs : total_tokens / block_size + 2 * num_seqs;
  const int range_blocks = one ? 0 : (num_seqs + kThreads - 1) / kThreads;
  const auto chunks = [](long long n, long long size) { return (n + size - 1) / size; };
  const auto head_chunks = [&] {
    return chunks(num_heads, p.heads) + chunks(num_kv_heads, p.heads) + chunks(num_kv_heads, p.key_heads);
  };
  // As many keys' heads a thread block, but 4 where their rows need several passes.
  const int longest = block_size < max_query_len ? block_size : max_query_len;
  const auto set_heads = [&](int n) {
    p.heads = n;
    p.key_heads = longest * (head_dim / 16) > kThreads ? kBatch : n;
  };
  // 32 heads a thread block, down to 8 while that leaves fewer than 8 blocks for each SM (24
  // prompts of up to 700 tokens, 32 + 2 x 8 heads: 43.6 us with 32, 44.5 with 16, 47.4 with 8)
  set_heads(32);
  while (!few && p.heads > 8 && (total_tokens / block_size + 1) * head_chunks() < 152 * 8)
    set_heads(p.heads / 2);
  const long long groups =
      few ? chunks((num_heads + 2ll * num_kv_heads) * (head_dim / 16), kThreads) : head_chunks();
  if (groups > 65535) return PA_ERR_INVALID_ARG;
  // 16 tokens of q and v a thread block, more only where a tile would need over 64 blocks
  p.split = (longest + 63) / 64 > 16 ? (longest + 63) / 64 : 16;
  const unsigned splits = few ? 1u : static_cast<unsigned>((longest + p.split - 1) / p.split);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles + range_blocks), static_cast<unsigned>(groups), splits);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (one)
    e = dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, kv_append_step_kernel<BF16, true>, p)
                         : cudaLaunchKernelEx(&cfg, kv_append_step_kernel<F16, true>, p);
  else if (few)
    e = dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, kv_append_step_kernel<BF16, false>, p)
                         : cudaLaunchKernelEx(&cfg, kv_append_step_kernel<F16, false>, p);
  else
    e = dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, kv_append_rope_kernel<BF16>, p)
                         : cudaLaunchKernelEx(&cfg, kv_append_rope_kernel<F16>, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
