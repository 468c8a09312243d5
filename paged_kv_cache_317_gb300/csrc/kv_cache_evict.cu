// Eviction: the kept tokens of each key head move to the front of their sequence.
//
// Place j of (sequence, key head) takes the row of K, of V and the weight that place kept[j] held.
// In place this is a gather within one array, safe in order: kept[j] >= j, so a row that is still to
// be read (for place j' > j, from a place >= j') is never one that place j overwrites.  Into other
// blocks, places without an entry take their own rows along.  K and V are moved apart.  A thread block, or for few lists a cluster, takes one list and goes through it in
// rounds: every thread loads its pieces of the round's rows into registers and looks up rows of the
// next round, a barrier, every thread stores its pieces.  Loads of later rounds may run ahead of the
// stores of earlier ones; only the loads of a round itself have to be over, which the barrier sees to.
// A move and nothing else: bound by HBM for batches (64 contexts of up to 16384 tokens, 8 heads, 1024 kept:
// 94 us for 556 MB, 5.9 TB/s), by a round's latency (list, tables, rows, barrier, stores) for one sequence (4096
// kept of 30,000: 11.4 us for 35 MB, two rounds a cluster).
#include <cuda_runtime.h>

#include "cluster.cuh"
#include "common.cuh"

namespace pagedkv {
namespace {

constexpr int kMaxCluster = 8;

// kThreads threads with kPieces 16-byte pieces each in flight: a round of a thread block.
template <int kThreads_, int kPieces_>
struct Round {
  static constexpr int kThreads = kThreads_, kPieces = kPieces_;
  static constexpr int kMaxRows = 2 * kThreads;  // rows that it looks up at most
  static constexpr int kBlocks = 512 / kThreads; // an SM, as registers allow
};
// Few lists: 64 KB, in clusters besides (8 + 8 lists of 4096 rows of 128 channels: 11.5 us, 29 with the other).
// Many: 16 KB, of which an SM has eight thread blocks whose loads and stores take turns (1024 lists of 1024 rows:
// 94 us, 99 with the other; 2048 of 128: 21 us, 31).
using Few = Round<256, 16>;
using Many = Round<64, 16>;
constexpr int kMany = 608;  // lists, four an SM

struct EvictParams {
  uint4* k;
  uint4* v;
  const int32_t* tables;
  const int32_t* new_tables;
  const int32_t* seq_lens;
  const int32_t* kept;
  float* weights;
  int32_t* err;
  long long weights_row;   // floats from (sequence, key head) to the next
  int num_kept, num_kv_heads, vecs, block_size, max_blocks, new_max_blocks, num_blocks;
  int rows;                // rows of a round and thread block
  unsigned inv_vecs;       // i / vecs = i * inv_vecs >> 20 for i < 4096, vecs <= 128
};

template <class R>
__global__ void __launch_bounds__(R::kThreads, R::kBlocks) kv_cache_evict_kernel(const EvictParams p) {
  constexpr int kThreads = R::kThreads, kPieces = R::kPieces, kMaxRows = R::kMaxRows;
  // rows of the caches seen as rows of head_dim: where a row of the round comes from (-1: it stays) and
  // goes to, of this round and the next
  __shared__ long long from[2][kMaxRows], to[2][kMaxRows];
  const int ranks = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int list = blockIdx.x / ranks, sh = list >> 1;
  const bool is_v = list & 1;
  const int seq = sh / p.num_kv_heads, head = sh - seq * p.num_kv_heads;
  int L = p.seq_lens[seq];
  const int cap = p.max_blocks * p.block_size;
  if (L < 0 || L > cap) {
    if (rank == 0 && threadIdx.x == 0 && head == 0 && !is_v) report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    L = min(max(L, 0), cap);
  }
  const int32_t* kept = p.kept + static_cast<size_t>(sh) * p.num_kept;
  const int32_t* table = p.tables + static_cast<size_t>(seq) * p.max_blocks;
  const int32_t* new_table = p.new_tables + static_cast<size_t>(seq) * p.new_max_blocks;
  float* weights = p.weights == nullptr || is_v ? nullptr : p.weights + sh * p.weights_row;
  uint4* cache = is_v ? p.v : p.k;
  const int places = min(p.num_kept, L);
  // whether place j has a block in other tables than its own: one that does not leaves the sequence
  auto renewed = [&](int j) -> bool {
    const int b = j / p.block_size;
    return p.new_tables != p.tables && b < p.new_max_blocks && new_table[b] != -1;
  };
  const bool uncut = L > 0 && L <= p.num_kept && renewed(L - 1);

  // the row of place j
  auto row_of = [&](const int32_t* t, int blocks, int j) -> long long {
    const int b = j / p.block_size;
    const int blk = b < blocks ? t[b] : -1;
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
      if (!is_v) report_error(p.err, PA_ERR_BAD_BLOCK, seq, blk);
      return -1;
    }
    return (static_cast<long long>(blk) * p.num_kv_heads + head) * p.block_size + (j - b * p.block_size);
  };
  // The rows of this block's places j0 on; a weight is moved by the thread that looks its row up, which
  // returns the place it was at, -1 for none (the weight becomes 0), -2 if it stays as it is.
  auto look_up = [&](int buf, int j0, int (&places_from)[kMaxRows / kThreads]) {
#pragma unroll
    for (int u = 0; u < kMaxRows / kThreads; ++u) {
      const int i = threadIdx.x + u * kThreads, j = j0 + i;
      long long src = -1, dst = -1;
      places_from[u] = -2;
      if (i < p.rows && j < places) {
        const int s = kept[j], b = j / p.block_size;
        bool moves = s >= j && s < L;
        // (a sequence that loses no tokens keeps its table, whose blocks a fork may read: its rows stay)
        if (uncut && s != j && table[b] == new_table[b]) moves = false;
        if (moves || renewed(j)) {
          src = row_of(table, p.max_blocks, moves ? s : j);
          dst = row_of(new_table, p.new_max_blocks, j);
        }
        if (moves) {
          if (src >= 0 && dst >= 0 && s != j) places_from[u] = s;  // a weight goes with its row, or stays
        } else if (s == -1) {
          places_from[u] = -1;
        } else if (!is_v) {
          report_error(p.err, PA_ERR_BAD_POSITION, sh, s);
        }
        if (dst < 0 || src == dst) src = -1;
      }
      if (i < p.rows) {
        from[buf][i] = src;
        to[buf][i] = dst;
      }
    }
  };
  int now[kMaxRows / kThreads], next[kMaxRows / kThreads];
  look_up(0, rank * p.rows, now);
  __syncthreads();
  const int step = ranks * p.rows;
  int buf = 0;
  for (int j0 = rank * p.rows; j0 - rank * p.rows < places; j0 += step, buf ^= 1) {
    uint4 piece[kPieces];
    float w[kMaxRows / kThreads];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = threadIdx.x + u * kThreads, row = i * p.inv_vecs >> 20;
      const long long src = row < p.rows ? from[buf][row] : -1;
      if (src >= 0) piece[u] = __ldcg(cache + src * p.vecs + (i - row * p.vecs));
    }
    if (weights != nullptr) {
#pragma unroll
      for (int u = 0; u < kMaxRows / kThreads; ++u) w[u] = now[u] >= 0 ? __ldcg(weights + now[u]) : 0.f;
    }
    look_up(buf ^ 1, j0 + step, next);
    if (ranks == 1) __syncthreads();
    else cluster_sync();
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = threadIdx.x + u * kThreads, row = i * p.inv_vecs >> 20;
      if (row < p.rows && from[buf][row] >= 0) cache[to[buf][row] * p.vecs + (i - row * p.vecs)] = piece[u];
    }
#pragma unroll
    for (int u = 0; u < kMaxRows / kThreads; ++u) {
      if (weights != nullptr && now[u] != -2) weights[j0 + static_cast<int>(threadIdx.x) + u * kThreads] = w[u];
      now[u] = next[u];
    }
    __syncthreads();  // the round's rows are used
  }
  // every weight has been read
  if (weights != nullptr)
    for (int j = places + rank * kThreads + static_cast<int>(threadIdx.x); j < L; j += ranks * kThreads)
      weights[j] = 0.f;
}

template <class R>
int launch(EvictParams p, int num_seqs, long long longest, cudaStream_t stream) {
  const int fit = R::kThreads * R::kPieces / p.vecs;
  p.rows = fit < R::kMaxRows ? fit : R::kMaxRows;
  // Few lists: clusters, as far as a round still has work for every block of them.
  const long long lists = 2ll * num_seqs * p.num_kv_heads;
  int ranks = 1;
  while (ranks < kMaxCluster && lists * ranks < 304 && longest > static_cast<long long>(ranks) * p.rows)
    ranks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(lists * ranks));
  cfg.blockDim = dim3(R::kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv_cache_evict_kernel<R>, p) != cudaSuccess || cudaGetLastError() != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int kv_cache_evict(void* k_cache, void* v_cache, const int32_t* block_tables,
                              const int32_t* new_tables, const int32_t* seq_lens, const int32_t* kept,
                              int num_kept, float* weights, int64_t weights_tokens, int num_seqs,
                              int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                              int new_max_blocks, int num_blocks, int dtype, int32_t* error_record,
                              void* stream) {
  NvtxRange range("kv_cache_evict");
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0 || num_kept <= 0 || (new_tables && new_max_blocks <= 0))
    return PA_ERR_INVALID_ARG;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (head_dim % 8 != 0 || head_dim > 1024) return PA_ERR_UNSUPPORTED;
  const long long cap = static_cast<long long>(max_blocks_per_seq) * block_size;
  if (cap > (1ll << 30) || num_seqs > 65535 || num_kept > (1 << 30) ||
      static_cast<long long>(num_seqs) * num_kv_heads > (1ll << 27))
    return PA_ERR_INVALID_ARG;
  if (weights && weights_tokens < cap) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !seq_lens || !kept) return PA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
  EvictParams p{};
  p.k = static_cast<uint4*>(k_cache);
  p.v = static_cast<uint4*>(v_cache);
  p.tables = block_tables;
  p.new_tables = new_tables ? new_tables : block_tables;
  p.new_max_blocks = new_tables ? new_max_blocks : max_blocks_per_seq;
  p.seq_lens = seq_lens;
  p.kept = kept;
  p.weights = weights;
  p.weights_row = weights_tokens;
  p.err = error_record;
  p.num_kept = num_kept;
  p.num_kv_heads = num_kv_heads;
  p.vecs = head_dim / 8;
  p.block_size = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.inv_vecs = ((1u << 20) + p.vecs - 1) / p.vecs;
  const long long longest = num_kept < cap ? num_kept : cap;
  return 2ll * num_seqs * num_kv_heads >= kMany
             ? launch<Many>(p, num_seqs, longest, static_cast<cudaStream_t>(stream))
             : launch<Few>(p, num_seqs, longest, static_cast<cudaStream_t>(stream));
}
