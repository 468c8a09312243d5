// Decode attention over listed blocks.
//
// A row is one (sequence, key head) with its list and the query heads that share the key
// head.  The tokens of the listed blocks are cut into chunks of 16; a cluster of thread
// blocks takes a row, and the chunks go round its warps, so that lists that end early
// still load every warp alike.
//  * Each warp runs a pipeline of its own: its lanes look up the next 32 of its chunks
//    (list entry, block table, length) at once, one lane starts the K and V copies of a
//    chunk (a 3-D TMA box of 16 rows x D channels in 128-byte swizzled columns) into the
//    warp's ring of stages, and the warp waits on the stage's barrier.  No warp waits for
//    another before the end.
//  * Per chunk the products and the softmax of warp_attn.cuh, tokens as the rows and query heads as
//    the columns.  Up to 8 query heads cost one product, up to 16 two; K and V are read once for all
//    of them.
//  * At the end the warps' (m, l, O) are joined in shared memory, and those of the cluster's
//    blocks over distributed shared memory, in a fixed order: the same bits on every run.  Only
//    where a few rows have long lists are a row's chunks spread over several clusters, whose sums
//    go through a workspace to a second kernel.
// Two operations per cached byte and query head: bound by HBM (64 sequences x 8 key heads x 8 query
// heads, lists of 128 blocks of 16, 527 MB: 81 us, 6.5 TB/s; 32 x 40 heads, 64 blocks, 672 MB: 100
// us, 6.7 TB/s).  One row alone is a chain of look-ups, copy, products and joins (8 rows of 64
// blocks: 5.6 us; one list of 2048 blocks over 32 clusters: 12.6 us, over one 166 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "cluster.cuh"
#include "common.cuh"
#include "tma.cuh"
#include "warp_attn.cuh"

namespace pagedkv {
namespace {

constexpr int kChunk = 16;       // tokens per stage
constexpr int kWarps = 4;        // warps per thread block
constexpr int kMaxStages = 8;
constexpr int kMaxCluster = 8;
constexpr int kMaxParts = 64;    // clusters per row
constexpr int kMaxShares = 1024; // clusters of all rows, where rows have several
constexpr int kWhole = 128;      // a list of at most so many chunks is one cluster's
constexpr int kAlign = 1024;     // a swizzled box must start on 1024 bytes
constexpr int kHeader = 1024;    // barriers and the chunks' row counts
constexpr float kLog2e = 1.4426950408889634f;

struct SparseParams {
  const void* q;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* selected;
  void* out;
  int32_t* err;
  int num_selected, num_heads, num_kv_heads, block_size, max_blocks, num_blocks;
  int group, tiles;     // query heads per key head; tiles of 8 NT of them
  int parts;            // clusters per row
  float* part_o;        // [row][part][8 NT][D], with parts > 1
  float2* part_ml;      // [row][part][8 NT]
  int out_dtype, stages;
  float qscale;         // scale * log2(e)
};

template <int D>
struct Geo {
  static constexpr int kTileBytes = kChunk * D * 2;  // one chunk of K or V
  static constexpr int kPitch = D + 4;               // floats per column of the joined O
};

template <class Tag, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32)
    paged_attn_sparse_kernel(const __grid_constant__ CUtensorMap tm_k,
                             const __grid_constant__ CUtensorMap tm_v, const SparseParams p) {
  using Gm = Geo<D>;
  using Attn = WarpAttn<Tag, D, NT>;
  constexpr int kCols = 8 * NT;
  if (threadIdx.x == 0) {  // arguments, not memory of the kernel before
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
  }
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int S = p.stages;
  const int cluster = blockIdx.x / ranks;
  const int row = cluster / p.parts, part = cluster - row * p.parts;  // row: (sequence, key head, tile)
  const int tile = row % p.tiles;
  const int sh = row / p.tiles;        // sequence * key heads + key head
  const int seq = sh / p.num_kv_heads, head = sh - seq * p.num_kv_heads;
  const int cols = min(kCols, p.group - tile * kCols);
  const size_t q0 = static_cast<size_t>(seq) * p.num_heads + head * p.group + tile * kCols;

  uint64_t* full = reinterpret_cast<uint64_t*>(smem) + warp * kMaxStages;
  int* rows_of = reinterpret_cast<int*>(smem + kWarps * kMaxStages * 8) + warp * kMaxStages;
  const uint32_t base = smem_addr(smem);
  uint8_t* ring0 = smem + (((base + kHeader + kAlign - 1) & ~uint32_t(kAlign - 1)) - base);
  uint8_t* ring = ring0 + static_cast<size_t>(warp) * S * 2 * Gm::kTileBytes;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncwarp();

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int L = p.seq_lens[seq];

  // ------------------------------------------------------- the warp's chunks
  // Chunk c of a row is 16 tokens of list entry c / (bs / 16), or with 8-token blocks
  // entries 2 c and 2 c + 1.  This warp takes c = me, me + all, ...; its lanes look up 32 of
  // them at a time and `mask` names those with tokens that are not issued yet.
  const int me = (part * ranks + rank) * kWarps + warp, all = p.parts * ranks * kWarps;
  const bool small = p.block_size == 8;
  const int sub = small ? 1 : p.block_size / kChunk;
  const int chunks = small ? (p.num_selected + 1) / 2 : p.num_selected * sub;
  const int32_t* list = p.selected + static_cast<size_t>(sh) * p.num_selected;
  const int32_t* table = p.block_tables + static_cast<size_t>(seq) * p.max_blocks;
  int next = me;  // chunk of lane 0 at the next look-up
  int b_lo, b_hi, blk_lo, blk_hi;
  // List entries and block numbers of the next 32 chunks.  The length is not needed for them.
  auto fetch = [&]() {
    const int c = next + lane * all;
    b_lo = b_hi = -1;
    if (c < chunks) {
      b_lo = list[small ? 2 * c : c / sub];
      if (small && 2 * c + 1 < p.num_selected) b_hi = list[2 * c + 1];
    }
    blk_lo = static_cast<unsigned>(b_lo) < static_cast<unsigned>(p.max_blocks) ? table[b_lo] : 0;
    blk_hi = static_cast<unsigned>(b_hi) < static_cast<unsigned>(p.max_blocks) ? table[b_hi] : 0;
  };
  fetch();
  const int cap = p.max_blocks * p.block_size;
  if (L < 0 || L > cap) {
    if (threadIdx.x == 0 && rank == 0 && part == 0 && head == 0 && tile == 0)
      report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    L = min(max(L, 0), cap);
  }
  // The tokens of block b from its row 16 from on, at most `height`, and their row in the cache
  // seen as rows of D.
  auto rows_in = [&](int b, int blk, int from, int height, int& y) -> int {
    if (b < -1 || b >= p.max_blocks) {
      if (from == 0 && tile == 0) report_error(p.err, PA_ERR_BAD_BLOCK, sh, b);
      return 0;
    }
    if (b < 0) return 0;
    const int rows = min(height, L - b * p.block_size - from * kChunk);
    if (rows <= 0) return 0;
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
      if (from == 0 && tile == 0) report_error(p.err, PA_ERR_BAD_BLOCK, seq, blk);
      blk = 0;
    }
    y = (blk * p.num_kv_heads + head) * p.block_size + from * kChunk;
    return rows;
  };
  unsigned mask = 0;
  int y_lo = 0, y_hi = 0, rows_lo = 0, rows_hi = 0;
  bool fetched = true;
  auto refill = [&]() {
    while (mask == 0 && next < chunks) {
      if (!fetched) fetch();
      fetched = false;
      const int c = next + lane * all;
      rows_lo = rows_hi = 0;
      if (small) {
        rows_lo = rows_in(b_lo, blk_lo, 0, 8, y_lo);
        rows_hi = rows_in(b_hi, blk_hi, 0, 8, y_hi);
      } else {
        const int rows = rows_in(b_lo, blk_lo, c % sub, 16, y_lo);
        rows_lo = min(rows, 8);
        rows_hi = rows - rows_lo;
      }
      mask = __ballot_sync(kFullMask, rows_lo + rows_hi > 0);
      next += 32 * all;
    }
  };
  // Starts the copies of the next chunk into a stage; false when there is none.
  auto issue = [&](int s) -> bool {
    if (mask == 0) refill();
    if (mask == 0) return false;
    const int j = __ffs(mask) - 1;
    mask &= mask - 1;
    const int ylo = __shfl_sync(kFullMask, y_lo, j), yhi = __shfl_sync(kFullMask, y_hi, j);
    const int rlo = __shfl_sync(kFullMask, rows_lo, j), rhi = __shfl_sync(kFullMask, rows_hi, j);
    if (lane == 0) {
      rows_of[s] = rlo | (rhi << 8);
      uint8_t* dst = ring + s * 2 * Gm::kTileBytes;
      if (!small) {
        mbar_arrive_expect_tx(&full[s], 2 * Gm::kTileBytes);
        tma_load_3d(dst, &tm_k, 0, ylo, 0, &full[s]);
        tma_load_3d(dst + Gm::kTileBytes, &tm_v, 0, ylo, 0, &full[s]);
      } else {
        constexpr int kHalf = Gm::kTileBytes / 2;
        mbar_arrive_expect_tx(&full[s], (rlo > 0 ? 2 * kHalf : 0) + (rhi > 0 ? 2 * kHalf : 0));
        if (rlo > 0) {
          tma_load_3d(dst, &tm_k, 0, ylo, 0, &full[s]);
          tma_load_3d(dst + Gm::kTileBytes, &tm_v, 0, ylo, 0, &full[s]);
        }
        if (rhi > 0) {
          tma_load_3d(dst + kHalf, &tm_k, 0, yhi, 0, &full[s]);
          tma_load_3d(dst + Gm::kTileBytes + kHalf, &tm_v, 0, yhi, 0, &full[s]);
        }
      }
    }
    return true;
  };
  int issued = 0, done = 0;
  while (issued < S && issue(issued)) ++issued;

  Attn at;
  at.init(static_cast<const typename Tag::T*>(p.q) + q0 * D, cols, small, lane);
  const uint32_t ring_addr = smem_addr(ring);

  bool aborted = false;
  while (done < issued) {
    const int s = done % S;
    if (!__all_sync(kFullMask, mbar_wait_bounded(&full[s], (done / S) & 1))) {
      if (lane == 0) report_error(p.err, PA_ERR_TIMEOUT, seq, done);
      aborted = true;
      break;
    }
    const int rows = rows_of[s];
    const int rlo = rows & 255, rhi = rows >> 8;
    const uint32_t kt = ring_addr + s * 2 * Gm::kTileBytes, vt = kt + Gm::kTileBytes;

    at.step(kt, vt, rlo, rhi, p.qscale, lane, [](int, const float (&)[4]) {});
    __syncwarp();  // the stage is read
    ++done;
    if (issue(s)) ++issued;
  }
  if (aborted) {  // no copy may land in shared memory after the block has exited
    for (int i = done; i < issued; ++i) mbar_wait_bounded(&full[i % S], (i / S) & 1);
  }

  // ------------------------------------------------------------------ the join
  // O of the warps as [warp][column][kPitch], then (m, l) as [warp][column]; the block's own
  // sums replace warp 0's.
  __syncthreads();
  float* jo = reinterpret_cast<float*>(ring0);
  float2* jml = reinterpret_cast<float2*>(jo + kWarps * kCols * Gm::kPitch);
  at.put(jo + warp * kCols * Gm::kPitch, Gm::kPitch, jml + warp * kCols, done > 0, lane);
  __syncthreads();
  // Column col, channels d .. d + 3 of the first n of up to kMost partials; their loads do not
  // wait for one another.
  auto join = [&](auto most, auto ml_of, auto o_of, int n, int col, int d, float& M, float& sum,
                  bool& tokens) {
    constexpr int kMost = decltype(most)::value;
    float2 ml[kMost];
    float4 v[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      ml[i] = i < n ? ml_of(i, col) : make_float2(-INFINITY, 0.f);
      if (i < n) v[i] = o_of(i, col, d);
    }
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMost; ++i) M = max_nan(M, ml[i].x);
    sum = 0.f;
    tokens = false;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      tokens |= ml[i].y < 0.f || ml[i].x != -INFINITY;
      if (ml[i].x != -INFINITY) {
        const float w = exp2f(ml[i].x - M);
        sum = fmaf(w, ml[i].y, sum);
        acc.x = fmaf(w, v[i].x, acc.x);
        acc.y = fmaf(w, v[i].y, acc.y);
        acc.z = fmaf(w, v[i].z, acc.z);
        acc.w = fmaf(w, v[i].w, acc.w);
      }
    }
    return acc;
  };
  constexpr std::integral_constant<int, kWarps> warps{};
  constexpr std::integral_constant<int, kMaxCluster> blocks{};
  auto finish = [&](float4 acc, float M, float sum, bool tokens, int col, int d) {
    const float inv = inverse_of(M, sum, tokens);
    const float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    store_out<4>(p.out, (q0 + col) * D + d, v, p.out_dtype);
  };
  auto ml_here = [&](int w, int col) { return jml[w * kCols + col]; };
  auto o_here = [&](int w, int col, int d) {
    return *reinterpret_cast<const float4*>(jo + (w * kCols + col) * Gm::kPitch + d);
  };
  if (ranks == 1) {
    for (int i = threadIdx.x; i < cols * (D / 4); i += kWarps * 32) {
      const int col = i / (D / 4), d = i % (D / 4) * 4;
      float M, sum;
      bool tokens;
      const float4 acc = join(warps, ml_here, o_here, kWarps, col, d, M, sum, tokens);
      finish(acc, M, sum, tokens, col, d);
    }
    return;
  }
  float2* block_ml = jml + kWarps * kCols;
  for (int i = threadIdx.x; i < cols * (D / 4); i += kWarps * 32) {
    const int col = i / (D / 4), d = i % (D / 4) * 4;
    float M, sum;
    bool tokens;
    const float4 acc = join(warps, ml_here, o_here, kWarps, col, d, M, sum, tokens);
    *reinterpret_cast<float4*>(jo + col * Gm::kPitch + d) = acc;  // only this thread reads it before
    if (d == 0) block_ml[col] = make_float2(M, M == -INFINITY && tokens ? -1.f : sum);
  }
  cluster_sync();
  const uint32_t o_addr = smem_addr(jo), ml_addr = smem_addr(block_ml);
  auto ml_peer = [&](int r, int col) { return ld_peer2(peer_addr(ml_addr + col * 8, r)); };
  auto o_peer = [&](int r, int col, int d) {
    return ld_peer4(peer_addr(o_addr + (col * Gm::kPitch + d) * 4, r));
  };
  // Each block finishes every ranks-th piece; it is done with its peers' memory before it stores.
  constexpr int kMine = (kCols * (D / 4) + kWarps * 32 - 1) / (kWarps * 32);
  float4 acc[kMine];
  float M[kMine], sum[kMine];
  bool tokens[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = (threadIdx.x + k * kWarps * 32) * ranks + rank;
    if (i < cols * (D / 4))
      acc[k] = join(blocks, ml_peer, o_peer, ranks, i / (D / 4), i % (D / 4) * 4, M[k], sum[k], tokens[k]);
  }
  cluster_arrive();
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = (threadIdx.x + k * kWarps * 32) * ranks + rank;
    if (i < cols * (D / 4)) {
      const int col = i / (D / 4), d = i % (D / 4) * 4;
      if (p.parts == 1) {
        finish(acc[k], M[k], sum[k], tokens[k], col, d);
      } else {
        const size_t at = static_cast<size_t>(cluster) * kCols + col;
        *reinterpret_cast<float4*>(p.part_o + at * D + d) = acc[k];
        if (d == 0) p.part_ml[at] = make_float2(M[k], M[k] == -INFINITY && tokens[k] ? -1.f : sum[k]);
      }
    }
  }
  cluster_wait();  // no block leaves while another may read its memory
}

// Joins the parts of a row: a thread block per query head, four channels a thread.
template <int D, int NT>
__global__ void __launch_bounds__(D / 4) paged_attn_sparse_join_kernel(const SparseParams p) {
  constexpr int kCols = 8 * NT, kAhead = 8;
  const int seq = blockIdx.x / p.num_heads, g = blockIdx.x - seq * p.num_heads;
  const int head = g / p.group, r = g - head * p.group;
  const size_t row = (static_cast<size_t>(seq) * p.num_kv_heads + head) * p.tiles + r / kCols;
  const size_t at = row * p.parts * kCols + r % kCols;
  const int d = threadIdx.x * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float M = -INFINITY, sum = 0.f;
  bool tokens = false;
#pragma unroll 8
  for (int i = 0; i < p.parts; ++i) M = max_nan(M, p.part_ml[at + i * kCols].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < p.parts; i0 += kAhead) {
    float2 ml[kAhead];
    float4 v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const size_t from = at + static_cast<size_t>(min(i0 + j, p.parts - 1)) * kCols;
      ml[j] = p.part_ml[from];
      v[j] = *reinterpret_cast<const float4*>(p.part_o + from * D + d);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j >= p.parts) break;
      tokens |= ml[j].y < 0.f || ml[j].x != -INFINITY;
      if (ml[j].x != -INFINITY) {
        const float w = exp2f(ml[j].x - M);
        sum = fmaf(w, ml[j].y, sum);
        acc.x = fmaf(w, v[j].x, acc.x);
        acc.y = fmaf(w, v[j].y, acc.y);
        acc.z = fmaf(w, v[j].z, acc.z);
        acc.w = fmaf(w, v[j].w, acc.w);
      }
    }
  }
  const float inv = inverse_of(M, sum, tokens);
  const float out[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
  store_out<4>(p.out, static_cast<size_t>(blockIdx.x) * D + d, out, p.out_dtype);
}

template <int D, int NT>
size_t smem_bytes(int stages) {
  const size_t ring = static_cast<size_t>(kWarps) * stages * 2 * Geo<D>::kTileBytes;
  const size_t join = static_cast<size_t>(kWarps) * 8 * NT * Geo<D>::kPitch * sizeof(float) +
                      (kWarps + 1) * 8 * NT * sizeof(float2);
  return kHeader + kAlign + (ring > join ? ring : join);
}

// Thread blocks per cluster, clusters per row and stages per ring: of the choices, the one with
// the least time by a model of the launch.  `slots` blocks are resident at a time and share the
// memory's rate; the blocks of the last, partly filled wave take what a warp's chunks take one after
// the other, if that is longer; each wave takes 2 us besides.  Of equals the deeper ring.
// Clusters wait for their slowest block and for free places on neighbouring SMs, which costs an
// eighth, so only launches of few rows have them; several clusters per row cost a second kernel,
// so only few rows with long lists do.  On GB300 (D = 128, us):
//   512 rows of 1 MB:     ranks 1 with stages 2: 97, 3: 82;  ranks 2: 91 and 95;  ranks 4: 93, 103
//   1280 rows of 0.5 MB:  ranks 1 with stages 2: 100, 3: 106 (two blocks an SM instead of three)
//   80 rows of 2 MB:      ranks 1 with stages 2: 54, 3: 55;  ranks 2: 34 and 34;  ranks 4: 30, 43
//   640 rows of 1 MB, D = 256:  ranks 1 with stages 1: 103, 2: 118 (one block an SM instead of three)
struct Shape {
  int ranks, parts, stages;
};
Shape shape_for(long long rows, long long chunks, const size_t (&smem_of)[3], double chunk_bytes,
                int most_per_sm, int most_parts) {
  constexpr double kRate = 6.8e6;              // bytes per us
  constexpr double kWait = 1.25, kStep = 0.85;  // us per chunk of a warp: copy and products, products
  const double row_bytes = chunks * chunk_bytes;
  Shape best{1, 1, 1};
  double least = 1e30;
  for (int stages = 1; stages <= 3; ++stages) {
    const size_t smem = smem_of[stages - 1];
    if (smem > 227 * 1024) continue;
    const int fit = static_cast<int>(228 * 1024 / (smem + 1024));
    const long long slots = 152ll * (fit < most_per_sm ? fit : most_per_sm);
    for (int all = 1; all <= kMaxCluster * most_parts; all *= 2) {  // blocks per row
      const long long blocks = rows * all, full = blocks / slots, rest = blocks - full * slots;
      const long long warps = static_cast<long long>(all) * kWarps;
      const long long each = (chunks + warps - 1) / warps;
      if (stages > 1 && stages > each) continue;  // nothing to fill them with
      const double alone = each * (stages == 1 ? kWait : kStep);
      const double bytes = row_bytes / all;
      const double shared = rest * bytes / kRate;
      double us = full * slots * bytes / kRate + (rest == 0 ? 0. : shared > alone ? shared : alone);
      us += 2. * (full + (rest > 0 ? 1 : 0));
      if (all > 1) us = us * 1.125 + 1.;
      if (all > kMaxCluster) us += 3.;
      if (us < least || (us == least && stages > best.stages)) {
        least = us;
        best = {all < kMaxCluster ? all : kMaxCluster, all <= kMaxCluster ? 1 : all / kMaxCluster, stages};
      }
    }
  }
  return best;
}

// The chunks of the longest list that holds no block twice.
long long chunks_of(int num_selected, int max_blocks, int block_size) {
  const long long held = num_selected < max_blocks ? num_selected : max_blocks;
  return (held * block_size + kChunk - 1) / kChunk;
}

// The clusters that a row may have.  kMaxShares in all fill the card several times over (39 rows of
// 19058 blocks of 16, 64 channels, 16 query heads: 503 us with 16 clusters a row, 551 us with 32).
int most_parts(long long rows, long long chunks) {
  if (chunks <= kWhole || rows > kMaxShares) return 1;
  return static_cast<int>(rows * kMaxParts < kMaxShares ? kMaxParts : kMaxShares / rows);
}

template <int D, int NT>
Shape shape_of(long long rows, int num_selected, int max_blocks, int block_size, bool parts) {
  const long long chunks = chunks_of(num_selected, max_blocks, block_size);
  // thread blocks an SM, as registers allow (64 channels, 8 heads: of 72 registers seven would fit)
  constexpr int kMost[3][2] = {{6, 4}, {4, 3}, {3, 2}};
  constexpr int most = kMost[D / 128][NT - 1];
  const size_t smem[3] = {smem_bytes<D, NT>(1), smem_bytes<D, NT>(2), smem_bytes<D, NT>(3)};
  return shape_for(rows, chunks, smem, 2 * Geo<D>::kTileBytes, most,
                   parts ? most_parts(rows, chunks) : 1);
}

long long rows_of(int num_seqs, int num_kv_heads, int group, int cols) {
  return static_cast<long long>(num_seqs) * num_kv_heads * ((group + cols - 1) / cols);
}

// Enough for the clusters of this call and of every one with fewer rows or shorter lists: what a
// call itself uses goes up and down with its rows (8 key heads, D = 128, lists of 8192 tokens: 40 shares
// of rows for 5 sequences, 24 for 6), and one buffer has to serve a batch whose sequences end.
template <int D, int NT>
size_t workspace_for(long long rows, long long chunks) {
  if (chunks <= kWhole) return 0;
  const long long shares = rows * kMaxParts < kMaxShares ? rows * kMaxParts : kMaxShares;
  return static_cast<size_t>(shares) * 8 * NT * (D * sizeof(float) + sizeof(float2));
}

template <class... Kernel, class... Args>
bool launch_dependent(void (*kernel)(Kernel...), dim3 grid, dim3 block, size_t smem, int cluster,
                      cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess && cudaGetLastError() == cudaSuccess;
}

template <class Tag, int D, int NT>
int launch(SparseParams p, const void* k_cache, const void* v_cache, int num_seqs, void* workspace,
           size_t workspace_bytes, cudaStream_t stream) {
  p.tiles = (p.group + 8 * NT - 1) / (8 * NT);
  const long long rows = rows_of(num_seqs, p.num_kv_heads, p.group, 8 * NT);
  const Shape shape = shape_of<D, NT>(rows, p.num_selected, p.max_blocks, p.block_size, workspace != nullptr);
  const int ranks = shape.ranks;
  p.stages = shape.stages;
  p.parts = shape.parts;
  if (rows * ranks * p.parts > 0x7fffffffll) return PA_ERR_INVALID_ARG;
  if (p.parts > 1) {
    if (workspace_bytes < workspace_for<D, NT>(rows, chunks_of(p.num_selected, p.max_blocks, p.block_size)))
      return PA_ERR_INVALID_ARG;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + rows * p.parts * 8 * NT * D);
  }
  // the caches as [D / 64][rows][64]: one box is a chunk, or half of one with 8-token blocks
  const cuuint64_t cache_rows = static_cast<cuuint64_t>(p.num_blocks) * p.num_kv_heads * p.block_size;
  const cuuint64_t dims[3] = {64, cache_rows, D / 64};
  const cuuint64_t strides[2] = {D * 2, 128};
  const cuuint32_t box[3] = {64, p.block_size == 8 ? 8u : 16u, D / 64};
  CUtensorMap tk, tv;
  const bool bf16 = std::is_same<Tag, BF16>::value;
  if (!encode_tensor_map(&tk, bf16, k_cache, 3, dims, strides, box) ||
      !encode_tensor_map(&tv, bf16, v_cache, 3, dims, strides, box))
    return PA_ERR_CUDA;
  const size_t smem = smem_bytes<D, NT>(p.stages);
  // Always the same value, so that concurrent callers never lower it for one another, and on
  // every launch that needs it (it is lost with the context).
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(paged_attn_sparse_kernel<Tag, D, NT>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
    return PA_ERR_CUDA;
  if (!launch_dependent(paged_attn_sparse_kernel<Tag, D, NT>,
                        dim3(static_cast<unsigned>(rows * ranks * p.parts)), dim3(kWarps * 32), smem,
                        ranks, stream, tk, tv, p))
    return PA_ERR_CUDA;
  if (p.parts > 1 &&
      !launch_dependent(paged_attn_sparse_join_kernel<D, NT>,
                        dim3(static_cast<unsigned>(num_seqs) * static_cast<unsigned>(p.num_heads)),
                        dim3(D / 4), 0, 1, stream, p))
    return PA_ERR_CUDA;
  return PA_OK;
}

template <class Tag, int D>
int launch_nt(const SparseParams& p, const void* k_cache, const void* v_cache, int num_seqs,
              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return p.group <= 8
             ? launch<Tag, D, 1>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, stream)
             : launch<Tag, D, 2>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, stream);
}

// f(D, NT) for the sizes of a call; 0 where there is no such call.
template <class F>
size_t for_sizes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                 int max_blocks_per_seq, int num_selected, F f) {
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      block_size <= 0 || max_blocks_per_seq <= 0 || num_selected <= 0)
    return 0;
  const auto with = [&](auto dim) {
    return num_heads / num_kv_heads <= 8 ? f(dim, std::integral_constant<int, 1>{})
                                         : f(dim, std::integral_constant<int, 2>{});
  };
  switch (head_dim) {
    case 64: return with(std::integral_constant<int, 64>{});
    case 128: return with(std::integral_constant<int, 128>{});
    case 256: return with(std::integral_constant<int, 256>{});
    default: return 0;
  }
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" size_t paged_attn_sparse_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                                   int head_dim, int block_size,
                                                   int max_blocks_per_seq, int num_selected) {
  return for_sizes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                   num_selected, [&](auto dim, auto nt) {
    constexpr int D = decltype(dim)::value, NT = decltype(nt)::value;
    return workspace_for<D, NT>(rows_of(num_seqs, num_kv_heads, num_heads / num_kv_heads, 8 * NT),
                                chunks_of(num_selected, max_blocks_per_seq, block_size));
  });
}

extern "C" size_t paged_attn_sparse_workspace_needed(int num_seqs, int num_heads, int num_kv_heads,
                                                     int head_dim, int block_size,
                                                     int max_blocks_per_seq, int num_selected) {
  return for_sizes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                   num_selected, [&](auto dim, auto nt) -> size_t {
    constexpr int D = decltype(dim)::value, NT = decltype(nt)::value;
    const long long rows = rows_of(num_seqs, num_kv_heads, num_heads / num_kv_heads, 8 * NT);
    if (shape_of<D, NT>(rows, num_selected, max_blocks_per_seq, block_size, true).parts == 1) return 0;
    return workspace_for<D, NT>(rows, chunks_of(num_selected, max_blocks_per_seq, block_size));
  });
}

extern "C" int paged_attn_sparse(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* block_tables, const int32_t* seq_lens,
                                 const int32_t* selected, int num_selected, int num_seqs,
                                 int num_heads, int num_kv_heads, int head_dim, int block_size,
                                 int max_blocks_per_seq, int num_blocks, float scale, int dtype,
                                 void* out, int out_dtype, void* workspace,
                                 size_t workspace_bytes, int32_t* error_record, void* stream) {
  NvtxRange range("paged_attn_sparse");
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || num_selected < 0)
    return PA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (block_size % 16 != 0 && block_size != 8) return PA_ERR_UNSUPPORTED;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (out_dtype != PA_F16 && out_dtype != PA_BF16 && out_dtype != PA_F32)
    return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size > (1ll << 30) || num_seqs > 65535 ||
      num_heads > 65535 ||
      static_cast<long long>(num_selected) * block_size > (1ll << 33))
    return PA_ERR_INVALID_ARG;
  if (static_cast<long long>(num_blocks) * num_kv_heads * block_size >= (1ll << 31))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !out ||
      (!selected && num_selected > 0))
    return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(workspace))
    return PA_ERR_INVALID_ARG;
  SparseParams p{};
  p.q = q;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.selected = selected;
  p.out = out;
  p.err = error_record;
  p.num_selected = num_selected;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.group = num_heads / num_kv_heads;
  p.out_dtype = out_dtype;
  p.qscale = scale * kLog2e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == PA_BF16) {
    switch (head_dim) {
      case 64: return launch_nt<BF16, 64>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, st);
      case 128: return launch_nt<BF16, 128>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, st);
      default: return launch_nt<BF16, 256>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, st);
    }
  }
  switch (head_dim) {
    case 64: return launch_nt<F16, 64>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, st);
    case 128: return launch_nt<F16, 128>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, st);
    default: return launch_nt<F16, 256>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, st);
  }
}
