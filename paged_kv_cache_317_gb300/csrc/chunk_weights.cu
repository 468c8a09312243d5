// The attention weight that the last rows of a chunk give each cached token, on the 5th-generation tensor
// cores (tcgen05 + TMEM + TMA):
//   weights[i][h][t] += sum over rows (token j, query head g of key head h) that see t of
//                       e^(scale <q, k_t> - lse of the row)
// with the rows' lse from the chunk's attention, so one pass over the keys does.
//
//  * Work item = (sequence, key head, 256 tokens).  S^T = K.Q^T: the tokens are the rows of the product
//    (TMEM lanes), so that a token's sum over rows is one thread's.  Two warpgroups take 128 tokens each, of
//    every 16 the first and the last 8 (a box of 16 rows then is one copy, whatever head_dim: 25 % faster
//    loads than a box for each 64 channels); the query rows, (token, head) packed 128 to a tile, go by as
//    columns.  A token's weight is added to by one thread, once: the same bits on every run.
//  * Persistent, one thread block an SM.  The items that exist are counted from the lengths, so that none
//    is dealt out in vain.  Where the window's tiles stay in shared memory a block takes a contiguous run
//    of items and loads them once a key head; else block b takes items b, 2 grid - 1 - b, 2 grid + b, ...,
//    heads innermost, so that the items of a causal triangle are shared out alike; few items of many tiles
//    are a cluster's each, whose blocks take its tiles in turn; some items a block go longest first.
//  * 11 warps: two softmax warpgroups, a producer (TMA boxes of 16 rows of K through the block table, boxes
//    of whole tiles of Q), an issuer of products for each warpgroup (one thread issues a product in about the
//    time that it runs, and has barriers to wait for besides: 32 sequences, 64 heads, window 32: 186 us with
//    one issuer, 165 with two).  Each warpgroup has two 128-column buffers of S in TMEM: one is read while
//    the next product runs.
//  * A token is seen from a column of a tile on: 32 columns are masked only where that column of one of the
//    warp's tokens lies among them, or the tile ends, and left out where no token is seen (the prompts below:
//    74 us, 92 with every tile of the diagonal masked).  Each warp has a copy of the rows' lse, so that it
//    waits for its products alone (72 prompts of 1500 rows: 772 us, 805 with a barrier a tile).
//  * Every wait is bounded (one second); on a timeout the block records PA_ERR_TIMEOUT, waits (bounded) for
//    its copies and products, frees its TMEM and returns.
// Bound by the hand-over between loads, products and softmax: a step of 256 tokens x 128 rows takes about 2300
// clocks (64 channels and passing rows: 2600), of which the products run for 1026 (513) and the exponentials
// for 1024.  Without exponentials and lse it still takes 85 % of the time, without any arithmetic on S 75-82 %;
// loads of S further ahead, of 16 or of 64 columns, make it slower.  32 sequences of up to 16384 tokens, 64
// heads on 8, window 32, 652 MB and 157 GFLOP: 151 us, 4.3 TB/s, 1.04 PFLOP/s.  12 whole prompts of up to 1500
// rows, 28 heads on 4, 64 channels, 17 GFLOP: 68 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "cluster.cuh"
#include "common.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace pagedkv {
namespace {

constexpr int kHalf = 128;                 // tokens of a warpgroup (MMA M)
constexpr int kTokens = 2 * kHalf;         // of an item
constexpr int kRows = 128;                 // query rows of a tile (MMA N)
constexpr int kWarpLoad = 8, kWarpMma = 9;  // and 10: an issuer for each warpgroup
constexpr int kThreads = 352;
constexpr int kMaxCluster = 4;
constexpr int kLists = 128;                // lists of sequences whose items are counted together
constexpr int kSorted = 256;               // (sequence, token tile) that are put in order
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kWide = D / 64;                    // 64-wide column groups, 128 bytes a row
  static constexpr int kKBytes = kTokens * D * 2;         // 32 / 64 / 128 KB
  static constexpr int kChunkBytes = 16 * D * 2;          // a box: 16 tokens of K
  static constexpr int kQBytes = kRows * D * 2;           // 16 / 32 / 64 KB
  static constexpr int kKStages = D == 64 ? 4 : D == 128 ? 2 : 1;
  static constexpr int kQStages = D == 256 ? 1 : 2;
  static constexpr int kOffQ = kKStages * kKBytes;
  static constexpr int kOffLse = kOffQ + kQStages * kQBytes;       // [warp][2][kRows] floats
  static constexpr int kOffSums = kOffLse + 8 * 2 * kRows * 4;  // [2][kMaxCluster][kTokens] floats
  static constexpr int kOffCount = kOffSums + 2 * kMaxCluster * kTokens * 4;  // [kLists] ints
  static constexpr int kOffOrder = kOffCount + kLists * 4;         // [kSorted] ints
  static constexpr int kOffBar = kOffOrder + kSorted * 4;
  static constexpr int kUsed = kOffBar + 512 + 1024;               // 1 KB to align the base
  // one block an SM, which takes all 512 TMEM columns
  static constexpr int kSmemBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static_assert(kSmemBytes <= 227 * 1024, "one block per SM");
};

struct Bars {
  uint64_t k_full[4], k_free[4], q_full[4], q_free[4];
  uint64_t s_full[2][2], s_free[2][2];  // [buffer][warpgroup]
  uint64_t sums_full[2], sums_free[2];  // the cluster's sums of even and odd items: all there; read
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

struct ChunkWeightsParams {
  const float* lse;
  const int32_t* query_start;
  const int32_t* seq_lens;
  const int32_t* block_tables;
  float* weights;
  int32_t* err;
  long long weights_row;  // floats from (sequence, key head) to the next
  int num_seqs, num_heads, num_kv_heads, block_size, max_blocks, num_blocks;
  int total_queries, max_query_len, window;
  int group, tile_tokens, inv_group;  // r / group = r * inv_group >> 16 for r < 128
  float qscale;                       // scale * log2(e)
};

// What a sequence has to do: its length, the rows of its window (0: nothing) and the first one's row in q.
struct Seq {
  int L, W, row0;
};

__device__ __forceinline__ Seq sequence(const ChunkWeightsParams& p, int seq, bool report) {
  Seq s{0, 0, 0};
  const int L = __ldg(p.seq_lens + seq);
  const int begin = __ldg(p.query_start + seq), end = __ldg(p.query_start + seq + 1);
  const int cap = p.max_blocks * p.block_size;
  const long long nq = static_cast<long long>(end) - begin;
  if (L < 0 || L > cap || nq < 0 || nq > L || nq > p.max_query_len || begin < 0 || end > p.total_queries) {
    if (report) report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    return s;
  }
  s.L = L;
  s.W = p.window > 0 ? min(p.window, static_cast<int>(nq)) : static_cast<int>(nq);
  s.row0 = end - s.W;
  return s;
}

__device__ __forceinline__ int tiles_of(const Seq& s) {
  return s.W > 0 ? (s.L + kTokens - 1) / kTokens : 0;
}

// The first tile of rows that sees a token of the tile at t0.
__device__ __forceinline__ int first_seeing(const ChunkWeightsParams& p, const Seq& s, int t0) {
  const int before = s.L - s.W;
  return t0 > before ? (t0 - before) / p.tile_tokens : 0;
}

// Items of one key head: its token tiles from `tile` to before `end`.
struct Run {
  Seq s;
  int seq, head, tile, end;
  int row_tiles;  // tiles of query rows

  __device__ __forceinline__ int first(const ChunkWeightsParams& p, int t0) const { return first_seeing(p, s, t0); }
};

// The items of a thread block or cluster, b of n, decoded alike by every warp, which look up what is next
// only from run to run: what each does once an item adds to every item's time.
// kResident: the window's tiles of rows stay in shared memory while a key head's tokens go by; else they go
// by for every item.
template <bool kResident>
struct Walk {
  const ChunkWeightsParams& p;
  const int* upto;  // [kLists]: items of the first lists of sequences
  const int* order; // (sequence, token tile), as 256 sequence + tile, in the order that they are dealt out; or NULL
  int list;         // sequences of a list
  int m, end, b, n;
  Run run;

  __device__ __forceinline__ Walk(const ChunkWeightsParams& p, const int* upto, const int* order, int list, int b,
                                  int n)
      : p(p), upto(upto), order(order), list(list), b(b), n(n) {
    const long long all = upto[kLists - 1];
    m = kResident ? static_cast<int>(all * b / n) : b;
    end = kResident ? static_cast<int>(all * (b + 1) / n) : static_cast<int>(all);
  }

  // The next run; false past the last.  By whole warps.
  __device__ __forceinline__ bool next() {
    if (m >= end) return false;
    if (!kResident && order != nullptr) {
      const int unit = m / p.num_kv_heads, u = order[unit];
      run.seq = u >> 8;
      run.s = sequence(p, run.seq, false);
      run.row_tiles = (run.s.W + p.tile_tokens - 1) / p.tile_tokens;
      run.head = m - unit * p.num_kv_heads;
      run.tile = u & 255;
      run.end = run.tile + 1;
      there_and_back();
      return true;
    }
    const int lane = threadIdx.x & 31;
    const int4 u = reinterpret_cast<const int4*>(upto)[lane];
    const int r = __reduce_add_sync(kFullMask, (u.x <= m) + (u.y <= m) + (u.z <= m) + (u.w <= m));
    int left = m - (r > 0 ? upto[r - 1] : 0);
    const int last = min(p.num_seqs, (r + 1) * list);
    for (int s0 = r * list; s0 < last; s0 += 32) {
      const int seq = s0 + lane;
      Seq s{0, 0, 0};
      if (seq < last) s = sequence(p, seq, false);
      const int items = tiles_of(s) * p.num_kv_heads;
      int sum = items;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(kFullMask, sum, off);
        if (lane >= off) sum += v;
      }
      const unsigned past = __ballot_sync(kFullMask, sum > left);
      if (past != 0) {
        const int at = __ffs(past) - 1;
        run.seq = s0 + at;
        run.s.L = __shfl_sync(kFullMask, s.L, at);
        run.s.W = __shfl_sync(kFullMask, s.W, at);
        run.s.row0 = __shfl_sync(kFullMask, s.row0, at);
        run.row_tiles = (run.s.W + p.tile_tokens - 1) / p.tile_tokens;
        left -= __shfl_sync(kFullMask, sum - items, at);
        break;
      }
      left -= __shfl_sync(kFullMask, sum, 31);
    }
    if constexpr (kResident) {  // a key head's tokens one after the other
      const int tiles = tiles_of(run.s);
      run.head = left / tiles;
      run.tile = left - run.head * tiles;
      run.end = min(tiles, run.tile + end - m);
      m += run.end - run.tile;
    } else {           // heads innermost
      run.tile = left / p.num_kv_heads;
      run.head = left - run.tile * p.num_kv_heads;
      run.end = run.tile + 1;
      there_and_back();
    }
    return true;
  }

  __device__ __forceinline__ void there_and_back() {  // a sequence's items get smaller
    b = n - 1 - b;
    m = (m / n + 1) * n + b;
  }
};

// e^(logit - lse) of 32 columns of S, added to the four sums; nl: shared address of -lse in base 2.
__device__ __forceinline__ void add_weights(const float (&s)[32], uint32_t nl, float qscale, float (&sum)[4]) {
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    const float4 v = ld_shared4(nl + 4 * c);
    float x0, x1, x2, x3;
    fma2(x0, x1, s[c], s[c + 1], qscale, v.x, v.y);
    fma2(x2, x3, s[c + 2], s[c + 3], qscale, v.z, v.w);
    add2(sum[0], sum[1], ex2_approx(x0), ex2_approx(x1));
    add2(sum[2], sum[3], ex2_approx(x2), ex2_approx(x3));
  }
}

// The same for the columns from `from` to before `cols` alone.  Others may hold anything.
__device__ __forceinline__ void add_seen_weights(const float (&s)[32], uint32_t nl, float qscale, int from, int cols,
                                                 float (&sum)[4]) {
  // bit c: column c is one of them
  const uint32_t seen = (from < 32 ? kFullMask << max(from, 0) : 0u) & (cols < 32 ? ~(kFullMask << cols) : kFullMask);
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    const float4 v = ld_shared4(nl + 4 * c);
    float x0, x1, x2, x3;
    fma2(x0, x1, s[c], s[c + 1], qscale, v.x, v.y);
    fma2(x2, x3, s[c + 2], s[c + 3], qscale, v.z, v.w);
    float e[4] = {ex2_approx(x0), ex2_approx(x1), ex2_approx(x2), ex2_approx(x3)};
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = seen & 1u << (c + i) ? e[i] : 0.f;
    add2(sum[0], sum[1], e[0], e[1]);
    add2(sum[2], sum[3], e[2], e[3]);
  }
}

template <bool BF16, int D, bool kResident>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k, const ChunkWeightsParams p) {
  using C = Cfg<D>;
  constexpr int KS = C::kKStages, QS = C::kQStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  float* lse_s = reinterpret_cast<float*>(smem + C::kOffLse);
  int* upto = reinterpret_cast<int*>(smem + C::kOffCount);
  int* order = reinterpret_cast<int*>(smem + C::kOffOrder);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  volatile int* abort_flag = &bars->abort;
  const bool half_blocks = p.block_size < 16;
  const int ranks = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());

  if (threadIdx.x == 0) {
    prefetch_tensor_map(&tm_q);
    prefetch_tensor_map(&tm_k);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_free[s], 2);  // both issuers
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_free[s], 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->drain[s], 1);
      mbar_init(&bars->sums_full[s], ranks > 1 ? (ranks - 1) * kTokens : 1);
      mbar_init(&bars->sums_free[s], kTokens);
    }
    for (int g = 0; g < 4; ++g) {
      mbar_init(&bars->s_full[g >> 1][g & 1], 1);
      mbar_init(&bars->s_free[g >> 1][g & 1], kHalf);
    }
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&bars->tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // The items of each list of sequences, then those of all lists up to each.
  const int list = (p.num_seqs + kLists - 1) / kLists;
  if (threadIdx.x < kLists) {
    int sum = 0;
    for (int s = threadIdx.x * list; s < min(p.num_seqs, (static_cast<int>(threadIdx.x) + 1) * list); ++s)
      sum += tiles_of(sequence(p, s, blockIdx.x == 0)) * p.num_kv_heads;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kFullMask, sum, off);
      if (lane >= off) sum += v;
    }
    upto[threadIdx.x] = sum;
  }
  __syncthreads();
  if (threadIdx.x < kLists) {
    int sum = upto[threadIdx.x];
    for (int w = 0; w < warp; ++w) sum += upto[w * 32 + 31];
    asm volatile("bar.sync 1, 128;" ::: "memory");
    upto[threadIdx.x] = sum;
  }
  tc_fence_before();
  __syncthreads();
  // Passing rows: a few items a block are dealt out longest first (12 sequences of 800 rows, 28 heads on 4: 58 us,
  // 71 in the order of sequences; 76 of 512, 17 items a cluster: 139 and 133).
  bool sorted = false;
  if constexpr (!kResident) {
    const int n = upto[kLists - 1] / p.num_kv_heads;  // (sequence, token tile)
    const int items = upto[kLists - 1], walkers = static_cast<int>(gridDim.x) / ranks;
    sorted = list == 1 && n <= kSorted && items > walkers && items <= 8 * walkers;
    if (sorted) {
      int* rows = reinterpret_cast<int*>(smem);  // tiles of rows of each; K's place, which nothing is in yet
      int* what = rows + kSorted;
      if (threadIdx.x < p.num_seqs) {
        const int seq = threadIdx.x, end = upto[seq] / p.num_kv_heads;
        const Seq s = sequence(p, seq, false);
        const int tiles = tiles_of(s), row_tiles = (s.W + p.tile_tokens - 1) / p.tile_tokens;
        for (int tile = 0; tile < tiles; ++tile) {
          rows[end - tiles + tile] = row_tiles - first_seeing(p, s, tile * kTokens);
          what[end - tiles + tile] = seq << 8 | tile;
        }
      }
      __syncthreads();
      if (threadIdx.x < n) {
        const int mine = rows[threadIdx.x];
        int place = 0;
        for (int i = 0; i < n; ++i) place += rows[i] > mine || (rows[i] == mine && i < threadIdx.x);
        order[place] = what[threadIdx.x];
      }
      fence_async_smem();  // TMA writes there
      __syncthreads();
    }
  }
  if (ranks > 1) cluster_sync();  // peers' barriers are set up
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  Walk<kResident> walk(p, upto, sorted ? order : nullptr, list, static_cast<int>(blockIdx.x) / ranks,
                       static_cast<int>(gridDim.x) / ranks);
  const Run& run = walk.run;

  int k_loads = 0, q_loads = 0;  // producer, issuer: tiles begun so far
  int mma_started = 0;
  if (warp == kWarpLoad) {
    // --------------------------------------------------------------- producer
    int good = 1;
    auto load_q = [&](int j) -> bool {
      const int qs = q_loads % QS;
      if (lane == 0) {
        if (q_loads >= QS) good = mbar_wait_bounded(&bars->q_free[qs], (q_loads / QS - 1) & 1);
        if (good) {
          mbar_arrive_expect_tx(&bars->q_full[qs], C::kWide * 128u * p.tile_tokens * p.group);
#pragma unroll
          for (int g = 0; g < C::kWide; ++g)
            tma_load_3d(smem + C::kOffQ + qs * C::kQBytes + g * (kRows * 128), &tm_q, 64 * g,
                        run.head * p.group, run.s.row0 + j * p.tile_tokens, &bars->q_full[qs]);
        }
      }
      ++q_loads;
      return __shfl_sync(kFullMask, good, 0) != 0 && __shfl_sync(kFullMask, *abort_flag, 0) == 0;
    };
    bool ok = true;
    while (ok && walk.next()) {
      const int32_t* table = p.block_tables + static_cast<size_t>(run.seq) * p.max_blocks;
      // lane l < 16 of a tile: the block of tokens t0 + 16 l on (with 8-token blocks also of the 8 after),
      // as a row of the cache seen as rows of D
      auto y_of = [&](int t) -> int {
        if (t >= run.s.L) return -1;
        const int b = t / p.block_size;
        int blk = __ldg(table + b);
        if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
          if (run.head == 0 && rank == 0 && t == b * p.block_size)
            report_error(p.err, PA_ERR_BAD_BLOCK, run.seq, blk);
          blk = 0;
        }
        return (blk * p.num_kv_heads + run.head) * p.block_size + (t - b * p.block_size);
      };
      bool with_q = kResident;
      for (int tile = run.tile; ok && tile < run.end; ++tile) {
        const int t0 = tile * kTokens;
        const int j0 = kResident ? 0 : run.first(p, t0) + rank;
        if (j0 >= run.row_tiles) break;  // other blocks of the cluster have its tiles
        int y = -1, y_hi = -1;
        if (lane < 16) {
          y = y_of(t0 + lane * 16);
          if (half_blocks) y_hi = y_of(t0 + lane * 16 + 8);
        }
        const int ks = k_loads % KS;
        if (lane == 0) {
          if (k_loads >= KS) good = mbar_wait_bounded(&bars->k_free[ks], (k_loads / KS - 1) & 1);
          const int unit = half_blocks ? 8 : 16;
          const int rows = (min(kTokens, run.s.L - t0) + unit - 1) / unit * unit;
          if (good) mbar_arrive_expect_tx(&bars->k_full[ks], static_cast<uint32_t>(rows) * D * 2);
        }
        ok = __shfl_sync(kFullMask, good, 0) != 0;
        if (!ok) break;
        uint8_t* dst = smem + ks * C::kKBytes + lane * C::kChunkBytes;
        if (y >= 0) tma_load_3d(dst, &tm_k, 0, y, 0, &bars->k_full[ks]);
        if (y_hi >= 0) tma_load_3d(dst + C::kChunkBytes / 2, &tm_k, 0, y_hi, 0, &bars->k_full[ks]);
        ++k_loads;
        if (__shfl_sync(kFullMask, *abort_flag, 0)) ok = false;
        if (!kResident || with_q)
          for (int j = j0; ok && j < run.row_tiles; j += ranks) ok = load_q(j);
        with_q = false;
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report_error(p.err, PA_ERR_TIMEOUT, run.seq, -1);
    }
  } else if (warp >= kWarpMma) {
    // ----------------------------------------------------- issuers, one a warpgroup
    const int g = warp - kWarpMma;
    constexpr uint32_t idesc = make_idesc(kHalf, kRows, BF16, false);
    // K: the same 8 rows of each of 16 chunks, one product's; from 8-token blocks a chunk is two boxes
    const uint64_t k_desc = smem_desc_sw128(smem, 16, C::kChunkBytes);
    const uint32_t k_half = half_blocks ? C::kChunkBytes / 2 : 1024, k_group = half_blocks ? 1024 : 2048;
    const uint64_t q_desc = smem_desc_sw128(smem + C::kOffQ, 16, 1024);
    // only the address, in the lower word, differs from product to product
    const uint32_t k_hi = static_cast<uint32_t>(k_desc >> 32), q_hi = static_cast<uint32_t>(q_desc >> 32);
    bool ok = true;
    int steps = 0;
    while (ok && walk.next()) {
      if (lane == 0) {
        const int held = q_loads;  // loads before the first of this run
        if constexpr (kResident) {
          q_loads += run.row_tiles;
          // (every load is waited for, its tile used or not, before its stage is handed back)
          for (int q = held; ok && q < q_loads; ++q) ok = mbar_wait_bounded(&bars->q_full[q % QS], (q / QS) & 1);
        }
        for (int tile = run.tile; ok && tile < run.end; ++tile) {
          const int first = run.first(p, tile * kTokens) + rank;
          if (first >= run.row_tiles) break;
          const int ks = k_loads % KS;
          const uint32_t k_lo = static_cast<uint32_t>(k_desc) + ((ks * C::kKBytes + g * k_half) >> 4);
          ok = mbar_wait_bounded(&bars->k_full[ks], (k_loads / KS) & 1);
          ++k_loads;
          for (int j = first; ok && j < run.row_tiles; j += ranks, ++steps) {
            const int q = kResident ? held + j : q_loads++, qs = q % QS, b = steps & 1;
            if (!kResident) ok = mbar_wait_bounded(&bars->q_full[qs], (q / QS) & 1);
            const uint32_t q_lo = static_cast<uint32_t>(q_desc) + (qs * C::kQBytes >> 4);
            if (ok && steps >= 2) ok = mbar_wait_bounded(&bars->s_free[b][g], ((steps >> 1) - 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_f16(tmem + (b * 2 + g) * kRows, k_hi, k_lo + (kk >> 2) * (k_group >> 4) + (kk & 3) * 2, q_hi,
                      q_lo + (((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4), idesc, kk > 0);
            mma_commit(&bars->s_full[b][g]);
            mma_started = 1;
            if (!kResident) mma_commit(&bars->q_free[qs]);
          }
          if (ok) mma_commit(&bars->k_free[ks]);
        }
        if (ok && kResident)
          for (int q = held; q < q_loads; ++q) mma_commit(&bars->q_free[q % QS]);
      }
      ok = __shfl_sync(kFullMask, ok, 0);
    }
    mma_started = __shfl_sync(kFullMask, mma_started, 0);
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report_error(p.err, PA_ERR_TIMEOUT, -1, -1);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int wg = warp >> 2, r = threadIdx.x & (kHalf - 1);
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + wg * kRows;
    const int at = (r >> 3) * 16 + wg * 8 + (r & 7);  // this thread's token of an item
    float* lse_warp = lse_s + warp * 2 * kRows;
    int steps = 0, items = 0, lse_loads = 0;
    bool ok = true;
    while (ok && walk.next()) {
      const size_t sh = static_cast<size_t>(run.seq) * p.num_kv_heads + run.head;
      // -lse in base 2 of rows lane, lane + 32, ... of tile j; 0 past the window's last, and where a row only
      // fills the tile up
      int tok[4];
      long long from_row[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = lane + 32 * k;
        tok[k] = row * p.inv_group >> 16;
        from_row[k] = (static_cast<long long>(run.s.row0) + tok[k]) * p.num_heads + run.head * p.group +
                      (row - tok[k] * p.group);
      }
      auto row_lse = [&](int j, float (&v)[4]) {
        const int tokens = min(p.tile_tokens, run.s.W - j * p.tile_tokens);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = tok[k] < tokens
                     ? -kLog2e * __ldg(p.lse + from_row[k] + static_cast<long long>(j) * p.tile_tokens * p.num_heads)
                     : 0.f;
      };
      if constexpr (kResident) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < QS; ++j) {
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          if (j < run.row_tiles) row_lse(j, v);
#pragma unroll
          for (int k = 0; k < 4; ++k) lse_warp[j * kRows + lane + 32 * k] = v[k];
        }
        __syncwarp();
      }
      for (int tile = run.tile; ok && tile < run.end; ++tile) {
        const int t0 = tile * kTokens, t = t0 + at;
        const int first = run.first(p, t0) + rank;
        float total = 0.f, next_lse[4];
        if (!kResident && first < run.row_tiles) row_lse(first, next_lse);
        for (int j = first; j < run.row_tiles; j += ranks, ++steps) {
          const int b = steps & 1;
          const float* lse = lse_warp + j * kRows;
          if constexpr (!kResident) {
            __syncwarp();  // the tile before the last is read
            float* mine = lse_warp + (lse_loads++ & 1) * kRows;
#pragma unroll
            for (int k = 0; k < 4; ++k) mine[lane + 32 * k] = next_lse[k];
            if (j + ranks < run.row_tiles) row_lse(j + ranks, next_lse);
            __syncwarp();
            lse = mine;
          }
          // the first row's place in the sequence: rows before it see less
          const int pos = run.s.L - run.s.W + j * p.tile_tokens;
          const int cols = min(p.tile_tokens, run.s.W - j * p.tile_tokens) * p.group;
          // Token t is seen from column (t - pos) group on; those of the warp lie between its first lane's,
          // from which all before are left out, and its last one's, from which on no column needs a mask.
          const int from = max(t - pos, 0) * p.group, warp_from = __shfl_sync(kFullMask, from, 0);
          const int warp_all = __shfl_sync(kFullMask, from, 31);
          const uint32_t at_s = lanes + b * 2 * kRows;
          const uint32_t nl = smem_addr(lse);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          ok = __all_sync(kFullMask, mbar_wait_bounded(&bars->s_full[b][wg], (steps >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          int c = warp_from & ~31;
#pragma unroll 1
          for (; c < min(warp_all, cols); c += 32) {
            float s[32];
            tmem_ld32(at_s + c, s);
            add_seen_weights(s, nl + 4 * c, p.qscale, from - c, cols - c, sum);
          }
#pragma unroll 1
          for (; c + 32 <= cols; c += 32) {
            float s[32];
            tmem_ld32(at_s + c, s);
            add_weights(s, nl + 4 * c, p.qscale, sum);
          }
          if (c < cols) {  // a tile whose rows are not a multiple of 32
            float s[32];
            tmem_ld32(at_s + c, s);
            add_seen_weights(s, nl + 4 * c, p.qscale, 0, cols - c, sum);
          }
          tc_fence_before();
          mbar_arrive(&bars->s_free[b][wg]);
          total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (__shfl_sync(kFullMask, *abort_flag, 0)) ok = false;
        if (ranks > 1) {
          // The cluster's sums meet in its first block, which adds them in order.
          const int buf = items & 1, use = items >> 1;
          ++items;
          float* sums = reinterpret_cast<float*>(smem + C::kOffSums) + buf * kMaxCluster * kTokens + at;
          if (rank == 0) {
            ok = ok && __all_sync(kFullMask, mbar_wait_cluster(&bars->sums_full[buf], use & 1));
            for (int i = 1; i < ranks; ++i) total += sums[i * kTokens];
            for (int i = 1; i < ranks; ++i) mbar_arrive_peer(&bars->sums_free[buf], i);
          } else {
            if (use > 0) ok = ok && __all_sync(kFullMask, mbar_wait_cluster(&bars->sums_free[buf], (use - 1) & 1));
            st_peer(smem_addr(sums + rank * kTokens), 0, total);
            mbar_arrive_peer(&bars->sums_full[buf], 0);
          }
        }
        // One thread adds to a weight, once: a reduction in L2 gives the same bits as a load, an add and a
        // store (but for numbers below 2^-126, which it may take for 0), and nothing waits for the load.
        if (ok && rank == 0 && t < run.s.L) atomicAdd(p.weights + sh * p.weights_row + t, total);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report_error(p.err, PA_ERR_TIMEOUT, -2, warp);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // Let every copy and product this block started finish before its shared memory and TMEM are
    // released (bounded waits).
    if (warp == kWarpLoad && lane == 0) {
      for (int s = 0; s < KS && s < k_loads; ++s)
        mbar_wait_bounded(&bars->k_full[s], ((k_loads - 1 - s) / KS) & 1);
      for (int s = 0; s < QS && s < q_loads; ++s)
        mbar_wait_bounded(&bars->q_full[s], ((q_loads - 1 - s) / QS) & 1);
    }
    if (warp >= kWarpMma && lane == 0 && mma_started) {
      mma_commit(&bars->drain[warp - kWarpMma]);
      mbar_wait_bounded(&bars->drain[warp - kWarpMma], 0);
    }
    __syncthreads();
  }
  if (ranks > 1) cluster_sync();  // no block leaves while another may write to its memory
  tc_fence_after();
  if (warp == kWarpMma) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

template <bool BF16, int D, bool kResident>
int launch(const ChunkWeightsParams& p, int most, const void* q, const void* k_cache,
           unsigned long long cache_rows, cudaStream_t stream) {
  using C = Cfg<D>;
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return PA_ERR_CUDA;
  CUtensorMap tq, tk;
  const cuuint64_t qdims[3] = {D, static_cast<cuuint64_t>(p.num_heads),
                               static_cast<cuuint64_t>(p.total_queries)};
  const cuuint64_t qstr[2] = {D * 2, static_cast<cuuint64_t>(D) * 2 * p.num_heads};
  const cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.tile_tokens)};
  // the cache as [D / 64][rows][64]: one box is a chunk, or half of one with 8-token blocks
  const cuuint64_t cdims[3] = {64, cache_rows, D / 64};
  const cuuint64_t cstr[2] = {D * 2, 128};
  const cuuint32_t cbox[3] = {64, p.block_size >= 16 ? 16u : 8u, D / 64};
  if (!encode_tensor_map(&tq, BF16, q, 3, qdims, qstr, qbox) ||
      !encode_tensor_map(&tk, BF16, k_cache, 3, cdims, cstr, cbox))
    return PA_ERR_CUDA;
  if (cudaFuncSetAttribute(chunk_weights_kernel<BF16, D, kResident>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::kSmemBytes) != cudaSuccess)
    return PA_ERR_CUDA;
  const long long tiles = (static_cast<long long>(p.max_blocks) * p.block_size + kTokens - 1) / kTokens;
  const long long items = p.num_seqs * tiles * p.num_kv_heads;
  // Few items of many tiles of rows: a cluster shares out an item's tiles.  Two tiles a block are enough where
  // every cluster has a place at once (4 key heads, 200 rows of 7 heads: 10.5 us, 13.1 with eight; of 12 such
  // sequences, where they do not: 18.1 us with two, 13.8 with eight).
  const int row_tiles = (most + p.tile_tokens - 1) / p.tile_tokens;
  int ranks = 1;
  while (!kResident && ranks < kMaxCluster && items * ranks < 4ll * sms &&
         row_tiles >= (items * 2 * ranks <= sms ? 2 : 8) * ranks)
    ranks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // as many clusters as find places at a time, whose SMs have to be neighbours
  int walkers = sms;
  if (ranks > 1) {
    cfg.gridDim = dim3(ranks);
    if (cudaOccupancyMaxActiveClusters(&walkers, chunk_weights_kernel<BF16, D, kResident>, &cfg) != cudaSuccess ||
        walkers <= 0)
      return PA_ERR_CUDA;
  }
  cfg.gridDim = dim3(static_cast<unsigned>((items < walkers ? items : walkers) * ranks));
  if (cudaLaunchKernelEx(&cfg, chunk_weights_kernel<BF16, D, kResident>, tq, tk, p) != cudaSuccess ||
      cudaGetLastError() != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

template <bool BF16, int D>
int launch(const ChunkWeightsParams& p, const void* q, const void* k_cache, unsigned long long cache_rows,
           cudaStream_t stream) {
  const int most = p.window > 0 && p.window < p.max_query_len ? p.window : p.max_query_len;
  return most <= Cfg<D>::kQStages * p.tile_tokens
             ? launch<BF16, D, true>(p, most, q, k_cache, cache_rows, stream)
             : launch<BF16, D, false>(p, most, q, k_cache, cache_rows, stream);
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int paged_chunk_weights(const void* q, const float* lse, const int32_t* query_start,
                                   int total_queries, int max_query_len, const void* k_cache,
                                   const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                                   int num_heads, int num_kv_heads, int head_dim, int block_size,
                                   int max_blocks_per_seq, int num_blocks, float scale, int dtype, int window,
                                   float* weights, int64_t weights_tokens, int32_t* error_record,
                                   void* stream) {
  NvtxRange range("paged_chunk_weights");
  if (num_seqs < 0 || total_queries < 0 || max_query_len < 0 || window < 0 || num_heads <= 0 ||
      num_kv_heads <= 0 || num_heads % num_kv_heads != 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  const int group = num_heads / num_kv_heads;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || (block_size % 16 != 0 && block_size != 8) ||
      group > kRows)
    return PA_ERR_UNSUPPORTED;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
  const long long cap = static_cast<long long>(max_blocks_per_seq) * block_size;
  const unsigned long long cache_rows =
      static_cast<unsigned long long>(num_blocks) * num_kv_heads * block_size;
  // (items are counted in an int, with a grid's worth of headroom)
  if (cap > (1ll << 30) || num_seqs > 65535 || weights_tokens < cap || cache_rows >= (1ull << 31) ||
      static_cast<long long>(num_seqs) * num_kv_heads > (1ll << 30) / ((cap + kTokens - 1) / kTokens))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_queries == 0 || max_query_len == 0) return PA_OK;
  if (!q || !lse || !query_start || !k_cache || !block_tables || !seq_lens || !weights)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache)) return PA_ERR_INVALID_ARG;
  ChunkWeightsParams p{};
  p.lse = lse;
  p.query_start = query_start;
  p.seq_lens = seq_lens;
  p.block_tables = block_tables;
  p.weights = weights;
  p.weights_row = weights_tokens;
  p.err = error_record;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.total_queries = total_queries;
  p.max_query_len = max_query_len < cap ? max_query_len : static_cast<int>(cap);  // (no more queries than tokens)
  p.window = window;
  p.group = group;
  p.tile_tokens = kRows / group;
  p.inv_group = (65536 + group - 1) / group;
  p.qscale = scale * kLog2e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch ((dtype == PA_BF16 ? 1 : 0) | (head_dim == 64 ? 0 : head_dim == 128 ? 2 : 4)) {
    case 0: return launch<false, 64>(p, q, k_cache, cache_rows, st);
    case 1: return launch<true, 64>(p, q, k_cache, cache_rows, st);
    case 2: return launch<false, 128>(p, q, k_cache, cache_rows, st);
    case 3: return launch<true, 128>(p, q, k_cache, cache_rows, st);
    case 4: return launch<false, 256>(p, q, k_cache, cache_rows, st);
    default: return launch<true, 256>(p, q, k_cache, cache_rows, st);
  }
}
