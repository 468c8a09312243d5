// The attention weight that the last rows of a chunk give each cached token, on the 5th-generation tensor
// cores (tcgen05 + TMEM + TMA):
//   weights[i][h][t] += sum over rows (token j, query head g of key head h) that see t of
//                       e^(scale <q, k_t> - lse of the row)
// with the rows' lse from the chunk's attention, so one pass over the keys does.
//
//  * Work item = (sequence, key head, 256 tokens).  S^T = K.Q^T: the tokens are the rows of the product
//    (TMEM lanes), so that a token's sum over rows is one thread's.  Two warpgroups take 128 tokens each;
//    the query rows, (token, head) packed 128 to a tile, go by as columns.  Every token is one thread's of
//    one item: no atomics, the same bits on every run.
//  * Persistent, one thread block an SM.  The items that exist are counted from the lengths, so that none
//    is dealt out in vain.  Where the window's tiles stay in shared memory a block takes a contiguous run
//    of items and loads them once a key head; else block b takes items b, b + grid, ...: heads innermost,
//    so that the items of a causal triangle are shared out alike.
//  * 10 warps: two softmax warpgroups, a producer (TMA boxes of 16 rows of K through the block table, boxes
//    of whole tiles of Q), an issuer of the products.  Each warpgroup has two 128-column buffers of S in
//    TMEM: one is read while the next product runs.
//  * Masks only where a tile of rows meets tokens that some of its rows do not see, or ends short.
//  * Every wait is bounded (one second); on a timeout the block records PA_ERR_TIMEOUT, waits (bounded) for
//    its copies and products, frees its TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace pagedkv {
namespace {

constexpr int kHalf = 128;                 // tokens of a warpgroup (MMA M)
constexpr int kTokens = 2 * kHalf;         // of an item
constexpr int kRows = 128;                 // query rows of a tile (MMA N)
constexpr int kWarpLoad = 8, kWarpMma = 9;
constexpr int kThreads = 320;
constexpr int kLists = 128;                // runs of sequences whose items are counted together
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kGroups = D / 64;                  // 64-wide column groups, 128 bytes a row
  static constexpr int kKBytes = kTokens * D * 2;         // 32 / 64 / 128 KB
  static constexpr int kQBytes = kRows * D * 2;           // 16 / 32 / 64 KB
  static constexpr int kKStages = D <= 128 ? 2 : 1;
  static constexpr int kQStages = D <= 128 ? 2 : 1;
  static constexpr int kOffQ = kKStages * kKBytes;
  static constexpr int kOffLse = kOffQ + kQStages * kQBytes;       // [warpgroup][2][kRows] floats
  static constexpr int kOffCount = kOffLse + 4 * kRows * 4;        // [kLists] ints
  static constexpr int kOffBar = kOffCount + kLists * 4;
  static constexpr int kUsed = kOffBar + 256 + 1024;               // 1 KB to align the base
  // one block an SM, which takes all 512 TMEM columns
  static constexpr int kSmemBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static_assert(kSmemBytes <= 227 * 1024, "one block per SM");
};

struct Bars {
  uint64_t k_full[2], k_free[2], q_full[2], q_free[2];
  uint64_t s_full[2][2], s_free[2][2];  // [warpgroup][buffer]
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

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
  int resident;                       // the window's tiles stay in shared memory
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

struct Item {
  Seq s;
  int seq, head, t0;
  int first, tiles;  // tiles of query rows: the first that sees a token of the item, and their number
};

// The items of a thread block, decoded alike by every warp.
struct Walk {
  const ChunkWeightsParams& p;
  const int* upto;   // [kLists]: items of the first runs of sequences
  int run;           // sequences of a run
  int m, end, step;
  Item it;
  int seq_begin, seq_items;  // the items of it.seq

  __device__ __forceinline__ Walk(const ChunkWeightsParams& p, const int* upto, int run)
      : p(p), upto(upto), run(run), seq_begin(0), seq_items(0) {
    const long long all = upto[kLists - 1];
    const int b = static_cast<int>(blockIdx.x), n = static_cast<int>(gridDim.x);
    step = p.resident ? 1 : n;
    m = p.resident ? static_cast<int>(all * b / n) : b;
    end = p.resident ? static_cast<int>(all * (b + 1) / n) : static_cast<int>(all);
  }

  // The next item; false past the last.  By whole warps.
  __device__ __forceinline__ bool next() {
    if (m >= end) return false;
    const int lane = threadIdx.x & 31;
    if (m - seq_begin >= seq_items) {
      const int4 u = reinterpret_cast<const int4*>(upto)[lane];
      const int r = __reduce_add_sync(kFullMask, (u.x <= m) + (u.y <= m) + (u.z <= m) + (u.w <= m));
      int left = m - (r > 0 ? upto[r - 1] : 0);
      for (int s0 = r * run;; s0 += 32) {
        const int seq = s0 + lane;
        Seq s{0, 0, 0};
        if (seq < min(p.num_seqs, (r + 1) * run)) s = sequence(p, seq, false);
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
          it.seq = s0 + at;
          it.s.L = __shfl_sync(kFullMask, s.L, at);
          it.s.W = __shfl_sync(kFullMask, s.W, at);
          it.s.row0 = __shfl_sync(kFullMask, s.row0, at);
          seq_items = __shfl_sync(kFullMask, items, at);
          seq_begin = m - (left - __shfl_sync(kFullMask, sum - items, at));
          break;
        }
        left -= __shfl_sync(kFullMask, sum, 31);
        if (s0 + 32 >= (r + 1) * run) return false;  // (not reached: the counts say there is one)
      }
    }
    const int at = m - seq_begin;
    int tile;
    if (p.resident) {
      const int tiles = seq_items / p.num_kv_heads;
      it.head = at / tiles;
      tile = at - it.head * tiles;
    } else {
      tile = at / p.num_kv_heads;
      it.head = at - tile * p.num_kv_heads;
    }
    it.t0 = tile * kTokens;
    it.tiles = (it.s.W + p.tile_tokens - 1) / p.tile_tokens;
    it.first = max(0, it.t0 - (it.s.L - it.s.W)) / p.tile_tokens;
    m += step;
    return true;
  }
};

template <bool BF16, int D>
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
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  volatile int* abort_flag = &bars->abort;
  const bool half_blocks = p.block_size < 16;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_free[s], 1);
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_free[s], 1);
      for (int g = 0; g < 2; ++g) {
        mbar_init(&bars->s_full[g][s], 1);
        mbar_init(&bars->s_free[g][s], kHalf);
      }
    }
    mbar_init(&bars->drain, 1);
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
  // The items of each run of sequences, then those of all runs up to each.
  const int run = (p.num_seqs + kLists - 1) / kLists;
  if (threadIdx.x < kLists) {
    int sum = 0;
    for (int s = threadIdx.x * run; s < min(p.num_seqs, (static_cast<int>(threadIdx.x) + 1) * run); ++s)
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
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  Walk walk(p, upto, run);
  const Item& it = walk.it;

  int k_loads = 0, q_loads = 0;  // producer, issuer: tiles begun so far
  int mma_started = 0;
  if (warp == kWarpLoad) {
    // --------------------------------------------------------------- producer
    bool ok = true;
    int held_seq = -1, held_head = -1;  // whose tiles of query rows are in shared memory
    while (ok && walk.next()) {
      const int32_t* table = p.block_tables + static_cast<size_t>(it.seq) * p.max_blocks;
      const int tokens = min(kTokens, it.s.L - it.t0);
      // lane l < 16: the block of tokens t0 + 16 l on (with 8-token blocks also of the 8 after)
      int y = 0, y_hi = 0;
      auto y_of = [&](int t) {
        const int b = t / p.block_size;
        int blk = __ldg(table + b);
        if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
          if (it.head == 0 && (t == b * p.block_size)) report_error(p.err, PA_ERR_BAD_BLOCK, it.seq, blk);
          blk = 0;
        }
        return (blk * p.num_kv_heads + it.head) * p.block_size + (t - b * p.block_size);
      };
      const bool mine = lane * 16 < tokens, mine_hi = half_blocks && lane * 16 + 8 < tokens;
      if (lane < 16) {
        if (mine) y = y_of(it.t0 + lane * 16);
        if (mine_hi) y_hi = y_of(it.t0 + lane * 16 + 8);
      }
      const int ks = k_loads % KS;
      int good = 1;
      if (lane == 0) {
        if (k_loads >= KS) good = mbar_wait_bounded(&bars->k_free[ks], (k_loads / KS - 1) & 1);
        const int unit = half_blocks ? 8 : 16;
        const int rows = (tokens + unit - 1) / unit * unit;
        if (good) mbar_arrive_expect_tx(&bars->k_full[ks], static_cast<uint32_t>(rows) * D * 2);
      }
      ok = __shfl_sync(kFullMask, good, 0);
      if (!ok) break;
      if (lane < 16) {
        uint8_t* dst = smem + ks * C::kKBytes + lane * 2048;
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
          if (mine) tma_load_2d(dst + g * (kTokens * 128), &tm_k, 64 * g, y, &bars->k_full[ks]);
          if (mine_hi) tma_load_2d(dst + g * (kTokens * 128) + 1024, &tm_k, 64 * g, y_hi, &bars->k_full[ks]);
        }
      }
      ++k_loads;
      if (!p.resident || it.seq != held_seq || it.head != held_head) {
        held_seq = it.seq;
        held_head = it.head;
        for (int j = p.resident ? 0 : it.first; ok && j < it.tiles; ++j) {
          const int qs = q_loads % QS;
          if (lane == 0) {
            if (q_loads >= QS) good = mbar_wait_bounded(&bars->q_free[qs], (q_loads / QS - 1) & 1);
            if (good) {
              mbar_arrive_expect_tx(&bars->q_full[qs], C::kGroups * 128u * p.tile_tokens * p.group);
#pragma unroll
              for (int g = 0; g < C::kGroups; ++g)
                tma_load_3d(smem + C::kOffQ + qs * C::kQBytes + g * (kRows * 128), &tm_q, 64 * g,
                            it.head * p.group, it.s.row0 + j * p.tile_tokens, &bars->q_full[qs]);
            }
          }
          ok = __shfl_sync(kFullMask, good, 0);
          if (ok) ++q_loads;
          if (__shfl_sync(kFullMask, *abort_flag, 0)) ok = false;
        }
      }
      if (__shfl_sync(kFullMask, *abort_flag, 0)) ok = false;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report_error(p.err, PA_ERR_TIMEOUT, it.seq, -1);
    }
  } else if (warp == kWarpMma) {
    // ----------------------------------------------------------------- issuer
    constexpr uint32_t idesc = make_idesc(kHalf, kRows, BF16, false);
    const uint64_t k_desc = smem_desc_sw128(smem, 16, 1024);
    const uint64_t q_desc = smem_desc_sw128(smem + C::kOffQ, 16, 1024);
    bool ok = true;
    int held_seq = -1, held_head = -1, held = 0;  // resident tiles: q loads before theirs
    int steps = 0;
    bool more = walk.next();
    while (ok && more) {
      const Item now = it;
      const bool fresh = !p.resident || now.seq != held_seq || now.head != held_head;
      if (fresh) {
        held_seq = now.seq;
        held_head = now.head;
        held = q_loads;
        q_loads += p.resident ? now.tiles : now.tiles - now.first;
      }
      more = walk.next();
      const bool last_use = !p.resident || !more || it.seq != now.seq || it.head != now.head;
      if (lane == 0) {
        const int ks = k_loads % KS;
        ok = mbar_wait_bounded(&bars->k_full[ks], (k_loads / KS) & 1);
        // (every load is waited for, its tile used or not, before its stage is handed back)
        for (int q = held; ok && fresh && p.resident && q < held + now.first; ++q)
          ok = mbar_wait_bounded(&bars->q_full[q % QS], (q / QS) & 1);
        for (int j = now.first; ok && j < now.tiles; ++j, ++steps) {
          const int q = held + (p.resident ? j : j - now.first), qs = q % QS, b = steps & 1;
          ok = mbar_wait_bounded(&bars->q_full[qs], (q / QS) & 1);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (ok && steps >= 2) ok = mbar_wait_bounded(&bars->s_free[g][b], ((steps >> 1) - 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t a = k_desc + static_cast<uint64_t>(
                  (ks * C::kKBytes + (kk >> 2) * (kTokens * 128) + g * (kHalf * 128) + (kk & 3) * 32) >> 4);
              const uint64_t bd = q_desc + static_cast<uint64_t>(
                  (qs * C::kQBytes + (kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4);
              mma_f16(tmem + (g * 2 + b) * kRows, a, bd, idesc, kk > 0);
            }
            mma_commit(&bars->s_full[g][b]);
            mma_started = 1;
          }
          if (ok && !p.resident) mma_commit(&bars->q_free[qs]);
        }
        if (ok) mma_commit(&bars->k_free[ks]);
        if (ok && p.resident && last_use)
          for (int j = 0; j < now.tiles; ++j) mma_commit(&bars->q_free[(held + j) % QS]);
      }
      ++k_loads;
      ok = __shfl_sync(kFullMask, ok, 0);
      steps = __shfl_sync(kFullMask, steps, 0);
      mma_started = __shfl_sync(kFullMask, mma_started, 0);
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report_error(p.err, PA_ERR_TIMEOUT, -1, -1);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int wg = warp >> 2, r = threadIdx.x & (kHalf - 1);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float* lse_wg = lse_s + wg * 2 * kRows;
    int steps = 0, held_seq = -1, held_head = -1, lse_loads = 0;
    const float* lse = lse_wg;
    bool ok = true;
    while (ok && walk.next()) {
      const int t = it.t0 + wg * kHalf + r;
      const size_t sh = static_cast<size_t>(it.seq) * p.num_kv_heads + it.head;
      float* to = p.weights + sh * p.weights_row + t;
      const float before = t < it.s.L ? *to : 0.f;
      float total = 0.f;
      for (int j = it.first; j < it.tiles; ++j, ++steps) {
        const int b = steps & 1;
        const int here = min(p.tile_tokens, it.s.W - j * p.tile_tokens), cols = here * p.group;
        // a key head's only tile: its rows' lse stay where they are
        if (!p.resident || it.tiles > 1 || it.seq != held_seq || it.head != held_head) {
          held_seq = it.seq;
          held_head = it.head;
          float v = 0.f;
          if (r < cols) {
            const int tok = r * p.inv_group >> 16;
            v = -kLog2e * p.lse[static_cast<size_t>(it.s.row0 + j * p.tile_tokens + tok) * p.num_heads +
                                it.head * p.group + (r - tok * p.group)];
          }
          // two buffers in turn: whoever is past the barrier of one load has done with the load before
          float* to = lse_wg + (lse_loads++ & 1) * kRows;
          to[r] = v;
          asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
          lse = to;
        }
        ok = __all_sync(kFullMask, mbar_wait_bounded(&bars->s_full[wg][b], (steps >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
        // the first row's place in the sequence: rows before it see less
        const int pos = it.s.L - it.s.W + j * p.tile_tokens;
        const bool seen = it.t0 + wg * kHalf + kHalf - 1 <= pos;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 32) {
          float s[32];
          tmem_ld32(tmem + lanes + (wg * 2 + b) * kRows + c0, s);
          const float4* nl = reinterpret_cast<const float4*>(lse + c0);
          if (seen && c0 + 32 <= cols) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 v = nl[c / 4];
              const float e0 = ex2_approx(fmaf(s[c], p.qscale, v.x));
              const float e1 = ex2_approx(fmaf(s[c + 1], p.qscale, v.y));
              const float e2 = ex2_approx(fmaf(s[c + 2], p.qscale, v.z));
              const float e3 = ex2_approx(fmaf(s[c + 3], p.qscale, v.w));
              add2(sum[0], sum[1], e0, e1);
              add2(sum[2], sum[3], e2, e3);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float e = ex2_approx(fmaf(s[c], p.qscale, lse[c0 + c]));
              const bool counts = c0 + c < cols && t <= pos + ((c0 + c) * p.inv_group >> 16);
              sum[c & 3] += counts ? e : 0.f;
            }
          }
        }
        total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tc_fence_before();
        mbar_arrive(&bars->s_free[wg][b]);
        if (__shfl_sync(kFullMask, *abort_flag, 0)) {
          ok = false;
          break;
        }
      }
      if (ok && t < it.s.L) *to = before + total;
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
    if (warp == kWarpMma && lane == 0 && mma_started) {
      mma_commit(&bars->drain);
      mbar_wait_bounded(&bars->drain, 0);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kWarpMma) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

template <bool BF16, int D>
int launch(ChunkWeightsParams p, const void* q, const void* k_cache, unsigned long long cache_rows,
           cudaStream_t stream) {
  using C = Cfg<D>;
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return PA_ERR_CUDA;
  const int most = p.window > 0 && p.window < p.max_query_len ? p.window : p.max_query_len;
  p.resident = most <= C::kQStages * p.tile_tokens;
  CUtensorMap tq, tk;
  const cuuint64_t qdims[3] = {D, static_cast<cuuint64_t>(p.num_heads),
                               static_cast<cuuint64_t>(p.total_queries)};
  const cuuint64_t qstr[2] = {D * 2, static_cast<cuuint64_t>(D) * 2 * p.num_heads};
  const cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.tile_tokens)};
  const cuuint64_t cdims[2] = {D, cache_rows};
  const cuuint64_t cstr[1] = {D * 2};
  const cuuint32_t cbox[2] = {64, p.block_size >= 16 ? 16u : 8u};
  if (!encode_tensor_map(&tq, BF16, q, 3, qdims, qstr, qbox) ||
      !encode_tensor_map(&tk, BF16, k_cache, 2, cdims, cstr, cbox))
    return PA_ERR_CUDA;
  if (cudaFuncSetAttribute(chunk_weights_kernel<BF16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::kSmemBytes) != cudaSuccess)
    return PA_ERR_CUDA;
  const long long tiles = (static_cast<long long>(p.max_blocks) * p.block_size + kTokens - 1) / kTokens;
  const long long items = p.num_seqs * tiles * p.num_kv_heads;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(items < sms ? items : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, chunk_weights_kernel<BF16, D>, tq, tk, p) != cudaSuccess ||
      cudaGetLastError() != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
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
  p.max_query_len = max_query_len;
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
