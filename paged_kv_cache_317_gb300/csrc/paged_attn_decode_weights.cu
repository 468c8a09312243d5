// Decode attention that keeps up what weight each cached token has had.
//
// A row is one (sequence, key head) and up to 8 NT of the query heads that share it.  Each warp runs a
// pipeline of its own over chunks of 16 tokens (see warp_attn.cuh): its lanes look up the blocks of 32
// chunks at once, one lane starts a chunk's K and V copies (TMA boxes of 16 rows) into the warp's ring
// of stages.  K and V are read once for all the heads.  A token's weight, sum over the heads of
// 2^(s - M) / l, can only be formed once M and l of the whole row are known, so the logits are kept
// until then:
//  * rows that fit, in shared memory: a thread block takes a row, joins its warps' sums, writes the
//    output and adds to the weights;
//  * else in the workspace: a row's chunks are shared out over `parts` thread blocks, whose sums and
//    logits a second kernel joins.
// Bound by HBM for batches: 64 x 40 rows of up to 2048 tokens of 128 channels, logits in shared memory: 206 us,
// 6.6 TB/s (97 % of a copy's rate).  64 x 8 rows of up to 16384 tokens, 8 heads each: 397 us, 5.8 TB/s of K, V and
// weights, 6.6 with the logits' way out (0.15 GB) and back, which is the price of reading K once.  One sequence
// of 30,000 tokens: 27 us for 125 MB, the ramp and the second kernel (4.6 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "tma.cuh"
#include "warp_attn.cuh"

namespace pagedkv {
namespace {

constexpr int kChunk = 16;      // tokens per stage
constexpr int kWarps = 4;       // warps per thread block
// 256 channels: one stage of 16 KB a warp lets three thread blocks onto an SM, two stages one (16 x 8 rows of
// up to 8000 tokens: 122 us, 168); 128 channels: two (64 x 40 rows of up to 2048: 206 us, with three 219).
template <int D>
constexpr int kStagesOf = D == 256 ? 1 : 2;
constexpr int kAlign = 1024;    // a swizzled box must start on 1024 bytes
constexpr int kHeader = 256;    // barriers
constexpr int kMaxParts = 64;   // thread blocks per row: 8 for each warp of the join
constexpr int kFew = 304;       // thread blocks of a few rows, and of more of them, which may be of unequal
constexpr int kShares = 4096;   // length (52 x 3 rows of up to 21,000 tokens, 16 heads: 200 us; over 304: 491)
constexpr int kFewRows = 19;
constexpr int kJoinThreads = 256;
constexpr int kJoinTokens = 2048;  // tokens of a join's thread block
constexpr int kJoinCols = 64;      // columns whose maxima and sums it holds at a time
constexpr float kLog2e = 1.4426950408889634f;

struct DecodeWeightsParams {
  const void* q;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  void* out;
  float* weights;
  int32_t* err;
  long long weights_row;  // floats from (sequence, key head) to the next
  int num_heads, num_kv_heads, block_size, max_blocks, num_blocks;
  int group, tiles;       // query heads per key head; tiles of 8 NT of them
  int cols;               // columns of the logits of a row
  int parts;              // thread blocks per row
  int pitch;              // floats from a column of the logits to the next
  float* logits;          // [row][cols][pitch], or NULL: in shared memory
  float* part_o;          // [row][part][8 NT][D]
  float2* part_ml;        // [row][part][8 NT]
  int out_dtype;
  float qscale;           // scale * log2(e)
};

__device__ __forceinline__ int length_of(const DecodeWeightsParams& p, int seq, bool report) {
  int L = p.seq_lens[seq];
  const int cap = p.max_blocks * p.block_size;
  if (L < 0 || L > cap) {
    if (report) report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    L = min(max(L, 0), cap);
  }
  return L;
}

// The rings, or the joined sums, which take their place.
template <int D, int NT>
constexpr size_t ring_bytes() {
  const size_t ring = static_cast<size_t>(kWarps) * kStagesOf<D> * 2 * kChunk * D * 2;
  const size_t join = static_cast<size_t>(kWarps) * 8 * NT * (D + 4) * sizeof(float) +
                      (kWarps + 1) * 8 * NT * sizeof(float2);
  return ring > join ? ring : join;
}

template <class Tag, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32)
    decode_weights_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const DecodeWeightsParams p) {
  using Attn = WarpAttn<Tag, D, NT>;
  constexpr int kCols = 8 * NT, kPitch = D + 4, kTile = Attn::kTileBytes, kStages = kStagesOf<D>;
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
  }
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
  const int tile = row % p.tiles, sh = row / p.tiles;
  const int seq = sh / p.num_kv_heads, head = sh - seq * p.num_kv_heads;
  const int cols = min(kCols, p.group - tile * kCols);
  const size_t q0 = static_cast<size_t>(seq) * p.num_heads + head * p.group + tile * kCols;

  uint64_t* full = reinterpret_cast<uint64_t*>(smem) + warp * kStages;
  const uint32_t base = smem_addr(smem);
  uint8_t* ring0 = smem + (((base + kHeader + kAlign - 1) & ~uint32_t(kAlign - 1)) - base);
  uint8_t* ring = ring0 + warp * kStages * 2 * kTile;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int L = length_of(p, seq, threadIdx.x == 0 && part == 0 && head == 0 && tile == 0);
  const int chunks = (L + kChunk - 1) / kChunk;
  const int begin = static_cast<int>(static_cast<long long>(chunks) * part / p.parts);
  const int end = static_cast<int>(static_cast<long long>(chunks) * (part + 1) / p.parts);
  const int mine = (end - begin - warp + kWarps - 1) / kWarps;  // chunks begin + warp, + kWarps, ...
  const bool small = p.block_size == 8;
  const int32_t* table = p.block_tables + static_cast<size_t>(seq) * p.max_blocks;

  // The blocks of the warp's next 32 chunks as rows of the cache seen as rows of D.
  int y_lo = 0, y_hi = 0;
  auto look_up = [&](int i) {
    const int t0 = (begin + warp + (i + lane) * kWarps) * kChunk;
    auto y_of = [&](int t) -> int {
      if (i + lane >= mine || t >= L) return 0;
      const int b = t / p.block_size;
      int blk = table[b];
      if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
        if (t == b * p.block_size && head == 0 && tile == 0) report_error(p.err, PA_ERR_BAD_BLOCK, seq, blk);
        blk = 0;
      }
      return (blk * p.num_kv_heads + head) * p.block_size + (t - b * p.block_size);
    };
    y_lo = y_of(t0);
    if (small) y_hi = y_of(t0 + 8);
  };
  auto rows_of = [&](int i) { return min(kChunk, L - (begin + warp + i * kWarps) * kChunk); };
  auto issue = [&](int i) {
    if ((i & 31) == 0) look_up(i);
    const int lo = __shfl_sync(kFullMask, y_lo, i & 31), hi = __shfl_sync(kFullMask, y_hi, i & 31);
    if (lane == 0) {
      const int s = i % kStages;
      uint8_t* dst = ring + s * 2 * kTile;
      const bool two = small && rows_of(i) > 8;
      const uint32_t bytes = small ? kTile / 2 : kTile;
      mbar_arrive_expect_tx(&full[s], 2 * bytes * (two ? 2 : 1));
      tma_load_3d(dst, &tm_k, 0, lo, 0, &full[s]);
      tma_load_3d(dst + kTile, &tm_v, 0, lo, 0, &full[s]);
      if (two) {
        tma_load_3d(dst + bytes, &tm_k, 0, hi, 0, &full[s]);
        tma_load_3d(dst + kTile + bytes, &tm_v, 0, hi, 0, &full[s]);
      }
    }
  };
  int issued = 0;
  while (issued < kStages && issued < mine) issue(issued++);

  Attn at;
  at.init(static_cast<const typename Tag::T*>(p.q) + q0 * D, cols, small, lane);
  const uint32_t ring_addr = smem_addr(ring);
  float* logits = p.logits != nullptr
                      ? p.logits + static_cast<size_t>(row) * p.cols * p.pitch
                      : reinterpret_cast<float*>(ring0 + ring_bytes<D, NT>());
  bool aborted = false;
  int done = 0;
  for (; done < mine; ++done) {
    const int s = done % kStages;
    if (!__all_sync(kFullMask, mbar_wait_bounded(&full[s], (done / kStages) & 1))) {
      if (lane == 0) report_error(p.err, PA_ERR_TIMEOUT, seq, done);
      aborted = true;
      break;
    }
    const int rows = rows_of(done), rlo = min(rows, 8), rhi = rows - rlo;
    const int t0 = (begin + warp + done * kWarps) * kChunk;
    at.step(ring_addr + s * 2 * kTile, ring_addr + s * 2 * kTile + kTile, rlo, rhi, p.qscale, lane,
            [&](int t, const float (&sc)[4]) {
      const int g = lane >> 2, col = t * 8 + 2 * (lane & 3);
      float* to = logits + static_cast<size_t>(col) * p.pitch + t0 + g;
      if (col < cols) {
        to[0] = sc[0];
        to[8] = sc[2];
      }
      if (col + 1 < cols) {
        to[p.pitch] = sc[1];
        to[p.pitch + 8] = sc[3];
      }
    });
    __syncwarp();  // the stage is read
    if (issued < mine) issue(issued++);
  }
  if (aborted) {  // no copy may land in shared memory after the block has exited
    for (int i = done; i < issued; ++i) mbar_wait_bounded(&full[i % kStages], (i / kStages) & 1);
  }

  // the warps' sums, over the ring: O as [warp][column][kPitch], then (m, l) as [warp][column]
  __syncthreads();
  float* jo = reinterpret_cast<float*>(ring0);
  float2* jml = reinterpret_cast<float2*>(jo + kWarps * kCols * kPitch);
  float2* stat = jml + kWarps * kCols;  // M and the factor of 2^(s - M), by column
  at.put(jo + warp * kCols * kPitch, kPitch, jml + warp * kCols, done > 0, lane);
  __syncthreads();
  for (int i = threadIdx.x; i < cols * (D / 4); i += kWarps * 32) {
    const int col = i / (D / 4), d = i % (D / 4) * 4;
    float M = -INFINITY, sum = 0.f;
    bool tokens = false;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = max_nan(M, jml[w * kCols + col].x);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = jml[w * kCols + col];
      tokens |= ml.y < 0.f || ml.x != -INFINITY;
      if (ml.x != -INFINITY) {
        const float f = exp2f(ml.x - M);
        const float4 v = *reinterpret_cast<const float4*>(jo + (w * kCols + col) * kPitch + d);
        sum = fmaf(f, ml.y, sum);
        acc[0] = fmaf(f, v.x, acc[0]);
        acc[1] = fmaf(f, v.y, acc[1]);
        acc[2] = fmaf(f, v.z, acc[2]);
        acc[3] = fmaf(f, v.w, acc[3]);
      }
    }
    if (p.logits != nullptr) {
      const size_t to = static_cast<size_t>(blockIdx.x) * kCols + col;
      *reinterpret_cast<float4*>(p.part_o + to * D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (d == 0) p.part_ml[to] = make_float2(M, M == -INFINITY && tokens ? -1.f : sum);
    } else {
      const float inv = inverse_of(M, sum, tokens);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= inv;
      store_out<4>(p.out, (q0 + col) * D + d, acc, p.out_dtype);
      if (d == 0) stat[col] = make_float2(M, inv * exp2f(Attn::kLift));
    }
  }
  if (p.logits != nullptr) return;
  __syncthreads();
  float* weights = p.weights + sh * p.weights_row;
  for (int t = threadIdx.x; t < L; t += kWarps * 32) {
    float sum = 0.f;
    for (int c = 0; c < cols; ++c) sum = fmaf(exp2f(logits[c * p.pitch + t] - stat[c].x), stat[c].y, sum);
    weights[t] += sum;
  }
}

// Joins the parts of the rows of a (sequence, key head): blocks of kJoinTokens tokens, which also share
// out the output's heads.  The last rows first: theirs are the logits most likely to be in L2 yet.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads, 4)
    decode_weights_join_kernel(const DecodeWeightsParams p, const int shares, const float lift) {
  constexpr int kCols = 8 * NT, kPer = kJoinTokens / kJoinThreads, kWarpsJoin = kJoinThreads / 32;
  constexpr int kVec = D / 32, kAhead = D == 256 ? 4 : 8;  // parts that a warp loads at a time
  __shared__ float2 stat[kJoinCols];
  __shared__ __align__(16) float slice[kWarpsJoin][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = static_cast<int>(gridDim.x - 1 - blockIdx.x);
  const int sh = block / shares, share = block - sh * shares;
  const int seq = sh / p.num_kv_heads, head = sh - seq * p.num_kv_heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int L = length_of(p, seq, false);
  const int t0 = share * kJoinTokens + static_cast<int>(threadIdx.x);
  if (share * kJoinTokens >= L && share >= p.group) return;  // neither tokens nor heads
  // (m, l) of column `col`'s parts, lane i's i and i + 32, and M and 1 / l of the whole
  struct Column {
    float w[2];  // 2^(m - M) of the lane's parts
    unsigned seen[2];  // the parts that have a weight: a NaN in them counts, however small it is
    float M, inv;
  };
  auto column = [&](int col, size_t at) -> Column {
    float2 ml[2];
    Column c;
    c.M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      ml[k] = i < p.parts ? p.part_ml[at + static_cast<size_t>(i) * kCols] : make_float2(-INFINITY, 0.f);
      c.M = max_nan(c.M, ml[k].x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) c.M = max_nan(c.M, __shfl_xor_sync(kFullMask, c.M, off));
    float l = 0.f;
    bool tokens = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      tokens |= ml[k].y < 0.f || ml[k].x != -INFINITY;
      c.seen[k] = __ballot_sync(kFullMask, ml[k].x != -INFINITY);
      c.w[k] = ml[k].x != -INFINITY ? exp2f(ml[k].x - c.M) : 0.f;
      if (ml[k].x != -INFINITY) l = fmaf(c.w[k], ml[k].y, l);
    }
    tokens = __any_sync(kFullMask, tokens);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(kFullMask, l, off);
    c.inv = inverse_of(c.M, l, tokens);
    return c;
  };
  auto first_part = [&](int col) -> size_t {
    const size_t row = static_cast<size_t>(sh) * p.tiles + col / kCols;
    return row * p.parts * kCols + col % kCols;
  };
  // ------------------------------------------------------------------ the weights
  float sum[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) sum[k] = 0.f;
  for (int c0 = 0; share * kJoinTokens < L && c0 < p.group; c0 += kJoinCols) {
    const int n = min(kJoinCols, p.group - c0);
    float s[4][kPer];
    auto load = [&](int c) {  // four columns' logits
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = c0 + min(c + i, n - 1);
        const size_t row = static_cast<size_t>(sh) * p.tiles + col / kCols;
        const float* from = p.logits + (row * p.cols + col % kCols) * p.pitch + t0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) s[i][k] = t0 + k * kJoinThreads < L ? __ldcs(from + k * kJoinThreads) : 0.f;
      }
    };
    load(0);  // on their way while the maxima and sums are joined
    __syncthreads();
    for (int c = warp; c < n; c += kWarpsJoin) {
      const Column col = column(c0 + c, first_part(c0 + c));
      if (lane == 0) stat[c] = make_float2(col.M, col.inv * lift);
    }
    __syncthreads();
    for (int c = 0; c < n; c += 4) {
      if (c > 0) load(c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c + i < n) {
          const float2 st = stat[c + i];
#pragma unroll
          for (int k = 0; k < kPer; ++k) sum[k] = fmaf(exp2f(s[i][k] - st.x), st.y, sum[k]);
        }
      }
    }
  }
  // One thread adds to a weight, once: a reduction in L2 gives the same bits as a load, an add and a store,
  // but for numbers below 2^-126, which it may take for 0.
  float* weights = p.weights + sh * p.weights_row + t0;
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (t0 + k * kJoinThreads < L) atomicAdd(weights + k * kJoinThreads, sum[k]);
  // ------------------------------------------------------------------- the output
  // A head's parts are shared out over the warps, whose sums meet in shared memory.
  for (int col = share; col < p.group; col += shares) {
    const size_t at = first_part(col);
    const Column c = column(col, at);
    float acc[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
    const float* o = p.part_o + at * D + lane * kVec;
#pragma unroll 1
    for (int k0 = 0; k0 < kMaxParts / kWarpsJoin && k0 * kWarpsJoin < p.parts; k0 += kAhead) {
      float v[kAhead][kVec];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = warp + (k0 + k) * kWarpsJoin;
        if (i < p.parts) {
          const float* from = o + static_cast<size_t>(i) * kCols * D;
#pragma unroll
          for (int e = 0; e < kVec; e += 2)
            *reinterpret_cast<float2*>(&v[k][e]) = *reinterpret_cast<const float2*>(from + e);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = warp + (k0 + k) * kWarpsJoin;
        const float f = __shfl_sync(kFullMask, i < 32 ? c.w[0] : c.w[1], i & 31);
        if ((i < 32 ? c.seen[0] : c.seen[1]) >> (i & 31) & 1) {  // (i < p.parts; one without tokens has no sums)
#pragma unroll
          for (int e = 0; e < kVec; ++e) acc[e] = fmaf(f, v[k][e], acc[e]);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kVec; ++e) slice[warp][lane * kVec + e] = acc[e];
    __syncthreads();
    const size_t to = (static_cast<size_t>(seq) * p.num_heads + head * p.group + col) * D;
    for (int d = threadIdx.x * 2; d < D; d += kJoinThreads * 2) {
      float out[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarpsJoin; ++w) {
        out[0] += slice[w][d];
        out[1] += slice[w][d + 1];
      }
      out[0] *= c.inv;
      out[1] *= c.inv;
      store_out<2>(p.out, to + d, out, p.out_dtype);
    }
  }
}

struct Shape {
  bool inside;       // logits in shared memory
  int parts, pitch;
  size_t smem;
};

template <int D, int NT>
Shape shape_for(long long rows, int tiles, int group, long long cap) {
  const int cols = group < 8 * NT ? group : 8 * NT;
  const int padded = static_cast<int>((cap + kChunk - 1) / kChunk * kChunk);
  Shape s{};
  const size_t bare = kHeader + kAlign + ring_bytes<D, NT>();
  // + 4: the columns of a warp's stores in different banks
  const size_t held = static_cast<size_t>(cols) * (padded + 4) * sizeof(float);
  // Only where there are many rows, or short ones: 32 x 8 rows of up to 4000 tokens of 64 channels take 75 us
  // so, 47 us in parts, 128 x 8 of up to 1000 of 128 channels 66 and 75.
  if (tiles == 1 && bare + held <= 113 * 1024 && (rows >= 1024 || cap <= 1024)) {
    s.inside = true;
    s.parts = 1;
    s.pitch = padded + 4;
    s.smem = bare + held;
    return s;
  }
  s.pitch = padded;
  s.smem = bare;
  const long long most = (cap + 255) / 256;
  long long parts = (rows <= kFewRows ? kFew : kShares) / rows;
  if (parts > most) parts = most;
  if (parts > kMaxParts) parts = kMaxParts;
  s.parts = static_cast<int>(parts < 1 ? 1 : parts);
  return s;
}

// Never falls as sequences or tables grow, the others alike.
template <int D, int NT>
size_t partials(long long rows) {
  const long long some = rows * kMaxParts < kShares ? rows * kMaxParts : kShares;
  return static_cast<size_t>(some > rows ? some : rows) * 8 * NT;
}

template <int D, int NT>
size_t workspace_for(long long sequences, int num_kv_heads, int group, long long cap) {
  const int tiles = (group + 8 * NT - 1) / (8 * NT), cols = group < 8 * NT ? group : 8 * NT;
  const long long rows = sequences * num_kv_heads * tiles, padded = (cap + kChunk - 1) / kChunk * kChunk;
  return partials<D, NT>(rows) * (D * sizeof(float) + sizeof(float2)) +
         static_cast<size_t>(rows) * cols * padded * sizeof(float);
}

template <class... Kernel, class... Args>
bool launch_dependent(void (*kernel)(Kernel...), unsigned grid, unsigned block, size_t smem,
                      cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess && cudaGetLastError() == cudaSuccess;
}

template <class Tag, int D, int NT>
int launch(DecodeWeightsParams p, const void* k_cache, const void* v_cache, int num_seqs, void* workspace,
           size_t workspace_bytes, cudaStream_t stream) {
  p.tiles = (p.group + 8 * NT - 1) / (8 * NT);
  p.cols = p.group < 8 * NT ? p.group : 8 * NT;
  const long long cap = static_cast<long long>(p.max_blocks) * p.block_size;
  const long long rows = static_cast<long long>(num_seqs) * p.num_kv_heads * p.tiles;
  const Shape shape = shape_for<D, NT>(rows, p.tiles, p.group, cap);
  const long long shares = (cap + kJoinTokens - 1) / kJoinTokens;
  if (rows * shape.parts > 0x7fffffffll || rows / p.tiles * shares > 0x7fffffffll) return PA_ERR_INVALID_ARG;
  p.parts = shape.parts;
  p.pitch = shape.pitch;
  if (!shape.inside) {
    if (!workspace || workspace_bytes < workspace_for<D, NT>(num_seqs, p.num_kv_heads, p.group, cap))
      return PA_ERR_INVALID_ARG;
    const size_t n = partials<D, NT>(rows);
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + n * D);
    p.logits = reinterpret_cast<float*>(p.part_ml + n);
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
  if (cudaFuncSetAttribute(decode_weights_kernel<Tag, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           227 * 1024) != cudaSuccess)
    return PA_ERR_CUDA;
  if (!launch_dependent(decode_weights_kernel<Tag, D, NT>, static_cast<unsigned>(rows * p.parts), kWarps * 32,
                        shape.smem, stream, tk, tv, p))
    return PA_ERR_CUDA;
  if (!shape.inside &&
      !launch_dependent(decode_weights_join_kernel<D, NT>, static_cast<unsigned>(rows / p.tiles * shares),
                        kJoinThreads, 0, stream, p, static_cast<int>(shares),
                        std::exp2(WarpAttn<Tag, D, NT>::kLift)))
    return PA_ERR_CUDA;
  return PA_OK;
}

// f(D, NT) for the sizes of a call; 0 where there is no such call.
template <class F>
size_t for_sizes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                 int max_blocks_per_seq, F f) {
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      block_size <= 0 || max_blocks_per_seq <= 0)
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

extern "C" size_t paged_attn_decode_weights_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                                           int head_dim, int block_size,
                                                           int max_blocks_per_seq) {
  return for_sizes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                   [&](auto dim, auto nt) {
    constexpr int D = decltype(dim)::value, NT = decltype(nt)::value;
    return workspace_for<D, NT>(num_seqs, num_kv_heads, num_heads / num_kv_heads,
                                static_cast<long long>(max_blocks_per_seq) * block_size);
  });
}

extern "C" size_t paged_attn_decode_weights_workspace_needed(int num_seqs, int num_heads, int num_kv_heads,
                                                             int head_dim, int block_size,
                                                             int max_blocks_per_seq) {
  return for_sizes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                   [&](auto dim, auto nt) -> size_t {
    constexpr int D = decltype(dim)::value, NT = decltype(nt)::value;
    const int group = num_heads / num_kv_heads, tiles = (group + 8 * NT - 1) / (8 * NT);
    const long long rows = static_cast<long long>(num_seqs) * num_kv_heads * tiles;
    const long long cap = static_cast<long long>(max_blocks_per_seq) * block_size;
    if (shape_for<D, NT>(rows, tiles, group, cap).inside) return 0;
    return workspace_for<D, NT>(num_seqs, num_kv_heads, group, cap);
  });
}

extern "C" int paged_attn_decode_weights(const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                                         int num_heads, int num_kv_heads, int head_dim, int block_size,
                                         int max_blocks_per_seq, int num_blocks, float scale, int dtype,
                                         void* out, int out_dtype, float* weights, int64_t weights_tokens,
                                         void* workspace, size_t workspace_bytes, int32_t* error_record,
                                         void* stream) {
  NvtxRange range("paged_attn_decode_weights");
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (block_size % 16 != 0 && block_size != 8) return PA_ERR_UNSUPPORTED;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (out_dtype != PA_F16 && out_dtype != PA_BF16 && out_dtype != PA_F32) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
  const long long cap = static_cast<long long>(max_blocks_per_seq) * block_size;
  if (cap > (1ll << 30) || num_seqs > 65535 || num_heads > 65535 || weights_tokens < cap)
    return PA_ERR_INVALID_ARG;
  if (static_cast<long long>(num_blocks) * num_kv_heads * block_size >= (1ll << 31))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !out || !weights) return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace))
    return PA_ERR_INVALID_ARG;
  DecodeWeightsParams p{};
  p.q = q;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.out = out;
  p.weights = weights;
  p.weights_row = weights_tokens;
  p.err = error_record;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.group = num_heads / num_kv_heads;
  p.out_dtype = out_dtype;
  p.qscale = scale * kLog2e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto with = [&](auto tag, auto dim) {
    using Tag = decltype(tag);
    constexpr int D = decltype(dim)::value;
    return p.group <= 8 ? launch<Tag, D, 1>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, st)
                        : launch<Tag, D, 2>(p, k_cache, v_cache, num_seqs, workspace, workspace_bytes, st);
  };
  const auto sized = [&](auto tag) {
    switch (head_dim) {
      case 64: return with(tag, std::integral_constant<int, 64>{});
      case 128: return with(tag, std::integral_constant<int, 128>{});
      default: return with(tag, std::integral_constant<int, 256>{});
    }
  };
  return dtype == PA_BF16 ? sized(BF16{}) : sized(F16{});
}
