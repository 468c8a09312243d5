// Channel-wise smallest and largest key of cached blocks, computed anew.
//
// A thread takes 8 channels (16 bytes) of one (sequence, block, key head) and walks the
// block's rows below the sequence's length, kBatch loads in flight at a time; past the last
// row it reads that row again, which changes no minimum.  Every key byte is read once from
// memory and two rows per block are written: the kernel is bound by HBM (32 sequences of up to
// 16384 tokens, 8 heads of 128, 639 MB: 95 us, 6.7 TB/s).
#include <cuda_runtime.h>

#include "common.cuh"
#include "rope.cuh"

namespace pagedkv {
namespace {

constexpr int kThreads = 256;

struct BoundsParams {
  const void* k_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* first_token;  // null: 0
  void* k_min;
  void* k_max;
  int32_t* err;
  int num_kv_heads, head_dim, block_size, max_blocks, num_blocks;
};

// A load that stays where it is written: left to itself the compiler moves the loads of a batch
// towards their uses, to save registers (the same case: 108 us, with the loads held 95 us).
__device__ __forceinline__ uint4 load(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <class Tag, int kBatch>
__global__ void __launch_bounds__(kThreads) kv_block_bounds_kernel(const BoundsParams p) {
  const int seq = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int L = p.seq_lens[seq];
  if (L < 0 || L > static_cast<long long>(p.max_blocks) * p.block_size) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_error(p.err, PA_ERR_BAD_SEQ_LEN, seq, L);
    return;
  }
  const int first = p.first_token ? max(p.first_token[seq], 0) : 0;
  const int pieces = p.head_dim / 8;                 // 16-byte pieces of a row
  const int per_block = p.num_kv_heads * pieces;     // threads of a block
  const int b0 = first / p.block_size;
  const int nb = (L + p.block_size - 1) / p.block_size;
  const long long total = static_cast<long long>(nb - b0) * per_block;
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += stride) {
    const int b = b0 + static_cast<int>(i / per_block);
    const int rem = static_cast<int>(i % per_block);
    const int head = rem / pieces, x = rem % pieces;
    const int blk = p.block_tables[static_cast<size_t>(seq) * p.max_blocks + b];
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
      if (rem == 0) report_error(p.err, PA_ERR_BAD_BLOCK, seq, blk);
      continue;
    }
    const int rows = min(p.block_size, L - b * p.block_size);
    const size_t bh = static_cast<size_t>(blk) * p.num_kv_heads + head;
    const uint4* src = static_cast<const uint4*>(p.k_cache) + bh * p.block_size * pieces + x;
    uint4 lo, hi;
    for (int r0 = 0; r0 < rows; r0 += kBatch) {
      uint4 u[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) u[j] = load(src + static_cast<size_t>(min(r0 + j, rows - 1)) * pieces);
      if (r0 == 0) lo = hi = u[0];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        lo = min8(lo, u[j], Tag{});
        hi = max8(hi, u[j], Tag{});
      }
    }
    static_cast<uint4*>(p.k_min)[bh * pieces + x] = lo;
    static_cast<uint4*>(p.k_max)[bh * pieces + x] = hi;
  }
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int kv_block_bounds(const void* k_cache, const int32_t* block_tables,
                               const int32_t* seq_lens, const int32_t* first_token, int num_seqs,
                               int num_kv_heads, int head_dim, int block_size,
                               int max_blocks_per_seq, int num_blocks, int dtype, void* k_min,
                               void* k_max, int32_t* error_record, void* stream) {
  NvtxRange range("kv_block_bounds");
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (head_dim % 8 != 0) return PA_ERR_UNSUPPORTED;
  const long long cap = static_cast<long long>(max_blocks_per_seq) * block_size;
  if (cap > (1ll << 30) || num_seqs > 65535 ||
      static_cast<long long>(num_kv_heads) * head_dim > (1 << 30))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!k_cache || !block_tables || !seq_lens || !k_min || !k_max) return PA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(k_min) || !aligned16(k_max)) return PA_ERR_INVALID_ARG;
  const BoundsParams p{k_cache, block_tables, seq_lens, first_token, k_min, k_max, error_record,
                       num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks};
  const long long work = static_cast<long long>(max_blocks_per_seq) * num_kv_heads * (head_dim / 8);
  const long long most = (152ll * 64 + num_seqs - 1) / num_seqs;
  const long long want = (work + kThreads - 1) / kThreads;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most), num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // as many loads in flight as a block has rows, up to 16 (32 sequences of up to 16384 tokens,
  // blocks of 16 rows: 95 us with 16, 106 us with 8)
  cudaError_t e;
  if (block_size <= 8)
    e = dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, kv_block_bounds_kernel<BF16, 8>, p)
                         : cudaLaunchKernelEx(&cfg, kv_block_bounds_kernel<F16, 8>, p);
  else
    e = dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, kv_block_bounds_kernel<BF16, 16>, p)
                         : cudaLaunchKernelEx(&cfg, kv_block_bounds_kernel<F16, 16>, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
