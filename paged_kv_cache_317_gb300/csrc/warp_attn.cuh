// One warp's attention over chunks of 16 cached tokens, on mma.sync m16n8k16 with the tokens as the
// rows and 8 NT query heads as the columns: S^T = K.Q^T in fp32, the running maximum and sum of each
// column in log2 units, O^T += V^T.P^T with P as a high and a low half-precision number (off by at
// most 2^-17 of a weight in bf16, 2^-23 in fp16; with one number it would be 2^-8, 2^-11).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "mma.cuh"

namespace pagedkv {

// 1 / l of a joined column; NaN where every logit was -infinity, 0 where there was no token.
__device__ __forceinline__ float inverse_of(float M, float l, bool tokens) {
  if (M == -INFINITY) return tokens ? NAN : 0.f;
  return 1.f / l;
}

// A chunk of K or V in shared memory, as TMA leaves it: [D / 64 column groups][16 rows][128 bytes],
// from 8-token blocks two of [D / 64][8][128]; token t's 16-byte piece c of a column group sits at
// c ^ (t & 7).
template <class Tag, int D, int NT>
struct WarpAttn {
  using T = typename Tag::T;
  static constexpr int kTileBytes = 16 * D * 2;
  // Weights are kept as 2^(s - m + kLift), sums and products alike: fp16 has no numbers below 2^-24,
  // and a long row's many small weights would be lost next to one of 1.
  static constexpr float kLift = std::is_same<Tag, F16>::value ? 12.f : 0.f;

  uint32_t qf[NT][D / 16][2];  // Q^T as B fragments: column g of an 8-column tile is query head g of it
  float o[NT][D / 16][4];      // O^T: channels (dd 16 + lane / 4) and 8 on, columns 2 (lane % 4), + 1
  float m[NT][2], l[NT][2];    // of columns 2 (lane % 4), + 1; l over this lane's tokens alone
  uint32_t k_row, v_row, group_bytes;
  int k_half, v_half, r8;

  // `q`: the first query head; those at or past `cols` are left out.
  __device__ __forceinline__ void init(const T* q, int cols, bool small, int lane) {
    const int g = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const bool have = t * 8 + g < cols;
      const T* src = q + static_cast<size_t>(have ? t * 8 + g : 0) * D + 2 * tq;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[t][kk][0] = have ? *reinterpret_cast<const uint32_t*>(src + kk * 16) : 0u;
        qf[t][kk][1] = have ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) : 0u;
      }
#pragma unroll
      for (int dd = 0; dd < D / 16; ++dd) o[t][dd][0] = o[t][dd][1] = o[t][dd][2] = o[t][dd][3] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
    // ldmatrix rows of this lane.  K (A operand): matrices (tokens 0-7, d + 0..7), (8-15, d + 0..7),
    // (0-7, d + 8..15), (8-15, d + 8..15).  V (A operand of V^T, transposed): (tokens 0-7, d + 0..7),
    // (0-7, d + 8..15), (8-15, d + 0..7), (8-15, d + 8..15).
    const int mi = lane >> 3;
    r8 = lane & 7;
    group_bytes = small ? 1024u : 2048u;
    const uint32_t half_bytes = small ? kTileBytes / 2 : 1024u;
    k_row = (mi & 1) * half_bytes + r8 * 128;
    v_row = (mi >> 1) * half_bytes + r8 * 128;
    k_half = mi >> 1;
    v_half = mi & 1;
  }

  // The chunk at shared addresses kt (K) and vt (V), of whose first and second 8 rows rlo and rhi hold
  // tokens.  logits(t, s): the logits in log2 units of tile t, s = (token lane / 4, column
  // 2 (lane % 4)), (the same, + 1), (token + 8, ...), -infinity in rows without a token.
  template <class F>
  __device__ __forceinline__ void step(uint32_t kt, uint32_t vt, int rlo, int rhi, float qscale, int lane,
                                       F logits) {
    const int g = lane >> 2, tq = lane & 3;
    float sc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t a[4];
      const int c = ((kk & 3) << 1) | k_half;
      ldsm_x4(kt + (kk >> 2) * group_bytes + k_row + ((c ^ r8) << 4), a);
#pragma unroll
      for (int t = 0; t < NT; ++t) mma(sc[t], a, qf[t][kk][0], qf[t][kk][1], Tag{});
    }
    const bool partial = rlo + rhi < 16;
    uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[t][e] *= qscale;
      if (partial) {
        if (g >= rlo) sc[t][0] = sc[t][1] = -INFINITY;
        if (g >= rhi) sc[t][2] = sc[t][3] = -INFINITY;
      }
      logits(t, sc[t]);
      float c0 = max_nan(sc[t][0], sc[t][2]), c1 = max_nan(sc[t][1], sc[t][3]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        c0 = max_nan(c0, __shfl_xor_sync(kFullMask, c0, off));
        c1 = max_nan(c1, __shfl_xor_sync(kFullMask, c1, off));
      }
      const float n0 = max_nan(m[t][0], c0), n1 = max_nan(m[t][1], c1);
      // all -infinity so far: any finite base gives them the weight 0
      const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
      const float a0 = exp2f(m[t][0] - b0), a1 = exp2f(m[t][1] - b1);
      const float s0 = kLift - b0, s1 = kLift - b1;
      const float p0 = exp2f(sc[t][0] + s0), p1 = exp2f(sc[t][1] + s1);
      const float p2 = exp2f(sc[t][2] + s0), p3 = exp2f(sc[t][3] + s1);
      l[t][0] = fmaf(l[t][0], a0, p0 + p2);
      l[t][1] = fmaf(l[t][1], a1, p1 + p3);
      if (__any_sync(kFullMask, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
        for (int dd = 0; dd < D / 16; ++dd) {
          o[t][dd][0] *= a0;
          o[t][dd][1] *= a1;
          o[t][dd][2] *= a0;
          o[t][dd][3] *= a1;
        }
      }
      m[t][0] = n0;
      m[t][1] = n1;
      uint32_t hi_a, lo_a, hi_b, lo_b;
      split2(p0, p1, hi_a, lo_a, Tag{});
      split2(p2, p3, hi_b, lo_b, Tag{});
      bh[t][0] = movmatrix_trans(hi_a);
      bh[t][1] = movmatrix_trans(hi_b);
      bl[t][0] = movmatrix_trans(lo_a);
      bl[t][1] = movmatrix_trans(lo_b);
    }
    // rows without a token may hold anything, NaN too: 0 in the product
    uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;
    if (partial) {
      keep_lo = (2 * tq < rlo ? 0xffffu : 0u) | (2 * tq + 1 < rlo ? 0xffff0000u : 0u);
      keep_hi = (2 * tq < rhi ? 0xffffu : 0u) | (2 * tq + 1 < rhi ? 0xffff0000u : 0u);
    }
#pragma unroll
    for (int dd = 0; dd < D / 16; ++dd) {
      uint32_t a[4];
      const int c = ((dd & 3) << 1) | v_half;
      ldsm_x4_trans(vt + (dd >> 2) * group_bytes + v_row + ((c ^ r8) << 4), a);
      if (partial) {
        a[0] &= keep_lo;
        a[1] &= keep_lo;
        a[2] &= keep_hi;
        a[3] &= keep_hi;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma(o[t][dd], a, bh[t][0], bh[t][1], Tag{});
        mma(o[t][dd], a, bl[t][0], bl[t][1], Tag{});
      }
    }
  }

  // The warp's sums to shared memory: columns of O as [8 NT][pitch], (m, l) of each.  m = -infinity
  // with l = 0 (no token) or l = -1 (tokens, every logit -infinity), which have no weight in a join;
  // m is NaN once a logit was.
  __device__ __forceinline__ void put(float* jo, int pitch, float2* jml, bool tokens, int lane) const {
    const int g = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[t][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(kFullMask, sum, off);
        const int col = t * 8 + 2 * tq + e;
        if (m[t][e] == -INFINITY && tokens) sum = -1.f;
        if (g == 0) jml[col] = make_float2(m[t][e], sum);
        float* dst = jo + col * pitch + g;
#pragma unroll
        for (int dd = 0; dd < D / 16; ++dd) {
          dst[dd * 16] = o[t][dd][e];
          dst[dd * 16 + 8] = o[t][dd][2 + e];
        }
      }
    }
  }
};

}  // namespace pagedkv
