// Rotary positions: the rotation of 8 pairs held as two 16-byte pieces, and packed
// minimum / maximum of 16-bit values (NaN if either is NaN).
#pragma once

#include <type_traits>

#include "common.cuh"

namespace pagedkv {

struct RopeParams {
  const float* cos_sin;  // null: no rotation
  const int32_t* positions;
  int max_position, rotary_dim, interleaved, num_axes, total_tokens;
  uint8_t pair_axis[128];  // head_dim <= 256
  uint8_t quad_axis[32];   // the axis of pairs 4 i .. 4 i + 3, kMixed if they differ
};
constexpr uint8_t kMixed = 255;

// Checks a caller's pa_rope and copies it; returns a pa_status.
inline int rope_params(const pa_rope& r, int head_dim, RopeParams& p) {
  if (r.max_position < 1 || r.rotary_dim < 1 || r.num_axes < 1 || r.num_axes > PA_ROPE_MAX_AXES ||
      !r.cos_sin || !aligned16(r.cos_sin))
    return PA_ERR_INVALID_ARG;
  if (r.rotary_dim % 16 != 0 || r.rotary_dim > head_dim) return PA_ERR_UNSUPPORTED;
  if (r.num_axes > 1 && (!r.positions || !r.pair_axis)) return PA_ERR_INVALID_ARG;
  p.cos_sin = r.cos_sin;
  p.positions = r.positions;
  p.max_position = r.max_position;
  p.rotary_dim = r.rotary_dim;
  p.interleaved = r.interleaved != 0;
  p.num_axes = r.num_axes;
  if (r.pair_axis) {
    for (int j = 0; j < r.rotary_dim / 2; ++j) {
      if (r.pair_axis[j] >= r.num_axes) return PA_ERR_INVALID_ARG;
      p.pair_axis[j] = r.pair_axis[j];
      if (j % 4 == 0) p.quad_axis[j / 4] = r.pair_axis[j];
      else if (p.quad_axis[j / 4] != r.pair_axis[j]) p.quad_axis[j / 4] = kMixed;
    }
  }
  return PA_OK;
}

// A token's position on an axis as given, then kept in range.
__device__ __forceinline__ int raw_position(const RopeParams& p, int axis, int token, int place) {
  return p.positions ? p.positions[static_cast<size_t>(axis) * p.total_tokens + token] : place;
}
__device__ __forceinline__ int position(const RopeParams& p, int axis, int token, int place) {
  return min(max(raw_position(p, axis, token, place), 0), p.max_position - 1);
}

__device__ inline void check_positions(const RopeParams& p, int token, int place, int32_t* err) {
  for (int a = 0; a < p.num_axes; ++a) {
    const int at = raw_position(p, a, token, place);
    if (at < 0 || at >= p.max_position) report_error(err, PA_ERR_BAD_POSITION, token, at);
  }
}

template <class Tag>
__device__ __forceinline__ uint4 from_float8(const float (&f)[8], Tag) {
  constexpr int kType = std::is_same<Tag, BF16>::value ? PA_BF16 : PA_F16;
  return make_uint4(pack2(f[0], f[1], kType), pack2(f[2], f[3], kType), pack2(f[4], f[5], kType),
                    pack2(f[6], f[7], kType));
}

// The cosines and sines of pairs j0 .. j0 + 7 of one token, each from its axis's row.
__device__ __forceinline__ void load_cos_sin(const RopeParams& p, int token, int place, int j0,
                                             float (&c)[8], float (&s)[8]) {
  const int half = p.rotary_dim / 2;
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    const int axis = p.num_axes == 1 ? 0 : p.quad_axis[(j0 + e) / 4];
    if (axis != kMixed) {
      const float* row = p.cos_sin +
                         static_cast<size_t>(position(p, axis, token, place)) * p.rotary_dim + j0 + e;
      const float4 u = *reinterpret_cast<const float4*>(row);
      const float4 w = *reinterpret_cast<const float4*>(row + half);
      c[e] = u.x; c[e + 1] = u.y; c[e + 2] = u.z; c[e + 3] = u.w;
      s[e] = w.x; s[e + 1] = w.y; s[e + 2] = w.z; s[e + 3] = w.w;
    } else {
#pragma unroll
      for (int i = e; i < e + 4; ++i) {
        const int at = position(p, p.pair_axis[j0 + i], token, place);
        const float* row = p.cos_sin + static_cast<size_t>(at) * p.rotary_dim + j0 + i;
        c[i] = row[0];
        s[i] = row[half];
      }
    }
  }
}

// Rotates 8 pairs of one token, in fp32, each result rounded once to the storage type.
// Half-split pairs: the first elements in a, the second ones in b; interleaved: a and b are 16
// consecutive elements, pair after pair.
template <class Tag>
__device__ __forceinline__ void rotate(const RopeParams& p, const float (&c)[8], const float (&s)[8],
                                       uint4& a, uint4& b, Tag) {
  float fa[8], fb[8];
  to_float8(a, fa, Tag{});
  to_float8(b, fb, Tag{});
  if (p.interleaved) {
    float x[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = fa[e];
      x[8 + e] = fb[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = x[2 * e], w = x[2 * e + 1];
      x[2 * e] = u * c[e] - w * s[e];
      x[2 * e + 1] = w * c[e] + u * s[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      fa[e] = x[e];
      fb[e] = x[8 + e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = fa[e], w = fb[e];
      fa[e] = u * c[e] - w * s[e];
      fb[e] = w * c[e] + u * s[e];
    }
  }
  a = from_float8(fa, Tag{});
  b = from_float8(fb, Tag{});
}

__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y, BF16) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                       *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y, F16) {
  const __half2 r =
      __hmin2_nan(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y, BF16) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                       *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y, F16) {
  const __half2 r =
      __hmax2_nan(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <class Tag>
__device__ __forceinline__ uint4 min8(const uint4& x, const uint4& y, Tag t) {
  return make_uint4(min2(x.x, y.x, t), min2(x.y, y.y, t), min2(x.z, y.z, t), min2(x.w, y.w, t));
}
template <class Tag>
__device__ __forceinline__ uint4 max8(const uint4& x, const uint4& y, Tag t) {
  return make_uint4(max2(x.x, y.x, t), max2(x.y, y.y, t), max2(x.z, y.z, t), max2(x.w, y.w, t));
}

}  // namespace pagedkv
