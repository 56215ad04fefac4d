// Rows of head vectors: norms and rotary positions of one row spread over
// lanes, shared by kv_append and the dense forms.
//
// A row (one head vector of D values) belongs to L = D / 16 lanes; lane i
// holds the 8-value chunks i and i + L, so that a full-width rotation in
// halves pairs values inside a lane, every access is 16 bytes and L lanes
// cover contiguous runs.
#pragma once

#include "kv.hpp"

namespace whtq {

struct KvRows {
  const uint8_t* p;
  int64_t tok, head;  // bytes
};
struct KvTurn {  // rotary positions; pos NULL: none
  const float *cos, *sin;
  const int32_t* pos;
  int64_t ld, max_pos;
  int rot, interleaved;
};
struct KvWeight {  // norm weights; p NULL: no norm
  const uint8_t* p;
  int64_t head;  // bytes; 0: one vector for all heads
};
struct KvNorm {
  KvWeight q, k;
  int dt;  // WHTQ_F32, or the 16-bit types
  float eps;
};

// The two chunks of a lane rotated in place (BACK: by the opposite angle).
// Each product and each sum is rounded by itself (no contraction), so the
// result is the same wherever it is computed.  `load` gives a chunk of the
// row as it was before the rotation.
template <int D, bool BACK = false, typename Load>
__device__ __forceinline__ void kv_rotate(float (&x)[16], const KvTurn& a, int64_t pos, int i, Load load) {
#pragma clang fp contract(off)
  constexpr int L = D / 16;
  const float* cs = a.cos + pos * a.ld;
  const float* sn = a.sin + pos * a.ld;
  if (!a.interleaved && a.rot == D) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 c = ldg<f32x4>(cs + 8 * i + 4 * h);
      f32x4 s = ldg<f32x4>(sn + 8 * i + 4 * h);
      if constexpr (BACK) s = -s;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = x[4 * h + e], w = x[8 + 4 * h + e];
        x[4 * h + e] = u * c[e] - w * s[e];
        x[8 + 4 * h + e] = w * c[e] + u * s[e];
      }
    }
    return;
  }
  const int pair = a.rot / 16;  // chunks in a half
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int ch = i + b * L;
    if (ch * 8 >= a.rot) continue;
    if (a.interleaved) {
      const f32x4 c = ldg<f32x4>(cs + 4 * ch);
      f32x4 s = ldg<f32x4>(sn + 4 * ch);
      if constexpr (BACK) s = -s;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = x[8 * b + 2 * e], w = x[8 * b + 2 * e + 1];
        x[8 * b + 2 * e] = u * c[e] - w * s[e];
        x[8 * b + 2 * e + 1] = w * c[e] + u * s[e];
      }
    } else {
      const bool low = ch < pair;
      const int at = low ? ch : ch - pair;
      float o[8];
      load(low ? ch + pair : ch - pair, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = cs[8 * at + e], s = BACK ? -sn[8 * at + e] : sn[8 * at + e], u = x[8 * b + e];
        const float os = o[e] * s;
        x[8 * b + e] = low ? u * c - os : u * c + os;
      }
    }
  }
}

template <int M>  // the value of the lane that differs in lane bit M = 1, 2, 4
__device__ __forceinline__ uint32_t kv_lane_xor(uint32_t x) {
  constexpr int QUAD = M == 1 ? 0xb1 : M == 2 ? 0x4e : 0x1b;  // quad_perm: lane ^ 1, ^ 2, ^ 3
  if constexpr (M == 4) x = __builtin_amdgcn_mov_dpp(x, 0x141, 0xf, 0xf, true);  // row_half_mirror: lane ^ 7
  return __builtin_amdgcn_mov_dpp(x, QUAD, 0xf, 0xf, true);
}
// Butterflies between lanes whose values differ in lane bit M.
template <int M>
__device__ __forceinline__ void kv_near_bfly(float (&x)[16], int i) {
  const float sg = i & M ? -1.f : 1.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = __builtin_fmaf(x[e], sg, as_f(kv_lane_xor<M>(as_u(x[e]))));
}

// Sum over the L lanes of a row, in every one of them.
template <int L>
__device__ __forceinline__ float kv_row_sum(float x) {
  x += as_f(kv_lane_xor<1>(as_u(x)));
  x += as_f(kv_lane_xor<2>(as_u(x)));
  if constexpr (L == 8) x += as_f(kv_lane_xor<4>(as_u(x)));
  return x;
}

// Eight weights, chunk ch of a head's.
__device__ __forceinline__ void kv_weight8(const uint8_t* w, int dt, int ch, float* f) {
  if (dt == 0) {
    const f32x4 a = ldg<f32x4>(w + 32 * ch), b = ldg<f32x4>(w + 32 * ch + 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = a[e];
      f[4 + e] = b[e];
    }
  } else if (dt == KV_BF16) {
    kv_widen8<KV_BF16>(ldg<u32x4>(w + 16 * ch), f);
  } else {
    kv_widen8<KV_F16>(ldg<u32x4>(w + 16 * ch), f);
  }
}
__device__ __forceinline__ void kv_weigh8(float* x, const uint8_t* w, int dt, int ch, float r) {
  float f[8];
  kv_weight8(w, dt, ch, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = x[e] * r * f[e];
}
// r = (mean x^2 + eps)^-1/2 of the row.
template <int D>
__device__ __forceinline__ float kv_rms(const float (&x)[16], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) ss = __builtin_fmaf(x[e], x[e], ss);
  return rsqrtf(kv_row_sum<D / 16>(ss) * (1.f / D) + eps);
}
// The lane's chunks times r and their weights; returns r.  Without weights the row is left as it is.
template <int D>
__device__ __forceinline__ float kv_norm(float (&x)[16], const uint8_t* w, int dt, float eps, int i) {
  const float r = kv_rms<D>(x, eps);
  if (w) {
    kv_weigh8(x, w, dt, i, r);
    kv_weigh8(x + 8, w, dt, i + D / 16, r);
  }
  return r;
}

}  // namespace whtq
