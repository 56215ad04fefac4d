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

// The ways of a rotation, each a kernel of its own where registers count: a
// whole row in halves, interleaved pairs, or halves of a part of the row.
enum KvWay : int { KV_STILL = 0, KV_HALVES = 1, KV_PAIRS = 2, KV_PART = 3 };
inline int kv_way(const KvTurn& a, int dim) {
  return !a.pos ? KV_STILL : a.interleaved ? KV_PAIRS : a.rot == dim ? KV_HALVES : KV_PART;
}
// The table's entries of a lane, taken beforehand (but for KV_PART, whose
// pairs lie in other lanes).
struct KvCs {
  f32x4 c[2], s[2];
};
template <int D, int WAY>
__device__ __forceinline__ void kv_load_cs(KvCs& t, const KvTurn& a, int64_t pos, int i) {
  if constexpr (WAY == KV_HALVES || WAY == KV_PAIRS) {
    const float* cs = a.cos + pos * a.ld;
    const float* sn = a.sin + pos * a.ld;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (an interleaved chunk that is not rotated has no entry: the first one is not used)
      const int at = WAY == KV_HALVES ? 8 * i + 4 * h : 8 * (i + h * (D / 16)) < a.rot ? 4 * (i + h * (D / 16)) : 0;
      t.c[h] = ldg<f32x4>(cs + at);
      t.s[h] = ldg<f32x4>(sn + at);
    }
  }
}
// The two chunks of a lane rotated in place (BACK: by the opposite angle).
// Each product and each sum is rounded by itself (no contraction), so the
// result is the same wherever it is computed.  `load` gives a chunk of the
// row as it was before the rotation (KV_PART).
template <int D, int WAY, bool BACK, typename Load>
__device__ __forceinline__ void kv_turn(float (&x)[16], const KvTurn& a, const KvCs& t, int64_t pos, int i, Load load) {
#pragma clang fp contract(off)
  if constexpr (WAY == KV_PART) {
    const float* cs = a.cos + pos * a.ld;
    const float* sn = a.sin + pos * a.ld;
    const int pair = a.rot / 16;  // chunks in a half
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int ch = i + b * (D / 16);
      if (ch * 8 >= a.rot) continue;
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
  if constexpr (WAY == KV_HALVES || WAY == KV_PAIRS) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (WAY == KV_PAIRS && 8 * (i + h * (D / 16)) >= a.rot) continue;
      const f32x4 c = t.c[h], s = BACK ? -t.s[h] : t.s[h];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float& p = x[WAY == KV_HALVES ? 4 * h + e : 8 * h + 2 * e];
        float& q = x[WAY == KV_HALVES ? 8 + 4 * h + e : 8 * h + 2 * e + 1];
        const float u = p, w = q;
        p = u * c[e] - w * s[e];
        q = w * c[e] + u * s[e];
      }
    }
  }
}
// Butterflies between lanes whose values differ in lane bit M.
template <int M>
__device__ __forceinline__ void kv_near_bfly(float (&x)[16], int i) {
  const float sg = i & M ? -1.f : 1.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = __builtin_fmaf(x[e], sg, as_f(kv_lane_xor<M>(as_u(x[e]))));
}

// The row x of head h, spread over the lanes, into its slot of the cache's keys or values.
template <int D, int T, bool INT4>
__device__ __forceinline__ void kv_keep(float (&x)[16], const KvCache& kv, const KvSide& c, int h, int64_t slot, bool ok, int i) {
  constexpr int L = D / 16;
  const int64_t page = slot >> kv.page_shift, off = slot & ((1 << kv.page_shift) - 1);
  if constexpr (!INT4) {
    if (!ok) return;
    uint8_t* o = c.p + page * c.page + h * c.head + off * c.tok;
    stg<u32x4>(o + 16 * i, kv_round8<T>(x));
    stg<u32x4>(o + 16 * (i + L), kv_round8<T>(x + 8));
  } else {
    if (kv.signs) {
      kv_sign8(x, (kv.signs[i >> 2] >> (8 * (i & 3))) & 255u);
      kv_sign8(x + 8, (kv.signs[(i + L) >> 2] >> (8 * ((i + L) & 3))) & 255u);
    }
    kv_bfly<8>(x);
    kv_bfly<8>(x + 8);
    kv_near_bfly<1>(x, i);
    kv_near_bfly<2>(x, i);
    if constexpr (D == 128) kv_near_bfly<4>(x, i);
#pragma unroll
    for (int e = 0; e < 8; ++e) bfly(x[e], x[8 + e]);
    // NaN stays the maximum: the row's scale is then NaN, and so is what it stands for
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] *= D == 64 ? 0.125f : 0.08838834764831845f;  // 1 / sqrt(D)
      top = __builtin_elementwise_maximum(top, fabsf(x[e]));
    }
#pragma unroll
    for (int m = 1; m < L; m *= 2) top = __builtin_elementwise_maximum(top, as_f(m == 1 ? kv_lane_xor<1>(as_u(top)) : m == 2 ? kv_lane_xor<2>(as_u(top)) : kv_lane_xor<4>(as_u(top))));
    const _Float16 s16 = (_Float16)(top / 7.0f);
    const float s = (float)s16, inv = s > 0.f ? 1.0f / s : 0.f;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int q = (int)__builtin_rintf(fminf(fmaxf(x[e] * inv, -7.f), 7.f));
      w[e >> 3] |= (uint32_t)(q & 15) << (4 * (e & 7));
    }
    if (!ok) return;
    uint8_t* o = c.p + page * c.page + h * c.head + off * c.tok;
    stg<uint32_t>(o + 4 * i, w[0]);
    stg<uint32_t>(o + 4 * (i + L), w[1]);
    if (i == 0) c.scale[page * c.s_page + h * c.s_head + off] = __builtin_bit_cast(uint16_t, s16);
  }
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
// The lane's chunks times r and their weights; returns r.
template <int D>
__device__ __forceinline__ float kv_norm(float (&x)[16], const uint8_t* w, int dt, float eps, int i) {
  const float r = kv_rms<D>(x, eps);
  kv_weigh8(x, w, dt, i, r);
  kv_weigh8(x + 8, w, dt, i + D / 16, r);
  return r;
}

}  // namespace whtq
