// kv_append and kv_gather: rows between dense tensors and a paged cache.
//
// A row (one head vector of D values) belongs to L = D / 16 lanes; lane i
// holds the 8-value chunks i and i + L, so that a full-width rotation in
// halves pairs values inside a lane, every access is 16 bytes and L lanes
// cover contiguous runs.  The transform of an INT4 row is then one butterfly
// between the two chunks, three inside a chunk and log2 L between lanes.
//
// Both kernels move bytes: what bounds them is memory (and, for a few
// tokens, the latency of the chain slot / position -> table row -> store).
// Rows of one token follow each other in the grid, so that a token's cos, sin
// and slot come from near caches.
//
// Measured (kernel times): a prompt of 8192 tokens, 32 + 2 x 8 heads of 128,
// bf16 pages: 205 MB in 41 us, 5.0 TB/s (a large copy moves 4.75).  4093
// tokens, 3 x 24 heads of 64, fp16 into INT4: 57 MB in 21 us, the vector
// pipes half busy with the transform, the rest latency of the one row a group
// of lanes has.  30011 entries of 8 INT4 heads of 128 read back: 155 MB in
// 33 us, 4.7 TB/s.  One token: 2.6 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kv.hpp"
#include "launch.hpp"

namespace whtq {

struct KvRows {
  const uint8_t* p;
  int64_t tok, head;  // bytes
};
struct KvAppendArgs {
  KvCache c;
  KvRows k, v, q, qo;
  const int64_t* slots;
  const float *cos, *sin;
  const int32_t* pos;
  int64_t ld_cs, max_pos, capacity;
  uint32_t rows;  // tokens * (heads + 2 kv_heads)
  int heads, rot, interleaved;
};

// The two chunks of a lane rotated in place.  Each product and each sum is
// rounded by itself (no contraction), so the result is the same wherever it
// is computed.
template <int D, int T>
__device__ __forceinline__ void kv_rotate(float (&x)[16], const KvAppendArgs& a, int64_t pos, int i, const uint8_t* row) {
#pragma clang fp contract(off)
  constexpr int L = D / 16;
  const float* cs = a.cos + pos * a.ld_cs;
  const float* sn = a.sin + pos * a.ld_cs;
  if (!a.interleaved && a.rot == D) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 c = ldg<f32x4>(cs + 8 * i + 4 * h), s = ldg<f32x4>(sn + 8 * i + 4 * h);
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
      const f32x4 c = ldg<f32x4>(cs + 4 * ch), s = ldg<f32x4>(sn + 4 * ch);
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
      kv_widen8<T>(ldg<u32x4>(row + 16 * (low ? ch + pair : ch - pair)), o);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = cs[8 * at + e], s = sn[8 * at + e], u = x[8 * b + e];
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

template <int D, int T, bool INT4>
__global__ __launch_bounds__(256) void k_kv_append(const KvAppendArgs a) {
  constexpr int L = D / 16, RB = 256 / L;
  const uint32_t r = blockIdx.x * RB + threadIdx.x / L;
  const int i = threadIdx.x % L;
  const uint32_t per = a.heads + 2 * a.c.kv_heads;
  const bool live = r < a.rows;
  const uint32_t t = live ? r / per : 0, hs = live ? r % per : 0;
  const int64_t pos = a.pos ? (int64_t)a.pos[t] : 0;
  // head slots of a token: its keys, its values, its queries
  const bool is_k = hs < (uint32_t)a.c.kv_heads, is_q = hs >= 2u * a.c.kv_heads;
  const int h = is_k ? hs : is_q ? hs - 2 * a.c.kv_heads : hs - a.c.kv_heads;
  const KvRows& in = is_k ? a.k : is_q ? a.q : a.v;
  const uint8_t* row = in.p + t * in.tok + h * in.head;
  float x[16];
  kv_widen8<T>(ldg<u32x4>(row + 16 * i), x);
  kv_widen8<T>(ldg<u32x4>(row + 16 * (i + L)), x + 8);
  bool ok = live;
  if (a.pos) ok = ok && pos >= 0 && pos < a.max_pos;
  if (a.pos && ok && (is_k || is_q)) kv_rotate<D, T>(x, a, pos, i, row);
  if (is_q) {
    if (ok) {
      uint8_t* o = const_cast<uint8_t*>(a.qo.p) + t * a.qo.tok + h * a.qo.head;
      stg<u32x4>(o + 16 * i, kv_round8<T>(x));
      stg<u32x4>(o + 16 * (i + L), kv_round8<T>(x + 8));
    }
    return;
  }
  const int64_t slot = a.slots[t];
  ok = ok && slot >= 0 && slot < a.capacity;
  const KvSide& c = is_k ? a.c.k : a.c.v;
  const int64_t page = slot >> a.c.page_shift, off = slot & ((1 << a.c.page_shift) - 1);
  if constexpr (!INT4) {
    if (!ok) return;
    uint8_t* o = c.p + page * c.page + h * c.head + off * c.tok;
    stg<u32x4>(o + 16 * i, kv_round8<T>(x));
    stg<u32x4>(o + 16 * (i + L), kv_round8<T>(x + 8));
  } else {
    if (a.c.signs) {
      kv_sign8(x, (a.c.signs[i >> 2] >> (8 * (i & 3))) & 255u);
      kv_sign8(x + 8, (a.c.signs[(i + L) >> 2] >> (8 * ((i + L) & 3))) & 255u);
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

// The unscaled transform of a row's codes, as whole numbers: at most 8 D = 1024
// in size, so fp16 holds every step exactly and two values go in one
// operation (in fp32 they kept the vector pipes 90 % busy over a long prefix).
// Lane i's words are its chunks' codes, pairs (j, j + 4).
template <int D>
__device__ __forceinline__ void kv_rht_codes(uint32_t c0, uint32_t c1, int i, float* x) {
  f16x2_t p[8];
  const u32x4 a = kv_codes8(c0), b = kv_codes8(c1);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t aw = a[w], bw = b[w];
    p[w] = __builtin_bit_cast(f16x2_t, aw);
    p[4 + w] = __builtin_bit_cast(f16x2_t, bw);
  }
#pragma unroll
  for (int h = 1; h < 8; h *= 2)  // index bits 0 and 1, and the chunks' bit
#pragma unroll
    for (int w = 0; w < 8; ++w)
      if (!(w & h)) {
        const f16x2_t u = p[w], v = p[w + h];
        p[w] = u + v;
        p[w + h] = u - v;
      }
  auto lanes = [&](auto m) {
    constexpr int M = decltype(m)::value;
    const _Float16 one = (_Float16)(i & M ? -1.f : 1.f);
#pragma unroll
    for (int w = 0; w < 8; ++w)
      p[w] = __builtin_elementwise_fma(p[w], f16x2_t{one, one},
                                       __builtin_bit_cast(f16x2_t, kv_lane_xor<M>(__builtin_bit_cast(uint32_t, p[w]))));
  };
  lanes(std::integral_constant<int, 1>{});
  lanes(std::integral_constant<int, 2>{});
  if constexpr (D == 128) lanes(std::integral_constant<int, 4>{});
#pragma unroll
  for (int w = 0; w < 8; ++w) {  // index bit 2, inside the pairs
    const _Float16 u = p[w][0], v = p[w][1];
    const f16x2_t y = __builtin_elementwise_fma(f16x2_t{v, v}, f16x2_t{(_Float16)1.f, (_Float16)-1.f}, f16x2_t{u, u});
    x[8 * (w >> 2) + (w & 3)] = (float)y[0];
    x[8 * (w >> 2) + (w & 3) + 4] = (float)y[1];
  }
}
// The signs of eight 16-bit floats in pairs turned by bits 0 .. 7 of b.
__device__ __forceinline__ void kv_sign_words(u32x4& w, uint32_t b) {
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] ^= (b << (15 - 2 * q) & 0x8000u) | (b << (30 - 2 * q) & 0x80000000u);
}

struct KvGatherArgs {
  KvCache c;
  KvRows k, v;
  const int64_t* slots;
  int64_t capacity;
  uint32_t rows;  // tokens * kv_heads
  int first, last;  // sides: 0 keys, 1 values
};

// A group of lanes has a token's key and value of one head: one slot is looked
// up for both and their loads are in flight together (30011 entries of 8 INT4
// heads of 128: 33 us against 39 with a group for each).  Where the machine
// holds a group for each at once, the two go apart (a grid of two rows; 61
// tokens of 8 INT4 heads of 128: 4 us against 5).  A slot outside the cache
// reads slot 0, whose place there is.
template <int D, int T, bool INT4>
__global__ __launch_bounds__(256) void k_kv_gather(const KvGatherArgs a) {
  constexpr int L = D / 16, RB = 256 / L;
  const uint32_t r = blockIdx.x * RB + threadIdx.x / L;
  const int i = threadIdx.x % L;
  const bool live = r < a.rows;
  const uint32_t t = live ? r / a.c.kv_heads : 0, h = live ? r % a.c.kv_heads : 0;
  const int64_t slot = a.slots[t];
  const bool ok = slot >= 0 && slot < a.capacity;
  const int64_t page = ok ? slot >> a.c.page_shift : 0, off = ok ? slot & ((1 << a.c.page_shift) - 1) : 0;
  const int first = a.first + blockIdx.y, last = gridDim.y == 2 ? first : a.last;
  u32x4 w[2][2];
  uint32_t codes[2][2];
  uint16_t sb[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    if (v < first || v > last) continue;
    const KvSide& c = v ? a.c.v : a.c.k;
    const uint8_t* e0 = c.p + page * c.page + h * c.head + off * c.tok;
    if constexpr (INT4) {
      codes[v][0] = ldg<uint32_t>(e0 + 4 * i);
      codes[v][1] = ldg<uint32_t>(e0 + 4 * (i + L));
      sb[v] = c.scale[page * c.s_page + h * c.s_head + off];
    } else {
      w[v][0] = ldg<u32x4>(e0 + 16 * i);
      w[v][1] = ldg<u32x4>(e0 + 16 * (i + L));
    }
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    if (v < first || v > last) continue;
    if constexpr (INT4) {
      float x[16];
      kv_rht_codes<D>(codes[v][0], codes[v][1], i, x);
      const float f = kv_scale(sb[v]) * (D == 64 ? 0.125f : 0.08838834764831845f);  // s / sqrt(D)
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= f;
      w[v][0] = kv_round8<T>(x);
      w[v][1] = kv_round8<T>(x + 8);
      if (a.c.signs) {
        kv_sign_words(w[v][0], a.c.signs[i >> 2] >> (8 * (i & 3)));
        kv_sign_words(w[v][1], a.c.signs[(i + L) >> 2] >> (8 * ((i + L) & 3)));
      }
    }
    if (!ok) w[v][0] = w[v][1] = u32x4{0u, 0u, 0u, 0u};
    if (live) {
      const KvRows& out = v ? a.v : a.k;
      uint8_t* o = const_cast<uint8_t*>(out.p) + t * out.tok + h * out.head;
      stg<u32x4>(o + 16 * i, w[v][0]);
      stg<u32x4>(o + 16 * (i + L), w[v][1]);
    }
  }
}

// Tokens of `per` rows of `lanes` threads, in as many launches as it takes; one
// in any ordinary call.  (A token is at most 3 x 65535 rows.)
template <typename F>
static hipError_t by_tokens(int64_t tokens, int64_t per, int lanes, F launch) {
  const int64_t most = kLaunchThreads / (per * lanes);
  for (int64_t t = 0; t < tokens; t += most) {
    launch(t, std::min(most, tokens - t));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

#define KV_DISPATCH(KERNEL, D, T, INT4, GRID, S, ARGS)                                                      \
  do {                                                                                                      \
    if ((D) == 128 && (T) == KV_BF16 && (INT4)) hipLaunchKernelGGL((KERNEL<128, KV_BF16, true>), GRID, dim3(256), 0, S, ARGS); \
    else if ((D) == 128 && (T) == KV_BF16) hipLaunchKernelGGL((KERNEL<128, KV_BF16, false>), GRID, dim3(256), 0, S, ARGS);     \
    else if ((D) == 128 && (INT4)) hipLaunchKernelGGL((KERNEL<128, KV_F16, true>), GRID, dim3(256), 0, S, ARGS);               \
    else if ((D) == 128) hipLaunchKernelGGL((KERNEL<128, KV_F16, false>), GRID, dim3(256), 0, S, ARGS);                        \
    else if ((T) == KV_BF16 && (INT4)) hipLaunchKernelGGL((KERNEL<64, KV_BF16, true>), GRID, dim3(256), 0, S, ARGS);           \
    else if ((T) == KV_BF16) hipLaunchKernelGGL((KERNEL<64, KV_BF16, false>), GRID, dim3(256), 0, S, ARGS);                    \
    else if ((INT4)) hipLaunchKernelGGL((KERNEL<64, KV_F16, true>), GRID, dim3(256), 0, S, ARGS);                              \
    else hipLaunchKernelGGL((KERNEL<64, KV_F16, false>), GRID, dim3(256), 0, S, ARGS);                                         \
  } while (0)

hipError_t launch_kv_append(const KvCache& c, int dim, int dt, bool int4, int64_t tokens, const void* k,
                            const int64_t* ks, const void* v, const int64_t* vs, const int64_t* slots,
                            int64_t capacity, const float* cos, const float* sin, const int32_t* pos, int64_t ld_cs,
                            int64_t max_pos, int rot, int interleaved, const void* q, const int64_t* qs, int heads,
                            void* qo, const int64_t* qos, hipStream_t s) {
  const int rb = 256 / (dim / 16);
  const int64_t per = (q ? heads : 0) + 2 * (int64_t)c.kv_heads;
  return by_tokens(tokens, per, dim / 16, [&](int64_t t0, int64_t n) {
    KvAppendArgs a{};
    a.c = c;
    a.k = {(const uint8_t*)k + t0 * ks[0] * 2, ks[0] * 2, ks[1] * 2};
    a.v = {(const uint8_t*)v + t0 * vs[0] * 2, vs[0] * 2, vs[1] * 2};
    if (q) {
      a.q = {(const uint8_t*)q + t0 * qs[0] * 2, qs[0] * 2, qs[1] * 2};
      a.qo = {(const uint8_t*)qo + t0 * qos[0] * 2, qos[0] * 2, qos[1] * 2};
      a.heads = heads;
    }
    a.slots = slots + t0;
    a.capacity = capacity;
    a.cos = cos;
    a.sin = sin;
    a.pos = pos ? pos + t0 : nullptr;
    a.ld_cs = ld_cs;
    a.max_pos = max_pos;
    a.rot = rot;
    a.interleaved = interleaved;
    a.rows = (uint32_t)(n * per);
    const dim3 grid((unsigned)((n * per + rb - 1) / rb));
    KV_DISPATCH(k_kv_append, dim, dt, int4, grid, s, a);
  });
}

hipError_t launch_kv_gather(const KvCache& c, int dim, int dt, bool int4, int64_t tokens, const int64_t* slots,
                            int64_t capacity, void* ko, const int64_t* ks, void* vo, const int64_t* vs,
                            hipStream_t s) {
  const int rb = 256 / (dim / 16);
  const int64_t per = c.kv_heads;
  return by_tokens(tokens, per, dim / 16, [&](int64_t t0, int64_t n) {
    KvGatherArgs a{};
    a.c = c;
    if (ko) a.k = {(const uint8_t*)ko + t0 * ks[0] * 2, ks[0] * 2, ks[1] * 2};
    if (vo) a.v = {(const uint8_t*)vo + t0 * vs[0] * 2, vs[0] * 2, vs[1] * 2};
    a.slots = slots + t0;
    a.capacity = capacity;
    a.first = ko ? 0 : 1;
    a.last = vo ? 1 : 0;
    a.rows = (uint32_t)(n * per);
    int dev = 0;
    (void)hipGetDevice(&dev);
    const bool apart = ko && vo && 2 * n * per * (dim / 16) <= 2048 * (int64_t)device_cu_count(dev);
    const dim3 grid((unsigned)((n * per + rb - 1) / rb), apart ? 2 : 1);
    KV_DISPATCH(k_kv_gather, dim, dt, int4, grid, s, a);
  });
}

}  // namespace whtq
