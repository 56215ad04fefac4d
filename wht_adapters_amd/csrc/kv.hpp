// Shared by the paged key/value cache kernels: kernel arguments, types of the
// 16-bit operands, and the transform of one head vector spread over lanes.
#pragma once

#include "common.hpp"

namespace whtq {

enum KvT : int { KV_BF16 = 1, KV_F16 = 2 };  // the values of WHTQ_BF16 / WHTQ_F16

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct KvSide {  // the keys or the values of a cache
  uint8_t* p;
  uint16_t* scale;
  int64_t page, head, tok;  // bytes
  int64_t s_page, s_head;   // elements
};
struct KvCache {
  KvSide k, v;
  const uint32_t* signs;
  int64_t num_pages;
  int page_shift, kv_heads;
};

// Load at a wave-uniform base plus a lane's 32-bit offset plus a constant, as
// a buffer load: the base is in scalar registers and no lane computes a 64-bit
// address.  (The buffer has no size of its own: offsets are checked by their
// callers, like any pointer's.)
template <typename V>
__device__ __forceinline__ V kv_load(const void* base, uint32_t off, int imm = 0) {
  const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, -1, 0x00027000);
  if constexpr (sizeof(V) == 16) return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(r, off + imm, 0, 0));
  else if constexpr (sizeof(V) == 8) return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b64(r, off + imm, 0, 0));
  else if constexpr (sizeof(V) == 4) return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b32(r, off + imm, 0, 0));
  else return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b16(r, off + imm, 0, 0));
}

template <int T>
__device__ __forceinline__ uint32_t kv_pack(float lo, float hi) {
  if constexpr (T == KV_BF16) return pack_bf16(lo, hi);
  else return pack_f16(lo, hi);
}
template <int T>
__device__ __forceinline__ void kv_widen8(u32x4 w, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = w[i];
    if constexpr (T == KV_BF16) {
      f[2 * i] = bf16lo(x);
      f[2 * i + 1] = bf16hi(x);
    } else {
      const f16x2_t h = __builtin_bit_cast(f16x2_t, x);
      f[2 * i] = (float)h[0];
      f[2 * i + 1] = (float)h[1];
    }
  }
}
template <int T>
__device__ __forceinline__ u32x4 kv_round8(const float* f) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = kv_pack<T>(f[2 * i], f[2 * i + 1]);
  return w;
}

// Butterflies of stride 1, 2, .., N / 2 among the lane's N values.
template <int N>
__device__ __forceinline__ void kv_bfly(float* v) {
#pragma unroll
  for (int h = 1; h < N; h *= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & h)) bfly(v[i], v[i + h]);
}
// The butterfly between lanes that differ in lane bit `m` (the lane with the
// bit clear holds the lower index).
template <int N>
__device__ __forceinline__ void kv_lane_bfly(float* v, int m, int lane) {
  const bool up = lane & m;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float o = __shfl_xor(v[i], m, 64);
    v[i] = up ? o - v[i] : v[i] + o;
  }
}

__device__ __forceinline__ void kv_sign8(float* v, uint32_t bits8) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = as_f(as_u(v[i]) ^ ((bits8 >> i) << 31));
}

// Eight INT4 codes (w: code i in bits [4i, 4i + 4), two's complement) to
// exact fp16, two operations a pair: offset by 8 they are whole numbers u in
// [0, 15]; 0x6400 | u is 1024 + u and 0x6400 | (u << 4) is 1024 + 16 u.  The
// pairs come out as codes (0,4), (1,5), (2,6), (3,7): position i of the eight
// holds code kv_perm(i), on both operands of a product or undone at its end.
__device__ __forceinline__ constexpr int kv_perm(int i) { return (i >> 1) | ((i & 1) << 2); }
__device__ __forceinline__ uint32_t kv_code_lo(uint32_t x) {  // x: u in bits 0..3 and 16..19
  const f16x2_t h = __builtin_bit_cast(f16x2_t, (x & 0x000f000fu) | 0x64006400u);
  return __builtin_bit_cast(uint32_t, h + f16x2_t{(_Float16)-1032.f, (_Float16)-1032.f});
}
__device__ __forceinline__ uint32_t kv_code_hi(uint32_t x) {  // x: u in bits 4..7 and 20..23
  const f16x2_t h = __builtin_bit_cast(f16x2_t, (x & 0x00f000f0u) | 0x64006400u);
  const f16x2_t c = {(_Float16)0.0625f, (_Float16)0.0625f}, o = {(_Float16)-72.f, (_Float16)-72.f};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(h, c, o));
}
__device__ __forceinline__ u32x4 kv_codes8(uint32_t w) {
  const uint32_t a = w ^ 0x88888888u, b = a >> 8;
  return u32x4{kv_code_lo(a), kv_code_hi(a), kv_code_lo(b), kv_code_hi(b)};
}

// The scale of an INT4 entry, from its bits.  An entry whose scale is not finite
// stands for NaN: an infinite scale must not make a score of -inf, which would
// hide its key.
__device__ __forceinline__ float kv_scale(uint16_t b) {
  const float s = (float)__builtin_bit_cast(_Float16, b);
  return fabsf(s) < 65536.f ? s : __builtin_nanf("");
}
// Two of them in a word, still fp16: x + 0 x.
__device__ __forceinline__ f16x2_t kv_scale2(uint32_t w) {
  const f16x2_t h = __builtin_bit_cast(f16x2_t, w), z = {(_Float16)0.f, (_Float16)0.f};
  return __builtin_elementwise_fma(h, z, h);
}

}  // namespace whtq
