// kv_gather: rows of a paged cache as dense tensors (kv_append, the way into
// it, is in qk_norm.hip).
//
// A row (one head vector of D values) belongs to L = D / 16 lanes; lane i
// holds the 8-value chunks i and i + L, so that every access is 16 bytes and L
// lanes cover contiguous runs.  The transform of an INT4 row is then one
// butterfly between the two chunks, three inside a chunk and log2 L between
// lanes.
//
// The kernel moves bytes: what bounds it is memory (and, for a few tokens, the
// latency of the chain slot -> entry -> store).
//
// Measured (kernel times): 30011 entries of 8 INT4 heads of 128 read back:
// 155 MB in 33 us, 4.7 TB/s (a large copy moves 4.75).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kv_rows.hpp"
#include "launch.hpp"

namespace whtq {

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

template <int D, int T, bool INT4>
static void gather_launch(const KvGatherArgs& a, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((k_kv_gather<D, T, INT4>), grid, dim3(256), 0, s, a);
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
    KV_PICK(gather_launch, dim, dt, int4, a, grid, s);
  });
}

}  // namespace whtq
