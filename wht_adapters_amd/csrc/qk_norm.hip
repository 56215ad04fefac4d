// kv_append (with norms or without), qk_norm_rope and its backward pass: norms
// of each head's queries and keys and their rotary positions, into a cache's
// slots and dense rows.
//
//   r = (mean x^2 + eps)^-1/2,  y = R (w o x r)
// and with g = R^T dy (the opposite rotation), u = w o g:
//   dw = sum g o x r  over tokens (and heads that share w),
//   dx = r (u - x r mean(u o x r)).
// The backward pass takes x again and computes r itself: two numbers a row
// less to keep, and x has to be read anyway.
//
// Both directions move bytes.  A row belongs to D / 16 lanes (kv_rows.hpp).
// Forward, the blocks of keys, values and queries are apart, so that a row's
// kind, its bases and strides are scalars.  Backward, a block walks rows of
// one weight vector, so that a lane's part of dw stays in registers; blocks
// leave one partial sum each, which a second kernel adds in a fixed order (no
// atomics: the same result every time).
//
// Measured (kernel times; 8192 tokens, 32 query and 8 key heads of 128, bf16):
// into a 16-bit cache 209 MB in 40 us, 5.2 TB/s (a large copy moves 4.9), without
// norms, from rows that lie close, 205 MB in 35; dense rows 176 MB in 36; backward
// 256 MB in 46 us, 5.5 TB/s, and 4.7 us for the join (a weight vector a head: 63
// us, a block walks one head's rows).  A kind's blocks together, with the
// rotation's kinds as branches, took 50 and 59 us, without norms 41: the branches
// keep registers of every kind.  2, 3 or 6 rows a group of lanes: 55 to 60 us
// against 45 at the time, fewer waves to wait side by side.  4093 tokens, 3 x 24
// heads of 64, fp16 into INT4 without norms: 57 MB in 17 us (21 with all kinds
// together), the vector pipes half busy with the transform, the rest latency of
// the one row a group of lanes has.  1 token, 48 heads: 3.3 us; 61 tokens of 80
// heads into INT4: 4.9 us; 333 tokens, 48 heads of 64 with a weight vector each:
// 3.9 us and 9.3 us, the latter the 11 rows in a row that a group of lanes has.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "qk_norm.hpp"

namespace whtq {

namespace {

__device__ __forceinline__ uint32_t kv_div(uint32_t n, const KvDiv& d) { return d.m ? __umulhi(n, d.m) >> d.s : n; }

template <int D, int T, bool INT4, int WAY>
__global__ __launch_bounds__(256) void k_qk_norm(const QkForwardArgs a) {
  constexpr int L = D / 16, RB = 256 / L;
  uint32_t b = blockIdx.x;
  const int kind = b < a.f[0].blocks ? 0 : b < a.f[0].blocks + a.f[1].blocks ? 1 : 2;
  if (kind > 0) b -= a.f[0].blocks;
  if (kind > 1) b -= a.f[1].blocks;
  const QkForward& f = a.f[kind];
  const uint32_t n = b * RB + threadIdx.x / L;
  const int i = threadIdx.x % L;
  const bool live = n < f.rows;
  const uint32_t t = live ? kv_div(n, f.heads) : 0, h = live ? n - t * f.heads.d : 0;
  const uint8_t* row = f.in.p + t * f.in.tok + h * f.in.head;
  const u32x4 raw0 = ldg<u32x4>(row + 16 * i), raw1 = ldg<u32x4>(row + 16 * (i + L));
  const int64_t pos = WAY ? (int64_t)a.turn.pos[t] : 0, slot = f.out.p ? 0 : a.slots[t];
  const bool ok = live && (!WAY || (pos >= 0 && pos < a.turn.max_pos));
  KvCs cs;
  if (f.turned) kv_load_cs<D, WAY>(cs, a.turn, ok ? pos : 0, i);
  float x[16];
  kv_widen8<T>(raw0, x);
  kv_widen8<T>(raw1, x + 8);
  const uint8_t* w = f.w.p ? f.w.p + h * f.w.head : nullptr;
  float r = 1.f;
  if (f.w.p) r = kv_norm<D>(x, w, a.dt, a.eps, i);
  if (f.turned && (WAY != KV_PART || ok))
    kv_turn<D, WAY, false>(x, a.turn, cs, pos, i, [&](int ch, float* o) {
      kv_widen8<T>(ldg<u32x4>(row + 16 * ch), o);
      if (w) kv_weigh8(o, w, a.dt, ch, r);
    });
  if (f.out.p) {
    if (!ok) {
      if (!live || !f.clear) return;
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.f;
    }
    uint8_t* o = const_cast<uint8_t*>(f.out.p) + t * f.out.tok + h * f.out.head;
    stg<u32x4>(o + 16 * i, kv_round8<T>(x));
    stg<u32x4>(o + 16 * (i + L), kv_round8<T>(x + 8));
  } else {
    kv_keep<D, T, INT4>(x, a.c, f.side, h, slot, ok && slot >= 0 && slot < a.capacity, i);
  }
}

template <int D, int T, int WAY>
__global__ __launch_bounds__(256) void k_qk_norm_back(const QkArgs a) {
  constexpr int L = D / 16, RB = 256 / L;
  const int i = threadIdx.x % L, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int qb = a.q.classes * a.q.blocks;
  const bool is_q = (int)blockIdx.x < qb;
  const QkSide& s = is_q ? a.q : a.k;
  const int b = is_q ? blockIdx.x : blockIdx.x - qb, cls = b / s.blocks, slot = b % s.blocks;
  const uint32_t per = s.classes == 1 ? s.heads : 1;  // rows of a token in this class
  const int64_t rows = a.tokens * per;
  float w[16], dw[16];
  const uint8_t* wp = s.w.p + cls * s.w.head;
  kv_weight8(wp, a.dt, i, w);
  kv_weight8(wp, a.dt, i + L, w + 8);
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.f;
  for (int64_t n = (int64_t)slot * RB + threadIdx.x / L; n < rows; n += (int64_t)s.blocks * RB) {
    const int64_t t = n >> 31 ? n / per : (int64_t)((uint32_t)n / per);
    const int h = per == 1 ? cls : (int)(n - t * per);
    const int64_t pos = WAY ? (int64_t)a.turn.pos[t] : 0;
    const uint8_t* xp = s.x.p + t * s.x.tok + h * s.x.head;
    const uint8_t* dp = s.dy.p + t * s.dy.tok + h * s.dy.head;
    const u32x4 x0 = ldg<u32x4>(xp + 16 * i), x1 = ldg<u32x4>(xp + 16 * (i + L));
    const u32x4 g0 = ldg<u32x4>(dp + 16 * i), g1 = ldg<u32x4>(dp + 16 * (i + L));
    uint8_t* o = const_cast<uint8_t*>(s.dx.p) + t * s.dx.tok + h * s.dx.head;
    if (WAY && (pos < 0 || pos >= a.turn.max_pos)) {
      if (s.clear) {
        stg<u32x4>(o + 16 * i, u32x4{0u, 0u, 0u, 0u});
        stg<u32x4>(o + 16 * (i + L), u32x4{0u, 0u, 0u, 0u});
      }
      continue;
    }
    KvCs cs;
    kv_load_cs<D, WAY>(cs, a.turn, pos, i);
    float x[16], g[16];
    kv_widen8<T>(x0, x);
    kv_widen8<T>(x1, x + 8);
    kv_widen8<T>(g0, g);
    kv_widen8<T>(g1, g + 8);
    const float r = kv_rms<D>(x, a.eps);
    kv_turn<D, WAY, true>(g, a.turn, cs, pos, i, [&](int ch, float* o) { kv_widen8<T>(ldg<u32x4>(dp + 16 * ch), o); });
    // x r first: of a row whose squares overflow r is 0, and so are x r and the gradients (x r^2 mean(u x) is 0 times
    // infinity there)
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] *= r;
      dw[e] = __builtin_fmaf(g[e], x[e], dw[e]);
      g[e] *= w[e];
      dot = __builtin_fmaf(g[e], x[e], dot);
    }
    dot = kv_row_sum<L>(dot) * (1.f / D);
#pragma unroll
    for (int e = 0; e < 16; ++e) g[e] = r * (g[e] - x[e] * dot);
    stg<u32x4>(o + 16 * i, kv_round8<T>(g));
    stg<u32x4>(o + 16 * (i + L), kv_round8<T>(g + 8));
  }
  // the block's sum: rows of a wave, then waves
  __shared__ __attribute__((aligned(16))) float sw[4][D];
#pragma unroll
  for (int e = 0; e < 16; ++e)
#pragma unroll
    for (int m = L; m < 64; m *= 2) dw[e] += __shfl_xor(dw[e], m, 64);
  if (lane < L) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) sw[wave][8 * (i + c * L) + e] = dw[8 * c + e];
  }
  __syncthreads();
  if ((int)threadIdx.x < D) {
    const float v = (sw[0][threadIdx.x] + sw[1][threadIdx.x]) + (sw[2][threadIdx.x] + sw[3][threadIdx.x]);
    float* to = a.part ? a.part + (int64_t)blockIdx.x * D : s.dw + cls * D;
    to[threadIdx.x] = v;
  }
}

// 16 columns of one weight vector's partial sums.
__global__ __launch_bounds__(1024) void k_qk_norm_join(const QkArgs a, int dim) {
  __shared__ float sw[64][17];
  const int pieces = dim / 16, cls = blockIdx.x / pieces, col = blockIdx.x % pieces * 16 + (threadIdx.x & 15), r = threadIdx.x >> 4;
  const bool is_q = cls < a.q.classes;
  const QkSide& s = is_q ? a.q : a.k;
  const int c = is_q ? cls : cls - a.q.classes;
  const float* p = a.part + ((int64_t)(is_q ? 0 : a.q.classes * a.q.blocks) + (int64_t)c * s.blocks) * dim + col;
  float v = 0.f;
  for (int b0 = r; b0 < s.blocks; b0 += 64 * 8) {
    float part[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) part[k] = p[(int64_t)min(b0 + 64 * k, s.blocks - 1) * dim];  // under way together
#pragma unroll
    for (int k = 0; k < 8; ++k) v += b0 + 64 * k < s.blocks ? part[k] : 0.f;
  }
  sw[r][threadIdx.x & 15] = v;
  __syncthreads();
  for (int m = 32; m; m >>= 1) {
    if (r < m) sw[r][threadIdx.x & 15] += sw[r + m][threadIdx.x & 15];
    __syncthreads();
  }
  if (r == 0) s.dw[(int64_t)c * dim + col] = sw[0][threadIdx.x & 15];
}

}  // namespace

// How many blocks walk the rows of a class: q.blocks and k.blocks of `a`; returns the partial sums to be kept (0: none).
int64_t qk_norm_split(QkArgs& a, int dim, int cus) {
  const int64_t rb = 256 / (dim / 16), all = std::max<int64_t>(1, a.tokens * (a.q.heads + a.k.heads));
  auto blocks = [&](QkSide& s) {
    if (!s.heads) {
      s.blocks = 0;
      return;
    }
    const int64_t rows = a.tokens * s.heads, need = (rows / s.classes + rb - 1) / rb;
    // a few turns of one block cost less than the joining kernel's launch (333 tokens, 2 x 24 heads of 64 with a weight
    // each: 6 turns 9.7 us, against 6.2 and 3.0)
    if (need <= 6) {
      s.blocks = 1;
      return;
    }
    const int64_t share = (4 * (int64_t)cus * rows / all + s.classes - 1) / s.classes;
    s.blocks = (int)std::max<int64_t>(1, std::min(need, share));
  };
  blocks(a.q);
  blocks(a.k);
  if (a.q.blocks <= 1 && a.k.blocks <= 1) return 0;
  return (int64_t)a.q.classes * a.q.blocks + (int64_t)a.k.classes * a.k.blocks;
}

static KvDiv kv_div_by(uint32_t d) {
  int l = 0;
  while ((1ull << l) < d) ++l;
  if (l == 0) return {0, 1, 0};
  // 2^(31 + l) / d rounded up is off by at most d 2^-(31 + l) of a quotient, less than 1 / d for n < 2^31
  return {(uint32_t)((1ull << (31 + l)) / d + 1), d, l - 1};
}

template <int D, int T, bool INT4>
static void forward_launch(const QkForwardArgs& a, dim3 grid, hipStream_t s) {
  switch (kv_way(a.turn, D)) {
    case KV_STILL: hipLaunchKernelGGL((k_qk_norm<D, T, INT4, KV_STILL>), grid, dim3(256), 0, s, a); break;
    case KV_HALVES: hipLaunchKernelGGL((k_qk_norm<D, T, INT4, KV_HALVES>), grid, dim3(256), 0, s, a); break;
    case KV_PAIRS: hipLaunchKernelGGL((k_qk_norm<D, T, INT4, KV_PAIRS>), grid, dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL((k_qk_norm<D, T, INT4, KV_PART>), grid, dim3(256), 0, s, a);
  }
}

// a: rows, divisions and blocks are set here
hipError_t launch_qk_norm(const QkForwardArgs& args, const int (&heads)[3], int64_t tokens, int dim, int dt, bool int4,
                          hipStream_t s) {
  const int64_t rb = 256 / (dim / 16), per = (int64_t)heads[0] + heads[1] + heads[2];
  const int64_t most = ((int64_t(1) << 31) - 1) / (per * (dim / 16));  // rows stay below 2^31, and so do threads
  for (int64_t t = 0; t < tokens; t += most) {
    const int64_t n = std::min(most, tokens - t);
    QkForwardArgs a = args;
    int64_t blocks = 0;
    for (int k = 0; k < 3; ++k) {
      QkForward& f = a.f[k];
      f.rows = (uint32_t)(n * heads[k]);
      f.blocks = (uint32_t)((n * heads[k] + rb - 1) / rb);
      f.heads = kv_div_by(std::max(heads[k], 1));
      f.in.p += t * f.in.tok;
      if (f.out.p) f.out.p += t * f.out.tok;
      blocks += f.blocks;
    }
    if (a.turn.pos) a.turn.pos += t;
    if (a.slots) a.slots += t;
    const dim3 grid((unsigned)blocks);
    KV_PICK(forward_launch, dim, dt, int4, a, grid, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int D, int T>
static void back_launch(const QkArgs& a, dim3 grid, hipStream_t s) {
  switch (kv_way(a.turn, D)) {
    case KV_STILL: hipLaunchKernelGGL((k_qk_norm_back<D, T, KV_STILL>), grid, dim3(256), 0, s, a); break;
    case KV_HALVES: hipLaunchKernelGGL((k_qk_norm_back<D, T, KV_HALVES>), grid, dim3(256), 0, s, a); break;
    case KV_PAIRS: hipLaunchKernelGGL((k_qk_norm_back<D, T, KV_PAIRS>), grid, dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL((k_qk_norm_back<D, T, KV_PART>), grid, dim3(256), 0, s, a);
  }
}

hipError_t launch_qk_norm_back(const QkArgs& a, int dim, int dt, hipStream_t s) {
  const dim3 grid((unsigned)(a.q.classes * a.q.blocks + a.k.classes * a.k.blocks));
  if (dim == 128) dt == KV_BF16 ? back_launch<128, KV_BF16>(a, grid, s) : back_launch<128, KV_F16>(a, grid, s);
  else dt == KV_BF16 ? back_launch<64, KV_BF16>(a, grid, s) : back_launch<64, KV_F16>(a, grid, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  hipLaunchKernelGGL(k_qk_norm_join, dim3((unsigned)((a.q.classes + a.k.classes) * (dim / 16))), dim3(1024), 0, s, a, dim);
  return hipGetLastError();
}

}  // namespace whtq
