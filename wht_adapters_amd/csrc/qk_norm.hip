// qk_norm_rope and its backward pass: norms of each head's queries and keys
// and their rotary positions on dense rows.
//
//   r = (mean x^2 + eps)^-1/2,  y = R (w o x r)
// and with g = R^T dy (the opposite rotation), u = w o g:
//   dw = sum g o x r  over tokens (and heads that share w),
//   dx = r (u - x r^2 mean(u o x)).
// The backward pass takes x again and computes r itself: two numbers a row
// less to keep, and x has to be read anyway.
//
// Both directions move bytes.  A row belongs to D / 16 lanes as in kv_append.
// Backward, a block walks rows of one weight vector, so that a lane's part of
// dw stays in registers; blocks leave one partial sum each, which a second
// kernel adds in a fixed order (no atomics: the same result every time).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "qk_norm.hpp"

namespace whtq {

namespace {

template <int D, int T>
__global__ __launch_bounds__(256) void k_qk_norm(const QkArgs a, uint32_t rows) {
  constexpr int L = D / 16, RB = 256 / L;
  const uint32_t n = blockIdx.x * RB + threadIdx.x / L;
  const int i = threadIdx.x % L;
  const uint32_t per = a.q.heads + a.k.heads;
  const bool live = n < rows;
  const uint32_t t = live ? n / per : 0, hs = live ? n % per : 0;
  const bool is_q = hs < (uint32_t)a.q.heads;
  const QkSide& s = is_q ? a.q : a.k;
  const int h = is_q ? hs : hs - a.q.heads;
  const uint8_t* row = s.x.p + t * s.x.tok + h * s.x.head;
  const uint8_t* w = s.w.p + h * s.w.head;
  const int64_t pos = a.turn.pos ? (int64_t)a.turn.pos[t] : 0;
  float x[16];
  kv_widen8<T>(ldg<u32x4>(row + 16 * i), x);
  kv_widen8<T>(ldg<u32x4>(row + 16 * (i + L)), x + 8);
  const float r = kv_norm<D>(x, w, a.dt, a.eps, i);
  if (!live) return;
  if (a.turn.pos) {
    if (pos < 0 || pos >= a.turn.max_pos) return;
    kv_rotate<D>(x, a.turn, pos, i, [&](int ch, float* o) {
      kv_widen8<T>(ldg<u32x4>(row + 16 * ch), o);
      kv_weigh8(o, w, a.dt, ch, r);
    });
  }
  uint8_t* o = const_cast<uint8_t*>(s.y.p) + t * s.y.tok + h * s.y.head;
  stg<u32x4>(o + 16 * i, kv_round8<T>(x));
  stg<u32x4>(o + 16 * (i + L), kv_round8<T>(x + 8));
}

template <int D, int T>
__global__ __launch_bounds__(256) void k_qk_norm_back(const QkArgs a) {
  constexpr int L = D / 16, RB = 256 / L;
  const int i = threadIdx.x % L, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int qb = a.q.classes * a.q.blocks;
  const bool is_q = (int)blockIdx.x < qb;
  const QkSide& s = is_q ? a.q : a.k;
  const int b = is_q ? blockIdx.x : blockIdx.x - qb, cls = b / s.blocks, slot = b % s.blocks;
  const uint32_t per = s.classes == 1 ? s.heads : 1;  // heads of a token in this class
  const int64_t rows = a.tokens * per;
  float w[16], dw[16];
  const uint8_t* wp = s.w.p + cls * s.w.head;
  kv_weight8(wp, a.dt, i, w);
  kv_weight8(wp, a.dt, i + L, w + 8);
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.f;
  for (int64_t n = (int64_t)slot * RB + threadIdx.x / L; n < rows; n += (int64_t)s.blocks * RB) {
    const int64_t t = n >> 31 ? n / per : (uint32_t)n / per;
    const int h = per == 1 ? cls : (int)(n - t * per);
    const int64_t pos = a.turn.pos ? (int64_t)a.turn.pos[t] : 0;
    if (a.turn.pos && (pos < 0 || pos >= a.turn.max_pos)) continue;
    const uint8_t* xp = s.x.p + t * s.x.tok + h * s.x.head;
    const uint8_t* dp = s.dy.p + t * s.dy.tok + h * s.dy.head;
    float x[16], g[16];
    kv_widen8<T>(ldg<u32x4>(xp + 16 * i), x);
    kv_widen8<T>(ldg<u32x4>(xp + 16 * (i + L)), x + 8);
    kv_widen8<T>(ldg<u32x4>(dp + 16 * i), g);
    kv_widen8<T>(ldg<u32x4>(dp + 16 * (i + L)), g + 8);
    const float r = kv_rms<D>(x, a.eps);
    if (a.turn.pos)
      kv_rotate<D, true>(g, a.turn, pos, i, [&](int ch, float* o) { kv_widen8<T>(ldg<u32x4>(dp + 16 * ch), o); });
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      dw[e] = __builtin_fmaf(g[e], x[e] * r, dw[e]);
      g[e] *= w[e];
      dot = __builtin_fmaf(g[e], x[e], dot);
    }
    dot = kv_row_sum<L>(dot) * (1.f / D) * r * r;
#pragma unroll
    for (int e = 0; e < 16; ++e) g[e] = r * (g[e] - x[e] * dot);
    uint8_t* o = const_cast<uint8_t*>(s.dx.p) + t * s.dx.tok + h * s.dx.head;
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
  for (int b = r; b < s.blocks; b += 64) v += p[(int64_t)b * dim];
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
    const int64_t share = (4 * (int64_t)cus * rows / all + s.classes - 1) / s.classes;
    s.blocks = (int)std::max<int64_t>(1, std::min(need, share));
  };
  blocks(a.q);
  blocks(a.k);
  if (a.q.blocks <= 1 && a.k.blocks <= 1) return 0;
  return (int64_t)a.q.classes * a.q.blocks + (int64_t)a.k.classes * a.k.blocks;
}

hipError_t launch_qk_norm(QkArgs a, int dim, int dt, hipStream_t s) {
  const int lanes = dim / 16, rb = 256 / lanes;
  const int64_t per = a.q.heads + a.k.heads, most = kLaunchThreads / (per * lanes), tokens = a.tokens;
  for (int64_t t = 0; t < tokens; t += most) {
    const int64_t n = std::min(most, tokens - t);
    const dim3 grid((unsigned)((n * per + rb - 1) / rb));
    QkArgs b = a;
    for (QkSide* x : {&b.q, &b.k}) {
      x->x.p += t * x->x.tok;
      x->y.p += t * x->y.tok;
    }
    if (b.turn.pos) b.turn.pos += t;
    const uint32_t rows = (uint32_t)(n * per);
    if (dim == 128 && dt == KV_BF16) hipLaunchKernelGGL((k_qk_norm<128, KV_BF16>), grid, dim3(256), 0, s, b, rows);
    else if (dim == 128) hipLaunchKernelGGL((k_qk_norm<128, KV_F16>), grid, dim3(256), 0, s, b, rows);
    else if (dt == KV_BF16) hipLaunchKernelGGL((k_qk_norm<64, KV_BF16>), grid, dim3(256), 0, s, b, rows);
    else hipLaunchKernelGGL((k_qk_norm<64, KV_F16>), grid, dim3(256), 0, s, b, rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_qk_norm_back(const QkArgs& a, int dim, int dt, hipStream_t s) {
  const dim3 grid((unsigned)(a.q.classes * a.q.blocks + a.k.classes * a.k.blocks));
  if (dim == 128 && dt == KV_BF16) hipLaunchKernelGGL((k_qk_norm_back<128, KV_BF16>), grid, dim3(256), 0, s, a);
  else if (dim == 128) hipLaunchKernelGGL((k_qk_norm_back<128, KV_F16>), grid, dim3(256), 0, s, a);
  else if (dt == KV_BF16) hipLaunchKernelGGL((k_qk_norm_back<64, KV_BF16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_qk_norm_back<64, KV_F16>), grid, dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  hipLaunchKernelGGL(k_qk_norm_join, dim3((unsigned)((a.q.classes + a.k.classes) * (dim / 16))), dim3(1024), 0, s, a, dim);
  return hipGetLastError();
}

}  // namespace whtq
