// token_logprobs and token_logprobs_backward: rows of logits to the log
// probabilities of given tokens, the entropy and the likeliest tokens, and
// the gradient of the logits.
//
// With z = scale x, m a value near the row's largest, S = sum e^(z - m) and
// T = sum e^(z - m) (z - m):
//   lse = m + log S,  logprob = (z_t - m) - log S,  entropy = log S - T / S,
// every term of the entropy of one sign.  Each lane keeps (m, S, T) of its
// own logits over one pass; m may lag behind the largest by 2^LP_LAG, so
// that S and T are rescaled a few times in a row and not for every vector.
//
// The likeliest tokens cost that pass one maximum over a group of logits
// (kept in memory, 4 bytes for 512 logits of a long row): the k largest, ties
// to the lower index, lie in the k groups whose maxima are the largest, ties
// to the lower group, because any other logit has k such maxima before it.
// The last kernel of a row picks those groups and reads only them again.
//
// What bounds both directions is memory.  Rows need no alignment beyond their
// elements': loads of 16 bytes are given their true alignment, and the last
// few logits of a row are loaded one by one.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "common.hpp"
#include "io.hpp"
#include "launch.hpp"
#include "logprob.hpp"

namespace whtq {

namespace {

constexpr float LP_NEG_INF = -__builtin_huge_valf();
constexpr float LP_LOG2E = 1.4426950408889634f, LP_LN2 = 0.6931471805599453f;
constexpr float LP_LAG = 6.f;
constexpr float LP_LEAST = -1e4f;  // 2^LP_LEAST is 0, and 0 times it is

template <int DT>
constexpr int LP_BYTES = DT == DT_F32 ? 4 : 2;

typedef u32x4 u32x4_by4 __attribute__((aligned(4)));
typedef u32x4 u32x4_by2 __attribute__((aligned(2)));

struct Lp8 {  // eight logits as loaded
  u32x4 w[2];
};
// Logits i .. i + 7 of a row; what lies behind its end is -inf.
template <int DT>
__device__ __forceinline__ void lp_load(const uint8_t* row, int i, int vocab, Lp8& r) {
  const uint8_t* p = row + (int64_t)i * LP_BYTES<DT>;
  if (i + 8 <= vocab) {
    if constexpr (DT == DT_F32) {
      r.w[0] = *reinterpret_cast<const u32x4_by4*>(p);
      r.w[1] = *reinterpret_cast<const u32x4_by4*>(p + 16);
    } else {
      r.w[0] = *reinterpret_cast<const u32x4_by2*>(p);
    }
    return;
  }
  constexpr uint32_t NONE = DT == DT_BF16 ? 0xff80u : 0xfc00u;
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.w[e >> 2][e & 3] = i + e < vocab ? reinterpret_cast<const uint32_t*>(p)[e] : 0xff800000u;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = i + 2 * e < vocab ? reinterpret_cast<const uint16_t*>(p)[2 * e] : NONE;
      const uint32_t hi = i + 2 * e + 1 < vocab ? reinterpret_cast<const uint16_t*>(p)[2 * e + 1] : NONE;
      r.w[0][e] = lo | hi << 16;
    }
  }
}
template <int DT>
__device__ __forceinline__ void lp_widen(const Lp8& r, float* f) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (DT == DT_F32) {
      const uint32_t x = r.w[e >> 2][e & 3];
      f[e] = as_f(x);
    } else {
      const uint32_t x = r.w[0][e >> 1];
      f[e] = widen16(x, e & 1, DT);
    }
  }
}
template <int DT>
__device__ __forceinline__ float lp_one(const uint8_t* row, int64_t i) {
  if constexpr (DT == DT_F32) return reinterpret_cast<const float*>(row)[i];
  else return widen16(reinterpret_cast<const uint16_t*>(row)[i], false, DT);
}

// Whole numbers in the order of the floats, above 0; -0 counts as 0.
__device__ __forceinline__ uint32_t lp_key(float x) {
  const uint32_t u = as_u(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float lp_value(uint32_t k) { return as_f(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// (m, S, T) of some logits; T in units of log 2.
struct LpSum {
  float m, s, t;
};
__device__ __forceinline__ LpSum lp_add(const LpSum& a, const LpSum& b, float c) {
  const float m = fmaxf(a.m, b.m);
  auto to = [&](const LpSum& x, float& s, float& t) {
    // of no logit above -inf the sums are 0, or NaN, which stays
    const bool none = x.m == LP_NEG_INF;
    const float d = none ? 0.f : fmaxf((x.m - m) * c, LP_LEAST), f = none ? 0.f : __builtin_amdgcn_exp2f(d);
    s = f * x.s;
    t = f * (x.t + d * x.s);
  };
  float sa, ta, sb, tb;
  to(a, sa, ta);
  to(b, sb, tb);
  return {m, sa + sb, ta + tb};
}
template <int N>  // over N lanes side by side
__device__ __forceinline__ LpSum lp_lanes(LpSum a, float c) {
#pragma unroll
  for (int x = 1; x < N; x *= 2) a = lp_add(a, {__shfl_xor(a.m, x, 64), __shfl_xor(a.s, x, 64), __shfl_xor(a.t, x, 64)}, c);
  return a;
}

// A row's outputs, by one thread.
template <int DT>
__device__ __forceinline__ void lp_finish(const LpArgs& a, int64_t row, const LpSum& r) {
  const bool none = r.s == 0.f;
  const float ls = logf(r.s);
  // lse as the sum of two floats: the gradient's exponent needs more than one where logits are large
  const double lse = none ? (double)LP_NEG_INF : (double)r.m * (double)a.scale + (double)ls;
  const float hi = (float)lse;
  if (a.lse) a.lse[row] = hi;
  if (a.lse_low) a.lse_low[row] = fabsf(hi) < __builtin_huge_valf() ? (float)(lse - (double)hi) : 0.f;
  if (a.entropy) a.entropy[row] = none ? 0.f : ls - r.t / r.s * LP_LN2;
  if (a.targets && a.logprob) {
    const int64_t t = a.targets[row];
    float lp = 0.f;
    if (t >= 0 && t < a.vocab) lp = none ? LP_NEG_INF : (lp_one<DT>(a.x + row * a.ld, t) - r.m) * a.scale - ls;
    a.logprob[row] = lp;
  }
}

// A block's share of a row: chunks c, c + 4, .. by each of its waves.
// TOP: the maxima of groups of LANES lanes' logits are kept.
template <int DT, int LANES>
__global__ __launch_bounds__(256) void k_lp_row(const LpArgs a) {
  constexpr int AHEAD = DT == DT_F32 ? 2 : 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % (uint32_t)a.splits;
  const int64_t row = a.row0 + blockIdx.x / (uint32_t)a.splits;
  const int chunks = (a.vocab + LP_CHUNK - 1) / LP_CHUNK;
  const int c0 = (int)((int64_t)chunks * split / a.splits), c1 = (int)((int64_t)chunks * (split + 1) / a.splits);
  const uint8_t* x = a.x + row * a.ld;
  const float c = a.scale * LP_LOG2E, lag = fminf(LP_LAG / c, 1e30f);
  LpSum r{LP_NEG_INF, 0.f, 0.f};
  Lp8 buf[AHEAD];
  auto take = [&](const Lp8& w, int ch) {
    float f[8];
    lp_widen<DT>(w, f);
    float top = fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));
    if constexpr (LANES > 0) {
      uint32_t k = lp_key(top == top ? top : LP_NEG_INF);  // (a NaN counts as -inf in the order)
      if constexpr (LANES == 64) {
        k = wave_max_u32(k);
        if (lane == 0) a.best[row * a.groups + ch] = k;
      } else {
#pragma unroll
        for (int m = 1; m < LANES; m *= 2) k = max(k, (uint32_t)__shfl_xor((int)k, m, 64));
        const int g = (ch * 64 + lane) / LANES;
        if (lane % LANES == 0 && g < a.groups) a.best[row * a.groups + g] = k;
      }
    }
    if (__any(top > r.m + lag)) {
      const float m = fmaxf(r.m, top);
      if (r.m == LP_NEG_INF) {
        r.m = m;
      } else if (m > r.m) {
        const float d = fmaxf((r.m - m) * c, LP_LEAST), f2 = __builtin_amdgcn_exp2f(d);
        r.t = f2 * (r.t + d * r.s);
        r.s *= f2;
        r.m = m;
      }
    }
    const float base = r.m == LP_NEG_INF ? 0.f : r.m;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float z = (f[e] - base) * c, p = __builtin_amdgcn_exp2f(z);
      r.s += p;
      r.t += p * fmaxf(z, LP_LEAST);
    }
  };
  int ch = c0 + wave;
#pragma unroll
  for (int u = 0; u < AHEAD; ++u)
    if (ch + 4 * u < c1) lp_load<DT>(x, (ch + 4 * u) * LP_CHUNK + 8 * lane, a.vocab, buf[u]);
  while (ch < c1) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (ch + 4 * u < c1) {
        take(buf[u], ch + 4 * u);
        const int next = ch + 4 * (u + AHEAD);
        if (next < c1) lp_load<DT>(x, next * LP_CHUNK + 8 * lane, a.vocab, buf[u]);
      }
    ch += 4 * AHEAD;
  }
  r = lp_lanes<64>(r, c);
  __shared__ LpSum sw[4];
  if (lane == 0) sw[wave] = r;
  __syncthreads();
  if (threadIdx.x == 0) {
    r = lp_add(lp_add(sw[0], sw[1], c), lp_add(sw[2], sw[3], c), c);
    if (a.splits == 1) {
      lp_finish<DT>(a, row, r);
    }
    if (a.splits > 1 || LANES > 0) {
      float* p = a.part + (row * a.splits + split) * 3;
      p[0] = r.m;
      p[1] = r.s;
      p[2] = r.t;
    }
  }
}

// Joins a row's shares, a wave a row.
template <int DT>
__global__ __launch_bounds__(256) void k_lp_join(const LpArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = a.row0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.rows) return;
  const float c = a.scale * LP_LOG2E;
  LpSum r{LP_NEG_INF, 0.f, 0.f};
  for (int s = lane; s < a.splits; s += 64) {
    const float* p = a.part + (row * a.splits + s) * 3;
    r = lp_add(r, {p[0], p[1], p[2]}, c);
  }
  r = lp_lanes<64>(r, c);
  if (lane == 0) lp_finish<DT>(a, row, r);
}

// The same for a row whose likeliest tokens are asked for, a block a row.
template <int DT>
__global__ __launch_bounds__(256) void k_lp_top(const LpArgs a) {
  constexpr int CAP = 256;  // candidates ranked at once
  __shared__ uint32_t key[LP_MOST_VOCAB / LP_CHUNK];
  __shared__ int pick[LP_MOST_TOP];
  __shared__ uint64_t cand[CAP], sbest[4];
  __shared__ uint32_t bar;
  __shared__ int count;
  __shared__ float sm, sls;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = a.row0 + blockIdx.x;
  const uint8_t* x = a.x + row * a.ld;
  const int n = min(a.top, a.groups);
  for (int i = threadIdx.x; i < a.groups; i += 256) key[i] = a.best[row * a.groups + i];
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  if (wave == 0) {
    // the n groups of largest maxima, one after another: lane i watches over its own run of groups
    const int per = (a.groups + 63) / 64, g0 = min(lane * per, a.groups), g1 = min(g0 + per, a.groups);
    uint32_t k = 0;
    int at = g0;
    auto look = [&] {
      k = 0;
      for (int g = g0; g < g1; ++g)
        if (key[g] > k) k = key[g], at = g;
    };
    look();
    for (int i = 0; i < n; ++i) {
      const uint32_t top = wave_max_u32(k);
      const int l = __builtin_ctzll(__ballot(k == top));
      if (lane == l) {
        pick[i] = at;
        key[at] = 0;
        look();
        if (i == n - 1) bar = n == a.top ? top : 0u;
      }
    }
  } else if (wave == 1) {
    const float c = a.scale * LP_LOG2E;
    LpSum r{LP_NEG_INF, 0.f, 0.f};
    for (int s = lane; s < a.splits; s += 64) {
      const float* p = a.part + (row * a.splits + s) * 3;
      r = lp_add(r, {p[0], p[1], p[2]}, c);
    }
    r = lp_lanes<64>(r, c);
    if (lane == 0) {
      if (a.splits > 1) lp_finish<DT>(a, row, r);
      sm = r.s == 0.f ? 0.f : r.m;
      sls = r.s == 0.f ? 0.f : logf(r.s);
    }
  }
  __syncthreads();
  // candidates: logits of those groups that reach the last one's maximum.
  // (value, index) as one number, larger first and the lower index first
  const int vecs = a.width / 8;
  auto each = [&](auto f) {
    for (int v = threadIdx.x; v < n * vecs; v += 256) {
      const int i = pick[v / vecs] * a.width + v % vecs * 8;
      if (i >= a.vocab) continue;
      Lp8 w;
      float y[8];
      lp_load<DT>(x, i, a.vocab, w);
      lp_widen<DT>(w, y);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < a.vocab) {
          const float z = y[e] == y[e] ? y[e] : LP_NEG_INF;
          f((uint64_t)lp_key(z) << 32 | ~(uint32_t)(i + e));
        }
    }
  };
  const uint64_t least = (uint64_t)bar << 32;
  each([&](uint64_t q) {
    if (q >= least) {
      const int at = atomicAdd(&count, 1);
      if (at < CAP) cand[at] = q;
    }
  });
  __syncthreads();
  auto put = [&](int i, uint64_t q) {
    const uint32_t id = ~(uint32_t)q;
    a.top_id[row * a.top + i] = id;
    a.top_logprob[row * a.top + i] = (lp_one<DT>(x, id) - sm) * a.scale - sls;
  };
  const int have = count;
  if (have <= CAP) {
    if ((int)threadIdx.x < have) {
      const uint64_t q = cand[threadIdx.x];
      int rank = 0;
      for (int i = 0; i < have; ++i) rank += cand[i] > q;
      if (rank < a.top) put(rank, q);
    }
    return;
  }
  // more than that are tied: one after another
  uint64_t last = ~0ull;
  for (int i = 0; i < a.top; ++i) {
    uint64_t q = 0;
    each([&](uint64_t p) { q = p < last && p > q ? p : q; });
#pragma unroll
    for (int m = 1; m < 64; m *= 2) q = max(q, (uint64_t)__shfl_xor((unsigned long long)q, m, 64));
    if (lane == 0) sbest[wave] = q;
    __syncthreads();
    last = max(max(sbest[0], sbest[1]), max(sbest[2], sbest[3]));
    if (threadIdx.x == 0) put(i, last);
    __syncthreads();
  }
}

// d logits = scale (g (onehot - p) - h p (log p + H)).
template <int DT>
__global__ __launch_bounds__(256) void k_lp_grad(const LpGradArgs a) {
  constexpr int U = 4;
  const int64_t row = a.row0 + blockIdx.x / (uint32_t)a.pieces;
  const int piece = blockIdx.x % (uint32_t)a.pieces;
  const uint8_t* x = a.x + row * a.ld;
  uint8_t* dx = a.dx + row * a.ldd;
  const int64_t t = a.targets ? a.targets[row] : -1;
  const bool given = t >= 0 && t < a.vocab;
  const float lse = a.lse[row], low = a.lse_low ? a.lse_low[row] : 0.f;
  const float g = given && a.dlogprob ? a.dlogprob[row] * a.scale : 0.f;
  const float h = a.dentropy ? a.dentropy[row] * a.scale : 0.f, ent = a.dentropy ? a.entropy[row] : 0.f;
  const bool none = lse == LP_NEG_INF;
  const int i0 = (piece * U * 256 + (int)threadIdx.x) * 8;
  Lp8 w[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (i0 + 2048 * u < a.vocab) lp_load<DT>(x, i0 + 2048 * u, a.vocab, w[u]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = i0 + 2048 * u;
    if (i >= a.vocab) break;
    float f[8];
    lp_widen<DT>(w[u], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float lp = __builtin_fmaf(f[e], a.scale, -lse) - low;
      const float p = __builtin_amdgcn_exp2f(lp * LP_LOG2E);
      float d = -p * (g + h * (fmaxf(lp, LP_LEAST) + ent));
      if (i + e == t) d += g;
      f[e] = none ? 0.f : d;
    }
    uint8_t* o = dx + (int64_t)i * LP_BYTES<DT>;
    if constexpr (DT == DT_F32) {
      if (i + 8 <= a.vocab) {
        *reinterpret_cast<u32x4_by4*>(o) = u32x4{as_u(f[0]), as_u(f[1]), as_u(f[2]), as_u(f[3])};
        *reinterpret_cast<u32x4_by4*>(o + 16) = u32x4{as_u(f[4]), as_u(f[5]), as_u(f[6]), as_u(f[7])};
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i + e < a.vocab) reinterpret_cast<float*>(o)[e] = f[e];
      }
    } else {
      u32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = DT == DT_BF16 ? pack_bf16(f[2 * q], f[2 * q + 1]) : pack_f16(f[2 * q], f[2 * q + 1]);
      if (i + 8 <= a.vocab) {
        *reinterpret_cast<u32x4_by2*>(o) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t y = v[e >> 1];
          if (i + e < a.vocab) reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(e & 1 ? y >> 16 : y & 0xffffu);
        }
      }
    }
  }
}

template <int DT>
hipError_t rows_launch(LpArgs a, hipStream_t s) {
  const int64_t most = kLaunchThreads / 256 / std::max(a.splits, 1);
  for (a.row0 = 0; a.row0 < a.rows; a.row0 += most) {
    const int64_t n = std::min(a.rows - a.row0, most);
    const dim3 grid((unsigned)(n * a.splits));
    if (!a.top) hipLaunchKernelGGL((k_lp_row<DT, 0>), grid, dim3(256), 0, s, a);
    else if (a.width == 8) hipLaunchKernelGGL((k_lp_row<DT, 1>), grid, dim3(256), 0, s, a);
    else if (a.width == 64) hipLaunchKernelGGL((k_lp_row<DT, 8>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_lp_row<DT, 64>), grid, dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.top) {
      hipLaunchKernelGGL((k_lp_top<DT>), dim3((unsigned)n), dim3(256), 0, s, a);
    } else if (a.splits > 1) {
      LpArgs b = a;
      b.rows = a.row0 + n;
      hipLaunchKernelGGL((k_lp_join<DT>), dim3((unsigned)((n + 3) / 4)), dim3(256), 0, s, b);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <int DT>
hipError_t grad_launch(LpGradArgs a, hipStream_t s) {
  a.pieces = (a.vocab + 8191) / 8192;
  const int64_t most = kLaunchThreads / 256 / a.pieces;
  for (a.row0 = 0; a.row0 < a.rows; a.row0 += most) {
    hipLaunchKernelGGL((k_lp_grad<DT>), dim3((unsigned)(std::min(a.rows - a.row0, most) * a.pieces)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_lp(const LpArgs& a, int dt, hipStream_t s) {
  return dt == DT_F32 ? rows_launch<DT_F32>(a, s) : dt == DT_BF16 ? rows_launch<DT_BF16>(a, s) : rows_launch<DT_F16>(a, s);
}
hipError_t launch_lp_grad(const LpGradArgs& a, int dt, hipStream_t s) {
  return dt == DT_F32 ? grad_launch<DT_F32>(a, s) : dt == DT_BF16 ? grad_launch<DT_BF16>(a, s) : grad_launch<DT_F16>(a, s);
}

}  // namespace whtq
