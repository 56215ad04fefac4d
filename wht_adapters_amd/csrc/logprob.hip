// token_logprobs and token_logprobs_backward: rows of logits to the log
// probabilities of given tokens, the entropy and the likeliest tokens, and
// the gradient of the logits.
//
// With z = scale x, m a logit near the row's largest, S = sum e^(z - scale m)
// and T = sum e^(z - scale m) (z - scale m):
//   lse = scale m + log S,  logprob = scale (x_t - m) - log S,
//   entropy = log S - T / S.
// Each lane keeps (m, S, T) of its own logits over one pass; m may lag behind
// the largest by LP_LAG, so that S and T are rescaled a few times in a row and
// not for every vector.  Terms above m are positive then, and what log S and
// T / S have in common, LP_LAG log 2 = 4.2 at most, cancels: a few 2^-24 times
// that of lse, logprob and entropy.  m is a logit of the row and keeps 1.5 % of
// the largest's weight, so that an entropy near 0 is only ever taken from the
// largest itself.  Exponents are differences of logits times a factor
// and never products that could overflow: rows masked with the type's lowest
// value, even all of a row, come out right.  The gradient takes m and S again
// rather than lse, whose rounding would be an error of every p.
//
// The likeliest tokens cost that pass one maximum over a group of logits
// (kept in memory, 4 bytes for 512 logits of a long row): the k largest, ties
// to the lower index, lie in the k groups whose maxima are the largest, ties
// to the lower group, because any other logit has k such maxima before it.
// The last kernel of a row picks those groups and reads only them again.
//
// What bounds both directions is memory.  Rows need no alignment beyond their
// elements': a row is taken by the aligned 16 bytes it lies in, and the few
// logits at its two ends are loaded one by one.
//
// Measured (kernel times, bf16): 2047 rows of 100003, five tokens: 410 MB in
// 80 to 85 us, 4.8 to 5.1 TB/s (a large copy moves 4.9), with the vector pipes
// 80 % busy (10 instructions a logit); 110 us before loads came streamed (past
// the caches) and without a branch between them and their use.  Forward and
// gradient of 8192 rows of 32000: 524 MB in 98 to 110 us (vector pipes 90 %)
// and 1049 MB in 180 us, 5.8 TB/s.  One row of
// 131072, 20 tokens: 4.8 us and 5.9 us for the likeliest, all latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

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
// A row by the aligned 16 bytes that hold it: logit i stands at place i + pad,
// places [pad, end) are the row's.
struct LpRow {
  const uint8_t* p;
  int pad, end;
};
template <int DT>
__device__ __forceinline__ LpRow lp_row(const uint8_t* x, int vocab) {
  const int off = (int)(reinterpret_cast<uintptr_t>(x) & 15u);
  return {x - off, off / LP_BYTES<DT>, vocab + off / LP_BYTES<DT>};
}
// Places i .. i + 7.  NT: read once, and not to be kept.
template <int DT, bool ALIGNED, bool NT>
__device__ __forceinline__ void lp_load8(const uint8_t* row, int i, Lp8& r) {
  const uint8_t* p = row + (int64_t)i * LP_BYTES<DT>;
  constexpr int N = DT == DT_F32 ? 2 : 1;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    using V = std::conditional_t<ALIGNED, u32x4, std::conditional_t<DT == DT_F32, u32x4_by4, u32x4_by2>>;
    const V* v = reinterpret_cast<const V*>(p) + k;
    if constexpr (NT) r.w[k] = __builtin_nontemporal_load(v);
    else r.w[k] = *v;
  }
}
// The same where some places may not be the row's: those give -inf.
template <int DT>
__device__ __forceinline__ void lp_load_edge(const LpRow& x, int i, Lp8& r) {
  if (i >= x.pad && i + 8 <= x.end) return lp_load8<DT, false, false>(x.p, i, r);
  const uint8_t* p = x.p + (int64_t)i * LP_BYTES<DT>;
  auto in = [&](int e) { return i + e >= x.pad && i + e < x.end; };
  constexpr uint32_t NONE = DT == DT_BF16 ? 0xff80u : 0xfc00u;
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.w[e >> 2][e & 3] = in(e) ? reinterpret_cast<const uint32_t*>(p)[e] : 0xff800000u;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = in(2 * e) ? reinterpret_cast<const uint16_t*>(p)[2 * e] : NONE;
      const uint32_t hi = in(2 * e + 1) ? reinterpret_cast<const uint16_t*>(p)[2 * e + 1] : NONE;
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

// The largest of eight (fmaxf would quiet each of them first, as many
// operations again).  A signalling NaN makes it NaN, other NaNs drop out.
__device__ __forceinline__ float lp_max8(const float* f) {
  float a, b;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(a) : "v"(f[0]), "v"(f[1]), "v"(f[2]));
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(b) : "v"(f[3]), "v"(f[4]), "v"(f[5]));
  asm("v_max3_f32 %0, %0, %1, %2" : "+v"(a) : "v"(f[6]), "v"(f[7]));
  asm("v_max_f32 %0, %0, %1" : "+v"(a) : "v"(b));
  return a;
}

// (m, S, T) of some logits; exponents are in units of log 2.
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
  if (a.lse) a.lse[row] = none ? LP_NEG_INF : (float)((double)r.m * (double)a.scale + (double)ls);
  if (a.ref) {
    a.ref[row] = none ? 0.f : r.m;
    a.sum[row] = r.s;
  }
  if (a.entropy) a.entropy[row] = none ? 0.f : ls - r.t / r.s * LP_LN2;
  if (a.targets && a.logprob) {
    const int64_t t = a.targets[row];
    float lp = 0.f;
    if (t >= 0 && t < a.vocab) lp = none ? LP_NEG_INF : (lp_one<DT>(a.x + row * a.ld, t) - r.m) * a.scale - ls;
    a.logprob[row] = lp;
  }
}

// A row's shares joined, by a wave.
__device__ __forceinline__ LpSum lp_shares(const LpArgs& a, int64_t row, int lane) {
  const float c = a.scale * LP_LOG2E;
  LpSum r{LP_NEG_INF, 0.f, 0.f};
  for (int s = lane; s < a.splits; s += 64) {
    const float* p = a.part + (row * a.splits + s) * 3;
    r = lp_add(r, {p[0], p[1], p[2]}, c);
  }
  return lp_lanes<64>(r, c);
}
template <int DT>
__global__ __launch_bounds__(256) void k_lp_join(const LpArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = a.row0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.rows) return;
  const LpSum r = lp_shares(a, row, lane);
  if (lane == 0) lp_finish<DT>(a, row, r);
}

// The n groups of largest maxima, ties to the lower group, by a wave; lane i
// holds PER groups side by side.  Bit by bit the largest number that n of the
// maxima reach: most of the time the count is n before the last bit, and the
// groups that reach it are the ones.  Returns a number that they reach and no
// other group exceeds.  A group may be several of those whose maxima were
// kept (`merge`).
template <int PER>
__device__ __forceinline__ uint32_t lp_pick(const uint32_t* best, int kept, int merge, int groups, int n, int lane, int* pick) {
  uint32_t key[PER];
  if (merge == 1) {
#pragma unroll
    for (int j = 0; j < PER; ++j) key[j] = best[min(lane * PER + j, groups - 1)];
#pragma unroll
    for (int j = 0; j < PER; ++j) key[j] = lane * PER + j < groups ? key[j] : 0u;
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int g = lane * PER + j;
      key[j] = 0;
      for (int k = g * merge; k < min((g + 1) * merge, kept); ++k) key[j] = max(key[j], best[k]);
    }
  }
  uint32_t bar = 0;
  int have = 0;
  for (uint32_t bit = 1u << 31; bit; bit >>= 1) {
    const uint32_t to = bar | bit;
    int c = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) c += __popcll(__ballot(key[j] >= to));
    if (c < n) continue;
    bar = to;
    have = c;
    if (c == n) break;
  }
  // (n groups are there, and their maxima are not 0: bar > 0)
  int spare = n, mine = 0;  // places for the last of equals; those of them before this lane's
  const uint64_t below = (1ull << lane) - 1;
  if (have > n) {
    int above = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      above += __popcll(__ballot(key[j] > bar));
      mine += __popcll(__ballot(key[j] == bar) & below);
    }
    spare = n - above;
  }
  int at = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool in = key[j] > bar || (key[j] == bar && (have == n || mine < spare));
    mine += key[j] == bar;
    const uint64_t m = __ballot(in);
    if (in) pick[at + __popcll(m & below)] = lane * PER + j;
    at += __popcll(m);
  }
  return bar;
}

// A row's likeliest tokens, by a block, from the maxima `best` of its groups.
// `sums` gives the row's sums, in one wave.
template <int DT, typename Sums>
__device__ __forceinline__ void lp_tops(const LpArgs& a, int64_t row, const LpRow& x, const uint32_t* best, Sums sums) {
  constexpr int CAP = 256, VECS = 128;  // candidates ranked at once, vectors that may hold any
  constexpr int MOST = 4;  // vectors of a thread under way (8 and fewer blocks a CU: 2047 rows 11.9 us against 9.4)
  __shared__ int pick[LP_MOST_TOP];
  __shared__ uint64_t cand[CAP], sbest[4];
  __shared__ __attribute__((aligned(16))) float vec[VECS][8];
  __shared__ int first[VECS], base[VECS];
  __shared__ uint32_t bar;
  __shared__ int vectors, count;
  __shared__ float sm, sls;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kept = (x.end + a.width - 1) / a.width;  // at most a.groups
  const int merge = kept <= 512 ? 1 : (kept + 511) / 512, groups = merge == 1 ? kept : (kept + merge - 1) / merge;
  const int n = min(a.top, groups);
  if (threadIdx.x == 0) vectors = count = 0;
  if (wave == 0) {
    const uint32_t reach = groups <= 64 ? lp_pick<1>(best, kept, merge, groups, n, lane, pick)
                          : groups <= 256 ? lp_pick<4>(best, kept, merge, groups, n, lane, pick)
                                          : lp_pick<8>(best, kept, merge, groups, n, lane, pick);
    if (lane == 0) bar = n == a.top ? reach : 0u;
  } else if (wave == 1) {
    const LpSum r = sums(lane);
    if (lane == 0) {
      lp_finish<DT>(a, row, r);
      sm = r.s == 0.f ? 0.f : r.m;
      sls = r.s == 0.f ? 0.f : logf(r.s);
    }
  }
  __syncthreads();
  // candidates: logits of those groups that reach `bar`; (value, index) as one
  // number, larger first and the lower index first
  const int shift = a.width == 8 ? 0 : a.width == 64 ? 3 : 6, all = n * merge << shift;
  auto at = [&](int v) {  // the first place of vector v
    const int u = v >> shift, in = v & ((1 << shift) - 1);
    return ((merge == 1 ? pick[u] : pick[u / merge] * merge + u % merge) << (shift + 3)) + 8 * in;
  };
  // vector v: its first place i, and the place from which 8 are loaded for it,
  // inside the row
  auto place = [&](int v, int& i, int& from) {
    i = v < all ? at(v) : x.end;
    from = max(min(i, x.end - 8), x.pad);
  };
  auto fetch = [&](Lp8& w, int from) __attribute__((always_inline)) {
    if (a.vocab < 8) lp_load_edge<DT>(x, from, w);
    else lp_load8<DT, false, false>(x.p, from, w);
  };
  const uint32_t least = bar;
  // 8 logits y from `from` on: f of the key and the token of those from i on
  auto one = [&](float y, int e, int i, int from, auto f) __attribute__((always_inline)) {
    const int id = from + e;
    if (id >= i && id < i + 8 && id < x.end) f(lp_key(y == y ? y : LP_NEG_INF), ~(uint32_t)(id - x.pad));
  };
  // vectors that may hold candidates first, then their logits side by side
  for (int v0 = 0; v0 < all; v0 += 256 * MOST) {
    Lp8 w[MOST];
    int i[MOST], from[MOST];
#pragma unroll
    for (int u = 0; u < MOST; ++u)  // all of them under way together
      if (v0 + 256 * u < all) {
        place(v0 + 256 * u + threadIdx.x, i[u], from[u]);
        fetch(w[u], from[u]);
      }
#pragma unroll
    for (int u = 0; u < MOST; ++u) {
      if (v0 + 256 * u >= all) break;
      float y[8];
      lp_widen<DT>(w[u], y);
      const float top = lp_max8(y);
      if (i[u] < x.end && (top != top || lp_key(top) >= least)) {  // (a NaN hides what is beside it)
        const int to = atomicAdd(&vectors, 1);
        if (to < VECS) {
          *reinterpret_cast<f32x4*>(&vec[to][0]) = f32x4{y[0], y[1], y[2], y[3]};
          *reinterpret_cast<f32x4*>(&vec[to][4]) = f32x4{y[4], y[5], y[6], y[7]};
          first[to] = i[u];
          base[to] = from[u];
        }
      }
    }
  }
  __syncthreads();
  if (vectors <= VECS) {
    for (int t = threadIdx.x; t < 8 * vectors; t += 256) {
      const int v = t >> 3;
      one(vec[v][t & 7], t & 7, first[v], base[v], [&](uint32_t k, uint32_t id) {
        if (k >= least) {
          const int to = atomicAdd(&count, 1);
          if (to < CAP) cand[to] = (uint64_t)k << 32 | id;
        }
      });
    }
  }
  __syncthreads();
  auto put = [&](int i, uint64_t q) {
    a.top_id[row * a.top + i] = ~(uint32_t)q;
    a.top_logprob[row * a.top + i] = (lp_value((uint32_t)(q >> 32)) - sm) * a.scale - sls;
  };
  const int have = vectors <= VECS ? count : CAP + 1;
  if (have <= CAP) {
    if ((int)threadIdx.x < have) {
      const uint64_t q = cand[threadIdx.x];
      int rank = 0;
#pragma unroll 4
      for (int i = 0; i < have; ++i) rank += cand[i] > q;
      if (rank < a.top) put(rank, q);
    }
    return;
  }
  // more than that are tied: one after another
  uint64_t last = ~0ull;
  for (int i = 0; i < a.top; ++i) {
    uint64_t q = 0;
    for (int v = threadIdx.x; v < all; v += 256) {
      Lp8 w;
      int k, from;
      place(v, k, from);
      fetch(w, from);
      float y[8];
      lp_widen<DT>(w, y);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        one(y[e], e, k, from, [&](uint32_t z, uint32_t id) {
          const uint64_t p = (uint64_t)z << 32 | id;
          q = p < last && p > q ? p : q;
        });
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) q = max(q, (uint64_t)__shfl_xor((unsigned long long)q, m, 64));
    if (lane == 0) sbest[wave] = q;
    __syncthreads();
    last = max(max(sbest[0], sbest[1]), max(sbest[2], sbest[3]));
    if (threadIdx.x == 0) put(i, last);
    __syncthreads();
  }
}

template <int DT>
__global__ __launch_bounds__(256) void k_lp_top(const LpArgs a) {
  const int64_t row = a.row0 + blockIdx.x;
  lp_tops<DT>(a, row, lp_row<DT>(a.x + row * a.ld, a.vocab), a.best + row * a.groups,
              [&](int lane) { return lp_shares(a, row, lane); });
}

// A block's share of a row: chunks c, c + 4, .. by each of its waves.
// LANES > 0: the maxima of groups of as many lanes' logits are kept.  WHOLE:
// the block has all of its row and goes on to the likeliest tokens itself.
template <int DT, int LANES, bool WHOLE>
__global__ __launch_bounds__(256, WHOLE ? 8 : 1) void k_lp_row(const LpArgs a) {
  constexpr int AHEAD = DT == DT_F32 ? 2 : 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % (uint32_t)a.splits;
  const int64_t row = a.row0 + blockIdx.x / (uint32_t)a.splits;
  const LpRow x = lp_row<DT>(a.x + row * a.ld, a.vocab);
  const int chunks = (x.end + LP_CHUNK - 1) / LP_CHUNK, first = x.pad > 0, whole = x.end / LP_CHUNK;  // [first, whole) are whole
  const int c0 = (int)((int64_t)chunks * split / a.splits), c1 = (int)((int64_t)chunks * (split + 1) / a.splits);
  const float c = a.scale * LP_LOG2E, lag = fminf(LP_LAG / c, 1e30f);
  __shared__ uint32_t mine[WHOLE ? LP_MOST_GROUPS : 1];
  uint32_t* best = WHOLE ? mine : a.best + row * a.groups;
  LpSum r{LP_NEG_INF, 0.f, 0.f};
  Lp8 buf[AHEAD];
  auto take = [&](const Lp8& w, int ch) __attribute__((always_inline)) {
    float f[8];
    lp_widen<DT>(w, f);
    const float top = lp_max8(f);
    if constexpr (LANES > 0) {
      float most = top;
      if (__any(top != top)) {  // a NaN counts as -inf in the order
        most = LP_NEG_INF;
#pragma unroll
        for (int e = 0; e < 8; ++e) most = f[e] > most ? f[e] : most;
      }
      uint32_t k = lp_key(most);
      if constexpr (LANES == 64) {
        k = wave_max_u32(k);
        if (lane == 0) best[ch] = k;
      } else {
#pragma unroll
        for (int m = 1; m < LANES; m *= 2) k = max(k, (uint32_t)__shfl_xor((int)k, m, 64));
        const int g = (ch * 64 + lane) / LANES;
        if (lane % LANES == 0 && g < a.groups) best[g] = k;
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
      r.t = __builtin_fmaf(p, fmaxf(z, LP_LEAST), r.t);
    }
  };
  // Whole chunks, each loaded AHEAD of its use; no branch between a load and
  // its use but at the end, so that every wait is for one load alone.
  auto load = [&](Lp8& w, int ch) __attribute__((always_inline)) { lp_load8<DT, true, true>(x.p, ch * LP_CHUNK + 8 * lane, w); };
  const int start = max(c0, first), end = min(c1, whole);
  int ch = start + wave;
  if (start < end) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load(buf[u], min(ch + 4 * u, end - 1));
  }
  for (; ch + 4 * (2 * AHEAD - 1) < end; ch += 4 * AHEAD)
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      take(buf[u], ch + 4 * u);
      load(buf[u], ch + 4 * (u + AHEAD));
    }
#pragma unroll
  for (int v = 0; v < 2; ++v, ch += 4 * AHEAD)
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (ch + 4 * u < end) take(buf[u], ch + 4 * u);
      if (v == 0 && ch + 4 * (u + AHEAD) < end) load(buf[u], ch + 4 * (u + AHEAD));
    }
  // the chunks at the row's ends (one, where it is short)
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const int at = e ? whole : 0;
    if (e ? whole == chunks || (first && whole == 0) : !first) continue;
    if (at < c0 || at >= c1 || (at + e) % 4 != wave) continue;
    lp_load_edge<DT>(x, at * LP_CHUNK + 8 * lane, buf[0]);
    take(buf[0], at);
  }
  r = lp_lanes<64>(r, c);
  __shared__ LpSum sw[4];
  if (lane == 0) sw[wave] = r;
  __syncthreads();
  auto sums = [&](int) { return lp_add(lp_add(sw[0], sw[1], c), lp_add(sw[2], sw[3], c), c); };
  if constexpr (WHOLE) {
    lp_tops<DT>(a, row, x, best, sums);
  } else if (threadIdx.x == 0) {
    r = sums(0);
    if (a.splits == 1) {
      lp_finish<DT>(a, row, r);
    } else {
      float* p = a.part + (row * a.splits + split) * 3;
      p[0] = r.m;
      p[1] = r.s;
      p[2] = r.t;
    }
  }
}

// d logits = scale (g (onehot - p) - h p (log p + H)), with p = e / S and
// log p = z - log S: e times a line in z, whose two numbers a row has.
template <int DT>
__global__ __launch_bounds__(256) void k_lp_grad(const LpGradArgs a) {
  constexpr int U = 4;
  const int64_t row = a.row0 + blockIdx.x / (uint32_t)a.pieces;
  const int piece = blockIdx.x % (uint32_t)a.pieces;
  // by the aligned 16 bytes of the gradient's row; the logits lie alike, or are loaded unaligned
  const LpRow o = lp_row<DT>(a.dx + row * a.ldd, a.vocab);
  const uint8_t* x = a.x + row * a.ld - o.pad * LP_BYTES<DT>;
  const int64_t t = a.targets ? a.targets[row] : -1;
  const bool given = t >= 0 && t < a.vocab;
  const float m = a.ref[row], sum = a.sum[row], c = a.scale * LP_LOG2E;
  const bool none = sum == 0.f;
  const float g = given && a.dlogprob && !none ? a.dlogprob[row] * a.scale : 0.f;
  const float h = a.dentropy ? a.dentropy[row] * a.scale : 0.f, ent = a.dentropy ? a.entropy[row] : 0.f;
  const float inv = none ? 0.f : -1.f / sum, ls = none ? 0.f : logf(sum);
  const float slope = h * LP_LN2 * inv, at0 = (g + h * (ent - ls)) * inv;
  const int64_t tp = given ? t + o.pad : -1;
  const int i0 = (piece * U * 256 + (int)threadIdx.x) * 8;
  auto inner = [&](int i) { return i >= o.pad && i + 8 <= o.end; };
  auto grad = [&](const Lp8& w, int i, float* f) __attribute__((always_inline)) {
    lp_widen<DT>(w, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float z = (f[e] - m) * c;
      const float d = __builtin_amdgcn_exp2f(z) * __builtin_fmaf(fmaxf(z, LP_LEAST), slope, at0);
      f[e] = i + e == tp ? d + g : d;
    }
  };
  Lp8 w[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (inner(i0 + 2048 * u)) lp_load8<DT, false, true>(x, i0 + 2048 * u, w[u]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = i0 + 2048 * u;
    float f[8];
    uint8_t* to = const_cast<uint8_t*>(o.p) + (int64_t)i * LP_BYTES<DT>;
    if (inner(i)) {
      grad(w[u], i, f);
      if constexpr (DT == DT_F32) {
        __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4*>(to));
        __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f32x4*>(to) + 1);
      } else {
        u32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = DT == DT_BF16 ? pack_bf16(f[2 * q], f[2 * q + 1]) : pack_f16(f[2 * q], f[2 * q + 1]);
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(to));
      }
    } else if (i < o.end) {  // the row's ends
      Lp8 y;
      lp_load_edge<DT>(LpRow{x, o.pad, o.end}, i, y);
      grad(y, i, f);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e >= o.pad && i + e < o.end) {
          if constexpr (DT == DT_F32) reinterpret_cast<float*>(to)[e] = f[e];
          else reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)((DT == DT_BF16 ? pack_bf16(f[e], 0.f) : pack_f16(f[e], 0.f)) & 0xffffu);
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
    const bool whole = a.top && a.splits == 1;
    if (!a.top) hipLaunchKernelGGL((k_lp_row<DT, 0, false>), grid, dim3(256), 0, s, a);
    else if (whole && a.width == 8) hipLaunchKernelGGL((k_lp_row<DT, 1, true>), grid, dim3(256), 0, s, a);
    else if (whole && a.width == 64) hipLaunchKernelGGL((k_lp_row<DT, 8, true>), grid, dim3(256), 0, s, a);
    else if (whole) hipLaunchKernelGGL((k_lp_row<DT, 64, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_lp_row<DT, 64, false>), grid, dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (whole) continue;
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
  a.pieces = (a.vocab + 7 + 8191) / 8192;  // (with a row's padding)
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
