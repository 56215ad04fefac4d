// Attention of one or a few new tokens over a paged cache (decode form), and
// the joining of split results.
//
// The rows of one key/value head (chunk tokens x the head's query group, at
// most 16 NQ) share every byte of cache read, so what bounds this kernel is
// reading the cache once.  A wave takes tiles of 32 keys straight from
// memory into registers, in the MFMA operand layouts (16 x 16 x 32):
//   S^T = K Q^T   A: lane (r, g) key r of 16, dims 8g .. 8g + 7 of each 32
//                 (INT4: dims gD/4 .. of the row, one 16-byte load);
//   O^T = V^T P^T B: lane (q, g) holds P of keys 4g .. 4g + 3 and 16 + 4g ..
//                 (its own scores), so A needs those 8 keys of one dim per
//                 lane: lane (r, g) loads dims r D/16 .. of the 8 keys (whole
//                 rows, 16 lanes x 16 bytes) and one v_perm a word pairs two
//                 keys' values: product i then yields dim r D/16 + i.
// Nothing goes through LDS until the four waves' results are joined at the
// end.  The keys are split over blocks until the grid covers the machine a
// few times; splits leave (maximum, sum, output) in fp32 and k_kv_join adds
// them in order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_attn.hpp"
#include "launch.hpp"

namespace whtq {

// The row transform x -> Hn S x over a group of D / N lanes with N values
// each: lane (sub) holds values N sub .. N sub + N - 1, lanes differ by
// `step` (a power of two).  SIGN_AFTER applies S last (the inverse).
template <int D, int N, bool SIGN_AFTER>
__device__ __forceinline__ void kv_row_rht(float* x, int sub, int step, int lane, const uint32_t* signs) {
  auto sign = [&] {
    if (!signs) return;
#pragma unroll
    for (int e = 0; e < N; e += 8) {
      const int at = N * sub + e;
      kv_sign8(x + e, (signs[at >> 5] >> (at & 31)) & 255u);
    }
  };
  if constexpr (!SIGN_AFTER) sign();
  kv_bfly<N>(x);
#pragma unroll
  for (int m = 1; m < D / N; m *= 2) kv_lane_bfly<N>(x, m * step, lane);
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] *= D == 64 ? 0.125f : 0.08838834764831845f;  // 1 / sqrt(D)
  if constexpr (SIGN_AFTER) sign();
}

// T: type of q and out; the operands of the products are T (dense) or fp16.
template <int D, int T, bool INT4, int NQ>
__global__ __launch_bounds__(256) void k_kv_step(const KvAttnArgs a) {
  constexpr int MT = INT4 ? KV_F16 : T;
  constexpr int KK = D / 32;   // products per 16 keys of S^T
  constexpr int DL = D / 16;   // dims a lane holds of a value row
  constexpr int VW = INT4 ? 1 : DL / 2;  // words of a value row in a lane
  constexpr int PAD = D + 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  int id = blockIdx.x;
  const int split = id % a.splits;
  id /= a.splits;
  const int h = id % a.c.kv_heads, b = id / a.c.kv_heads;

  const int q0 = a.q_start[b], nq = min(a.q_start[b + 1] - q0, (16 * NQ) / a.group);
  const int rows = nq * a.group;
  const int kv = min(a.kv_len[b], (int)min<int64_t>((int64_t)a.table_width << a.c.page_shift, INT32_MAX));
  if (rows <= 0) return;
  const int chunk = a.q_start[b + 1] - q0;  // positions count from the whole chunk
  const int p0 = kv - chunk;
  // keys any row of the block sees: [first, last]
  int first = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
  int last = a.causal ? min(kv - 1, p0 + nq - 1) : kv - 1;
  const int lo = split * a.split_keys, hi = split == a.splits - 1 ? INT32_MAX : lo + a.split_keys - 1;
  const int kfirst = max(first, lo), klast = min(last, hi);
  const int32_t* table = a.table + b * a.table_stride;

  // the lane's queries (column r of each block of 16) and what they see
  int qpos[NQ];
  bool qlive[NQ];
  u32x4 qf[NQ][KK];
  float qs[NQ];  // scale of the scores
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int row = 16 * n + r, tok = row / a.group;
    qlive[n] = row < rows && (uint32_t)(q0 + tok) < (uint64_t)a.q_tokens;
    qpos[n] = p0 + tok;
    qs[n] = a.scale;
    const uint8_t* qp = a.q + (int64_t)(q0 + tok) * a.q_tok + (int64_t)(h * a.group + row % a.group) * a.q_head;
    if constexpr (!INT4) {
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
        qf[n][kk] = qlive[n] ? ldg<u32x4>(qp + 64 * kk + 16 * g) : u32x4{0u, 0u, 0u, 0u};
    } else {
      float x[D / 4];
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
        kv_widen8<T>(qlive[n] ? ldg<u32x4>(qp + g * (D / 2) + 16 * kk) : u32x4{0u, 0u, 0u, 0u}, x + 8 * kk);
      kv_row_rht<D, D / 4, false>(x, g, 16, lane, a.c.signs);
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < D / 4; ++e) top = fmaxf(top, fabsf(x[e]));
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      // an exact power of two brings the row's largest value to [1, 2)
      const int ex = top > 0.f && top < __builtin_huge_valf() ? max(-126, min(126, __builtin_amdgcn_frexp_expf(top) - 1)) : 0;
      const float down = __builtin_ldexpf(1.f, -ex);
      qs[n] = a.scale * __builtin_ldexpf(1.f, ex);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
          qf[n][kk][w] = pack_f16(x[8 * kk + kv_perm(2 * w)] * down, x[8 * kk + kv_perm(2 * w + 1)] * down);
      }
    }
  }

  float m[NQ], l[NQ];
  f32x4 o[NQ][DL];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = KV_NEG_INF;
    l[n] = 0.f;
#pragma unroll
    for (int i = 0; i < DL; ++i) o[n][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  int ve = -30;  // INT4: the outputs are in units of 2^ve (fp16's least scale is 2^-24)

  const uint8_t* kbase = a.c.k.p + h * a.c.k.head;
  const uint8_t* vbase = a.c.v.p + h * a.c.v.head;
  constexpr int KL = INT4 ? 1 : KK;  // 16-byte loads of a lane's key share (INT4, D = 64: 8 bytes)
  struct Tile {
    u32x4 k[2][KL];
    uint32_t v[8][VW];
    u32x2 ks[2], vs[2];
  };
  // 16 keys lie in one page; lane kb holds the page of the tile's half kb
  auto look_up = [&](int key0) {
    const int k = min(max(key0 + 16 * (lane & 1), kfirst), klast);
    return kv_page(a, table[k >> a.c.page_shift]);
  };
  auto fetch = [&](Tile& t, int key0, int pages) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const int kk0 = key0 + 16 * kb;
      const int64_t page = __builtin_amdgcn_readlane(pages, kb);
      const int off = kk0 & ((1 << a.c.page_shift) - 1);
      const uint8_t* kp = kbase + page * a.c.k.page + (off + r) * a.c.k.tok;
      if constexpr (!INT4) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) t.k[kb][kk] = ldg_global<u32x4>(kp + 64 * kk + 16 * g);
      } else if constexpr (D == 128) {
        t.k[kb][0] = ldg_global<u32x4>(kp + 16 * g);
      } else {
        const u32x2 w = ldg_global<u32x2>(kp + 8 * g);
        t.k[kb][0] = u32x4{w.x, w.y, 0u, 0u};
      }
      const uint8_t* vp = vbase + page * a.c.v.page + (off + 4 * g) * a.c.v.tok + r * (INT4 ? DL / 2 : 2 * DL);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* p = vp + j * a.c.v.tok;
        if constexpr (!INT4 && D == 128) {
          const u32x4 w = ldg_global<u32x4>(p);
#pragma unroll
          for (int i = 0; i < 4; ++i) t.v[4 * kb + j][i % VW] = w[i];
        } else if constexpr (!INT4) {
          const u32x2 w = ldg_global<u32x2>(p);
          t.v[4 * kb + j][0] = w.x;
          t.v[4 * kb + j][1 % VW] = w.y;
        } else if constexpr (D == 128) {
          t.v[4 * kb + j][0] = ldg_global<uint32_t>(p);
        } else {
          t.v[4 * kb + j][0] = ldg_global<uint16_t>(p);
        }
      }
      if constexpr (INT4) {
        t.ks[kb] = ldg_global<u32x2>(a.c.k.scale + page * a.c.k.s_page + h * a.c.k.s_head + off + 4 * g);
        t.vs[kb] = ldg_global<u32x2>(a.c.v.scale + page * a.c.v.s_page + h * a.c.v.s_head + off + 4 * g);
      }
    }
  };

  const int t0 = kfirst >> 5, t1 = klast >> 5;  // tiles of 32 keys; kfirst > klast: none
  Tile cur, nxt;
  int t = t0 + wave;
  const bool work = kfirst <= klast;
  int ahead = 0;
  if (work && t <= t1) {
    fetch(cur, 32 * t, look_up(32 * t));
    ahead = look_up(32 * (t + 4));
  }
  for (; work && t <= t1; t += 4) {
    const bool more = t + 4 <= t1;
    if (more) {
      fetch(nxt, 32 * (t + 4), ahead);
      ahead = look_up(32 * (t + 8));
    }
    const int key0 = 32 * t;
    // every row sees the whole tile? (wave-uniform)
    const bool full = key0 >= (a.window > 0 ? max(kfirst, p0 + nq - a.window) : kfirst) &&
                      key0 + 31 <= (a.causal ? min(klast, p0) : klast);
    // what lies outside [kfirst, klast] may be anything: the values become 0
    if constexpr (!INT4) {
      if (key0 < kfirst || key0 + 31 > klast) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int key = key0 + (s < 4 ? 0 : 16) + 4 * g + (s & 3);
          const bool in = key >= kfirst && key <= klast;
#pragma unroll
          for (int w = 0; w < VW; ++w) cur.v[s][w] = in ? cur.v[s][w] : 0u;
        }
      }
    }
    float ks[8], vs[8];
    if constexpr (INT4) {
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint32_t kw = cur.ks[s >> 2][(s >> 1) & 1], vw = cur.vs[s >> 2][(s >> 1) & 1];
        ks[s] = (float)__builtin_bit_cast(_Float16, (uint16_t)(s & 1 ? kw >> 16 : kw & 0xffffu));
        vs[s] = (float)__builtin_bit_cast(_Float16, (uint16_t)(s & 1 ? vw >> 16 : vw & 0xffffu));
      }
      // the largest value scale of the tile, as a power of two, sets the unit
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int key = key0 + (s < 4 ? 0 : 16) + 4 * g + (s & 3);
        if (key >= kfirst && key <= klast && vs[s] < 65536.f) top = fmaxf(top, vs[s]);
      }
      if (__any(top >= __builtin_ldexpf(1.f, ve + 1))) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const int e = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(top) - 1);
        const float f = __builtin_ldexpf(1.f, ve - e);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int i = 0; i < DL; ++i) o[n][i] *= f;
        ve = e;
      }
      const float unit = __builtin_ldexpf(1.f, -ve);
#pragma unroll
      for (int s = 0; s < 8; ++s) vs[s] *= unit;
    }
    // S^T: s[n][4 kb + e] is key 16 kb + 4 g + e
    float sc[NQ][8];
    {
      u32x4 kf[2][KK];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          if constexpr (INT4) kf[kb][kk] = kv_codes8(cur.k[kb][0][kk]);
          else kf[kb][kk] = cur.k[kb][kk];
        }
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) acc = kv_mfma16<MT>(kf[kb][kk], qf[n][kk], acc);
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][4 * kb + e] = acc[e];
        }
    }
    u32x4 pf[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = KV_NEG_INF;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        sc[n][s] *= INT4 ? qs[n] * ks[s] : qs[n];
        if (!full) {
          const int key = key0 + (s < 4 ? 0 : 16) + 4 * g + (s & 3);
          const bool in = key >= kfirst && key <= klast && (!a.causal || key <= qpos[n]) &&
                          (a.window <= 0 || key > qpos[n] - a.window);
          sc[n][s] = in ? sc[n][s] : KV_NEG_INF;
        }
        top = fmaxf(top, sc[n][s]);
      }
      if (__any(top > m[n] + KV_LAG)) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float mn = fmaxf(m[n], top);
        const float al = kv_alpha(m[n], mn);
        l[n] *= al;
#pragma unroll
        for (int i = 0; i < DL; ++i) o[n][i] *= al;
        m[n] = mn;
      }
      const float base = kv_base(m[n]);
      float p[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        p[s] = __builtin_amdgcn_exp2f(sc[n][s] - base);
        l[n] += p[s];
        if constexpr (INT4) p[s] = sc[n][s] == KV_NEG_INF ? 0.f : p[s] * vs[s];
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) pf[n][w] = kv_pack<MT>(p[2 * w], p[2 * w + 1]);
    }
    // O^T: product i yields dim DL r + i
    auto value = [&](int i, auto keep) {  // A operand of product i; keep(s): whether slot s counts
      u32x4 f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x0 = keep(2 * w) ? cur.v[2 * w][i / 2 % VW] : 0u;
        const uint32_t x1 = keep(2 * w + 1) ? cur.v[2 * w + 1][i / 2 % VW] : 0u;
        f[w] = __builtin_amdgcn_perm(x1, x0, (i & 1) ? 0x07060302u : 0x05040100u);
      }
      return f;
    };
    if constexpr (INT4) {
#pragma unroll
      for (int s = 0; s < 8; ++s) cur.v[s][0] ^= 0x88888888u;
#pragma unroll
      for (int i = 0; i < DL; i += 2) {
        u32x4 f0, f1;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // byte i / 2 of two keys' words, each alone in a half
          const uint32_t x = __builtin_amdgcn_perm(cur.v[2 * w + 1][0], cur.v[2 * w][0], 0x0c040c00u + 0x00010001u * (i / 2));
          f0[w] = kv_code_lo(x);
          f1[w] = kv_code_hi(x);
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          o[n][i] = kv_mfma16<MT>(f0, pf[n], o[n][i]);
          o[n][i + 1] = kv_mfma16<MT>(f1, pf[n], o[n][i + 1]);
        }
      }
    } else {
      bool bad = false;
      if (!full && nq > 1) {
        // a masked probability of 0 does not hide a value that is not finite
        u16x2 top = {0, 0};
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int w = 0; w < VW; ++w) top = absmax16(top, cur.v[s][w]);
        bad = __any(kv_not_finite<T>(top));
      }
      if (!bad) {
#pragma unroll
        for (int i = 0; i < DL; ++i) {
          const u32x4 f = value(i, [](int) { return true; });
#pragma unroll
          for (int n = 0; n < NQ; ++n) o[n][i] = kv_mfma16<MT>(f, pf[n], o[n][i]);
        }
      } else {
        // once per token of the chunk, with the keys it does not see cleared
        for (int tok = 0; tok < nq; ++tok) {
          const int pos = p0 + tok;
          auto keep = [&](int s) {
            const int key = key0 + (s < 4 ? 0 : 16) + 4 * g + (s & 3);
            return (!a.causal || key <= pos) && (a.window <= 0 || key > pos - a.window);
          };
#pragma unroll
          for (int i = 0; i < DL; ++i) {
            const u32x4 f = value(i, keep);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              const f32x4 one = kv_mfma16<MT>(f, pf[n], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
              for (int e = 0; e < 4; ++e) o[n][i][e] += qpos[n] == pos ? one[e] : 0.f;
            }
          }
        }
      }
    }
    if (more) cur = nxt;
  }

  // join the four waves: rows of 16 queries at a time through LDS
  __shared__ __attribute__((aligned(16))) float so[4][16][PAD];
  __shared__ float sm[4][16], sl[4][16];
  __shared__ int se[4];
  constexpr int LR = D / 8;  // lanes of a row in the join
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float ls = l[n];
    ls += __shfl_xor(ls, 16, 64);
    ls += __shfl_xor(ls, 32, 64);
    if (n) __syncthreads();
    // lane (q = r, g): dims (4 g + e) DL + i
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < DL; i += 4)
        *reinterpret_cast<f32x4*>(&so[wave][r][(4 * g + e) * DL + i]) =
            f32x4{o[n][i][e], o[n][i + 1][e], o[n][i + 2][e], o[n][i + 3][e]};
    if (g == 0) {
      sm[wave][r] = m[n];
      sl[wave][r] = ls;
    }
    if (lane == 0) se[wave] = ve;
    __syncthreads();
    const int row = 16 * n + (int)threadIdx.x / LR, i0 = threadIdx.x % LR;
    if ((int)threadIdx.x < 16 * LR && row < rows) {
      const int q = row & 15, tok = row / a.group, head = h * a.group + row % a.group;
      float mx = KV_NEG_INF;
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = fmaxf(mx, sm[w][q]);
      float sum = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(sm[w][q] - kv_base(mx));
        sum += f * sl[w][q];
        const float fo = INT4 ? f * __builtin_ldexpf(1.f, se[w]) : f;
        // a wave that saw nothing for this row adds nothing
        const bool none = sm[w][q] == KV_NEG_INF && sl[w][q] == 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += none ? 0.f : fo * so[w][q][8 * i0 + e];
      }
      if ((uint32_t)(q0 + tok) < (uint64_t)a.q_tokens) {
        const int64_t gr = (int64_t)(q0 + tok) * a.heads + head;
        if (a.splits == 1) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= inv;
          if constexpr (INT4) kv_row_rht<D, 8, true>(x, i0, 1, lane, a.c.signs);
          stg<u32x4>(a.out + (int64_t)(q0 + tok) * a.o_tok + (int64_t)head * a.o_head + 16 * i0, kv_round8<T>(x));
          if (a.lse && i0 == 0)
            a.lse[gr] = sum == 0.f ? KV_NEG_INF : (mx + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
        } else {
          const int64_t pr = (int64_t)split * a.q_tokens * a.heads + gr;
          stg<f32x4>(a.part_o + pr * D + 8 * i0, f32x4{x[0], x[1], x[2], x[3]});
          stg<f32x4>(a.part_o + pr * D + 8 * i0 + 4, f32x4{x[4], x[5], x[6], x[7]});
          if (i0 == 0) {
            a.part_ml[2 * pr] = mx;
            a.part_ml[2 * pr + 1] = sum;
          }
        }
      }
    }
  }
}

// Adds the splits of each row in order of the keys.  GR groups of D / 8
// lanes share a row when there are few rows and many splits.
template <int D, int T, bool INT4>
__global__ __launch_bounds__(256) void k_kv_join(const KvAttnArgs a, int gr) {
  constexpr int LR = D / 8, PAD = D + 4;
  __shared__ __attribute__((aligned(16))) float so[256 / LR][PAD];
  __shared__ float sm[256 / LR], sl[256 / LR];
  const int grp = threadIdx.x / LR, i0 = threadIdx.x % LR, lane = threadIdx.x & 63;
  const int per = (256 / LR) / gr;  // rows of the block
  const int64_t rows = a.q_tokens * a.heads;
  const int64_t row = (int64_t)blockIdx.x * per + grp / gr;
  const int part = grp % gr;
  float mx = KV_NEG_INF, sum = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto add = [&](float m1, float l1, const float* y) {
    const float mn = fmaxf(mx, m1), f0 = __builtin_amdgcn_exp2f(mx - kv_base(mn)), f1 = __builtin_amdgcn_exp2f(m1 - kv_base(mn));
    const bool none = m1 == KV_NEG_INF && l1 == 0.f;  // its output was not written
    sum = f0 * sum + (none ? 0.f : f1 * l1);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = f0 * x[e] + (none ? 0.f : f1 * y[e]);
    mx = mn;
  };
  if (row < rows)
    for (int s = part; s < a.splits; s += gr) {
      const int64_t pr = (int64_t)s * rows + row;
      const f32x4 u = ldg<f32x4>(a.part_o + pr * D + 8 * i0), w = ldg<f32x4>(a.part_o + pr * D + 8 * i0 + 4);
      const float y[8] = {u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]};
      add(a.part_ml[2 * pr], a.part_ml[2 * pr + 1], y);
    }
  if (gr > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) so[grp][8 * i0 + e] = x[e];
    if (i0 == 0) {
      sm[grp] = mx;
      sl[grp] = sum;
    }
    __syncthreads();
    if (part) return;
    for (int p = 1; p < gr; ++p) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = so[grp + p][8 * i0 + e];
      add(sm[grp + p], sl[grp + p], y);
    }
  }
  if (row >= rows) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= inv;
  if constexpr (INT4) kv_row_rht<D, 8, true>(x, i0, 1, lane, a.c.signs);
  const int64_t tok = row / a.heads, head = row % a.heads;
  stg<u32x4>(a.out + tok * a.o_tok + head * a.o_head + 16 * i0, kv_round8<T>(x));
  if (a.lse && i0 == 0) a.lse[row] = sum == 0.f ? KV_NEG_INF : (mx + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

template <int D, int T, bool INT4>
static hipError_t step_launch(const KvAttnArgs& a, int nq, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.seqs * a.c.kv_heads * a.splits));
  if (nq == 1) hipLaunchKernelGGL((k_kv_step<D, T, INT4, 1>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_kv_step<D, T, INT4, 2>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}
template <int D, int T, bool INT4>
static hipError_t join_launch(const KvAttnArgs& a, hipStream_t s) {
  int gr = 1;
  const int most = 256 / (D / 8);
  const int64_t rows = a.q_tokens * a.heads;
  while (gr < most && gr < a.splits && rows * gr < 8192) gr *= 2;
  const int per = most / gr;
  hipLaunchKernelGGL((k_kv_join<D, T, INT4>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, a, gr);
  return hipGetLastError();
}

#define KV_PICK(F, DIM, T, INT4, ...)                                                            \
  ((DIM) == 128 ? ((T) == KV_BF16 ? ((INT4) ? F<128, KV_BF16, true>(__VA_ARGS__) : F<128, KV_BF16, false>(__VA_ARGS__)) \
                                  : ((INT4) ? F<128, KV_F16, true>(__VA_ARGS__) : F<128, KV_F16, false>(__VA_ARGS__)))  \
                : ((T) == KV_BF16 ? ((INT4) ? F<64, KV_BF16, true>(__VA_ARGS__) : F<64, KV_BF16, false>(__VA_ARGS__))   \
                                  : ((INT4) ? F<64, KV_F16, true>(__VA_ARGS__) : F<64, KV_F16, false>(__VA_ARGS__))))

hipError_t launch_kv_step(const KvAttnArgs& a, int dim, int dt, bool int4, int nq, hipStream_t s) {
  return KV_PICK(step_launch, dim, dt, int4, a, nq, s);
}
hipError_t launch_kv_join(const KvAttnArgs& a, int dim, int dt, bool int4, hipStream_t s) {
  return KV_PICK(join_launch, dim, dt, int4, a, s);
}

}  // namespace whtq
