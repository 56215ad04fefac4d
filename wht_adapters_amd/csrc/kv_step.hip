// Attention of one or a few new tokens over a paged cache (decode form), and
// the joining of split results.
//
// The rows of one key/value head (chunk tokens x the head's query group, at
// most 16 NQ) share every byte of cache read, so what bounds this kernel is
// reading the cache once.  A wave takes tiles of 32 or 64 keys straight from
// memory into registers, in the MFMA operand layouts (16 x 16 x 32):
//   S^T = K Q^T   A: lane (r, g) key r of 16, dims 8g .. 8g + 7 of each 32
//                 (INT4: dims gD/4 .. of the row, one 16-byte load);
//   O^T = V^T P^T B: lane (q, g) holds P of keys 4g .. 4g + 3 and 16 + 4g ..
//                 (its own scores), so A needs those 8 keys of one dim per
//                 lane: lane (r, g) loads dims r D/16 .. of the 8 keys (whole
//                 rows, 16 lanes x 16 bytes) and one v_perm a word pairs two
//                 keys' values: product i then yields dim r D/16 + i.
// Softmax in one pass: a row's maximum may lag (KV_LAG), sums are fp32 of the
// unrounded probabilities.  An operand register is loaded again for the next
// tile as soon as its product has used it; nothing goes through LDS until the
// waves' results are joined at the end.  The keys of all sequences are dealt
// to the blocks in equal runs (see the comment below), so that ragged lengths
// keep all of them busy; the price is the join: pieces of a sequence leave
// (maximum, sum, output) in fp32 and k_kv_step_join adds them in the order of
// the keys.
//
// Measured (kernel times): 64 sequences of 17 to 8191 keys, 32 heads on 8 of
// 128, bf16: 363 MB in 80 us, 4.6 TB/s (a large copy moves 4.75), and 4.7 us
// for the join.  Two INT4 contexts of 100003 and 131072 keys, 64 heads on 8:
// 244 MB in 62 us, 3.9 TB/s, the vector pipes 55 % busy unpacking codes, and
// 7.1 us for the join.  One token over 777 keys: 8.6 + 4.1 us, all latency.
// Registers: the INT4 builds keep about 100 scalars in vector lanes, two column
// blocks (17 to 32 rows) leave one wave a SIMD, and the 16-bit build for several
// tokens has up to 24 vector registers in scratch (take_out, unrolled over the
// tile): the 64 sequences with 4 tokens each take 114 us.
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

// Work of a call.  A sequence's keys are counted in units of one tile for
// every wave of a block, at least one unit where it has queries.
//  - whole (a.blocks == 0): a block is one sequence and head.
//  - shared: a.blocks blocks a head take equal runs of all sequences' units
//    (run i starts at unit i T / n).  A run that holds a sequence whole writes
//    its result; other pieces leave (maximum, sum, output) in slot i + b,
//    which no other piece has (a step to the right adds to i or to b), and
//    the run with a sequence's first unit notes the runs it reaches over.
struct KvSpan {  // a sequence's share of the work
  int q0, nq, chunk, p0, first, last, units;
};
__device__ __forceinline__ KvSpan kv_span(const KvAttnArgs& a, int q0, int q1, int kv_len, int unit) {
  KvSpan s;
  s.q0 = q0;
  s.chunk = q1 - q0;
  s.nq = min(s.chunk, a.rows / a.group);  // at most max_q_len
  const int kv = kv_held(a, kv_len);
  s.p0 = kv - s.chunk;  // position of the first query
  s.first = a.window > 0 ? max(0, s.p0 - a.window + 1) : 0;  // the keys any of its queries sees
  s.last = a.causal ? min(kv - 1, s.p0 + s.nq - 1) : kv - 1;
  s.units = s.nq <= 0 ? 0 : max(1, s.last / unit - s.first / unit + 1);
  if (s.last < s.first) s.units = s.nq > 0;
  return s;
}

// n runs of a number of units, the first `more` of them one longer.
struct KvRuns {
  int64_t each, more;
  __device__ __forceinline__ KvRuns() {}
  __device__ __forceinline__ KvRuns(int64_t total, int n) {
    each = total >> 31 ? total / n : (uint32_t)total / (uint32_t)n;  // (a 64-bit division takes a microsecond)
    more = total - each * n;
  }
  __device__ __forceinline__ int64_t start(int run) const { return run * each + min<int64_t>(run, more); }
  __device__ __forceinline__ int of(int64_t unit) const {  // the run a unit is in
    const int64_t big = more * (each + 1), x = unit < big ? unit : unit - big, d = unit < big ? each + 1 : each;
    return (int)((unit < big ? 0 : more) + (x >> 31 || d >> 31 ? x / d : (int64_t)((uint32_t)x / (uint32_t)d)));
  }
};

// Values every lane has alike, kept as such (scalar registers and branches).
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t scalar(int64_t x) {
  return (int64_t)((uint64_t)(uint32_t)scalar((int)(x >> 32)) << 32 | (uint32_t)scalar((int)x));
}

// T: type of q and out; the operands of the products are T (dense) or fp16.
// MANY: chunks of more than one token (values that are not finite need care
// there: a kernel of its own keeps its registers out of the single token's).
template <int D, int T, bool INT4, int NQ, int NW, bool MANY>
__global__ __launch_bounds__(64 * NW, NQ == 1 ? 2 : 1) void k_kv_step(const KvAttnArgs a) {
  constexpr int MT = INT4 ? KV_F16 : T;
  constexpr bool LOW = INT4 && T == KV_F16;  // the queries' low parts count, see qf
  constexpr int KK = D / 32;   // products per 16 keys of S^T
  constexpr int DL = D / 16;   // dims a lane holds of a value row
  constexpr int VW = INT4 ? 1 : DL / 2;  // words of a value row in a lane
  constexpr int KL = INT4 ? 1 : KK;      // loads of a lane's key share
  constexpr int KP = (D == 128 && !INT4) ? 1 : 2;  // pairs of 16 keys in a tile
  constexpr int TK = 32 * KP, UNIT = TK * NW;
  constexpr int PAD = D + 4;
  constexpr int LR = D / 8;  // lanes of a row in the join
  __shared__ __attribute__((aligned(16))) float so[NW][16][PAD];
  __shared__ float sm[NW][16], sl[NW][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;

  // the block's run of units [u, u1), starting `at` units into sequence b
  int b, run = 0, runs = 1;
  const int h = blockIdx.x % a.c.kv_heads;
  int64_t u = 0, u1 = 1, at = 0, total = 1;
  KvRuns share{};
  KvSpan sp;
  if (a.blocks == 0) {
    b = blockIdx.x / a.c.kv_heads;
    sp = kv_span(a, scalar(a.q_start[b]), scalar(a.q_start[b + 1]), scalar(a.kv_len[b]), UNIT);
  } else {
    run = blockIdx.x / a.c.kv_heads;
    // lane i looks at sequence s + i
    KvSpan mine;
    auto look = [&](int s) {
      const int i = s + lane;
      mine = i < a.seqs ? kv_span(a, a.q_start[i], a.q_start[i + 1], a.kv_len[i], UNIT) : KvSpan{};
      int sum = mine.units;  // of the lanes up to this one
#pragma unroll
      for (int m = 1; m < 64; m *= 2) {
        const int o = __shfl_up(sum, m, 64);
        if (lane >= m) sum += o;
      }
      return sum;
    };
    int sum = look(0);
    total = scalar(__builtin_amdgcn_readlane(sum, 63));
    for (int s = 64; s < a.seqs; s += 64) total += scalar(__builtin_amdgcn_readlane(look(s), 63));
    runs = (int)min<int64_t>(a.blocks, total);
    if (run >= runs) return;
    share = KvRuns(total, runs);
    u = share.start(run);
    u1 = share.start(run + 1);
    int64_t before = 0;
    for (b = 0;; b += 64) {  // ends: u < total
      if (a.seqs > 64) sum = look(b);
      const uint64_t past = __ballot(before + sum > u);
      if (past) {
        const int i = __builtin_ctzll(past);
        auto of = [&](int x) { return __builtin_amdgcn_readlane(x, i); };
        sp = {of(mine.q0), of(mine.nq), of(mine.chunk), of(mine.p0), of(mine.first), of(mine.last), of(mine.units)};
        at = u - before - (of(sum) - sp.units);
        b += i;
        break;
      }
      before += __builtin_amdgcn_readlane(sum, 63);
    }
    b = scalar(b);
    at = scalar(at);
  }

  for (bool one = true; u < u1; ++b, one = false) {
    if (!one) sp = kv_span(a, scalar(a.q_start[b]), scalar(a.q_start[b + 1]), scalar(a.kv_len[b]), UNIT);
    if (sp.units == 0) {
      if (a.blocks == 0) return;
      continue;
    }
    const int q0 = sp.q0, nq = sp.nq, p0 = sp.p0, rows = nq * a.group;
    // this piece: units [at, at + take) of the sequence
    const int from = (int)at;
    const int take = a.blocks == 0 ? sp.units : (int)min<int64_t>(sp.units - from, u1 - u);
    const bool whole = take == sp.units;
    const int base_key = sp.first / UNIT * UNIT;
    const int kfirst = max(sp.first, base_key + from * UNIT);
    const int klast = min(sp.last, base_key + (from + take) * UNIT - 1);
    const int32_t* table = a.table + b * a.table_stride;

    const uint8_t* kbase = a.c.k.p + h * a.c.k.head;
    const uint8_t* vbase = a.c.v.p + h * a.c.v.head;
    // a lane's places in 16 keys (a page's extent is below 2^31 bytes)
    const uint32_t klane = r * (uint32_t)a.c.k.tok + g * (INT4 ? D / 8 : 16);
    const uint32_t vlane = 4 * g * (uint32_t)a.c.v.tok + r * (INT4 ? DL / 2 : 2 * DL);
    const int pmask = (1 << a.c.page_shift) - 1;

    // keys and scales, and values, of the tile at hand; each is loaded again
    // for the next tile as soon as it was used
    u32x4 kr[2 * KP][KL];
    uint32_t vr[8 * KP][VW];
    u32x2 ksr[2 * KP], vsr[2 * KP];
    // 16 keys lie in one page; lane i holds the page of the tile's i-th 16
    auto look_up = [&](int key0) {
      const int k = min(max(key0 + 16 * (lane & (2 * KP - 1)), kfirst), klast);
      return table[k >> a.c.page_shift];
    };
    auto fetch_k = [&](int key0, int pages) {
#pragma unroll
      for (int kb = 0; kb < 2 * KP; ++kb) {
        const int64_t page = __builtin_amdgcn_readlane(pages, kb);
        const int off = (key0 + 16 * kb) & pmask;
        const uint8_t* kp = kbase + (page * a.c.k.page + off * a.c.k.tok);
        if constexpr (!INT4) {
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) kr[kb][kk] = ldg_global<u32x4>(kp + (klane + 64 * kk));
        } else if constexpr (D == 128) {
          kr[kb][0] = kv_load<u32x4>(kp, klane);
        } else {
          const u32x2 w = kv_load<u32x2>(kp, klane);
          kr[kb][0] = u32x4{w.x, w.y, 0u, 0u};
        }
        if constexpr (INT4)
          ksr[kb] = kv_load<u32x2>(a.c.k.scale + (page * a.c.k.s_page + h * a.c.k.s_head + off), 8 * g);
      }
    };
    auto fetch_v = [&](int key0, int pages) {
#pragma unroll
      for (int kb = 0; kb < 2 * KP; ++kb) {
        const int64_t page = __builtin_amdgcn_readlane(pages, kb);
        const int off = (key0 + 16 * kb) & pmask;
        const uint8_t* vp = vbase + (page * a.c.v.page + off * a.c.v.tok);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t p = vlane + j * (uint32_t)a.c.v.tok;
          uint32_t* to = vr[4 * kb + j];
          if constexpr (!INT4 && D == 128) {
            const u32x4 w = ldg_global<u32x4>(vp + p);
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i % VW] = w[i];
          } else if constexpr (!INT4) {
            const u32x2 w = kv_load<u32x2>(vp, p);
            to[0] = w.x;
            to[1 % VW] = w.y;
          } else if constexpr (D == 128) {
            to[0] = kv_load<uint32_t>(vp, p);
          } else {
            to[0] = kv_load<uint16_t>(vp, p);
          }
        }
        if constexpr (INT4)
          vsr[kb] = kv_load<u32x2>(a.c.v.scale + (page * a.c.v.s_page + h * a.c.v.s_head + off), 8 * g);
      }
    };

    const bool work = kfirst <= klast;
    const int t1 = klast / TK;
    // memory answers in order: the next tile's table entries are asked for
    // before this tile's keys and values, and so are there with them
    int t = kfirst / TK + wave, entry = 0;
    if (work && t <= t1) {
      const int pages = kv_page(a, look_up(t * TK));
      entry = look_up((t + NW) * TK);
      fetch_k(t * TK, pages);
      fetch_v(t * TK, pages);
    }
    // the lane's queries (column r of each block of 16) and what they see
    // INT4: the rotated query is rounded to fp16 for its product, 2^-12 of each
    // value.  bf16 outputs hide that (it adds 1 % to their own 2^-9); fp16
    // outputs would be off by twice their own rounding, so there what the
    // rounding dropped goes into a second product.
    int qpos[NQ];
    u32x4 qf[NQ][KK], ql[NQ][LOW ? KK : 1];
    float qs[NQ];  // the scores are kept in units of 1 / qs, qs > 0; a negative scale turns q around
    const uint32_t turn = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int row = 16 * n + r, tok = row / a.group;
      const bool live = row < rows && (uint32_t)(q0 + tok) < (uint64_t)a.q_tokens;
      qpos[n] = p0 + tok;
      // 0 would turn a masked -inf into NaN; the results are the same (a score in
      // these units is below 2^27 where INT4's power of two takes part)
      qs[n] = fmaxf(fabsf(a.scale), 1e-30f);
      const uint8_t* qp = a.q + (int64_t)(q0 + tok) * a.q_tok + (int64_t)(h * a.group + row % a.group) * a.q_head;
      if constexpr (!INT4) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
          qf[n][kk] = live ? ldg<u32x4>(qp + 64 * kk + 16 * g) ^ turn : u32x4{0u, 0u, 0u, 0u};
      } else {
        float x[D / 4];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
          kv_widen8<T>(live ? ldg<u32x4>(qp + g * (D / 2) + 16 * kk) : u32x4{0u, 0u, 0u, 0u}, x + 8 * kk);
        kv_row_rht<D, D / 4, false>(x, g, 16, lane, a.c.signs);
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < D / 4; ++e) top = fmaxf(top, fabsf(x[e]));
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        // an exact power of two brings the row's largest value to [1, 2)
        const int ex = top > 0.f && top < __builtin_huge_valf() ? max(-126, min(126, __builtin_amdgcn_frexp_expf(top) - 1)) : 0;
        const float down = __builtin_ldexpf(1.f, -ex);
        qs[n] = fmaxf(qs[n] * __builtin_ldexpf(1.f, ex), 1e-30f);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float x0 = x[8 * kk + kv_perm(2 * w)] * down, x1 = x[8 * kk + kv_perm(2 * w + 1)] * down;
            const uint32_t hi = pack_f16(x0, x1);
            qf[n][kk][w] = hi ^ turn;
            if constexpr (LOW) ql[n][kk][w] = kv_low(hi, x0, x1) ^ turn;
          }
        }
      }
    }

    float m[NQ], l[NQ], lag[NQ];
    f32x4 o[NQ][DL];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      m[n] = KV_NEG_INF;
      lag[n] = KV_LAG / qs[n];
      l[n] = 0.f;
#pragma unroll
      for (int i = 0; i < DL; ++i) o[n][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // INT4: sums and outputs are in units of 2^ve, 2^ve the power of two below the
    // largest value scale seen: the products stay inside fp16 (whose least is 2^-24)
    int ve = -30;

    // Values that are not finite, taken out of a tile that some query does not
    // see whole: the outputs of the queries that see them become what they are
    // (the sum's result whatever the probability), 16 keys at a time through
    // the wave's rows of `so`, and the tile holds 0 in their place.
    constexpr uint32_t EXPO = T == KV_BF16 ? 0x7f80u : 0x7c00u;
    auto take_out = [&](int key0) {
#pragma unroll
      for (int kb = 0; kb < 2 * KP; ++kb) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            uint32_t& x = vr[4 * kb + j][w];
            const uint32_t lo = x & 0xffffu, hi = x >> 16;
            const bool bl = (lo & EXPO) == EXPO, bh = (hi & EXPO) == EXPO;
            float f[8];
            kv_widen8<T>(u32x4{x, 0u, 0u, 0u}, f);
            so[wave][4 * g + j][DL * r + 2 * w] = bl ? f[0] : 0.f;
            so[wave][4 * g + j][DL * r + 2 * w + 1] = bh ? f[1] : 0.f;
            x = (bl ? 0u : lo) | (bh ? 0u : hi << 16);
          }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
        for (int k = 0; k < 16; ++k) {
          const int key = key0 + 16 * kb + k;
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            const bool in = key >= kfirst && key <= klast && (!a.causal || key <= qpos[n]) &&
                            (a.window <= 0 || key > qpos[n] - a.window);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int i = 0; i < DL; i += 4) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(&so[wave][k][(4 * g + e) * DL + i]);
#pragma unroll
                for (int x = 0; x < 4; ++x) o[n][i + x][e] += in ? v[x] : 0.f;
                asm volatile("" ::: "memory");
              }
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
    };
    for (; work && t <= t1; t += NW) {
      // the last tile is loaded again (from near caches) rather than nothing:
      // without branches around the loads each wait is for its own data alone
      const int key0 = TK * t, next0 = t + NW <= t1 ? key0 + TK * NW : key0;
      // every row sees the whole tile? (wave-uniform)
      const bool full = key0 >= (a.window > 0 ? max(kfirst, p0 + nq - a.window) : kfirst) &&
                        key0 + TK - 1 <= (a.causal ? min(klast, p0) : klast);
      auto key_of = [&](int s) { return key0 + 16 * (s >> 2) + 4 * g + (s & 3); };
      float ks[8 * KP], vs[8 * KP];
      if constexpr (INT4) {
#pragma unroll
        for (int s = 0; s < 8 * KP; s += 2) {
          const uint32_t w = ksr[s >> 2][(s >> 1) & 1];
          const f16x2_t h = kv_scale2(w);
          ks[s] = (float)h[0];
          ks[s + 1] = (float)h[1];
        }
      }
      // S^T: sc[n][4 kb + e] is key 16 kb + 4 g + e
      float sc[NQ][8 * KP];
#pragma unroll
      for (int kb = 0; kb < 2 * KP; ++kb) {
        u32x4 kf[KK];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          if constexpr (INT4) kf[kk] = kv_codes8(kr[kb][0][kk]);
          else kf[kk] = kr[kb][kk];
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) {
            acc = kv_mfma16<MT>(kf[kk], qf[n][kk], acc);
            if constexpr (LOW) acc = kv_mfma16<MT>(kf[kk], ql[n][kk], acc);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][4 * kb + e] = acc[e];
        }
      }
      const int pages = kv_page(a, entry);
      entry = look_up(next0 + TK * NW);
      fetch_k(next0, pages);
      const bool inner = key0 >= kfirst && key0 + TK - 1 <= klast;  // wave-uniform
      if constexpr (INT4) {
        // the scales' largest, as bits: they are not negative
        u16x2 big = {0, 0};
#pragma unroll
        for (int kb = 0; kb < 2 * KP; ++kb) {
          const uint32_t w0 = vsr[kb].x, w1 = vsr[kb].y;
          big = absmax16(absmax16(big, w0), w1);
        }
#pragma unroll
        for (int s = 0; s < 8 * KP; ++s) {
          const uint32_t w = vsr[s >> 2][(s >> 1) & 1];
          vs[s] = (float)__builtin_bit_cast(_Float16, (uint16_t)(s & 1 ? w >> 16 : w & 0xffffu));
        }
        float top = (float)__builtin_bit_cast(_Float16, (uint16_t)absmax16(big));
        if (__any(!(top < __builtin_ldexpf(1.f, ve + 1)))) {
          // of the keys that count, without infinities and NaN
          top = 0.f;
#pragma unroll
          for (int s = 0; s < 8 * KP; ++s)
            if (key_of(s) >= kfirst && key_of(s) <= klast && vs[s] < 65536.f) top = fmaxf(top, vs[s]);
#pragma unroll
          for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x, 64));
          // (of 0 the exponent would be 0: the largest may be that of a key which does not count)
          const int e = top > 0.f ? max(ve, __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(top) - 1)) : ve;
          const float f = __builtin_ldexpf(1.f, ve - e);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            l[n] *= f;
#pragma unroll
            for (int i = 0; i < DL; ++i) o[n][i] *= f;
          }
          ve = e;
        }
      } else if (!inner) {
        // what lies outside [kfirst, klast] may be anything: the values become 0
#pragma unroll
        for (int s = 0; s < 8 * KP; ++s) {
          const bool in = key_of(s) >= kfirst && key_of(s) <= klast;
#pragma unroll
          for (int w = 0; w < VW; ++w) vr[s][w] = in ? vr[s][w] : 0u;
        }
      }
      u32x4 pf[NQ][KP];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float top = KV_NEG_INF;
#pragma unroll
        for (int s = 0; s < 8 * KP; ++s) {
          if constexpr (INT4) sc[n][s] *= ks[s];
          if (!full) {
            const int key = key_of(s);
            const bool in = key >= kfirst && key <= klast && (!a.causal || key <= qpos[n]) &&
                            (a.window <= 0 || key > qpos[n] - a.window);
            sc[n][s] = in ? sc[n][s] : KV_NEG_INF;
          }
          top = fmaxf(top, sc[n][s]);
        }
        if (__any(top > m[n] + lag[n])) {
          top = fmaxf(top, __shfl_xor(top, 16, 64));
          top = fmaxf(top, __shfl_xor(top, 32, 64));
          const float mn = fmaxf(m[n], top);
          const float al = m[n] == KV_NEG_INF ? 1.f : __builtin_amdgcn_exp2f((m[n] - mn) * qs[n]);  // 1: l and o are 0
          l[n] *= al;
#pragma unroll
          for (int i = 0; i < DL; ++i) o[n][i] *= al;
          m[n] = mn;
        }
        const float base = -kv_base(m[n]) * qs[n] - (INT4 ? (float)ve : 0.f) + KV_UP<MT>;
        float p[8 * KP];
#pragma unroll
        for (int s = 0; s < 8 * KP; ++s) {
          p[s] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][s], qs[n], base));
          l[n] += p[s];
          if constexpr (INT4) p[s] *= vs[s];
        }
        if (INT4 && !full) {  // whatever the scale of a masked place is
#pragma unroll
          for (int s = 0; s < 8 * KP; ++s) p[s] = sc[n][s] == KV_NEG_INF ? 0.f : p[s];
        }
#pragma unroll
        for (int w = 0; w < 4 * KP; ++w) pf[n][w / 4][w % 4] = kv_pack<MT>(p[2 * w], p[2 * w + 1]);
      }
      // O^T: product i yields dim DL r + i
      if constexpr (INT4) {
#pragma unroll
        for (int kp = 0; kp < KP; ++kp)
#pragma unroll
          for (int i = 0; i < DL; i += 2) {
            u32x4 f0, f1;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              // byte i / 2 of two keys' words, each alone in a half, offset by 8
              const int s = 8 * kp + 2 * w;
              const uint32_t x = __builtin_amdgcn_perm(vr[s + 1][0], vr[s][0], 0x0c040c00u + 0x00010001u * (i / 2)) ^ 0x00880088u;
              f0[w] = kv_code_lo(x);
              f1[w] = kv_code_hi(x);
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              o[n][i] = kv_mfma16<MT>(f0, pf[n][kp], o[n][i]);
              o[n][i + 1] = kv_mfma16<MT>(f1, pf[n][kp], o[n][i + 1]);
            }
          }
      } else {
        if (MANY && !full && nq > 1) {
          // a masked probability of 0 does not hide a value that is not finite
          u16x2 top = {0, 0};
#pragma unroll
          for (int s = 0; s < 8 * KP; ++s)
#pragma unroll
            for (int w = 0; w < VW; ++w) top = absmax16(top, vr[s][w]);
          if (__any(kv_not_finite<T>(top))) take_out(key0);
        }
#pragma unroll
        for (int kp = 0; kp < KP; ++kp)
#pragma unroll
          for (int i = 0; i < DL; ++i) {
            u32x4 f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int s = 8 * kp + 2 * w;
              f[w] = __builtin_amdgcn_perm(vr[s + 1][i / 2 % VW], vr[s][i / 2 % VW], (i & 1) ? 0x07060302u : 0x05040100u);
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n) o[n][i] = kv_mfma16<MT>(f, pf[n][kp], o[n][i]);
          }
      }
      fetch_v(next0, pages);
    }

    // join the waves, 16 queries at a time, through LDS
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float ls = l[n];
      ls += __shfl_xor(ls, 16, 64);
      ls += __shfl_xor(ls, 32, 64);
      __syncthreads();  // the rows of the last round, or sequence, have been read
      // lane (q = r, g): dims (4 g + e) DL + i
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < DL; i += 4)
          *reinterpret_cast<f32x4*>(&so[wave][r][(4 * g + e) * DL + i]) =
              f32x4{o[n][i][e], o[n][i + 1][e], o[n][i + 2][e], o[n][i + 3][e]};
      if (g == 0) {
        sm[wave][r] = m[n] == KV_NEG_INF ? m[n] : m[n] * qs[n] + (INT4 ? (float)ve : 0.f) - KV_UP<MT>;
        sl[wave][r] = ls;
      }
      __syncthreads();
      const int row = 16 * n + (int)threadIdx.x / LR, i0 = threadIdx.x % LR;
      if ((int)threadIdx.x < 16 * LR && row < rows) {
        const int q = row & 15, tok = row / a.group, head = h * a.group + row % a.group;
        float mx = KV_NEG_INF;
#pragma unroll
        for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm[w][q]);
        float sum = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = __builtin_amdgcn_exp2f(sm[w][q] - kv_base(mx));
          sum += f * sl[w][q];
          // a wave that saw nothing for this row adds nothing
          const bool none = sm[w][q] == KV_NEG_INF && sl[w][q] == 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] += none ? 0.f : f * so[w][q][8 * i0 + e];
        }
        if ((uint32_t)(q0 + tok) < (uint64_t)a.q_tokens) {
          if (whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= inv;
            if constexpr (INT4) kv_row_rht<D, 8, true>(x, i0, 1, lane, a.c.signs);
            stg<u32x4>(a.out + (int64_t)(q0 + tok) * a.o_tok + (int64_t)head * a.o_head + 16 * i0, kv_round8<T>(x));
            if (a.lse && i0 == 0)
              a.lse[(int64_t)(q0 + tok) * a.heads + head] =
                  sum == 0.f ? KV_NEG_INF : (mx + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
          } else {
            const int64_t pr = ((int64_t)(run + b) * a.c.kv_heads + h) * a.rows + row;
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
    if (a.blocks == 0) return;
    if (from == 0 && h == 0 && threadIdx.x == 0) {
      a.reach[2 * b] = run;
      a.reach[2 * b + 1] = share.of(u + sp.units - 1);  // the run with its last unit
    }
    u += take;
    at = 0;
    // `so` has been read: the next sequence's take_out writes it before its first barrier
    if (MANY && u < u1) __syncthreads();
  }
}

// Joins the pieces a row's keys were split into, in order of the keys.
// Pieces of a row are at piece(i), i in [0, n); `gr` groups of D / 8 lanes
// share a row when there are few rows and many pieces.
template <int D, int T, bool INT4, typename P>
__device__ __forceinline__ void kv_join_row(const KvAttnArgs& a, int64_t tok, int head, bool live, int n, int gr, P piece) {
  constexpr int LR = D / 8, PAD = D + 4;
  __shared__ __attribute__((aligned(16))) float so[256 / LR][PAD];
  __shared__ float sm[256 / LR], sl[256 / LR];
  const int grp = threadIdx.x / LR, i0 = threadIdx.x % LR, lane = threadIdx.x & 63;
  const int part = grp % gr;
  float mx = KV_NEG_INF, sum = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto add = [&](float m1, float l1, const float* y) {
    const float mn = fmaxf(mx, m1), f0 = __builtin_amdgcn_exp2f(mx - kv_base(mn)), f1 = __builtin_amdgcn_exp2f(m1 - kv_base(mn));
    const bool none = m1 == KV_NEG_INF && l1 == 0.f;  // saw nothing
    const bool old = mx == KV_NEG_INF && sum == 0.f;
    sum = (old ? 0.f : f0 * sum) + (none ? 0.f : f1 * l1);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (old ? 0.f : f0 * x[e]) + (none ? 0.f : f1 * y[e]);
    mx = mn;
  };
  if (live)
    for (int s = part; s < n; s += gr) {
      const int64_t pr = piece(s);
      const float m1 = a.part_ml[2 * pr], l1 = a.part_ml[2 * pr + 1];
      const f32x4 u = ldg<f32x4>(a.part_o + pr * D + 8 * i0), w = ldg<f32x4>(a.part_o + pr * D + 8 * i0 + 4);
      const float y[8] = {u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]};
      add(m1, l1, y);
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
    for (int p = 1; p < min(gr, n); ++p) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = so[grp + p][8 * i0 + e];
      add(sm[grp + p], sl[grp + p], y);
    }
  }
  if (!live) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= inv;
  if constexpr (INT4) kv_row_rht<D, 8, true>(x, i0, 1, lane, a.c.signs);
  stg<u32x4>(a.out + tok * a.o_tok + head * a.o_head + 16 * i0, kv_round8<T>(x));
  if (a.lse && i0 == 0) a.lse[tok * a.heads + head] = sum == 0.f ? KV_NEG_INF : (mx + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

// of the chunk kernel: pieces by split, one row of the call after another
template <int D, int T, bool INT4>
__global__ __launch_bounds__(256) void k_kv_join(const KvAttnArgs a, int gr) {
  const int64_t rows = a.q_tokens * a.heads;
  const int64_t row = (int64_t)blockIdx.x * (256 / (D / 8) / gr) + threadIdx.x / (D / 8) / gr;
  // (a 64-bit division takes a microsecond)
  const int64_t tok = rows >> 31 ? row / a.heads : (uint32_t)row / (uint32_t)a.heads;
  kv_join_row<D, T, INT4>(a, tok, (int)(row - tok * a.heads), row < rows, a.splits, gr,
                          [&](int s) { return (int64_t)s * rows + row; });
}
// of the step kernel: a block per sequence, head and `16 or 32 / gr` of its rows
template <int D, int T, bool INT4>
__global__ __launch_bounds__(256) void k_kv_step_join(const KvAttnArgs a, int gr, int parts) {
  const int part = blockIdx.x % parts, h = blockIdx.x / parts % a.c.kv_heads, b = a.launched + blockIdx.x / parts / a.c.kv_heads;
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], i0 = a.reach[2 * b], i1 = a.reach[2 * b + 1];
  const int rows = min(q1 - q0, a.rows / a.group) * a.group;  // as kv_span counts them: with none there is no reach
  if (rows <= 0 || i0 == i1) return;
  const int row = part * (256 / (D / 8) / gr) + threadIdx.x / (D / 8) / gr;
  const int tok = q0 + row / a.group;
  const bool live = row < rows && (uint32_t)tok < (uint64_t)a.q_tokens;
  kv_join_row<D, T, INT4>(a, tok, h * a.group + row % a.group, live, i1 - i0 + 1, gr, [&](int s) {
    return ((int64_t)(i0 + s + b) * a.c.kv_heads + h) * a.rows + row;
  });
}

template <int D, int T, bool INT4>
static hipError_t step_launch(KvAttnArgs a, int nq, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.c.kv_heads * (a.blocks ? a.blocks : a.seqs)));
  // 16-bit pages: at most 16 rows, INT4: at most 32 and one kernel for single tokens and chunks
  const bool many = !INT4 && a.rows > a.group;
  if (nq == 1 && !many && a.blocks == 0) hipLaunchKernelGGL((k_kv_step<D, T, INT4, 1, 8, false>), grid, dim3(512), 0, s, a);
  else if (nq == 1 && !many) hipLaunchKernelGGL((k_kv_step<D, T, INT4, 1, 4, false>), grid, dim3(256), 0, s, a);
  if constexpr (INT4) {
    if (nq == 2) hipLaunchKernelGGL((k_kv_step<D, T, true, 2, 4, false>), grid, dim3(256), 0, s, a);
  } else {
    if (many && a.blocks == 0) hipLaunchKernelGGL((k_kv_step<D, T, false, 1, 8, true>), grid, dim3(512), 0, s, a);
    else if (many) hipLaunchKernelGGL((k_kv_step<D, T, false, 1, 4, true>), grid, dim3(256), 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.blocks == 0) return e;
  // as many groups a row as keep the machine busy
  int gr = 1;
  const int most = 256 / (D / 8);
  const int64_t rows = a.q_tokens * a.heads;
  while (gr < most && gr < a.blocks && rows * gr < 8192) gr *= 2;
  const int per = most / gr, parts = (a.rows + per - 1) / per;
  const int most_seqs = (int)std::min<int64_t>(a.seqs, kLaunchThreads / 256 / ((int64_t)a.c.kv_heads * parts));
  for (a.launched = 0; e == hipSuccess && a.launched < a.seqs; a.launched += most_seqs) {
    const int n = std::min(a.seqs - a.launched, most_seqs);
    hipLaunchKernelGGL((k_kv_step_join<D, T, INT4>), dim3((unsigned)(n * a.c.kv_heads * parts)), dim3(256), 0, s, a, gr, parts);
    e = hipGetLastError();
  }
  return e;
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

// Keys of a unit of the step kernel (one tile for each wave of a block).
int kv_step_unit(int dim, bool int4, bool whole) { return (dim == 128 && !int4 ? 32 : 64) * (whole ? 8 : 4); }

hipError_t launch_kv_step(const KvAttnArgs& a, int dim, int dt, bool int4, int nq, hipStream_t s) {
  return KV_PICK(step_launch, dim, dt, int4, a, nq, s);
}
hipError_t launch_kv_join(const KvAttnArgs& a, int dim, int dt, bool int4, hipStream_t s) {
  return KV_PICK(join_launch, dim, dt, int4, a, s);
}

}  // namespace whtq
