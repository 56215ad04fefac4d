// Attention of a chunk of new tokens over a paged cache.
//
// A block owns 32 NW rows (chunk tokens x query group of one key/value head,
// the group innermost) and walks the keys they see in tiles of 64, double
// buffered in LDS; each of its NW waves owns 32 rows, one per lane column.
// MFMA 32 x 32 x 16:
//   S^T = K Q^T   A: 16-byte row reads of the K tile, B: Q^T kept in registers;
//   O^T = V^T P^T A: ds_read_b64_tr_b16 of the V tile (4 keys of one dim per
//                 lane), B: the lane's own probabilities, keys in the order
//                 the scores came out in.
// Tiles are swizzled (16-byte chunk index XOR row) so that the row reads and
// the transposing reads spread over the banks.  16-bit pages are copied to
// LDS directly; INT4 codes go through registers and are stored as exact fp16.
// Softmax in one pass: a row's maximum may lag (KV_LAG), sums are fp32 of the
// unrounded probabilities.  32 rows a wave, because 64 (half the LDS reads)
// need more registers than there are at two waves a SIMD.
//
// Measured (kernel times): a prompt of 8192 tokens, 32 heads of 128, bf16:
// 550 GFLOP in 580 to 620 us in a row, 660 among other kernels, 835 to 950
// TFLOP/s (a large bf16 product of the library: 1300);
// the matrix pipes are busy half the time and the vector pipes (32 exp2 and
// about 170 other operations a tile and lane) the other half, the two blocks of
// a CU overlapping little, at about 1.9 GHz.  512 tokens over 33000 INT4 keys,
// 64 heads on 8 of 128: 549 GFLOP in 600 to 675 us and 10 us for the join.  Six
// fp16 chunks of 5 to 1500 tokens under a window of 1000, 24 heads on 8 of
// 64: 35 us, 1.25 us a tile of two waves a SIMD, about 10 us before and after.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kv_attn.hpp"
#include "launch.hpp"

namespace whtq {

constexpr int KV_TILE = 64;
constexpr int KB = KV_TILE / 32;

// the kernel's parts are lambdas, written once and used in several places
#define KV_INLINE __attribute__((always_inline))

typedef short kv_s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 kv_tr_read(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) kv_s16x4*)p));
}

// Chunk (16 bytes) of a tile row at which chunk c is kept.  LDS has 64 banks,
// 256 bytes: a tile row of D = 128, two of D = 64.  K is read as one chunk of
// 16 rows at a time, V as 32 bytes of 4 rows twice side by side; either way
// the reads of a quarter or half wave fall on different banks.
template <int D>
__device__ __forceinline__ int kv_k_at(int row, int c) {
  return D == 128 ? c ^ (row & 15) : c ^ ((row >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int kv_v_at(int row, int c) {
  return D == 128 ? c ^ (4 * (row & 3)) ^ (2 * ((row >> 2) & 1)) : c ^ (4 * ((row >> 1) & 1));
}

// INT4: the order in which the lane that unpacks unit c (32 codes, 4 chunks) of
// a row stores them: chunk j ^ this at step j.
template <int D>
__device__ __forceinline__ int kv_turn(bool v, int row, int c) {
  return (D == 128 ? c & 2 : 2 * (row & 1)) | (v ? c & 1 : 0);
}

template <int D, int T, bool INT4, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_kv_chunk(const KvAttnArgs a) {
  constexpr int MT = INT4 ? KV_F16 : T;
  constexpr bool LOW = INT4 && T == KV_F16;  // the queries' low parts count, see qf
  constexpr int ROWS = 32 * NW, CH = D / 8, ROWB = 2 * D;  // 16-byte chunks and bytes of a tile row
  constexpr int KK = D / 16, DB = D / 32;
  constexpr int TILEB = KV_TILE * ROWB;
  // Each buffer is a variable of its own and the walk is written for both, so
  // that the compiler can tell a read of one from a copy into the other:
  // otherwise it waits for the copies of the next tile before it reads this one.
  __shared__ __attribute__((aligned(16))) uint8_t sk0[TILEB], sk1[TILEB], sv0[TILEB], sv1[TILEB];
  __shared__ __attribute__((aligned(16))) float sks[2][INT4 ? KV_TILE : 1], svs[2][INT4 ? KV_TILE : 1];
  __shared__ u32x4 sql[NW][LOW ? D / 16 : 1][64];
  auto skb = [&](auto buf) KV_INLINE -> uint8_t* { return buf.value ? sk1 : sk0; };
  auto svb = [&](auto buf) KV_INLINE -> uint8_t* { return buf.value ? sv1 : sv0; };

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int qc = lane & 31, hf = lane >> 5;

  // block -> (tile of rows, head, split).  Blocks are dealt to the 8 XCDs in
  // turn; whole groups of one head and split go to one XCD each, so that its
  // L2 holds their keys (groups beyond a multiple of 8 are spread over all).
  // Later tiles of a causal chunk are longer and go first.
  const int groups = a.c.kv_heads * a.splits, per = a.grid / groups, whole = groups / 8 * 8;
  const int block = a.launched + blockIdx.x;
  int hs, slot;
  if (block < whole * per) {
    const int i = block >> 3;
    hs = i / per * 8 + (block & 7);
    slot = i % per;
  } else {
    const int i = block - whole * per;
    hs = whole + i / per;
    slot = i % per;
  }
  slot = per - 1 - slot;
  const int h = hs % a.c.kv_heads, split = hs / a.c.kv_heads;
  // sequence b owns the slots from q_start[b] * group / ROWS + b on (rounded
  // down: at least as many as its rows fill)
  int b = 0;
  for (int step = 1 << (31 - __builtin_clz(a.seqs)); step; step >>= 1)
    if (b + step < a.seqs && (int64_t)a.q_start[b + step] * a.group / ROWS + b + step <= slot) b += step;
  const int q0 = a.q_start[b], chunk = a.q_start[b + 1] - q0;
  // (rows of a head are below 2^30, so that these are 32-bit)
  const int row0 = (int)(slot - ((int64_t)q0 * a.group / ROWS + b)) * ROWS;
  const int rows = chunk * a.group;
  if (row0 < 0 || row0 >= rows) return;
  const int kv = kv_held(a, a.kv_len[b]);
  const int p0 = kv - chunk;
  const int32_t* table = a.table + b * a.table_stride;

  // first and last position among rows [r0, r0 + n) that exist
  const int tok0 = row0 / a.group, tok1 = (min(row0 + ROWS, rows) - 1) / a.group;
  const int first = a.window > 0 ? max(0, p0 + tok0 - a.window + 1) : 0;
  const int last = a.causal ? min(kv - 1, p0 + tok1) : kv - 1;
  // the split's share of the block's tiles
  const int b0 = first / KV_TILE, bn = max(0, last / KV_TILE - b0 + 1);
  const int kfirst = max(first, (b0 + (int)((int64_t)bn * split / a.splits)) * KV_TILE);
  const int klast = min(last, (b0 + (int)((int64_t)bn * (split + 1) / a.splits)) * KV_TILE - 1);
  // The lane's query.  Its scores are kept in units of 1 / qs, qs > 0 (0 would
  // turn a masked -inf into NaN; 1e-30 gives the same results, for INT4, whose
  // power of two takes part, because a score is below 2^27): a negative scale
  // turns q around.
  const int row = row0 + 32 * wave + qc;
  const int tok = row / a.group, head = h * a.group + row % a.group;
  const bool live = row < rows && (uint32_t)(q0 + tok) < (uint64_t)a.q_tokens;
  const int pos = p0 + tok;
  // INT4: the rotated query is rounded to fp16 for its product, 2^-12 of each
  // value.  bf16 outputs hide that (it adds 1 % to their own 2^-9); fp16
  // outputs would be off by twice their own rounding, so there what the
  // rounding dropped goes into a second product, from LDS.
  float qs = fmaxf(fabsf(a.scale), 1e-30f);
  u32x4 qf[KK];
  {
    const uint32_t turn = a.scale < 0.f ? 0x80008000u : 0u;
    const uint8_t* qp = a.q + (int64_t)(q0 + tok) * a.q_tok + (int64_t)head * a.q_head;
    u32x4 raw[KK];
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) raw[kk] = live ? ldg<u32x4>(qp + 32 * kk + 16 * hf) : u32x4{0u, 0u, 0u, 0u};
    if constexpr (!INT4) {
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) qf[kk] = raw[kk] ^ turn;
    } else {
      // the lane holds chunks 2 kk + hf of its row: chunk bit 0 is the lane's half
      float x[8 * KK];
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        kv_widen8<T>(raw[kk], x + 8 * kk);
        const int c = 2 * kk + hf;
        if (a.c.signs) kv_sign8(x + 8 * kk, (a.c.signs[c >> 2] >> (8 * (c & 3))) & 255u);
      }
      kv_bfly<8 * KK>(x);
      kv_lane_bfly<8 * KK>(x, 32, lane);
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8 * KK; ++e) {
        x[e] *= D == 64 ? 0.125f : 0.08838834764831845f;  // 1 / sqrt(D)
        top = fmaxf(top, fabsf(x[e]));
      }
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      // an exact power of two brings the row's largest value to [1, 2)
      const int ex = top > 0.f && top < __builtin_huge_valf() ? max(-126, min(126, __builtin_amdgcn_frexp_expf(top) - 1)) : 0;
      const float down = __builtin_ldexpf(1.f, -ex);
      qs = fmaxf(qs * __builtin_ldexpf(1.f, ex), 1e-30f);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        u32x4 low;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float x0 = x[8 * kk + kv_perm(2 * w)] * down, x1 = x[8 * kk + kv_perm(2 * w + 1)] * down;
          const uint32_t hi = pack_f16(x0, x1);
          qf[kk][w] = hi ^ turn;
          if constexpr (LOW) low[w] = kv_low(hi, x0, x1) ^ turn;
        }
        if constexpr (LOW) sql[wave][kk][lane] = low;
      }
    }
  }
  const float lag = KV_LAG / qs;
  float m = KV_NEG_INF, l = 0.f;
  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  int ve = -30;  // INT4: the outputs are in units of 2^ve (fp16's least scale is 2^-24)

  const uint8_t* kbase = a.c.k.p + h * a.c.k.head;
  const uint8_t* vbase = a.c.v.p + h * a.c.v.head;

  // --- tile loads.  Keys outside [kfirst, klast] are replaced by the nearest
  // inside, so a tile holds only keys that some row sees.
  constexpr int CR = 64 / CH;                  // rows of one copy instruction (4 or 8; in one page)
  constexpr int COPIES = KV_TILE / (CR * NW);  // copy instructions of a wave for K, and for V
  const int lr = lane / CH, pmask = (1 << a.c.page_shift) - 1;
  // a lane's 16 bytes among the rows of a copy; the swizzle depends on the
  // row of the tile, (n NW + wave) CR + lr, which is the same modulo 16 for all n
  const int trl = wave * CR + lr;
  static_assert(NW * CR % 16 == 0, "swizzle alike for every copy");
  const uint32_t kswz = 16 * kv_k_at<D>(trl, lane % CH), vswz = 16 * kv_v_at<D>(trl, lane % CH);
  const uint32_t ktok = (uint32_t)a.c.k.tok, vtok = (uint32_t)a.c.v.tok;
  auto copy_key = [&](int n, int key0) KV_INLINE {  // first key of copy n, wave-uniform for a given n
    return min(max(key0 + (n * NW + wave) * CR, kfirst & ~(CR - 1)), klast & ~(CR - 1));
  };
  const uint32_t klane = lr * ktok + kswz, vlane = lr * vtok + vswz;
  // dense: lane n finds the places of copy n of K and of V (`page` there), the
  // others read them
  auto copy = [&](auto buf, int key0, int page) KV_INLINE {
    uint64_t from[2][COPIES];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint64_t at = (uint64_t)(v ? vbase : kbase) + (uint64_t)((int64_t)page * (v ? a.c.v.page : a.c.k.page)) +
                          (uint32_t)(copy_key(lane % COPIES, key0) & pmask) * (uint64_t)(v ? vtok : ktok);
#pragma unroll
      for (int n = 0; n < COPIES; ++n)
        from[v][n] = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(at >> 32), n) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane((int)at, n);
    }
    auto go = [&](int v, int n, uint32_t off) KV_INLINE {
      const __attribute__((address_space(1))) uint8_t* g = reinterpret_cast<const __attribute__((address_space(1))) uint8_t*>(from[v][n]);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(g + off),
                                       (__attribute__((address_space(3))) void*)((v ? svb(buf) : skb(buf)) + (n * NW + wave) * CR * ROWB),
                                       16, 0, 0);
    };
    if (key0 >= kfirst && key0 + KV_TILE - 1 <= klast) {
#pragma unroll
      for (int i = 0; i < 2 * COPIES; ++i) go(i / COPIES, i % COPIES, i / COPIES ? vlane : klane);
    } else {
#pragma unroll
      for (int n = 0; n < COPIES; ++n) {
        const int k0 = copy_key(n, key0);
        const uint32_t r = min(max(lr, kfirst - k0), klast - k0);
        go(0, n, r * ktok + kswz);
        go(1, n, r * vtok + vswz);
      }
    }
  };
  // INT4: unit u of a tile is 16 bytes (32 codes) of one row, first K's units,
  // then V's; wave 0 holds the keys' scales, wave 1 the values'
  constexpr int UR = D / 32;                   // units of a row
  constexpr int UNITS = KV_TILE * UR, UT = (2 * UNITS + 64 * NW - 1) / (64 * NW);
  u32x4 code[INT4 ? UT : 1];
  uint16_t scl = 0;
  auto unit_row = [&](int n) KV_INLINE { return (n * 64 * NW + (int)threadIdx.x) / UR % KV_TILE; };
  auto unit_of_v = [&](int n) KV_INLINE { return n * NW + wave >= UNITS / 64; };  // wave-uniform
  auto has_unit = [&](int n) KV_INLINE { return n * NW + wave < UNITS / 32; };
  auto inside = [&](int key) KV_INLINE { return min(max(key, kfirst), klast); };
  const bool has_scale = wave < 2;
  // Table entries of a tile, held by the lanes that need them: dense, copy n's
  // in lane n; INT4, of the thread's units and of its scale.  Memory answers
  // in order: they are asked for before the copies of the tile before.
  struct Pages {
    int at[INT4 ? UT + 1 : 1];
  };
  auto look_up = [&](Pages& p, int key0) KV_INLINE {
    if constexpr (INT4) {
#pragma unroll
      for (int n = 0; n < UT; ++n) p.at[n] = table[inside(key0 + unit_row(n)) >> a.c.page_shift];
      p.at[UT] = table[inside(key0 + lane) >> a.c.page_shift];
    } else {
      p.at[0] = table[copy_key(lane % COPIES, key0) >> a.c.page_shift];
    }
  };
  // Checked as soon as this tile has landed, before new loads go out: the
  // compiler then has nothing to wait for.
  auto check = [&](Pages& p) KV_INLINE {
#pragma unroll
    for (int n = 0; n < (INT4 ? UT + 1 : 1); ++n) {
      p.at[n] = kv_page(a, p.at[n]);
      asm volatile("" : "+v"(p.at[n]));
    }
  };
  auto fetch = [&](auto buf, int key0, const Pages& p) KV_INLINE {
    if constexpr (!INT4) {
      copy(buf, key0, p.at[0]);
    } else {
#pragma unroll
      for (int n = 0; n < UT; ++n)
        if (has_unit(n)) {
          const bool v = unit_of_v(n);
          code[n] = ldg_global<u32x4>((v ? vbase : kbase) + (int64_t)p.at[n] * (v ? a.c.v.page : a.c.k.page) +
                                      ((uint32_t)(inside(key0 + unit_row(n)) & pmask) * (v ? vtok : ktok) +
                                       16 * (threadIdx.x % UR)));
        }
      if (has_scale) {
        const KvSide& c = wave ? a.c.v : a.c.k;
        scl = c.scale[p.at[UT] * c.s_page + h * c.s_head + (inside(key0 + lane) & pmask)];
      }
    }
  };
  // INT4: the fetched codes and scales to LDS.  Stores of 16 bytes go 8 lanes
  // at a time, here 8 units of a row or two, in an order of its own each: they
  // fall on different banks.
  auto spread = [&](auto buf) KV_INLINE {
    if constexpr (INT4) {
#pragma unroll
      for (int n = 0; n < UT; ++n)
        if (has_unit(n)) {
          const bool v = unit_of_v(n);
          const int tr = unit_row(n), c = threadIdx.x % UR;
          const int turn = kv_turn<D>(v, tr, c);
          uint8_t* rowp = (v ? svb(buf) : skb(buf)) + tr * ROWB;
          u32x4 w = code[n];
          if (turn & 2) w = u32x4{w[2], w[3], w[0], w[1]};
          if (turn & 1) w = u32x4{w[1], w[0], w[3], w[2]};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = 4 * c + (j ^ turn);
            *reinterpret_cast<u32x4*>(rowp + 16 * (v ? kv_v_at<D>(tr, at) : kv_k_at<D>(tr, at))) = kv_codes8(w[j]);
          }
        }
      if (has_scale) (wave ? svs : sks)[buf][lane] = kv_scale(scl);
    }
  };

  // the keys [low, low + span] that the lane's row sees here
  int low = a.window > 0 ? max(kfirst, pos - a.window + 1) : kfirst;
  const int high = a.causal ? min(klast, pos) : klast;
  const uint32_t span = high < low ? 0u : (uint32_t)(high - low);
  if (high < low) low = INT32_MAX;  // none
  auto sees = [&](int key) KV_INLINE { return (uint32_t)(key - low) <= span; };
  // A probability of 0 does not hide a value that is not finite, so in a
  // tile that some row does not see whole such values are taken out: the
  // outputs of the rows that see them become what they are (the sum's result
  // whatever the probability), and the tile holds 0 in their place.
  auto wild = [&](auto buf) KV_INLINE {  // whether this thread's part of the V tile holds any
    bool any = false;
    if constexpr (INT4) {
      any = wave == 0 && !(svs[buf][lane] < 65536.f);
    } else {
      for (int i = threadIdx.x; i < TILEB / 16; i += 64 * NW) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(svb(buf) + 16 * i);
        u16x2 big = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = w[e];
          big = absmax16(big, x);
        }
        any = any || kv_not_finite<T>(big);
      }
    }
    return any;
  };
  constexpr uint32_t EXPO = T == KV_BF16 ? 0x7f80u : 0x7c00u;
  auto take_out = [&](auto buf, int key0) KV_INLINE {
#pragma unroll 1
    for (int j = 0; j < KV_TILE; ++j) {
      const uint8_t* rp = svb(buf) + j * ROWB;
      {
        const bool mine = sees(key0 + j);
        if constexpr (INT4) {
          const float bad = mine && !(svs[buf][j] < 65536.f) ? __builtin_nanf("") : 0.f;
#pragma unroll
          for (int d = 0; d < DB; ++d) o[d] += bad;
        } else {
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const u32x2 w = *reinterpret_cast<const u32x2*>(rp + 16 * kv_v_at<D>(j, 4 * d + jj) + 8 * hf);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t x = w[e >> 1], b = e & 1 ? x >> 16 : x & 0xffffu;
                const float v = T == KV_BF16 ? as_f(b << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)b);
                o[d][4 * jj + e] += mine && (b & EXPO) == EXPO ? v : 0.f;
              }
            }
        }
      }
    }
    __syncthreads();
    if constexpr (INT4) {
      if (wave == 0 && !(svs[buf][lane] < 65536.f)) svs[buf][lane] = 0.f;
    } else {
      for (int i = threadIdx.x; i < TILEB / 4; i += 64 * NW) {
        uint32_t* p = reinterpret_cast<uint32_t*>(svb(buf)) + i;
        const uint32_t x = *p;
        *p = ((x & EXPO) == EXPO ? 0u : x & 0xffffu) | ((x >> 16 & EXPO) == EXPO ? 0u : x & 0xffff0000u);
      }
    }
    __syncthreads();
  };
  const int ln = lane & 15, dg = (lane >> 4) & 1;
  auto scores = [&](f32x16 (&s)[KB], auto buf) KV_INLINE {
    // S^T: lane (qc, hf), s[kb][4 j + e] is key 32 kb + 8 j + 4 hf + e.  Reads
    // run AHEAD products before their use, the order laid down.
    constexpr int AHEAD = LOW ? 4 : 8;
    u32x4 f[KB][KK], low[LOW ? KK : 1];
    auto read = [&](int i) KV_INLINE {
      const int kb = i % KB, kk = i / KB, tr = 32 * kb + qc;
      f[kb][kk] = *reinterpret_cast<const u32x4*>(skb(buf) + tr * ROWB + 16 * kv_k_at<D>(tr, 2 * kk + hf));
      if constexpr (LOW)
        if (kb == 0) low[kk] = sql[wave][kk][lane];
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) read(i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[kb][e] = 0.f;
#pragma unroll
    for (int i = 0; i < KB * KK; ++i) {
      s[i % KB] = kv_mfma32<MT>(f[i % KB][i / KB], qf[i / KB], s[i % KB]);
      if constexpr (LOW) s[i % KB] = kv_mfma32<MT>(f[i % KB][i / KB], low[i / KB], s[i % KB]);
      if (i + AHEAD < KB * KK) read(i + AHEAD);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // the new scores masked and (INT4) scaled, and the maximum they call for;
  // both stay in units of 1 / qs
  auto settle = [&](f32x16 (&s)[KB], auto buf, int key0, bool masked) KV_INLINE {
    if constexpr (INT4) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 ksc = *reinterpret_cast<const f32x4*>(&sks[buf][32 * kb + 8 * j + 4 * hf]);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[kb][4 * j + e] *= ksc[e];
        }
    }
    if (masked) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          s[kb][e] = sees(key0 + 32 * kb + 8 * (e >> 2) + 4 * hf + (e & 3)) ? s[kb][e] : KV_NEG_INF;
    }
    float top = KV_NEG_INF;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[kb][e]);
    if (__any(top > m + lag)) {
      const float mn = fmaxf(m, fmaxf(top, __shfl_xor(top, 32, 64)));
      const float al = m == KV_NEG_INF ? 1.f : __builtin_amdgcn_exp2f((m - mn) * qs);  // 1: l is 0, o 0 or not finite
      l *= al;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= al;
      m = mn;
    }
  };
  // probabilities from settled scores, as the second product's operand: slots
  // 0..7 of 16 keys are words 4 j', 4 j' + 2 of their scores
  auto probs = [&](f32x16 (&s)[KB], u32x4 (&pf)[2 * KB], auto buf) KV_INLINE {
    if constexpr (INT4) {
      // INT4: sum and outputs are in units of 2^ve, 2^ve the power of two below
      // the largest value scale seen: the products stay inside fp16
      float vtop = svs[buf][lane % KV_TILE];
      vtop = vtop < 65536.f ? vtop : 0.f;
      if (__any(vtop >= __builtin_ldexpf(1.f, ve + 1))) {
#pragma unroll
        for (int x = 1; x < 64; x *= 2) vtop = fmaxf(vtop, __shfl_xor(vtop, x, 64));
        const int e = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(vtop) - 1);
        const float f = __builtin_ldexpf(1.f, ve - e);
        l *= f;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] *= f;
        ve = e;
      }
    }
    const float base = -kv_base(m) * qs - (INT4 ? (float)ve : 0.f) + KV_UP<MT>;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][4 * j + e], qs, base));
#pragma unroll
        for (int e = 0; e < 4; ++e) l += p[e];  // before they are rounded: lse is good to fp32
        if constexpr (INT4) {
          const f32x4 vsc = *reinterpret_cast<const f32x4*>(&svs[buf][32 * kb + 8 * j + 4 * hf]);
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] *= vsc[e];
        }
        pf[2 * kb + j / 2][2 * (j & 1)] = kv_pack<MT>(p[0], p[1]);
        pf[2 * kb + j / 2][2 * (j & 1) + 1] = kv_pack<MT>(p[2], p[3]);
      }
  };
  auto outputs = [&](u32x4 (&pf)[2 * KB], auto buf) KV_INLINE {
    // O^T: product of 16 keys: lane (dim qc of 32, hf) needs keys 4 hf .. and 8 + 4 hf ..
#pragma unroll
    for (int ks = 0; ks < 2 * KB; ++ks)
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        u32x4 f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tr = 16 * ks + 8 * u + 4 * hf + (ln >> 2);
          const int cc = 4 * d + 2 * dg + ((ln & 3) >> 1);
          const u32x2 w = kv_tr_read(svb(buf) + tr * ROWB + 16 * kv_v_at<D>(tr, cc) + 8 * (ln & 1));
          f[2 * u] = w.x;
          f[2 * u + 1] = w.y;
        }
        o[d] = kv_mfma32<MT>(f, pf[ks], o[d]);
      }
  };

  const bool work = kfirst <= klast;
  const int t0 = kfirst / KV_TILE, t1 = klast / KV_TILE;
  // Among tokens [i0, i1]: tiles [f0, f1) that every one sees whole, and tiles
  // [n0, n1] that one of them sees any of.
  struct Range {
    int f0, f1, n0, n1;
  };
  auto range = [&](int i0, int i1) KV_INLINE {
    const int w0 = a.window > 0 ? max(kfirst, p0 + i1 - a.window + 1) : kfirst, w1 = a.causal ? min(klast, p0 + i0) : klast;
    const int s0 = a.window > 0 ? max(kfirst, p0 + i0 - a.window + 1) : kfirst, s1 = a.causal ? min(klast, p0 + i1) : klast;
    // (w1 and s1 may be negative: none)
    return Range{(w0 + KV_TILE - 1) / KV_TILE, (w1 + 1) / KV_TILE, s0 / KV_TILE, s1 < s0 ? -1 : s1 / KV_TILE};
  };
  const Range br = range(tok0, tok1);
  const int wrow = row0 + 32 * wave;
  Range wr = range(wrow / a.group, (min(wrow + 32, rows) - 1) / a.group);
  if (wrow >= rows) wr.n1 = -1;
  auto masked = [&](const Range& r, int t) KV_INLINE { return t < r.f0 || t >= r.f1; };
  constexpr std::false_type B0{};
  constexpr std::true_type B1{};
  f32x16 s[KB];
  u32x4 pf[2 * KB];
  // Tiles go to the two buffers in turn; the next one is asked for before
  // this one is worked on.
  Pages later = {};  // table entries of the next tile to be asked for
  auto ask = [&](int t, auto buf) KV_INLINE {
    Pages now = later;
    check(now);
    look_up(later, (t + 1) * KV_TILE);
    fetch(buf, t * KV_TILE, now);
  };
  auto visit = [&](int t, auto buf, auto other) KV_INLINE {
    // this tile has landed, and every wave is done with the other buffer
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (t < t1) ask(t + 1, other);
    if (masked(br, t) && __syncthreads_or(wild(buf))) take_out(buf, t * KV_TILE);
    if (t >= wr.n0 && t <= wr.n1) {
      scores(s, buf);
      settle(s, buf, t * KV_TILE, masked(wr, t));
      probs(s, pf, buf);
      outputs(pf, buf);
    }
    if (t < t1) spread(other);
  };
  if (work) {
    look_up(later, t0 * KV_TILE);
    ask(t0, B0);
    spread(B0);
    for (int t = t0; t <= t1; t += 2) {
      visit(t, B0, B1);
      if (t < t1) visit(t + 1, B1, B0);
    }
  }

  // lane (qc, hf): o[d][4 j + e] is position 32 d + 8 j + 4 hf + e of its row
  {
    l += __shfl_xor(l, 32, 64);
    const bool one = a.splits == 1;
    const float inv = one ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] *= inv;
    if constexpr (INT4) {
      // positions of eight hold dims kv_perm: back to natural order, the lane
      // keeping dims 8 (4 d + j) + 4 hf + e.  Position 4 hf + e is dim
      // {0, 4, 1, 5}[e] + 2 hf: the halves swap what the other one keeps.
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = o[d][4 * j], x1 = o[d][4 * j + 1], x2 = o[d][4 * j + 2], x3 = o[d][4 * j + 3];
          // hf 0 holds dims 0, 4, 1, 5 and keeps 0..3; hf 1 holds 2, 6, 3, 7 and keeps 4..7
          const float g0 = __shfl_xor(hf ? x0 : x1, 32, 64), g1 = __shfl_xor(hf ? x2 : x3, 32, 64);
          o[d][4 * j] = hf ? g0 : x0;
          o[d][4 * j + 1] = hf ? g1 : x2;
          o[d][4 * j + 2] = hf ? x1 : g0;
          o[d][4 * j + 3] = hf ? x3 : g1;
        }
      if (one) {
        // S Hn over the row: dim bits 0, 1 are e, bit 2 the lane's half, the rest j and d
        float x[16 * DB];
#pragma unroll
        for (int e = 0; e < 16 * DB; ++e) x[e] = o[e >> 4][e & 15];
        kv_bfly<16 * DB>(x);
        kv_lane_bfly<16 * DB>(x, 32, lane);
#pragma unroll
        for (int e = 0; e < 16 * DB; ++e) {
          const int dim = 8 * (e >> 2) + 4 * hf + (e & 3);
          const uint32_t sg = a.c.signs ? (a.c.signs[dim >> 5] >> (dim & 31)) << 31 : 0u;
          o[e >> 4][e & 15] = as_f(as_u(x[e] * (D == 64 ? 0.125f : 0.08838834764831845f)) ^ sg);  // 1 / sqrt(D)
        }
      }
    }
    if (live) {
      const int64_t gr = (int64_t)(q0 + tok) * a.heads + head;
      if (one) {
        uint8_t* op = a.out + (int64_t)(q0 + tok) * a.o_tok + (int64_t)head * a.o_head;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            stg<u32x2>(op + 2 * (32 * d + 8 * j + 4 * hf), u32x2{kv_pack<T>(o[d][4 * j], o[d][4 * j + 1]),
                                                                 kv_pack<T>(o[d][4 * j + 2], o[d][4 * j + 3])});
        if (a.lse && hf == 0)
          a.lse[gr] = l == 0.f ? KV_NEG_INF : (m * qs + (INT4 ? (float)ve : 0.f) - KV_UP<MT> + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
      } else {
        const int64_t pr = (int64_t)split * a.q_tokens * a.heads + gr;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            stg<f32x4>(a.part_o + pr * D + 32 * d + 8 * j + 4 * hf,
                       f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]});
        if (hf == 0) {
          a.part_ml[2 * pr] = m == KV_NEG_INF ? m : m * qs + (INT4 ? (float)ve : 0.f) - KV_UP<MT>;
          a.part_ml[2 * pr + 1] = l;
        }
      }
    }
  }
}

template <int D, int T, bool INT4>
static hipError_t chunk_launch(KvAttnArgs a, int waves, hipStream_t s) {
  const int most = (int)(kLaunchThreads / (64 * waves));  // (a multiple of 8: blocks keep their XCDs)
  for (a.launched = 0;;) {
    const int n = std::min(a.grid - a.launched, most);
    if (INT4 && waves == 8) hipLaunchKernelGGL((k_kv_chunk<D, T, INT4, INT4 ? 8 : 4>), dim3(n), dim3(512), 0, s, a);
    else hipLaunchKernelGGL((k_kv_chunk<D, T, INT4, 4>), dim3(n), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || n == a.grid - a.launched) return e;
    a.launched += n;
  }
}

// waves: 4, or for INT4 8; 32 rows each
hipError_t launch_kv_chunk(const KvAttnArgs& a, int dim, int dt, bool int4, int waves, hipStream_t s) {
  if (dim == 128) {
    if (dt == KV_BF16) return int4 ? chunk_launch<128, KV_BF16, true>(a, waves, s) : chunk_launch<128, KV_BF16, false>(a, waves, s);
    return int4 ? chunk_launch<128, KV_F16, true>(a, waves, s) : chunk_launch<128, KV_F16, false>(a, waves, s);
  }
  if (dt == KV_BF16) return int4 ? chunk_launch<64, KV_BF16, true>(a, waves, s) : chunk_launch<64, KV_BF16, false>(a, waves, s);
  return int4 ? chunk_launch<64, KV_F16, true>(a, waves, s) : chunk_launch<64, KV_F16, false>(a, waves, s);
}

}  // namespace whtq
