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
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kv_attn.hpp"
#include "launch.hpp"

namespace whtq {

constexpr int KV_TILE = 64;

typedef short kv_s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 kv_tr_read(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) kv_s16x4*)p));
}

template <int D, int T, bool INT4, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_kv_chunk(const KvAttnArgs a) {
  constexpr int MT = INT4 ? KV_F16 : T;
  constexpr int ROWS = 32 * NW, CH = D / 8, ROWB = 2 * D;  // 16-byte chunks and bytes of a tile row
  constexpr int KK = D / 16, DB = D / 32;
  constexpr int TILEB = KV_TILE * ROWB;
  constexpr int KSW = CH - 1, VSW = CH / 2 - 1;            // swizzles: chunk ^ (row & KSW), chunk ^ 2 (row & VSW)
  __shared__ __attribute__((aligned(16))) uint8_t sk[2][TILEB], sv[2][TILEB];
  __shared__ __attribute__((aligned(16))) float sks[2][INT4 ? KV_TILE : 1], svs[2][INT4 ? KV_TILE : 1];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int qc = lane & 31, hf = lane >> 5;

  // block -> (tile of rows, head, split).  Blocks are dealt to the 8 XCDs in
  // turn; whole groups of one head and split go to one XCD each, so that its
  // L2 holds their keys (groups beyond a multiple of 8 are spread over all).
  // Later tiles of a causal chunk are longer and go first.
  const int groups = a.c.kv_heads * a.splits, per = gridDim.x / groups, whole = groups / 8 * 8;
  int hs, slot;
  if ((int)blockIdx.x < whole * per) {
    const int i = blockIdx.x >> 3;
    hs = i / per * 8 + (blockIdx.x & 7);
    slot = i % per;
  } else {
    const int i = blockIdx.x - whole * per;
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
  const int64_t row0 = (slot - ((int64_t)q0 * a.group / ROWS + b)) * ROWS;
  const int64_t rows = (int64_t)chunk * a.group;
  if (row0 < 0 || row0 >= rows) return;
  const int kv = min(a.kv_len[b], (int)min<int64_t>((int64_t)a.table_width << a.c.page_shift, INT32_MAX));
  const int p0 = kv - chunk;
  const int32_t* table = a.table + b * a.table_stride;

  // first and last position among rows [r0, r0 + n) that exist
  const int tok0 = (int)(row0 / a.group), tok1 = (int)((min<int64_t>(row0 + ROWS, rows) - 1) / a.group);
  const int first = a.window > 0 ? max(0, p0 + tok0 - a.window + 1) : 0;
  const int last = a.causal ? min(kv - 1, p0 + tok1) : kv - 1;
  const int lo = split * a.split_keys, hi = split == a.splits - 1 ? INT32_MAX : lo + a.split_keys - 1;
  const int kfirst = max(first, lo), klast = min(last, hi);
  // the same for the wave's rows
  const int64_t wr0 = row0 + 32 * wave;
  const bool wlive = wr0 < rows;
  const int wt0 = (int)(wr0 / a.group), wt1 = (int)((min<int64_t>(wr0 + 32, rows) - 1) / a.group);
  const int wany0 = a.window > 0 ? max(kfirst, p0 + wt0 - a.window + 1) : kfirst;   // some row sees keys of [wany0, wany1]
  const int wany1 = a.causal ? min(klast, p0 + wt1) : klast;

  // the lane's query
  const int64_t row = wr0 + qc;
  const int tok = (int)(row / a.group), head = h * a.group + (int)(row % a.group);
  const bool live = row < rows && (uint32_t)(q0 + tok) < (uint64_t)a.q_tokens;
  const int pos = p0 + tok;
  // the scores are kept in units of 1 / qs, qs >= 0: a negative scale turns q around
  float qs = fabsf(a.scale);
  const uint32_t turn = a.scale < 0.f ? 0x80008000u : 0u;
  u32x4 qf[KK];
  {
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
      qs *= __builtin_ldexpf(1.f, ex);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int w = 0; w < 4; ++w)
          qf[kk][w] = pack_f16(x[8 * kk + kv_perm(2 * w)] * down, x[8 * kk + kv_perm(2 * w + 1)] * down) ^ turn;
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
  constexpr int CR = 64 / CH;                     // rows of one copy instruction (4 or 8; in one page)
  constexpr int COPIES = KV_TILE / (CR * NW);     // copy instructions of a wave for K, and for V
  auto copy_key = [&](int n, int key0) {          // first key of copy n, wave-uniform for a given n
    return min(max(key0 + (n * NW + wave) * CR, kfirst & ~(CR - 1)), klast & ~(CR - 1));
  };
  auto copy = [&](int buf, int key0, int entry) {  // dense; lane n holds the table entry of copy n
    const int pages = kv_page(a, entry);
#pragma unroll
    for (int n = 0; n < COPIES; ++n) {
      const int r0 = (n * NW + wave) * CR, lr = lane / CH;
      const int k0 = copy_key(n, key0);
      const int64_t page = __builtin_amdgcn_readlane(pages, n);
      const int off = (k0 & ((1 << a.c.page_shift) - 1)) + min(max(lr, kfirst - k0), klast - k0);
      const int tr = r0 + lr, cc = lane % CH;
      const uint8_t* kp = kbase + page * a.c.k.page + off * a.c.k.tok + 16 * (cc ^ (tr & KSW));
      const uint8_t* vp = vbase + page * a.c.v.page + off * a.c.v.tok + 16 * (cc ^ (2 * (tr & VSW)));
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)kp,
                                       (__attribute__((address_space(3))) void*)(sk[buf] + r0 * ROWB), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)vp,
                                       (__attribute__((address_space(3))) void*)(sv[buf] + r0 * ROWB), 16, 0, 0);
    }
  };
  // INT4: unit u of a tile is 16 bytes (32 codes) of one row of K or V
  constexpr int UR = D / 32;                                  // units of a row
  constexpr int UNITS = 2 * KV_TILE * UR, UT = UNITS / (64 * NW);
  static_assert(UNITS % (64 * NW) == 0, "whole units a thread");
  u32x4 code[INT4 ? UT : 1];
  uint16_t scl = 0;
  auto unit_row = [&](int n) { return (n * 64 * NW + (int)threadIdx.x) % (UNITS / 2) / UR; };
  auto inside = [&](int key) { return min(max(key, kfirst), klast); };
  // Table entries of a tile, held by the lanes that need them: dense, copy n's
  // in lane n; INT4, of the thread's units and of its scale.  Memory answers
  // in order: they are asked for before the copies of the tile before.
  struct Pages {
    int at[INT4 ? UT + 1 : 1];
  };
  auto look_up = [&](Pages& p, int key0) {
    if constexpr (INT4) {
#pragma unroll
      for (int n = 0; n < UT; ++n) p.at[n] = table[inside(key0 + unit_row(n)) >> a.c.page_shift];
      p.at[UT] = table[inside(key0 + (int)(threadIdx.x % KV_TILE)) >> a.c.page_shift];
    } else {
      p.at[0] = table[copy_key(lane % COPIES, key0) >> a.c.page_shift];
    }
  };
  auto fetch = [&](int key0, const Pages& p) {
    if constexpr (INT4) {
#pragma unroll
      for (int n = 0; n < UT; ++n) {
        const int u = n * 64 * NW + threadIdx.x, c = u % UR;
        const int64_t page = kv_page(a, p.at[n]);
        const int off = inside(key0 + unit_row(n)) & ((1 << a.c.page_shift) - 1);
        code[n] = u >= UNITS / 2 ? ldg_global<u32x4>(vbase + page * a.c.v.page + off * a.c.v.tok + 16 * c)
                                 : ldg_global<u32x4>(kbase + page * a.c.k.page + off * a.c.k.tok + 16 * c);
      }
      if (threadIdx.x < 2 * KV_TILE) {
        const int64_t page = kv_page(a, p.at[UT]);
        const int off = inside(key0 + (int)(threadIdx.x % KV_TILE)) & ((1 << a.c.page_shift) - 1);
        scl = threadIdx.x < KV_TILE ? a.c.k.scale[page * a.c.k.s_page + h * a.c.k.s_head + off]
                                    : a.c.v.scale[page * a.c.v.s_page + h * a.c.v.s_head + off];
      }
    }
  };
  auto spread = [&](int buf) {
    if constexpr (INT4) {
#pragma unroll
      for (int n = 0; n < UT; ++n) {
        const int u = n * 64 * NW + threadIdx.x, tr = unit_row(n), c = u % UR;
        const bool isv = u >= UNITS / 2;
        uint8_t* rowp = (isv ? sv[buf] : sk[buf]) + tr * ROWB;
        const int sw = isv ? 2 * (tr & VSW) : tr & KSW;
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<u32x4*>(rowp + 16 * ((4 * c + j) ^ sw)) = kv_codes8(code[n][j]);
      }
      if (threadIdx.x < 2 * KV_TILE) {
        const float s = (float)__builtin_bit_cast(_Float16, scl);
        if (threadIdx.x < KV_TILE) sks[buf][threadIdx.x] = s;
        else svs[buf][threadIdx.x - KV_TILE] = s;
      }
    }
  };

  auto sees = [&](int key) {
    return key >= kfirst && key <= klast && (!a.causal || key <= pos) && (a.window <= 0 || key > pos - a.window);
  };
  // A probability of 0 does not hide a value that is not finite, so in a
  // tile that some row does not see whole such values are taken out: the
  // outputs of the rows that see them become what they are (the sum's result
  // whatever the probability), and the tile holds 0 in their place.
  auto wild = [&](int buf) {  // whether this thread's part of the V tile holds any
    bool any = false;
    for (int i = threadIdx.x; i < TILEB / 16; i += 64 * NW) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(sv[buf] + 16 * i);
      u16x2 big = {0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = w[e];
        big = absmax16(big, x);
      }
      any = any || kv_not_finite<T>(big);
    }
    return any;
  };
  constexpr uint32_t EXPO = T == KV_BF16 ? 0x7f80u : 0x7c00u;
  auto take_out = [&](int buf, int key0) {
#pragma unroll 1
    for (int j = 0; j < KV_TILE; ++j) {
      const bool mine = wlive && sees(key0 + j);
      const uint8_t* rp = sv[buf] + j * ROWB;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(rp + 16 * ((4 * d + jj) ^ (2 * (j & VSW))) + 8 * hf);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x = w[e >> 1], b = e & 1 ? x >> 16 : x & 0xffffu;
            const float v = T == KV_BF16 ? as_f(b << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)b);
            o[d][4 * jj + e] += mine && (b & EXPO) == EXPO ? v : 0.f;
          }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < TILEB / 4; i += 64 * NW) {
      uint32_t* p = reinterpret_cast<uint32_t*>(sv[buf]) + i;
      const uint32_t x = *p;
      *p = ((x & EXPO) == EXPO ? 0u : x & 0xffffu) | ((x >> 16 & EXPO) == EXPO ? 0u : x & 0xffff0000u);
    }
    __syncthreads();
  };
  // --- one tile.  MASK: some row of the block does not see all of it.
  auto tile = [&](auto mask, int buf, int key0) {
    constexpr bool MASK = decltype(mask)::value;
    if (!wlive) return;
    if (MASK && (key0 > wany1 || key0 + KV_TILE - 1 < wany0)) return;
    // S^T: lane (qc, hf), s[kb][4 j + e] is key 32 kb + 8 j + 4 hf + e
    f32x16 s[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const int tr = 32 * kb + qc;
      const uint8_t* rp = sk[buf] + tr * ROWB;
#pragma unroll
      for (int e = 0; e < 16; ++e) s[kb][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
        s[kb] = kv_mfma32<MT>(*reinterpret_cast<const u32x4*>(rp + 16 * ((2 * kk + hf) ^ (tr & KSW))), qf[kk], s[kb]);
    }
    float top = KV_NEG_INF;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (INT4) {
          const f32x4 ksc = *reinterpret_cast<const f32x4*>(&sks[buf][32 * kb + 8 * j + 4 * hf]);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[kb][4 * j + e] *= ksc[e];
        }
        if constexpr (MASK) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[kb][4 * j + e] = sees(key0 + 32 * kb + 8 * j + 4 * hf + e) ? s[kb][4 * j + e] : KV_NEG_INF;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[kb][4 * j + e]);
      }
    // scores are in units of 1 / qs here; the maximum too
    if (__any(top > m + lag)) {
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float mn = fmaxf(m, top);
      const float al = m == KV_NEG_INF ? 1.f : __builtin_amdgcn_exp2f((m - mn) * qs);  // 1: l is 0, o 0 or not finite
      l *= al;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= al;
      m = mn;
    }
    float unit = 1.f;
    if constexpr (INT4) {
      float vtop = svs[buf][lane];
      vtop = vtop < 65536.f ? vtop : 0.f;
      if (__any(vtop >= __builtin_ldexpf(1.f, ve + 1))) {
#pragma unroll
        for (int x = 1; x < 64; x *= 2) vtop = fmaxf(vtop, __shfl_xor(vtop, x, 64));
        const int e = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(vtop) - 1);
        const float f = __builtin_ldexpf(1.f, ve - e);
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] *= f;
        ve = e;
      }
      unit = __builtin_ldexpf(1.f, -ve);
    }
    const float base = -kv_base(m) * qs;
    u32x4 pf[4];  // slots 0..7 of 16 keys: words 4 j', 4 j' + 2 of their scores
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 vsc = {1.f, 1.f, 1.f, 1.f};
        if constexpr (INT4) vsc = *reinterpret_cast<const f32x4*>(&svs[buf][32 * kb + 8 * j + 4 * hf]);
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = s[kb][4 * j + e];
          p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x, qs, base));
          if constexpr (MASK) p[e] = x == KV_NEG_INF ? 0.f : p[e];
          l += p[e];
          if constexpr (INT4) p[e] = MASK && x == KV_NEG_INF ? 0.f : p[e] * (vsc[e] * unit);
        }
        pf[2 * kb + j / 2][2 * (j & 1)] = kv_pack<MT>(p[0], p[1]);
        pf[2 * kb + j / 2][2 * (j & 1) + 1] = kv_pack<MT>(p[2], p[3]);
      }
    // O^T: product of 16 keys: lane (dim qc of 32, hf) needs keys 4 hf .. and 8 + 4 hf ..
    const int ln = lane & 15, dg = (lane >> 4) & 1;
    auto value = [&](int ks, int d) {
      u32x4 f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tr = 16 * ks + 8 * u + 4 * hf + (ln >> 2);
        const int cc = 4 * d + 2 * dg + ((ln & 3) >> 1);
        const u32x2 w = kv_tr_read(sv[buf] + tr * ROWB + 16 * (cc ^ (2 * (tr & VSW))) + 8 * (ln & 1));
        f[2 * u] = w.x;
        f[2 * u + 1] = w.y;
      }
      return f;
    };
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] = kv_mfma32<MT>(value(ks, d), pf[ks], o[d]);
  };

  const bool work = kfirst <= klast;
  const int t0 = kfirst / KV_TILE, t1 = work ? klast / KV_TILE : t0 - 1;
  // tiles [f0, f1) that every row of the block sees whole
  const int bfull0 = a.window > 0 ? max(kfirst, p0 + tok1 - a.window + 1) : kfirst;
  const int bfull1 = a.causal ? min(klast, p0 + tok0) : klast;
  const int f0 = min(max(t0, (bfull0 + KV_TILE - 1) / KV_TILE), t1 + 1);
  const int f1 = min(max(f0, (bfull1 + 1) / KV_TILE), t1 + 1);
  Pages ahead = {};
  if (work) {
    Pages now;
    look_up(now, t0 * KV_TILE);
    look_up(ahead, (t0 + 1) * KV_TILE);
    if constexpr (INT4) {
      fetch(t0 * KV_TILE, now);
      spread(0);
    } else {
      copy(0, t0 * KV_TILE, now.at[0]);
    }
  }
  int buf = 0;
  auto walk = [&](auto mask, int from, int to) {
    for (int t = from; t < to; ++t) {
      // this tile has landed, and every wave is done with the other buffer
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (t < t1) {
        const Pages now = ahead;
        look_up(ahead, (t + 2) * KV_TILE);
        if constexpr (INT4) fetch((t + 1) * KV_TILE, now);
        else copy(buf ^ 1, (t + 1) * KV_TILE, now.at[0]);
      }
      if constexpr (decltype(mask)::value && !INT4) {
        if (__syncthreads_or(wild(buf))) take_out(buf, t * KV_TILE);
      }
      tile(mask, buf, t * KV_TILE);
      if constexpr (INT4) {
        if (t < t1) spread(buf ^ 1);
      }
      buf ^= 1;
    }
  };
  if (f0 > t0) walk(std::true_type{}, t0, f0);
  walk(std::false_type{}, f0, f1);
  walk(std::true_type{}, f1, t1 + 1);

  // lane (qc, hf): o[d][4 j + e] is position 32 d + 8 j + 4 hf + e of its row
  if (!wlive) return;
  l += __shfl_xor(l, 32, 64);
  const bool one = a.splits == 1;
  const float inv = one ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
  const float out_scale = INT4 ? inv * __builtin_ldexpf(1.f, ve) : inv;
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] *= out_scale;
  const int64_t gr = (int64_t)(q0 + tok) * a.heads + head;
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
  if (!live) return;
  if (one) {
    uint8_t* op = a.out + (int64_t)(q0 + tok) * a.o_tok + (int64_t)head * a.o_head;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        stg<u32x2>(op + 2 * (32 * d + 8 * j + 4 * hf),
                   u32x2{kv_pack<T>(o[d][4 * j], o[d][4 * j + 1]), kv_pack<T>(o[d][4 * j + 2], o[d][4 * j + 3])});
    if (a.lse && hf == 0) a.lse[gr] = l == 0.f ? KV_NEG_INF : (m * qs + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
  } else {
    const int64_t pr = (int64_t)split * a.q_tokens * a.heads + gr;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        stg<f32x4>(a.part_o + pr * D + 32 * d + 8 * j + 4 * hf,
                   f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]});
    if (hf == 0) {
      a.part_ml[2 * pr] = m == KV_NEG_INF ? m : m * qs;
      a.part_ml[2 * pr + 1] = l;
    }
  }
}

template <int D, int T, bool INT4>
static hipError_t chunk_launch(const KvAttnArgs& a, int64_t tiles, hipStream_t s) {
  const dim3 grid((unsigned)(tiles * a.c.kv_heads * a.splits));
  hipLaunchKernelGGL((k_kv_chunk<D, T, INT4, 4>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

int kv_chunk_rows() { return 128; }

hipError_t launch_kv_chunk(const KvAttnArgs& a, int dim, int dt, bool int4, int64_t tiles, hipStream_t s) {
  if (dim == 128) {
    if (dt == KV_BF16) return int4 ? chunk_launch<128, KV_BF16, true>(a, tiles, s) : chunk_launch<128, KV_BF16, false>(a, tiles, s);
    return int4 ? chunk_launch<128, KV_F16, true>(a, tiles, s) : chunk_launch<128, KV_F16, false>(a, tiles, s);
  }
  if (dt == KV_BF16) return int4 ? chunk_launch<64, KV_BF16, true>(a, tiles, s) : chunk_launch<64, KV_BF16, false>(a, tiles, s);
  return int4 ? chunk_launch<64, KV_F16, true>(a, tiles, s) : chunk_launch<64, KV_F16, false>(a, tiles, s);
}

}  // namespace whtq
