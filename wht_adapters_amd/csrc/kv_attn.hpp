// Shared by the attention kernels over a paged cache: arguments, the keys a
// query sees, and the softmax of scores held as S^T.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T, so that a lane's
// column is ONE query: its scores, maximum, sum and outputs stay in that
// lane (and the few lanes that share the column), the probabilities are
// already the second product's operand, and no score crosses lanes but for
// the maximum.  The order of the keys inside a product is free, so the
// values are read in the order the scores came out in.
#pragma once

#include "kv.hpp"

namespace whtq {

struct KvAttnArgs {
  KvCache c;
  const uint8_t* q;
  uint8_t* out;
  int64_t q_tok, q_head, o_tok, o_head;  // bytes
  float* lse;
  const int32_t *q_start, *kv_len, *table;
  int64_t table_stride;
  // partial results in fp32 (maximum and sum apart from the outputs): chunk
  // kernel [split][q_tokens * heads], step kernel [run + sequence][kv_heads][rows]
  float *part_o, *part_ml;
  int* reach;  // step kernel: first and last run of each sequence
  int64_t q_tokens;
  int table_width, heads, group, seqs, causal, window;
  int splits, grid;        // chunk kernel: splits of the keys, blocks in all
  int blocks, rows;        // step kernel: runs a head (0: a block per sequence), rows of a sequence and head (max_q_len * group)
  int launched;            // blocks (chunk kernel) or sequences (joining of steps) in the launches before this one
  float scale;  // times log2(e)
};

constexpr float KV_NEG_INF = -__builtin_huge_valf();

// exp2 of a score against the running maximum (a maximum of -inf means that
// nothing was seen yet: the score is -inf too and gives 0).
__device__ __forceinline__ float kv_base(float m) { return m == KV_NEG_INF ? 0.f : m; }
// Scores are compared with a maximum that may lag behind by up to 2^KV_LAG:
// the accumulators are rescaled only when a score exceeds it by more.  The
// final division by the sum makes the result the same.
constexpr float KV_LAG = 6.f;
// Probabilities that become fp16 operands are kept times 2^8: with the lag and
// INT4's value scale (below 2 in the outputs' unit) they stay below 2^15, and
// their least is 2^-32 of the maximum's instead of 2^-24, so that a hundred
// thousand keys of small weight beside one of large weight keep theirs (131064
// keys of 2^-25.1: they were all 0, 0.05 % of the weight and the whole result
// where the heavy keys' values are 0).  Sums and outputs are in the same unit,
// maxima leave the kernel in it.  bf16 has fp32's range and needs none of it.
template <int MT>
constexpr float KV_UP = MT == KV_F16 ? 8.f : 0.f;

// The page a table entry names; entries outside the cache read page 0.  The
// kernels load entries one tile of keys ahead of the keys themselves, so that
// a tile's copies never wait for them.
__device__ __forceinline__ int kv_page(const KvAttnArgs& a, int entry) {
  return (uint32_t)entry < (uint64_t)a.c.num_pages ? entry : 0;
}

// A sequence's length, held to [0, what its row of the table covers] and to
// 2^30 keys: sums of a position, a window and a tile stay inside 32 bits.
__device__ __forceinline__ int kv_held(const KvAttnArgs& a, int len) {
  return max(0, min(len, (int)min<int64_t>((int64_t)a.table_width << a.c.page_shift, 1 << 30)));
}

template <int T>
__device__ __forceinline__ f32x4 kv_mfma16(u32x4 x, u32x4 y, f32x4 c) {
  if constexpr (T == KV_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x), __builtin_bit_cast(bf16x8_t, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, x), __builtin_bit_cast(f16x8_t, y), c, 0, 0, 0);
}
template <int T>
__device__ __forceinline__ f32x16 kv_mfma32(u32x4 x, u32x4 y, f32x16 c) {
  if constexpr (T == KV_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, x), __builtin_bit_cast(bf16x8_t, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, x), __builtin_bit_cast(f16x8_t, y), c, 0, 0, 0);
}

// What rounding x0, x1 to the fp16 pair hi dropped, as a pair.
__device__ __forceinline__ uint32_t kv_low(uint32_t hi, float x0, float x1) {
  const f16x2_t h = __builtin_bit_cast(f16x2_t, hi);
  return pack_f16(x0 - (float)h[0], x1 - (float)h[1]);
}

// Whether any 16-bit float among the words folded into m (absmax16) is an
// infinity or NaN.
template <int T>
__device__ __forceinline__ bool kv_not_finite(u16x2 m) {
  return absmax16(m) >= (T == KV_BF16 ? 0x7f80u : 0x7c00u);
}

}  // namespace whtq
