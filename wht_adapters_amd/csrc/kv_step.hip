// Instances of the step kernel without sinks, and the joining of split results.
#include "kv_step.hpp"

namespace whtq {

hipError_t launch_kv_step_sinks(const KvAttnArgs& a, int dim, int dt, bool int4, int nq, hipStream_t s);

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
  if constexpr (INT4) kv_row_rht<D, 8, 1, true>(x, i0, lane, a.c.signs);
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
hipError_t step_join_launch(KvAttnArgs a, hipStream_t s) {
  // as many groups a row as keep the machine busy
  int gr = 1;
  const int most = 256 / (D / 8);
  const int64_t rows = a.q_tokens * a.heads;
  while (gr < most && gr < a.blocks && rows * gr < 8192) gr *= 2;
  const int per = most / gr, parts = (a.rows + per - 1) / per;
  const int most_seqs = (int)std::min<int64_t>(a.seqs, kLaunchThreads / 256 / ((int64_t)a.c.kv_heads * parts));
  hipError_t e = hipSuccess;
  for (a.launched = 0; e == hipSuccess && a.launched < a.seqs; a.launched += most_seqs) {
    const int n = std::min(a.seqs - a.launched, most_seqs);
    hipLaunchKernelGGL((k_kv_step_join<D, T, INT4>), dim3((unsigned)(n * a.c.kv_heads * parts)), dim3(256), 0, s, a, gr, parts);
    e = hipGetLastError();
  }
  return e;
}
template hipError_t step_join_launch<64, KV_BF16, false>(KvAttnArgs, hipStream_t);
template hipError_t step_join_launch<64, KV_BF16, true>(KvAttnArgs, hipStream_t);
template hipError_t step_join_launch<64, KV_F16, false>(KvAttnArgs, hipStream_t);
template hipError_t step_join_launch<64, KV_F16, true>(KvAttnArgs, hipStream_t);
template hipError_t step_join_launch<128, KV_BF16, false>(KvAttnArgs, hipStream_t);
template hipError_t step_join_launch<128, KV_BF16, true>(KvAttnArgs, hipStream_t);
template hipError_t step_join_launch<128, KV_F16, false>(KvAttnArgs, hipStream_t);
template hipError_t step_join_launch<128, KV_F16, true>(KvAttnArgs, hipStream_t);
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

// Keys of a unit of the step kernel (one tile for each wave of a block).
int kv_step_unit(int dim, bool int4, bool whole) { return (dim == 128 && !int4 ? 32 : 64) * (whole ? 8 : 4); }

template <int D, int T, bool INT4>
static hipError_t plain_launch(const KvAttnArgs& a, int nq, hipStream_t s) { return step_launch<D, T, INT4, false>(a, nq, s); }
hipError_t launch_kv_step(const KvAttnArgs& a, int dim, int dt, bool int4, int nq, hipStream_t s) {
  if (a.sinks > 0) return launch_kv_step_sinks(a, dim, dt, int4, nq, s);
  return KV_PICK(plain_launch, dim, dt, int4, a, nq, s);
}
hipError_t launch_kv_join(const KvAttnArgs& a, int dim, int dt, bool int4, hipStream_t s) {
  return KV_PICK(join_launch, dim, dt, int4, a, s);
}

}  // namespace whtq
