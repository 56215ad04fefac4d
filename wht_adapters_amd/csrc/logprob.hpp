// Log probabilities of rows of logits: kernel arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace whtq {

constexpr int LP_MOST_VOCAB = 1 << 20, LP_MOST_TOP = 32;  // (WHTQ_TOP_MOST)
constexpr int LP_CHUNK = 512;  // logits a wave takes at a time, 8 a lane
constexpr int LP_MOST_GROUPS = (LP_MOST_VOCAB + 7) / LP_CHUNK + 1;  // of a row

struct LpArgs {
  const uint8_t* x;
  int64_t ld, rows;  // ld in bytes
  int vocab;
  float scale;
  const int64_t* targets;
  float *logprob, *lse, *ref, *sum, *entropy;
  int top;
  float* top_logprob;
  int64_t* top_id;
  int splits, width, groups;  // blocks of a row; logits of a group whose maximum is kept (top > 0), and groups of a row
  float* part;                // [rows][splits][3]: maximum, sum, weighted sum
  uint32_t* best;             // [rows][groups]
  int64_t row0;               // rows in the launches before this one
};
struct LpGradArgs {
  const uint8_t* x;
  uint8_t* dx;
  int64_t ld, ldd, rows;  // bytes
  int vocab, pieces;      // blocks of a row
  float scale;
  const int64_t* targets;
  const float *ref, *sum, *entropy, *dlogprob, *dentropy;
  int64_t row0;
};

}  // namespace whtq
