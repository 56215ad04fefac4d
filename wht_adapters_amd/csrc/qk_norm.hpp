// Norms and rotary positions of query and key rows: kernel arguments.
#pragma once

#include "kv_rows.hpp"

namespace whtq {

// Unsigned division of numbers below 2^31 by d, as a product (m 0: by 1).
struct KvDiv {
  uint32_t m, d;
  int s;
};

// forward: rows of one kind (queries, keys, values) and where they go
struct QkForward {
  KvRows in, out;  // out.p NULL: into the cache
  KvSide side;
  KvWeight w;      // p NULL: neither normed
  bool turned;     // rotated
  KvDiv heads;
  uint32_t rows, blocks;
  bool clear;      // rows of out whose token is outside the positions become 0
};
struct QkForwardArgs {
  QkForward f[3];
  KvCache c;
  const int64_t* slots;
  int64_t capacity;
  KvTurn turn;
  int dt;  // of the weights
  float eps;
};

struct QkSide {  // backward: queries or keys; heads 0: none
  KvRows x, dy, dx;  // dy the outputs' gradient, dx the rows'
  KvWeight w;
  float* dw;    // [classes][dim]
  int heads;
  int classes;  // weight vectors: 1 or heads
  int blocks;   // blocks of a class
  bool clear;   // rows of dx whose token is outside the positions become 0
};
struct QkArgs {
  QkSide q, k;
  KvTurn turn;
  int64_t tokens;
  int dt;
  float eps;
  float* part;  // [blocks of q's classes, then of k's][dim]; NULL: a block a class, which writes dw itself
};

}  // namespace whtq
