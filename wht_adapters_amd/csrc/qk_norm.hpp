// Norms and rotary positions of dense query and key rows: kernel arguments.
#pragma once

#include "kv_rows.hpp"

namespace whtq {

struct QkSide {  // queries or keys; heads 0: none
  KvRows x, y, dy, dx;  // backward: dy the outputs' gradient, dx the rows'
  KvWeight w;
  float* dw;    // [classes][dim]
  int heads;
  int classes;  // weight vectors: 1 or heads
  int blocks;   // backward: blocks of a class
};
struct QkArgs {
  QkSide q, k;
  KvTurn turn;
  int64_t tokens;
  int dt;  // of the weights
  float eps;
  float* part;  // backward: [blocks of q's classes, then of k's][dim]; NULL: a block a class, which writes dw itself
};

}  // namespace whtq
