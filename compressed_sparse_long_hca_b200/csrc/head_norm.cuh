// Arguments of the head-norm launch, shared by its kernel and the C ABI.
#pragma once
#include <stdint.h>

namespace csa {

struct HeadNormPart {                  // the query heads, or the key heads
  const void* x;
  void* y;
  const float* weight;                 // [dim], or null (ones)
  int64_t x_tok, x_head, y_tok, y_head;   // strides in elements
  int heads, f32, rotate;
  int vec, block_heads, blocks;        // set by the launch
};

struct HeadNormArgs {
  int64_t n_tok;
  const int64_t* positions;
  const double* theta;                 // [rope / 2]
  double eps;
  int dim, rope;
  int lanes;                           // lanes of a head (set by the launch)
  HeadNormPart part[2];
};

}  // namespace csa
