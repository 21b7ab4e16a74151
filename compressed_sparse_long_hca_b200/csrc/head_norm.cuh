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
  int vec, block_heads, block0, blocks;   // set by the launch: its blocks of a token are block0, ..., block_heads heads each
};

struct HeadNormArgs {
  int64_t n_tok;
  const int64_t* positions;
  const double* theta;                 // [rope / 2]
  double eps;
  int dim, rope;
  int lanes, blocks;                   // lanes of a head, blocks of a token (set by the launch)
  int group;                           // for blocks with runs of tokens, set by the launch: the tokens whose sines are
  int64_t share;                       // kept at once, and the cost a block takes
  HeadNormPart part[2];
};

}  // namespace csa
