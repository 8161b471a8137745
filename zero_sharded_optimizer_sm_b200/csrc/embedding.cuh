// The embedding at a model's entrance: the lookup of a batch's rows and the
// gradient of the whole table.
//
//   out[t] = scale * table[token[t]]
//   dtable[v] = scale * sum over the t with token[t] = v of dy[t]
//
// A token outside [0, vocab) stands for padding: a row of zeros, no gradient.
#pragma once

#include "mx4.cuh"

namespace zsm {

struct EmbeddingArgs {
  const void* tokens;  // n of token_bytes each
  int token_bytes;     // 4 or 8
  int64_t n, vocab, cols;
  const void* table;   // of `type`, ld elements between rows; or an MX4 matrix:
  MxMatrix from;       //   (codes set)
  int type;
  int64_t ld;
  float scale;
  void* out;
  int out_type;
  int64_t ld_out;
};

struct EmbeddingBackwardArgs {
  const void* dy;
  int type;
  int64_t n, cols, ld_dy;
  const void* tokens;
  int token_bytes;
  int64_t vocab;
  float scale;
  void* dtable;
  int dtable_type;
  int64_t ld;
  int accumulate;   // 1: added to what dtable holds
  void* workspace;  // embedding_backward_workspace bytes
};

cudaError_t launch_embedding(const EmbeddingArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_embedding_backward(const EmbeddingBackwardArgs& a, int sm_count, cudaStream_t s);
int64_t embedding_backward_workspace(int64_t n, int64_t cols);

}  // namespace zsm
