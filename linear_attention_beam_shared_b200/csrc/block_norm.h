// Internal declarations of the norms around a block.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace onela {

struct BlockNormParams {
  int64_t N, y_stride, gate_stride, x_stride;
  int D, group;
  int y_bf16, bf16;  // element types: of y; of gate, x and the outputs
  int act;
  float alpha, eps;
  const void *y, *gate, *x;                // any may be null
  const float *w_post, *scale, *w_pre;
  void *x_out, *n_out;
};

cudaError_t launch_block_norm(const BlockNormParams &p, cudaStream_t s);

}  // namespace onela
