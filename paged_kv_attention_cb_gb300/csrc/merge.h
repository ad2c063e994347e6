// The log-sum-exp merge of query rows whose keys were attended in several pieces.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace cb {

// Output row t is merged from na partial rows a, a + a_step, ... and nb rows b, b + b_step, ...
// of the partial arrays.
struct MergeRow {
  int t;
  int a, a_step, na;
  int b, b_step, nb;
};

constexpr int kMergeThreads = 256;

struct MergeArgs {
  void* out;             // [T, Hq, D]
  int dtype;
  int num_q_heads, head_dim;
  const float* part_o;   // [row][Hq][D] unnormalised
  const float2* part_ml; // [row][Hq] (running maximum in log2 units, sum)
  int parts;             // threads per output, each over a share of the pieces
};

// Threads per output for rows of up to `pieces` pieces.
int merge_parts(int pieces);
// `rows`: n rows, in as many launches as they need.
cudaError_t launch_merge(const MergeArgs& m, const MergeRow* rows, int n, cudaStream_t stream);

}  // namespace cb
