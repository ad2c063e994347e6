// Host-side checks and error reporting shared by the entry points.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "cb.h"

namespace cb {

// Record the message (and the CUDA error) for cb_last_error_message and return the status.
cb_status report_error(cb_status s, const char* msg);
cb_status report_cuda_error(cudaError_t e, const char* what);

// Arrays in a workspace start at multiples of 32 bytes whatever the workspace's own address (16-byte
// aligned): the widest stores take 32. A workspace has kWorkspaceAlign bytes to spare for it.
constexpr size_t kWorkspaceAlign = 32;
inline uint8_t* align_workspace(void* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + kWorkspaceAlign - 1) & ~(uintptr_t)(kWorkspaceAlign - 1));
}

inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The sizes of a step: signs, supported head_dim / group / block_size / dtype, host mirrors given.
cb_status check_step_sizes(int32_t num_requests, int32_t num_tokens, int32_t num_blocks,
                           int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                           int32_t head_dim, int32_t block_table_stride, int32_t dtype,
                           const int32_t* h_query_start_loc, const int32_t* h_seq_lens);

// The host mirrors: query_start_loc[0] = 0, non-decreasing, 0 <= q_len <= seq_len. max_pages:
// the most pages a request has.
cb_status check_step_mirrors(const int32_t* h_query_start_loc, const int32_t* h_seq_lens,
                             int32_t num_requests, int32_t block_size, int64_t* max_pages);

}  // namespace cb
